// route_common.cuh -- the routing of one token by one warp (the method is
// described at the top of route.cu), shared by the routing kernels and the
// few-token layer.
#pragma once

#include <cfloat>
#include <climits>

#include "moe_ptx.cuh"

namespace moe {

// Warp argmax of (key, id): larger key wins, equal keys go to the lower id.
__device__ __forceinline__ void warp_argmax(float &key, int &id) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float k2 = __shfl_xor_sync(0xffffffffu, key, o);
        const int i2 = __shfl_xor_sync(0xffffffffu, id, o);
        if (k2 > key || (k2 == key && i2 < id)) {
            key = k2;
            id = i2;
        }
    }
}

__device__ __forceinline__ float sigmoid_exact(float z) {
    return (float)(1.0 / (1.0 + exp(-(double)z)));
}

// Fills slot j = lane (< k) of token t from the selected id and its score.
__device__ __forceinline__ void write_weights(int t, int k, int lane, int my_id, float my_s,
                                             float scaling, int32_t *ids, float *w, float *ssel) {
    double S = 0.0;
    for (int j = 0; j < k; ++j) S += (double)__shfl_sync(0xffffffffu, my_s, j);
    if (lane < k) {
        const size_t o = (size_t)t * k + lane;
        ids[o] = my_id;
        ssel[o] = my_s;
        w[o] = S > 0.0 ? (float)((double)scaling * (double)my_s / S) : 0.0f;
    }
}

// The top-k of one token from its logits: lane l holds the logits zv[i] and
// biases bv[i] of experts l + 32 i (read below E only).  lst_*: 32 entries of
// shared memory of this warp each.  Lane j < k gets the id and the score of
// slot j.  Every lane of the warp calls it.
template <int EPL>
__device__ __forceinline__ void route_topk_token(const float (&zv)[EPL], const float (&bv)[EPL],
                                                 int lane, int E, int k, int *lst_e, float *lst_z,
                                                 float *lst_b, int &my_id, float &my_s) {
    float key[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        key[i] = -INFINITY;
        if (lane + 32 * i < E) {
            const float s = 1.0f / (1.0f + expf(-zv[i]));
            const float kk = s + bv[i];
            key[i] = (kk == kk) ? kk : -FLT_MAX;  // NaN ranks last
        }
    }
        // pass 1: approximate k-th key
        uint32_t taken = 0;
        float kth = INFINITY;
        for (int j = 0; j < k; ++j) {
            float bk = -INFINITY;
            int be = INT_MAX;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const int e = lane + 32 * i;
                if (e < E && !(taken >> i & 1u) && (key[i] > bk || (key[i] == bk && e < be))) {
                    bk = key[i];
                    be = e;
                }
            }
            warp_argmax(bk, be);
            if (be != INT_MAX && (be & 31) == lane) taken |= 1u << (be >> 5);
            kth = bk;
        }
        // error bound of the approximate key: expf, 1+e and the division add a
        // few ulp of the score; the two key additions half an ulp of the key each
        const float tol = 4e-6f * fmaxf(1.0f, fabsf(kth));
        const float thr = kth - 2.0f * tol;
        // pass 2: exact keys inside the window, then the exact top-k.  The
        // window's experts are first packed one per lane, so that the warp
        // evaluates the fp64 sigmoid once for all of them.
        bool cand[EPL];
        int ncand = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = lane + 32 * i;
            cand[i] = e < E && key[i] >= thr;
            ncand += __popc(__ballot_sync(0xffffffffu, cand[i]));
        }
        my_id = 0;
        my_s = 0.0f;
        if (ncand <= 32) {
            int base = 0;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const unsigned m = __ballot_sync(0xffffffffu, cand[i]);
                if (cand[i]) {
                    const int pos = base + __popc(m & ((1u << lane) - 1u));
                    lst_e[pos] = lane + 32 * i;
                    lst_z[pos] = zv[i];
                    lst_b[pos] = bv[i];
                }
                base += __popc(m);
            }
            __syncwarp();
            int ce = INT_MAX;
            float cs = 0.0f, ck = -INFINITY;
            if (lane < ncand) {
                ce = lst_e[lane];
                cs = sigmoid_exact(lst_z[lane]);
                const float kk = __fadd_rn(cs, lst_b[lane]);
                ck = (kk == kk) ? kk : -FLT_MAX;
            }
            __syncwarp();
            for (int j = 0; j < k; ++j) {
                float bk = ck;
                int be = ce;
                warp_argmax(bk, be);
                const unsigned owner = __ballot_sync(0xffffffffu, ce == be && be != INT_MAX);
                const int ol = owner ? __ffs(owner) - 1 : 0;
                const float sv = __shfl_sync(0xffffffffu, cs, ol);
                if (lane == ol) {
                    ck = -INFINITY;
                    ce = INT_MAX;
                }
                if (lane == j) {
                    my_id = be == INT_MAX ? 0 : be;
                    my_s = sv;
                }
            }
        } else {
            // many exact ties in the window: every lane evaluates its own experts
            float ek[EPL], es[EPL];
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                es[i] = 0.0f;
                ek[i] = -INFINITY;
                if (cand[i]) {
                    es[i] = sigmoid_exact(zv[i]);
                    const float kk = __fadd_rn(es[i], bv[i]);
                    ek[i] = (kk == kk) ? kk : -FLT_MAX;
                }
            }
            taken = 0;
            for (int j = 0; j < k; ++j) {
                float bk = -INFINITY;
                int be = INT_MAX;
#pragma unroll
                for (int i = 0; i < EPL; ++i) {
                    const int e = lane + 32 * i;
                    if (e < E && !(taken >> i & 1u) && (ek[i] > bk || (ek[i] == bk && e < be))) {
                        bk = ek[i];
                        be = e;
                    }
                }
                warp_argmax(bk, be);
                float sv = 0.0f;
                if (be != INT_MAX && (be & 31) == lane) {
                    const int i = be >> 5;
                    taken |= 1u << i;
#pragma unroll
                    for (int ii = 0; ii < EPL; ++ii)
                        if (ii == i) sv = es[ii];
                }
                const int owner = be == INT_MAX ? 0 : (be & 31);
                sv = __shfl_sync(0xffffffffu, sv, owner);
                if (lane == j) {
                    my_id = be == INT_MAX ? 0 : be;
                    my_s = sv;
                }
            }
        }
}

}  // namespace moe
