// balance.cu -- the balance loss of the router with each expert's load, and its
// gradient at the gate's logits.
//
// For sequence q with N valid tokens (f is a constant of the gradient, as is usual):
//   count[e] = slots of the valid tokens that chose e,  f[e] = E count[e] / (k N)
//   s = sigmoid(z) or exp(z - max z),  p = s / sum_e s  (zeros where the sum is zero)
//   seq_loss = sum_e f[e] mean_t p[t, e],  loss = alpha / n_seq sum_q seq_loss
//   dz[t, j] = dloss alpha / (n_seq N) p_j (f_j - sum_e f_e p_e) (1 - s_j for sigmoid)
// (Text and vision, or any other share of the tokens, are balanced apart by giving each
// as sequences of its own: "HyperParallel加速DeepSeek-V4.1多模态1M长序列训练" §01 item 5.)
//
// Sums are fp32 in a fixed order, so that results do not depend on the schedule: a lane's
// tokens, the warps of a chunk of tokens, the chunks of a sequence (32 interleaved sums).
// (fp64 for the last two cost more than the rest of a small call: this GPU adds two of
// them a cycle.)  Bound by HBM: the logits are read once in
// each direction, and their gradient is written once.  Measured at 65536 x 384 in 16 sequences,
// sigmoid: backward 34 us (87 % of the copy bandwidth by the rows of all tokens), forward 28.5: 22
// of the pass over the tokens, 67 % (it issues in 60 % of its cycles and waits for its loads in
// most others), the rest of the sequences' sums, which begin when the last chunk ends.
// Smallest call: 3.9 and 2.4 us.
#include <cstring>

#include "fp8_common.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr int kOneWarps = 16, kOneTokens = 128;   // of the one CTA that takes a small call

struct BalanceParams {
    int T, E, k, n_seq, chunk, n_chunks;
    bool one;   // one CTA takes all tokens
    float alpha;
    const float *logits;
    const int32_t *ids, *seq_offsets;
    const uint8_t *valid;
    int32_t *counts, *tokens;
    float *load, *seq_loss, *loss;
    const float *dloss;
    float *dlogits;
    // partial sums: one slot for each (chunk, sequence) that meet, at chunk + sequence,
    // which is another number for every such pair
    float *part_p;     // [slots, E]
    int32_t *part_c;   // [slots, E]
    int32_t *part_n;   // [slots]
    unsigned *done;    // sequences that are finished
    unsigned *descend; // the sequences' offsets do
    int *status;
};

__device__ __forceinline__ int seq_begin(const BalanceParams &p, int q) {
    return p.seq_offsets ? min(max(__ldg(p.seq_offsets + q), 0), p.T) : q == 0 ? 0 : p.T;
}

// The first sequence that ends behind token t (n_seq: none); called by a whole warp, which
// looks at 32 places at a time (each look costs a trip to L2).
__device__ __forceinline__ int first_seq(const BalanceParams &p, int t) {
    int lo = 0, hi = p.n_seq;
    while (lo < hi) {
        const int width = (hi - lo + 31) >> 5, at = lo + (threadIdx.x & 31) * width;
        const bool before = at < hi && seq_begin(p, min(at + width, hi)) <= t;
        lo += __popc(__ballot_sync(0xffffffffu, before)) * width;
        if (width == 1) break;
        hi = min(hi, lo + width);
    }
    return min(lo, p.n_seq);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Writes expert e's count and load in sequence q of n valid tokens; returns its term of the
// loss, from its count and the sum of its shares.
__device__ __forceinline__ float finish(const BalanceParams &p, int q, int e, int n, int count,
                                        float shares) {
    const float inv = n ? 1.0f / (float)n : 0.0f;
    const float f = (float)count * inv * ((float)p.E / (float)p.k);
    p.counts[(size_t)q * p.E + e] = count;
    p.load[(size_t)q * p.E + e] = f;
    return n ? f * (shares * inv) : 0.0f;   // (no token: no share, whatever they hold)
}

// A lane's columns: VEC consecutive ones from VEC (lane + 32 i), i < N.
template <int VEC, int N>
struct Row {
    float z[N][VEC];

    __device__ __forceinline__ void load(const float *src, int E) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = VEC * (lane + 32 * i);
#pragma unroll
            for (int j = 0; j < VEC; ++j) z[i][j] = -INFINITY;
            if (c < E) {
                if constexpr (VEC == 4) {
                    const float4 v = __ldg(reinterpret_cast<const float4 *>(src + c));
                    z[i][0] = v.x;
                    z[i][1] = v.y;
                    z[i][2] = v.z;
                    z[i][3] = v.w;
                } else {
                    z[i][0] = __ldg(src + c);
                }
            }
        }
    }
};

// Sigmoids that are all small lose bits below fp32's normal range, and their sum's reciprocal
// may be none (logits of -88 and less).  Below this sum (above it a score that fp32 cannot
// hold is a share below 2^-105) the scores of the row r of such a token are taken relative to
// the largest, s e^-m = e^(z - m) (1 - s), whose common factor leaves p as it is.
constexpr float kLowSum = 0x1p-20f;
template <int VEC, int N>
__device__ __forceinline__ float low_shares(const Row<VEC, N> &r, float (&p)[N][VEC]) {
    float m = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) m = fmaxf(m, r.z[i][j]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (m == -INFINITY) m = 0.0f;   // nothing is left: every term is zero
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const float z = r.z[i][j];   // (below zero)
            p[i][j] = __fdividef(__expf(z - m), 1.0f + __expf(z));
            sum += p[i][j];
        }
    sum = warp_sum(sum);
    return sum == 0.0f ? 0.0f : 1.0f / sum;
}

// z -> s (columns outside E: zeros), p is s times what it returns; slope = 1 - s for the
// sigmoid, 1 otherwise.  low: the scores have to be low_shares().
template <bool SOFTMAX, int VEC, int N>
__device__ __forceinline__ float shares(const Row<VEC, N> &r, float (&p)[N][VEC],
                                       float (&slope)[N][VEC], bool &low) {
    float sum = 0.0f;
    if constexpr (SOFTMAX) {
        float m = -INFINITY;   // (a NaN makes the sum one)
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) m = fmaxf(m, r.z[i][j]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (m == -INFINITY) m = 0.0f;   // nothing is left: every term is zero
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                p[i][j] = __expf(r.z[i][j] - m);
                slope[i][j] = 1.0f;
                sum += p[i][j];
            }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                // both s and 1 - s without cancellation or overflow
                const float z = r.z[i][j], t = __expf(-fabsf(z));
                const float big = __fdividef(1.0f, 1.0f + t);
                // (its own rounding wherever this is used: `low` below has one answer for a row)
                const float small = __fmul_rn(t, big);
                p[i][j] = z < 0.0f ? small : big;
                slope[i][j] = z < 0.0f ? big : small;
                sum += p[i][j];
            }
    }
    sum = warp_sum(sum);
    low = !SOFTMAX && sum < kLowSum;
    return (SOFTMAX ? sum == 0.0f : low) ? 0.0f : 1.0f / sum;
}

// CTA: one chunk of tokens, sequence by sequence; its warps take tokens in turn (UNROLL
// of them at a time, whose loads are issued together), a lane sums its columns' shares in
// registers.  ONE: the chunk is all there is, and the CTA finishes its sums itself.
template <bool SOFTMAX, int VEC, int N, bool ONE>
__global__ void __launch_bounds__(32 * (ONE ? kOneWarps : kWarps), !ONE && N * VEC <= 16 ? 4 : 1)
    balance_part_kernel(const BalanceParams p) {
    constexpr int WARPS = ONE ? kOneWarps : kWarps;
    constexpr int UNROLL = N * VEC <= 16 ? 2 : 1;
    extern __shared__ float sm[];   // [kWarps, E] shares, [E] counts
    __shared__ int n_valid;
    __shared__ float term[WARPS];
    wait_for_kernels_ahead();
    let_kernels_behind_begin();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int32_t *hist = reinterpret_cast<int32_t *>(sm + kWarps * p.E);
    if (!ONE && blockIdx.x == 0 && threadIdx.x == 0) *p.done = 0;
    // Offsets that descend leave the slots of some (chunk, sequence) unwritten and give others
    // to two of them: nothing is counted then.
    bool descend = false;
    if (blockIdx.x == 0 && p.seq_offsets) {
        for (int q = threadIdx.x; q <= p.n_seq; q += blockDim.x) {
            const int o = p.seq_offsets[q];
            const bool down = q > 0 && seq_begin(p, q - 1) > seq_begin(p, q);
            if (o < 0 || o > p.T || down) record_status(p.status, MOE_ERR_INVALID_ARG);
            descend = descend || down;
        }
    }
    const int end = min(p.T, (int)(blockIdx.x + 1) * p.chunk);
    int a = blockIdx.x * p.chunk;
    float loss = 0.0f;
    for (int q = ONE ? 0 : first_seq(p, a); q < p.n_seq && (ONE || a < end); ++q) {
        const int b = max(a, min(end, seq_begin(p, q + 1)));
        a = min(b, max(a, seq_begin(p, q)));
        if (!ONE && a >= b) continue;
        __syncthreads();   // the last sequence's sums have been read
        for (int e = threadIdx.x; e < p.E; e += blockDim.x) hist[e] = 0;
        if (threadIdx.x == 0) n_valid = 0;
        __syncthreads();
        float acc[N][VEC] = {};
        int n = 0;
        for (int t0 = a + warp; t0 < b; t0 += WARPS * 32) {
            // the valid ones of the warp's next 32 tokens (a flag each before its row would
            // be a second trip to memory for every token)
            const int tl = t0 + lane * WARPS;
            unsigned left = __ballot_sync(0xffffffffu, tl < b && (!p.valid || __ldg(p.valid + tl)));
            [[maybe_unused]] bool any_low = false;
            n += __popc(left);
            while (left) {
                Row<VEC, N> r[UNROLL];
                bool live[UNROLL];
                int id[UNROLL];
#pragma unroll
                for (int u = 0; u < UNROLL; ++u) {
                    live[u] = left != 0;
                    if (!live[u]) continue;
                    const int t = t0 + (__ffs(left) - 1) * WARPS;
                    left &= left - 1;
                    r[u].load(p.logits + (size_t)t * p.E, p.E);
                    id[u] = lane < p.k ? __ldg(p.ids + (size_t)t * p.k + lane) : 0;
                }
#pragma unroll
                for (int u = 0; u < UNROLL; ++u) {
                    if (!live[u]) continue;
                    float s[N][VEC], slope[N][VEC];
                    bool is_low;
                    const float inv = shares<SOFTMAX>(r[u], s, slope, is_low);
                    any_low |= is_low;
#pragma unroll
                    for (int i = 0; i < N; ++i)
#pragma unroll
                        for (int j = 0; j < VEC; ++j) acc[i][j] = fmaf(s[i][j], inv, acc[i][j]);
                    if (lane < p.k) {
                        if ((unsigned)id[u] < (unsigned)p.E) atomicAdd(hist + id[u], 1);
                        else record_status(p.status, MOE_ERR_INVALID_ARG);
                    }
                }
            }
            if constexpr (!SOFTMAX) {
                // the low ones, all of them looked at again (which leaves the loop above its
                // registers)
                left = any_low ? __ballot_sync(0xffffffffu, tl < b && (!p.valid || __ldg(p.valid + tl)))
                               : 0;
                for (; left; left &= left - 1) {
                    const int t = t0 + (__ffs(left) - 1) * WARPS;
                    Row<VEC, N> r;
                    r.load(p.logits + (size_t)t * p.E, p.E);
                    float s[N][VEC], slope[N][VEC];
                    bool is_low;
                    shares<false>(r, s, slope, is_low);
                    if (!is_low) continue;
                    const float inv = low_shares(r, s);
#pragma unroll
                    for (int i = 0; i < N; ++i)
#pragma unroll
                        for (int j = 0; j < VEC; ++j) acc[i][j] = fmaf(s[i][j], inv, acc[i][j]);
                }
            }
        }
        if (lane == 0 && n) atomicAdd(&n_valid, n);
        // (eight warps' worth of shared memory: further warps add to the first ones')
        for (int w0 = 0; w0 < WARPS; w0 += kWarps) {
            if (warp >= w0 && warp < w0 + kWarps) {
#pragma unroll
                for (int i = 0; i < N; ++i)
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        const int c = VEC * (lane + 32 * i) + j;
                        if (c >= p.E) continue;
                        float *dst = sm + (warp - w0) * p.E + c;
                        *dst = w0 ? *dst + acc[i][j] : acc[i][j];
                    }
            }
            __syncthreads();
        }
        bool counted = true;
        if constexpr (ONE) counted = !__syncthreads_or(descend);
        n = counted ? n_valid : 0;
        if constexpr (ONE) {
            float mine = 0.0f;
            for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
                float v = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) v += sm[w * p.E + e];
                mine += finish(p, q, e, n, counted ? hist[e] : 0, v);
            }
            mine = warp_sum(mine);
            if (lane == 0) term[warp] = mine;
            __syncthreads();
            if (threadIdx.x == 0) {
                float t = 0.0f;
                for (int w = 0; w < WARPS; ++w) t += term[w];
                p.seq_loss[q] = t;
                p.tokens[q] = n;
                loss += t;
            }
        } else {
            const size_t slot = (size_t)blockIdx.x + q;
            for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
                float s = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) s += sm[w * p.E + e];
                p.part_p[slot * p.E + e] = s;
                p.part_c[slot * p.E + e] = hist[e];
            }
            if (threadIdx.x == 0) p.part_n[slot] = n;
        }
        a = b;
    }
    if constexpr (ONE) {
        if (threadIdx.x == 0) p.loss[0] = p.alpha * loss / (float)p.n_seq;
    } else if (blockIdx.x == 0) {
        descend = __syncthreads_or(descend);
        if (threadIdx.x == 0) *p.descend = descend;
    }
}

// A cluster for each sequence, a CTA of it for 128 columns: 32 warps take the sequence's
// slots in turn, a lane four columns of them; then the warps' sums and the CTAs' terms are
// added up in order.  (A CTA for each sequence alone took 60 us of the 77 of 65536 x 384 in 16
// sequences.)
constexpr int kSeqWarps = 32, kSeqCols = 128;

__global__ void __launch_bounds__(32 * kSeqWarps) balance_seq_kernel(const BalanceParams p) {
    __shared__ float sum[kSeqWarps][kSeqCols];
    __shared__ int32_t cnt[kSeqWarps][kSeqCols];
    __shared__ float term[kSeqCols / 32];
    __shared__ float terms[8];   // of the first CTA: one for each CTA of the cluster
    __shared__ int n_all;
    const int q = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) n_all = 0;
    cluster_sync_all();   // the cluster's CTAs have begun: the first one's memory takes the terms
    wait_for_kernels_ahead();
    let_kernels_behind_begin();
    const int a = seq_begin(p, q), b = seq_begin(p, q + 1);
    const bool counted = *p.descend == 0;
    const int c0 = a / p.chunk, c1 = counted && b > a ? (b - 1) / p.chunk : c0 - 1;
    int n = 0;
    for (int c = c0 + threadIdx.x; c <= c1; c += blockDim.x) n += p.part_n[c + q];
    float s[4] = {};
    int32_t k[4] = {};
    const int col = blockIdx.x * kSeqCols + lane;
#pragma unroll 4
    for (int c = c0 + warp; c <= c1; c += kSeqWarps) {
        const size_t at = (size_t)(c + q) * p.E;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (col + 32 * j < p.E) {
                s[j] += p.part_p[at + col + 32 * j];
                k[j] += p.part_c[at + col + 32 * j];
            }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        sum[warp][lane + 32 * j] = s[j];
        cnt[warp][lane + 32 * j] = k[j];
    }
    if (n) atomicAdd(&n_all, n);
    __syncthreads();
    n = n_all;
    if (threadIdx.x < kSeqCols) {
        const int e = blockIdx.x * kSeqCols + threadIdx.x;
        float v = 0.0f;
        int32_t c = 0;
#pragma unroll
        for (int w = 0; w < kSeqWarps; ++w) {
            v += sum[w][threadIdx.x];
            c += cnt[w][threadIdx.x];
        }
        const float mine = warp_sum(e < p.E ? finish(p, q, e, n, c, v) : 0.0f);
        if (lane == 0) term[warp] = mine;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        float t = 0.0f;
        for (int i = 0; i < kSeqCols / 32; ++i) t += term[i];
        dsmem_st_u32(dsmem_map(&terms[blockIdx.x], 0), __float_as_uint(t));
    }
    cluster_sync_all();
    if (blockIdx.x != 0 || warp != 0) return;
    bool last = false;
    if (lane == 0) {
        float t = 0.0f;
        for (int i = 0; i < (int)gridDim.x; ++i) t += terms[i];
        p.seq_loss[q] = t;
        p.tokens[q] = n;
        __threadfence();
        last = atomicAdd(p.done, 1u) == (unsigned)p.n_seq - 1;
    }
    if (!__any_sync(0xffffffffu, last)) return;
    // the sequence that is finished last takes the mean of all, in their order: each lane's sum
    // compensated, as it can be long
    __threadfence();
    float sum_q = 0.0f, c = 0.0f;
    for (int i = lane; i < p.n_seq; i += 32) {
        const float v = __ldcg(p.seq_loss + i) - c, u = sum_q + v;
        c = (u - sum_q) - v;
        sum_q = u;
    }
    sum_q = warp_sum(sum_q);
    if (lane == 0) p.loss[0] = p.alpha * sum_q / (float)p.n_seq;
}

// A warp takes `chunk` consecutive tokens; a sequence's load stays in its registers.  (Narrow
// rows at 32 registers a thread: 30000 x 128 8.9 us, at the 39 that the compiler takes 10.9.)
template <bool SOFTMAX, int VEC, int N>
__global__ void __launch_bounds__(32 * kWarps, N * VEC <= 4 ? 8 : 0)
    balance_bwd_kernel(const BalanceParams p) {
    wait_for_kernels_ahead();
    let_kernels_behind_begin();
    const int lane = threadIdx.x & 31;
    const long long first =
        ((long long)blockIdx.x * kWarps + (threadIdx.x >> 5)) * p.chunk;
    if (first >= p.T) return;
    const int a = (int)first, b = (int)min((long long)p.T, first + p.chunk);
    int q = first_seq(p, a);
    int begin = q < p.n_seq ? seq_begin(p, q) : p.T;
    int end = q < p.n_seq ? seq_begin(p, q + 1) : p.T;
    const float g = (p.dloss ? __ldg(p.dloss) : 1.0f) * p.alpha;
    float f[N][VEC], coef = 0.0f;
    bool loaded = false;
    for (int t = a; t < b; ++t) {
        while (q < p.n_seq && t >= end) {
            ++q;
            loaded = false;
            begin = q < p.n_seq ? seq_begin(p, q) : p.T;
            end = q < p.n_seq ? seq_begin(p, q + 1) : p.T;
        }
        float *dst = p.dlogits + (size_t)t * p.E;
        const bool live = q < p.n_seq && t >= begin && (!p.valid || __ldg(p.valid + t));
        float out[N][VEC] = {};
        if (live) {
            if (!loaded) {
                Row<VEC, N> l;
                l.load(p.load + (size_t)q * p.E, p.E);
#pragma unroll
                for (int i = 0; i < N; ++i)
#pragma unroll
                    for (int j = 0; j < VEC; ++j)
                        f[i][j] = VEC * (lane + 32 * i) + j < p.E ? l.z[i][j] : 0.0f;
                coef = g / ((float)p.n_seq * (float)max(1, __ldg(p.tokens + q)));
                loaded = true;
            }
            Row<VEC, N> r;
            r.load(p.logits + (size_t)t * p.E, p.E);
            float s[N][VEC], slope[N][VEC];
            bool low;
            float inv = shares<SOFTMAX>(r, s, slope, low);
            if (low) {
                r.load(p.logits + (size_t)t * p.E, p.E);   // (again, for fewer registers)
                inv = low_shares(r, s);
            }
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int j = 0; j < VEC; ++j) s[i][j] *= inv;
            float dot = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int j = 0; j < VEC; ++j) dot = fmaf(f[i][j], s[i][j], dot);
            dot = warp_sum(dot);
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int j = 0; j < VEC; ++j)
                    out[i][j] = coef * (s[i][j] * (f[i][j] - dot) * slope[i][j]);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = VEC * (lane + 32 * i);
            if (c >= p.E) continue;
            if constexpr (VEC == 4)
                *reinterpret_cast<float4 *>(dst + c) =
                    make_float4(out[i][0], out[i][1], out[i][2], out[i][3]);
            else
                dst[c] = out[i][0];
        }
    }
}

// Tokens of a chunk: four CTAs an SM, at least a token for each warp.
int part_chunk(int T) {
    const int c = (int)(((long long)T + 4LL * num_sms() - 1) / (4LL * num_sms()));
    return c < 2 * kWarps ? 2 * kWarps : c;
}

BalanceParams params(const moe_balance_args *a) {
    BalanceParams p;
    std::memset(&p, 0, sizeof p);
    p.T = a->T;
    p.E = a->E;
    p.k = a->k;
    p.n_seq = a->n_seq;
    p.alpha = a->alpha;
    p.logits = a->logits;
    p.ids = a->ids;
    p.seq_offsets = a->seq_offsets;
    p.valid = a->valid;
    p.counts = a->counts;
    p.tokens = a->tokens;
    p.load = a->load;
    p.seq_loss = a->seq_loss;
    p.loss = a->loss;
    p.dloss = a->dloss;
    p.dlogits = a->dlogits;
    return p;
}

// Instances by the columns of a lane: four at a time where rows are whole 16 bytes.
template <template <bool, int, int> class L>
moe_status by_columns(const moe_balance_args *a, const BalanceParams &p, cudaStream_t st) {
    const bool soft = a->score == MOE_SCORE_SOFTMAX;
    const int E = a->E;
#define MOE_BALANCE(V, N) return soft ? L<true, V, N>::go(p, st) : L<false, V, N>::go(p, st)
    if (E % 4 == 0) {
        if (E <= 128) MOE_BALANCE(4, 1);
        if (E <= 256) MOE_BALANCE(4, 2);
        if (E <= 384) MOE_BALANCE(4, 3);
        if (E <= 512) MOE_BALANCE(4, 4);
        MOE_BALANCE(4, 8);
    }
    if (E <= 32) MOE_BALANCE(1, 1);
    if (E <= 128) MOE_BALANCE(1, 4);
    if (E <= 256) MOE_BALANCE(1, 8);
    if (E <= 512) MOE_BALANCE(1, 16);
    MOE_BALANCE(1, 32);
#undef MOE_BALANCE
}

template <bool S, int V, int N>
struct PartLaunch {
    static moe_status go(const BalanceParams &p, cudaStream_t st) {
        const int smem = (kWarps + 1) * p.E * 4;
        if (p.one) return launch_early(balance_part_kernel<S, V, N, true>, dim3(1), 32 * kOneWarps,
                                       smem, st, p);
        return launch_early(balance_part_kernel<S, V, N, false>, dim3(p.n_chunks), 32 * kWarps,
                            smem, st, p);
    }
};
template <bool S, int V, int N>
struct BwdLaunch {
    static moe_status go(const BalanceParams &p, cudaStream_t st) {
        const long long ctas = ((long long)p.T + (long long)p.chunk * kWarps - 1) /
                               ((long long)p.chunk * kWarps);
        return launch_early(balance_bwd_kernel<S, V, N>, dim3((unsigned)ctas), 32 * kWarps, 0, st,
                            p);
    }
};

}  // namespace

size_t balance_workspace_bytes(int T, int E, int n_seq) {
    const int C = part_chunk(T);
    const size_t slots = (size_t)((T + C - 1) / C) + n_seq;
    return slots * E * 8 + slots * 4 + 8;
}

moe_status launch_balance(const moe_balance_args *a, cudaStream_t st) {
    BalanceParams p = params(a);
    p.status = device_status_ptr();
    if (!p.status) return MOE_ERR_CUDA;
    p.chunk = part_chunk(a->T);
    // Few tokens and sequences: one launch of one CTA instead of two of many.  A token takes the
    // one CTA as long as E + 300 numbers, a sequence as long as 28 tokens.  Measured, one sequence,
    // us in one launch / in two: 64 tokens of 16 experts 3.7 / 7.3, 128 tokens of 384 7.7 / 7.9,
    // 64 of 1024 8.7 / 8.6, 128 of 1024 13.4 / 8.6; four: 128 of 16 8.7 / 8.7, 32 of 384 9.3 / 9.8,
    // 64 of 384 10.8 / 10.6, 8 of 1024 12.7 / 9.4.
    p.one = a->T <= kOneTokens && (a->T + 28LL * (a->n_seq - 1)) * (a->E + 300) <= 88000;
    if (p.one) {
        p.chunk = kOneTokens;
        return by_columns<PartLaunch>(a, p, st);
    }
    p.n_chunks = (a->T + p.chunk - 1) / p.chunk;
    const size_t slots = (size_t)p.n_chunks + a->n_seq;
    p.part_p = static_cast<float *>(a->ws);
    p.part_c = reinterpret_cast<int32_t *>(p.part_p + slots * a->E);
    p.part_n = p.part_c + slots * a->E;
    p.done = reinterpret_cast<unsigned *>(p.part_n + slots);
    p.descend = p.done + 1;
    if (p.n_chunks == 0) p.n_chunks = 1;   // (no token: it sets `done` and `descend`)
    const moe_status s = by_columns<PartLaunch>(a, p, st);
    if (s != MOE_OK) return s;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (a->E + kSeqCols - 1) / kSeqCols;   // at most 8
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(at[1].val.clusterDim.x, a->n_seq);
    cfg.blockDim = dim3(32 * kSeqWarps);
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, balance_seq_kernel, p) != cudaSuccess) return MOE_ERR_CUDA;
    return cuda_status(cudaGetLastError());
}

moe_status launch_balance_bwd(const moe_balance_args *a, cudaStream_t st) {
    BalanceParams p = params(a);
    const long long warps = (long long)num_sms() * 4 * kWarps;
    p.chunk = (int)(((long long)a->T + warps - 1) / warps);
    return by_columns<BwdLaunch>(a, p, st);
}

}  // namespace moe
