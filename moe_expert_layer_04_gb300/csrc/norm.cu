// norm.cu -- the root-mean-square norm ahead of the layer, with the residual's
// addition before it and the rows' quantisation behind it, and its backward.
//
//   v    = bf16(x + residual)                    (x alone without a residual)
//   rstd = 1 / sqrt( mean_i v_i^2 + eps )
//   u    = v rstd w                              fp32
//   y    = bf16(u),  codes and scales of u in FP8 (1 x 128), MXFP8 or MXFP4
//
//   vh = v rstd,  a = w dy
//   dx = bf16( d_residual + rstd (a - vh mean_i(a_i vh_i)) )   (for x and the residual)
//   dw = sum over the rows of dy vh
//
// (The rows are those of the MoE layer: "HyperParallel加速DeepSeek-V4.1多模态1M长序列
// 训练" §2.3, MegaMHC's residual update and norm ahead of it.)  Sums are fp32 in a
// fixed order.  Both directions are bound by HBM: each row is held in registers
// between its sum and its use, so that every value crosses once.
#include <cstring>

#include "fp8_common.cuh"
#include "mx_common.cuh"

namespace moe {
namespace {

__device__ __forceinline__ void unpack8(const uint4 v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

// Sum over the `warps` warps that share a row (all of the CTA's rows at once); `part`
// holds a float for each warp of the CTA.
__device__ __forceinline__ float row_sum(float s, int warps, float *part) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (warps == 1) return s;
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) part[warp] = s;
    __syncthreads();
    const int first = warp / warps * warps;
    s = 0.0f;
    for (int i = 0; i < warps; ++i) s += part[first + i];
    return s;
}

struct NormRows {
    int T, d8, threads;   // threads of a row, a multiple of 32
    float eps, inv_d;
    int format;
    int *status;
    const uint4 *x, *residual;
    const float *weight;
    uint4 *residual_out, *y;
    float *rstd;
    uint8_t *q;
    void *scales;
    int scale_pitch;      // scales of a row
};

// The largest of |u| as bits, over the `lanes` lanes of a block.  NAN_COUNTS: a NaN is larger than
// every number (0x7FFFFFFF), else it is left out.  (Three inputs an instruction: as integer
// maxima of masked bits these were a seventh of the norm's instructions.)
template <bool NAN_COUNTS>
__device__ __forceinline__ uint32_t block_max(const float (&u)[8], int lanes) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        if constexpr (NAN_COUNTS)
            asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(u[i]), "f"(u[i + 1]));
        else
            asm("max.abs.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(u[i]), "f"(u[i + 1]));
    }
    uint32_t b = __float_as_uint(m);
#pragma unroll
    for (int o = 1; o < lanes; o <<= 1) b = max(b, __shfl_xor_sync(0xffffffffu, b, o));
    return b;
}

// u times r in E4M3.
__device__ __forceinline__ uint2 e4m3_of(const float (&u)[8], float r) {
    return make_uint2(e4m3x4(u[0] * r, u[1] * r, u[2] * r, u[3] * r),
                      e4m3x4(u[4] * r, u[5] * r, u[6] * r, u[7] * r));
}

// Codes and scales of the eight values u, elements 8 c .. of row `row`; called by
// whole warps, whose lanes hold consecutive vectors (a block of 128 is sixteen lanes,
// one of 32 four).
template <int FORMAT>
__device__ __forceinline__ void store_codes(const NormRows &p, size_t row, int c, bool live,
                                            const float (&u)[8]) {
    if constexpr (FORMAT == MOE_ROWS_FP8) {
        const Fp8Scale f = fp8_scale(block_max<true>(u, 16));
        if (!live) return;
        *reinterpret_cast<uint2 *>(p.q + (row * p.d8 + c) * 8) = e4m3_of(u, f.r);
        if ((c & 15) == 0)
            static_cast<float *>(p.scales)[row * p.scale_pitch + (c >> 4)] = f.s;
    } else if constexpr (FORMAT == MOE_ROWS_MXFP8) {
        const uint32_t code = mx_scale_code(__uint_as_float(block_max<false>(u, 4)));
        if (!live) return;
        *reinterpret_cast<uint2 *>(p.q + (row * p.d8 + c) * 8) = e4m3_of(u, mx_inv_scale(code));
        if ((c & 3) == 0)
            static_cast<uint8_t *>(p.scales)[row * p.scale_pitch + (c >> 2)] = (uint8_t)code;
    } else {
        const uint32_t code = mx4_scale_code(block_max<true>(u, 4));
        if (!live) return;
        *reinterpret_cast<uint32_t *>(p.q + (row * p.d8 + c) * 4) = e2m1x8(u, mx4_inv_scale(code));
        if ((c & 3) == 0)
            static_cast<uint8_t *>(p.scales)[row * p.scale_pitch + (c >> 2)] = (uint8_t)code;
    }
}

// Few rows, or long ones: a CTA for each (or for a few short ones).  A row's `threads`
// threads hold V vectors of eight elements each.
template <int V>
__global__ void __launch_bounds__(1024) rmsnorm_kernel(const NormRows p) {
    __shared__ float part[32];
    wait_for_kernels_ahead();
    let_kernels_behind_begin();
    const int in_row = threadIdx.x % p.threads;
    const long long row = (long long)blockIdx.x * (blockDim.x / p.threads) +
                          threadIdx.x / p.threads;
    const bool has = row < p.T;
    uint4 v[V];
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int c = in_row + j * p.threads;
        v[j] = make_uint4(0, 0, 0, 0);
        if (has && c < p.d8) {
            v[j] = __ldg(p.x + row * p.d8 + c);
            if (p.residual) {
                const uint4 b = __ldg(p.residual + row * p.d8 + c);
                float f[8], g[8];
                unpack8(v[j], f);
                unpack8(b, g);
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] += g[i];
                v[j] = pack8(f);
                p.residual_out[row * p.d8 + c] = v[j];
            }
        }
        float f[8];
        unpack8(v[j], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
    }
    ss = row_sum(ss, p.threads >> 5, part);
    const float r = 1.0f / sqrtf(fmaf(ss, p.inv_d, p.eps));
    if (has && in_row == 0 && p.rstd) p.rstd[row] = r;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int c = in_row + j * p.threads;
        const bool live = has && c < p.d8;
        float f[8];
        unpack8(v[j], f);
        if (live) {
            const float4 w0 = __ldg(reinterpret_cast<const float4 *>(p.weight) + 2 * c);
            const float4 w1 = __ldg(reinterpret_cast<const float4 *>(p.weight) + 2 * c + 1);
            const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = f[i] * r * w[i];
            if (p.y) p.y[row * p.d8 + c] = pack8(f);
        }
        if (p.format == MOE_ROWS_FP8) store_codes<MOE_ROWS_FP8>(p, (size_t)row, c, live, f);
        else if (p.format == MOE_ROWS_MXFP8) store_codes<MOE_ROWS_MXFP8>(p, (size_t)row, c, live, f);
        else if (p.format == MOE_ROWS_MXFP4) store_codes<MOE_ROWS_MXFP4>(p, (size_t)row, c, live, f);
    }
}

// ------------------------------------------------------- many rows, in a ring
//
// A CTA takes every gridDim.x-th group of rows (one row, or as many short ones as its threads
// hold, two vectors each) and has the next kRing groups on their way into shared memory by
// bulk copies, so that the loads do not stop while a row is summed and written, and the
// weight stays in registers.  The barrier of a row's sum is also what frees its place in the
// ring.  Measured, of the copy bandwidth: backward of 16384 x 4096 83 us, 96 % (103 with a
// row's loads into registers), of 4096 x 512 7.2 us (23 with one row a CTA); forward of
// 4096 x 4096 with the residual 23 us, 86 %, with FP8 rows 27.7 us, 81 %: half of what the codes
// add is their bytes, half the instructions that make them.  The forward takes three CTAs an
// SM and four rows ahead (23.2 and 28.3 us; four CTAs and two ahead 23.3 and 28.7, four and
// three 24.0 and 29.1, three and two 24.0 and 30.0).
constexpr int kRing = 4;
constexpr int kFwdCtas = 3, kBwdCtas = 2;   // to an SM
constexpr int kRingThreads = 256;
// The forward's ring takes rows that nearly fill its threads' two vectors, where there are more
// of them than the SMs hold CTAs of the other kernel at once, and not so many that its
// waves' ends no longer count.
constexpr int kFwdVecs = 7 * kRingThreads / 4, kFwdMore = 6, kFwdMost = 64;   // rows to an SM

struct Ring {
    uint64_t *full;      // [kRing]
    volatile int *abort;
    int *status;
    int arrays;          // rows of so many arrays make a group
    const uint4 *src[3];
    uint4 *smem;
    int group;           // vectors of a group of one array
};

__device__ __forceinline__ void ring_load(const Ring &r, int slot, long long row, int rows, int d8) {
    const uint32_t bytes = (uint32_t)rows * d8 * 16;
    mbar_arrive_expect_tx(&r.full[slot], r.arrays * bytes);
    for (int i = 0; i < r.arrays; ++i)
        bulk_load(r.smem + (slot * r.arrays + i) * r.group, r.src[i] + row * d8, bytes,
                  &r.full[slot]);
}

// The group in `slot` has come: the same answer for the whole CTA.  Where the wait ran out,
// the copies still in flight (of the groups from row `base` on) are waited for as well.
__device__ __forceinline__ bool ring_wait(const Ring &r, int slot, uint32_t parity, long long base,
                                          long long step, long long T) {
    const WaitCtl wc{r.abort, r.status, kWaitLimitCycles};
    if (__syncthreads_and(mbar_wait(&r.full[slot], parity, wc))) return true;
    if (threadIdx.x == 0)
        for (int i = 0; i < kRing; ++i)
            if (base + i * step < T)
                mbar_wait_teardown(&r.full[(slot + i) % kRing],
                                   slot + i < kRing ? parity : parity ^ 1u, kWaitLimitCycles);
    __syncthreads();
    return false;
}

// Pairs of fp32 in one instruction: the forward of the ring is bound by its instructions as
// much as by HBM (4096 x 4096 with FP8 rows took 28.8 us one element at a time).
__device__ __forceinline__ uint64_t pair_of(uint32_t bf16x2) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(bf16x2 << 16), "r"(bf16x2 & 0xFFFF0000u));
    return v;
}
__device__ __forceinline__ uint64_t pair_f(float lo, float hi) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
    return v;
}
__device__ __forceinline__ float2 two(uint64_t v) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint32_t bf16_of(uint64_t v) {
    const float2 f = two(v);
    return pack_bf16x2(f.x, f.y);
}

template <int V, int FORMAT>
__global__ void __launch_bounds__(kRingThreads, kFwdCtas) rmsnorm_ring_kernel(const NormRows p) {
    extern __shared__ uint4 ring_smem[];
    __shared__ uint64_t full[kRing];
    __shared__ int abort_s;
    __shared__ float part[2][8];
    const Ring r{full, &abort_s, p.status, p.residual ? 2 : 1, {p.x, p.residual, nullptr}, ring_smem,
                 p.d8};
    if (threadIdx.x == 0) {
        for (int i = 0; i < kRing; ++i) mbar_init(&full[i], 1);
        abort_s = 0;
        fence_barrier_init();
    }
    __syncthreads();
    wait_for_kernels_ahead();
    let_kernels_behind_begin();
    const long long step = gridDim.x;
    auto load = [&](int slot, long long row) {
        if (row < p.T) ring_load(r, slot, row, 1, p.d8);
    };
    if (threadIdx.x == 0)
        for (int i = 0; i < kRing; ++i) load(i, blockIdx.x + i * step);
    uint64_t w[V][4];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int c = threadIdx.x + j * blockDim.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = c < p.d8 ? __ldg(reinterpret_cast<const float2 *>(p.weight) + 4 * c + i)
                                      : make_float2(0.0f, 0.0f);
            w[j][i] = pair_f(f.x, f.y);
        }
    }
    int slot = 0, turn = 0;
    uint32_t ph = 0;
    for (long long row = blockIdx.x; row < p.T; row += step, turn ^= 1) {
        if (!ring_wait(r, slot, ph, row, step, p.T)) return;
        const uint4 *at = ring_smem + slot * r.arrays * r.group;
        uint64_t f[V][4], ss = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = threadIdx.x + j * blockDim.x;
            const bool live = c < p.d8;
            uint4 v = live ? at[c] : make_uint4(0, 0, 0, 0);
            if (p.residual && live) {
                const uint4 b = at[r.group + c];
                v.x = bf16_of(add2(pair_of(v.x), pair_of(b.x)));
                v.y = bf16_of(add2(pair_of(v.y), pair_of(b.y)));
                v.z = bf16_of(add2(pair_of(v.z), pair_of(b.z)));
                v.w = bf16_of(add2(pair_of(v.w), pair_of(b.w)));
                p.residual_out[row * p.d8 + c] = v;
            }
            f[j][0] = pair_of(v.x);
            f[j][1] = pair_of(v.y);
            f[j][2] = pair_of(v.z);
            f[j][3] = pair_of(v.w);
#pragma unroll
            for (int i = 0; i < 4; ++i) ss = fma2(f[j][i], f[j][i], ss);
        }
        const float2 s2 = two(ss);
        const float sum = row_sum(s2.x + s2.y, blockDim.x >> 5, part[turn]);
        if (threadIdx.x == 0) load(slot, row + kRing * step);
        if (++slot == kRing) { slot = 0; ph ^= 1u; }
        const float rs = 1.0f / sqrtf(fmaf(sum, p.inv_d, p.eps));
        if (threadIdx.x == 0 && p.rstd) p.rstd[row] = rs;
        const uint64_t rs2 = pair_f(rs, rs);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = threadIdx.x + j * blockDim.x;
            const bool live = c < p.d8;
            uint64_t u2[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) u2[i] = mul2(mul2(f[j][i], rs2), w[j][i]);
            if (live && p.y)
                p.y[row * p.d8 + c] =
                    make_uint4(bf16_of(u2[0]), bf16_of(u2[1]), bf16_of(u2[2]), bf16_of(u2[3]));
            if constexpr (FORMAT != MOE_ROWS_NONE) {
                float u[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 t = two(u2[i]);
                    u[2 * i] = t.x;
                    u[2 * i + 1] = t.y;
                }
                store_codes<FORMAT>(p, (size_t)row, c, live, u);
            }
        }
    }
}

__device__ __forceinline__ void add_to(float4 &s, const float4 v) {
    s.x += v.x;
    s.y += v.y;
    s.z += v.z;
    s.w += v.w;
}

struct NormBwd {
    int T, d8, threads;
    int *status;
    float inv_d;
    const uint4 *x, *dy, *d_residual;
    const float *weight, *rstd;
    uint4 *dx;
    float *part;   // [CTAs, d]: each one's sums
};

template <int V>
__global__ void __launch_bounds__(kRingThreads, kBwdCtas) rmsnorm_bwd_ring_kernel(const NormBwd p) {
    extern __shared__ uint4 ring_smem[];
    __shared__ uint64_t full[kRing];
    __shared__ int abort_s;
    __shared__ float part[2][8];
    const int per = blockDim.x / p.threads;
    const int in_row = threadIdx.x % p.threads, my = threadIdx.x / p.threads;
    const Ring r{full, &abort_s, p.status, p.d_residual ? 3 : 2, {p.x, p.dy, p.d_residual}, ring_smem,
                 per * p.d8};
    if (threadIdx.x == 0) {
        for (int i = 0; i < kRing; ++i) mbar_init(&full[i], 1);
        abort_s = 0;
        fence_barrier_init();
    }
    __syncthreads();
    wait_for_kernels_ahead();
    let_kernels_behind_begin();
    const long long first = (long long)blockIdx.x * per, step = (long long)gridDim.x * per;
    auto load = [&](int slot, long long base) {
        if (base < p.T) ring_load(r, slot, base, (int)min((long long)per, p.T - base), p.d8);
    };
    if (threadIdx.x == 0)
        for (int i = 0; i < kRing; ++i) load(i, first + i * step);
    float w[V][8], dw[V][8];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int c = in_row + j * p.threads;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            w[j][i] = c < p.d8 ? __ldg(p.weight + 8 * c + i) : 0.0f;
            dw[j][i] = 0.0f;
        }
    }
    int slot = 0, turn = 0;
    uint32_t ph = 0;
    for (long long base = first; base < p.T; base += step, turn ^= 1) {
        const long long row = base + my;
        const bool has = row < p.T;
        const float rs = has ? __ldg(p.rstd + row) : 0.0f;
        if (!ring_wait(r, slot, ph, base, step, p.T)) return;
        const uint4 *at = ring_smem + slot * r.arrays * r.group + my * p.d8;
        uint4 v[V], dr[V];
        float a[V][8];
        float dot = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = in_row + j * p.threads;
            const bool live = has && c < p.d8;
            v[j] = dr[j] = make_uint4(0, 0, 0, 0);
            uint4 dy = make_uint4(0, 0, 0, 0);
            if (live) {
                v[j] = at[c];
                dy = at[r.group + c];
                if (p.d_residual) dr[j] = at[2 * r.group + c];
            }
            float f[8], g[8];
            unpack8(v[j], f);
            unpack8(dy, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float vh = f[i] * rs;
                dw[j][i] = fmaf(g[i], vh, dw[j][i]);
                a[j][i] = g[i] * w[j][i];
                dot = fmaf(a[j][i], vh, dot);
            }
        }
        const float m = row_sum(dot, p.threads >> 5, part[turn]) * p.inv_d;
        if (p.threads == 32) __syncthreads();
        if (threadIdx.x == 0) load(slot, base + kRing * step);
        if (++slot == kRing) { slot = 0; ph ^= 1u; }
        if (!has) continue;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = in_row + j * p.threads;
            if (c >= p.d8) continue;
            float f[8], g[8];
            unpack8(v[j], f);
            unpack8(dr[j], g);
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] += rs * (a[j][i] - f[i] * rs * m);
            p.dx[row * p.d8 + c] = pack8(g);
        }
    }
    // the rows' sums of this CTA, added up in order
    float4 *sum = reinterpret_cast<float4 *>(ring_smem);
    const int d4 = 2 * p.d8;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int c = in_row + j * p.threads;
        if (c >= p.d8) continue;
        sum[my * d4 + 2 * c] = make_float4(dw[j][0], dw[j][1], dw[j][2], dw[j][3]);
        sum[my * d4 + 2 * c + 1] = make_float4(dw[j][4], dw[j][5], dw[j][6], dw[j][7]);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < d4; c += blockDim.x) {
        float4 s = sum[c];
        for (int i = 1; i < per; ++i) add_to(s, sum[i * d4 + c]);
        reinterpret_cast<float4 *>(p.part)[(size_t)blockIdx.x * d4 + c] = s;
    }
}

// Long rows: a cluster of CL CTAs takes each gridDim.x / CL-th row, a CTA up to 1024 vectors of
// it, two a thread.  The next row's loads are issued before this row's sum, which goes
// through the CTAs' shared memory.  Measured, of the copy bandwidth: 4096 x 7168 43 us, 80 %, 2048 x
// 16384 62 us, 64 %, 1024 x 32768 68 us, 58 % (115 and 476 us with a CTA a row, whose four or
// eight vectors a thread spill).
template <int CL>
__global__ void __launch_bounds__(512) rmsnorm_bwd_kernel(const NormBwd p) {
    constexpr int V = 2;
    __shared__ float part[2][16];
    __shared__ float sums[2][CL];   // of the cluster's CTAs
    if constexpr (CL > 1) cluster_sync_all();   // they have begun
    wait_for_kernels_ahead();
    let_kernels_behind_begin();
    const int slots = gridDim.x / CL, slot = blockIdx.x / CL;
    const int rank = CL > 1 ? (int)cluster_ctarank() : 0, slice = (p.d8 + CL - 1) / CL;
    const int c0 = rank * slice, c1 = min(p.d8, c0 + slice);
    float w[V][8], dw[V][8];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int c = c0 + threadIdx.x + j * blockDim.x;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            w[j][i] = c < c1 ? __ldg(p.weight + 8 * c + i) : 0.0f;
            dw[j][i] = 0.0f;
        }
    }
    const uint4 zero = make_uint4(0, 0, 0, 0);
    uint4 nv[V], nd[V], nr[V];
    float nrstd = 0.0f;
    auto load = [&](long long row) {
        const bool has = row < p.T;
        nrstd = has ? __ldg(p.rstd + row) : 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = c0 + threadIdx.x + j * blockDim.x;
            const bool live = has && c < c1;
            nv[j] = live ? __ldg(p.x + row * p.d8 + c) : zero;
            nd[j] = live ? __ldg(p.dy + row * p.d8 + c) : zero;
            nr[j] = live && p.d_residual ? __ldg(p.d_residual + row * p.d8 + c) : zero;
        }
    };
    load(slot);
    int turn = 0;
    for (long long row = slot; row < p.T; row += slots, turn ^= 1) {
        const float r = nrstd;
        uint4 v[V], dr[V];
        float a[V][8];
        float dot = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            v[j] = nv[j];
            dr[j] = nr[j];
            float f[8], g[8];
            unpack8(nv[j], f);
            unpack8(nd[j], g);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float vh = f[i] * r;
                dw[j][i] = fmaf(g[i], vh, dw[j][i]);
                a[j][i] = g[i] * w[j][i];
                dot = fmaf(a[j][i], vh, dot);
            }
        }
        load(row + slots);
        float m = row_sum(dot, blockDim.x >> 5, part[turn]);
        if constexpr (CL > 1) {
            if (threadIdx.x < CL)
                dsmem_st_u32(dsmem_map(&sums[turn][rank], threadIdx.x), __float_as_uint(m));
            cluster_sync_all();
            m = 0.0f;
#pragma unroll
            for (int i = 0; i < CL; ++i) m += sums[turn][i];
        }
        m *= p.inv_d;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = c0 + threadIdx.x + j * blockDim.x;
            if (c >= c1) continue;
            float f[8], g[8];
            unpack8(v[j], f);
            unpack8(dr[j], g);
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] += r * (a[j][i] - f[i] * r * m);
            p.dx[row * p.d8 + c] = pack8(g);
        }
    }
    float4 *dst = reinterpret_cast<float4 *>(p.part + (size_t)slot * p.d8 * 8);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int c = c0 + threadIdx.x + j * blockDim.x;
        if (c >= c1) continue;
        dst[2 * c] = make_float4(dw[j][0], dw[j][1], dw[j][2], dw[j][3]);
        dst[2 * c + 1] = make_float4(dw[j][4], dw[j][5], dw[j][6], dw[j][7]);
    }
}

// dw = the sum of the CTAs' rows: a CTA takes 128 columns, its 32 warps every 32nd row, added
// up in order.
constexpr int kDwWarps = 32;
__global__ void __launch_bounds__(32 * kDwWarps)
    rmsnorm_dw_kernel(const float4 *__restrict__ part, int slots, int d4, float4 *__restrict__ dw) {
    __shared__ float4 sums[kDwWarps][32];
    wait_for_kernels_ahead();
    let_kernels_behind_begin();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (c < d4) {
#pragma unroll 4
        for (int i = warp; i < slots; i += kDwWarps) add_to(s, part[(size_t)i * d4 + c]);
    }
    sums[warp][lane] = s;
    __syncthreads();
    if (warp != 0 || c >= d4) return;
#pragma unroll
    for (int i = 1; i < kDwWarps; ++i) add_to(s, sums[i][lane]);
    dw[c] = s;
}

// Threads of a row of d8 vectors, V of them each, and rows of a CTA: V a power of two, no
// more than `most` threads a row, CTAs of 128 at least.
struct RowShape {
    int V, threads, rows;
};
RowShape row_shape(int d8, int most) {
    RowShape s;
    s.V = 1;
    while (d8 > s.V * most) s.V *= 2;
    s.threads = ((d8 + s.V - 1) / s.V + 31) / 32 * 32;
    s.rows = s.threads < 128 ? 128 / s.threads : 1;
    return s;
}

// Rows that the ring kernels take: V <= 2 vectors for each of 256 threads.
constexpr int kRingVecs = 2 * kRingThreads;
RowShape ring_shape(int d8) {
    RowShape s;
    s.V = 2;
    s.threads = (d8 + 63) / 64 * 32;
    s.rows = kRingThreads / s.threads;
    return s;
}

// CTAs that share a row of the backward.
int wide_cluster(int d8) { return d8 <= 1024 ? 1 : d8 <= 2048 ? 2 : 4; }

// Rows of partial sums of the backward, one for each CTA or cluster: as many as the SMs take at
// once, no more than there are groups of rows.
int bwd_parts(int T, int d8) {
    const bool ring = d8 <= kRingVecs;
    const int rows = ring ? ring_shape(d8).rows : 1;
    const long long want = ((long long)T + rows - 1) / rows;
    const long long most = ring ? (long long)num_sms() * kBwdCtas : num_sms() / wide_cluster(d8);
    return (int)(want < most ? want : most);
}

// The clusters that the GPU holds at once, where they are fewer than `parts`, become it.
template <int CL>
moe_status launch_wide(int &parts, const NormBwd &p, cudaStream_t st) {
    static int resident[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
    if (dev < 0 || dev >= 64) return MOE_ERR_UNSUPPORTED;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = CL;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(num_sms() / CL * CL);
    cfg.blockDim = dim3(512);
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    if (!resident[dev]) {
        int n = num_sms();
        if (CL > 1 && (cudaOccupancyMaxActiveClusters(&n, rmsnorm_bwd_kernel<CL>, &cfg) !=
                           cudaSuccess ||
                       n < 1))
            return MOE_ERR_CUDA;
        resident[dev] = n;
    }
    if (parts > resident[dev]) parts = resident[dev];
    const int slice = (p.d8 + CL - 1) / CL;
    cfg.gridDim = dim3(parts * CL);
    cfg.blockDim = dim3((slice + 63) / 64 * 32);
    if (cudaLaunchKernelEx(&cfg, rmsnorm_bwd_kernel<CL>, p) != cudaSuccess) return MOE_ERR_CUDA;
    return cuda_status(cudaGetLastError());
}

template <auto KERN, typename P>
moe_status launch_ring(int ctas, const RowShape &s, int arrays, int d, cudaStream_t st, const P &p) {
    static bool attr_set[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
    if (dev < 0 || dev >= 64) return MOE_ERR_UNSUPPORTED;
    if (!attr_set[dev]) {
        if (cudaFuncSetAttribute(KERN, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kRing * 3 * kRingVecs * 16) != cudaSuccess)
            return MOE_ERR_CUDA;
        attr_set[dev] = true;
    }
    return launch_early(KERN, dim3(ctas), s.threads * s.rows, kRing * arrays * s.rows * d * 2, st, p);
}

}  // namespace

moe_status launch_rmsnorm(const moe_norm_args *a, cudaStream_t st) {
    const int d8 = a->d / 8;
    // Rows of 3584 to 4096: with many of them a thread holds two vectors, so that more rows are
    // on their way in an SM (700 rows of 4096 4.1 us against 5.3, with FP8 rows 16384
    // 102 us against 106), with few of them one (300 rows 2.9 us against 3.1; other
    // widths: 2000 rows of 2304 7.9 us against 8.5).
    const bool wide = d8 >= kFwdVecs && d8 <= kRingVecs;
    // Longer rows likewise, four vectors a thread where that leaves 192 threads or more (2048
    // rows of 8192 28.1 us, two 30.3, one 32.0; of 16384 53.0 and, two, 68.0; 4096 rows of 7168
    // 47.1, 52.7 and 52.6, but of 5120 33.8, 32.2 and 33.6).
    const bool many = a->T > 2 * num_sms();
    const int most = !many ? 1024
                     : wide || (d8 > 3 * kRingThreads && d8 <= 4 * kRingThreads) ? kRingThreads
                     : d8 > kRingVecs && d8 <= 4 * 512 ? 512
                                                       : 1024;
    const RowShape s = row_shape(d8, most);
    NormRows p;
    std::memset(&p, 0, sizeof p);
    p.T = a->T;
    p.d8 = a->d / 8;
    p.threads = s.threads;
    p.eps = a->eps;
    p.inv_d = 1.0f / (float)a->d;
    p.format = a->format;
    p.x = reinterpret_cast<const uint4 *>(a->x);
    p.residual = reinterpret_cast<const uint4 *>(a->residual);
    p.weight = a->weight;
    p.residual_out = reinterpret_cast<uint4 *>(a->residual_out);
    p.y = reinterpret_cast<uint4 *>(a->y);
    p.rstd = a->rstd;
    p.q = a->q;
    p.scales = a->scales;
    p.scale_pitch = a->format == MOE_ROWS_FP8 ? fp8_blocks(a->d) : mx_sf_pitch(a->d);
    p.status = device_status_ptr();
    if (!p.status) return MOE_ERR_CUDA;
    // The ring: 2000 rows of 4096 12.2 us there, 14.4 in the other kernel (with FP8 rows 14.9
    // and 16.5), 4096 rows 23.3 and 25.4 (28.3 and 29.3), 16384 rows 90 and 88 (111 and 102);
    // narrower rows leave threads idle: 2000 rows of 1536 5.5 and 5.0.
    if (wide && a->T > kFwdMore * num_sms() && a->T <= kFwdMost * num_sms()) {
        const RowShape r = ring_shape(d8);
        const int ctas = kFwdCtas * num_sms(), arrays = a->residual ? 2 : 1;
#define MOE_RING(F) return launch_ring<rmsnorm_ring_kernel<2, F>>(ctas, r, arrays, a->d, st, p)
        switch (a->format) {
        case MOE_ROWS_FP8: MOE_RING(MOE_ROWS_FP8);
        case MOE_ROWS_MXFP8: MOE_RING(MOE_ROWS_MXFP8);
        case MOE_ROWS_MXFP4: MOE_RING(MOE_ROWS_MXFP4);
        default: MOE_RING(MOE_ROWS_NONE);
        }
#undef MOE_RING
    }
    const dim3 grid((unsigned)(((long long)a->T + s.rows - 1) / s.rows));
    const int threads = s.threads * s.rows;
    if (s.V == 1) return launch_early(rmsnorm_kernel<1>, grid, threads, 0, st, p);
    if (s.V == 2) return launch_early(rmsnorm_kernel<2>, grid, threads, 0, st, p);
    return launch_early(rmsnorm_kernel<4>, grid, threads, 0, st, p);
}

size_t rmsnorm_bwd_workspace_bytes(int T, int d) {
    return (size_t)bwd_parts(T, d / 8) * d * sizeof(float);
}

moe_status launch_rmsnorm_bwd(const moe_norm_bwd_args *a, cudaStream_t st) {
    NormBwd p;
    std::memset(&p, 0, sizeof p);
    p.T = a->T;
    p.d8 = a->d / 8;
    p.inv_d = 1.0f / (float)a->d;
    p.x = reinterpret_cast<const uint4 *>(a->x);
    p.dy = reinterpret_cast<const uint4 *>(a->dy);
    p.d_residual = reinterpret_cast<const uint4 *>(a->d_residual);
    p.weight = a->weight;
    p.rstd = a->rstd;
    p.dx = reinterpret_cast<uint4 *>(a->dx);
    p.part = static_cast<float *>(a->ws);
    p.status = device_status_ptr();
    if (!p.status) return MOE_ERR_CUDA;
    int parts = bwd_parts(a->T, p.d8);
    moe_status r = MOE_OK;
    if (parts > 0 && p.d8 <= kRingVecs) {
        const RowShape s = ring_shape(p.d8);
        p.threads = s.threads;
        r = launch_ring<rmsnorm_bwd_ring_kernel<2>>(parts, s, a->d_residual ? 3 : 2, a->d, st, p);
    } else if (parts > 0) {
        const int cl = wide_cluster(p.d8);
        r = cl == 1 ? launch_wide<1>(parts, p, st)
                    : cl == 2 ? launch_wide<2>(parts, p, st) : launch_wide<4>(parts, p, st);
    }
    if (r != MOE_OK) return r;
    // without rows: zeros
    const int d4 = a->d / 4;
    return launch_early(rmsnorm_dw_kernel, dim3((d4 + 31) / 32), 32 * kDwWarps, 0, st,
                        reinterpret_cast<const float4 *>(a->ws), parts, d4,
                        reinterpret_cast<float4 *>(a->d_weight));
}

}  // namespace moe
