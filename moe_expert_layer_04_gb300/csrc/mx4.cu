// mx4.cu -- MXFP4 quantisation of bf16 rows (weights, or token rows in place and through
// the dispatch), and the values of quantised rows in bf16.  Format: mx_common.cuh; codes
// q [rows, K/2], scales sf [rows, mx_sf_pitch(K)] as for MXFP8.
//
// A lane owns eight consecutive elements, 16 bytes of bf16 and a word of codes, four
// lanes a block: every load and store of a warp is contiguous, and a block's largest
// magnitude is two shuffles away.  All loads of a lane are issued before the first use.
// Bound by HBM: 2 bytes read, 1/2 + 1/32 written an element, and the reverse.  Measured at
// 36864 rows of 4096: quantised in 55.6 us, the values in 56.1, 101 and 100 % of the copy
// bandwidth (70 and 61 with a grid-stride loop and a scale's byte stored by each fourth lane);
// one row of 4096 1.6 us.
#include "fp8_common.cuh"
#include "mx_common.cuh"

namespace moe {
namespace {

constexpr int kU = 4;   // vectors of eight elements of a lane (own_block() says four)

// Codes and scale code of a vector; every lane of the warp calls it.
__device__ __forceinline__ uint32_t quantise8(const uint4 v, uint32_t &code) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const uint32_t lo = m & 0xFFFFu, hi = m >> 16;
    code = mx4_scale_code((lo > hi ? lo : hi) << 16);   // bf16 bits order as magnitudes
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
    }
    return e2m1x8(f, mx4_inv_scale(code));
}

// A warp's scale codes: lane l holds that of its block l / 4 of each of kU = 4 vectors.
// Block 8 u + l / 4 of the warp's 32 is stored (and, for the values, loaded) by lane
// 4 (l / 4) + u: 32 consecutive bytes where the row's scales are.
__device__ __forceinline__ int own_block(int lane) { return (lane & 3) * 8 + (lane >> 2); }

// Place of the scale of block b (of all rows); kb blocks a row, sfp bytes.
__device__ __forceinline__ long long scale_at(long long b, int kb, int sfp) {
    if (kb == sfp) return b;
    const long long r = b / kb;
    return r * sfp + (b - r * kb);
}

// n8 = all vectors of the matrix; kb = blocks of a row.  A warp: 32 kU vectors.
__global__ void __launch_bounds__(256)
    mx4_quantize_kernel(const uint4 *__restrict__ src, long long n8, int kb, int sfp,
                        uint32_t *__restrict__ q, uint8_t *__restrict__ sf) {
    wait_for_kernels_ahead();
    let_kernels_behind_begin();
    const int lane = threadIdx.x & 31;
    const long long w0 = ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * 32 * kU;
    if (w0 >= n8) return;
    uint4 v[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        const long long i = w0 + 32 * u + lane;
        v[u] = i < n8 ? __ldcs(src + i) : make_uint4(0, 0, 0, 0);
    }
    uint32_t own = 0;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        const long long i = w0 + 32 * u + lane;
        uint32_t code;
        const uint32_t w = quantise8(v[u], code);
        if (i < n8) q[i] = w;
        if ((lane & 3) == u) own = code;
    }
    const long long b = w0 / 4 + own_block(lane);
    if (4 * b < n8) sf[scale_at(b, kb, sfp)] = (uint8_t)own;
}

__global__ void __launch_bounds__(256)
    mx4_dequantize_kernel(const uint32_t *__restrict__ q, const uint8_t *__restrict__ sf,
                          long long n8, int kb, int sfp, uint4 *__restrict__ out) {
    wait_for_kernels_ahead();
    let_kernels_behind_begin();
    const int lane = threadIdx.x & 31;
    const long long w0 = ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * 32 * kU;
    if (w0 >= n8) return;
    const long long b = w0 / 4 + own_block(lane);
    uint32_t own = 0, w[kU];
    if (4 * b < n8) own = __ldg(sf + scale_at(b, kb, sfp));
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        const long long i = w0 + 32 * u + lane;
        w[u] = i < n8 ? __ldcs(q + i) : 0u;
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        const long long i = w0 + 32 * u + lane;
        const float x = mx4_scale(__shfl_sync(0xffffffffu, own, (lane & ~3) + u));
        uint32_t h[4], o[4];
        e2m1x8_f16(w[u], h);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[j]));
            o[j] = pack_bf16x2(f.x * x, f.y * x);
        }
        if (i < n8) out[i] = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// The dispatch: a warp takes kU * 256 elements of one token, quantises them once and
// writes them to the token's k routed rows and to row T k + t.
__global__ void __launch_bounds__(256)
    mx4_gather_kernel(const uint4 *__restrict__ x, const int32_t *__restrict__ slot_row, int T,
                      int d8, int k, int sfp, uint32_t *__restrict__ q,
                      uint8_t *__restrict__ sf) {
    wait_for_kernels_ahead();
    let_kernels_behind_begin();
    const int lane = threadIdx.x & 31;
    const int chunks = (d8 + 32 * kU - 1) / (32 * kU);
    const long long units = (long long)T * chunks, S = (long long)T * k;
    for (long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); i < units;
         i += (long long)gridDim.x * 8) {
        const long long t = i / chunks;
        const int c0 = (int)(i - t * chunks) * (32 * kU) + lane;
        long long row = 0;
        if (lane < k) row = slot_row[t * k + lane];
        uint4 v[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int c = c0 + 32 * u;
            v[u] = c < d8 ? __ldg(x + t * d8 + c) : make_uint4(0, 0, 0, 0);
        }
        uint32_t w[kU], code[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) w[u] = quantise8(v[u], code[u]);
        for (int j = 0; j <= k; ++j) {
            long long r = __shfl_sync(0xffffffffu, row, j & 31);
            if (j == k) r = S + t;
            else if (r < 0 || r >= S) continue;   // not a routed row
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int c = c0 + 32 * u;
                if (c >= d8) continue;
                q[r * d8 + c] = w[u];
                if ((lane & 3) == 0) sf[r * sfp + (c >> 2)] = (uint8_t)code[u];
            }
        }
    }
}

unsigned blocks_for(long long warps) {
    const long long want = (warps + 7) / 8, most = (long long)num_sms() * 64;
    return (unsigned)(want < most ? want : most);
}

}  // namespace

moe_status launch_mx4_quantize(const uint16_t *src, long long rows, int K, uint8_t *q, uint8_t *sf,
                               cudaStream_t st) {
    const long long n8 = rows * (K / 8), ctas = (n8 + 256 * kU - 1) / (256 * kU);
    if (ctas > 0x7FFFFFFFLL) return MOE_ERR_UNSUPPORTED;
    return launch_early(mx4_quantize_kernel, dim3((unsigned)ctas), 256, 0, st, reinterpret_cast<const uint4 *>(src), n8, K / 32, mx_sf_pitch(K),
                        reinterpret_cast<uint32_t *>(q), sf);
}

moe_status launch_mx4_dequantize(const uint8_t *q, const uint8_t *sf, long long rows, int K,
                                 uint16_t *out, cudaStream_t st) {
    const long long n8 = rows * (K / 8), ctas = (n8 + 256 * kU - 1) / (256 * kU);
    if (ctas > 0x7FFFFFFFLL) return MOE_ERR_UNSUPPORTED;
    return launch_early(mx4_dequantize_kernel, dim3((unsigned)ctas), 256, 0, st, reinterpret_cast<const uint32_t *>(q), sf, n8, K / 32,
                        mx_sf_pitch(K), reinterpret_cast<uint4 *>(out));
}

moe_status launch_mx4_gather(const uint16_t *x, const int32_t *slot_row, int T, int d, int k,
                             uint8_t *q, uint8_t *sf, cudaStream_t st) {
    const int d8 = d / 8;
    const long long units = (long long)T * ((d8 + 32 * kU - 1) / (32 * kU));
    return launch_early(mx4_gather_kernel, dim3(blocks_for(units)), 256, 0, st,
                        reinterpret_cast<const uint4 *>(x), slot_row, T, d8, k, mx_sf_pitch(d),
                        reinterpret_cast<uint32_t *>(q), sf);
}

}  // namespace moe
