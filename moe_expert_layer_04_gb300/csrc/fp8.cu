// fp8.cu -- FP8 quantisation with one fp32 scale per block of 128 (the format
// is in fp8_common.cuh): token rows in 1 x 128 blocks, in place or through the
// dispatch; weights in 128 x 128 blocks in both orientations; and the
// operands of the weight gradient, quantised along each group's rows.
#include "fp8_common.cuh"

namespace moe {
namespace {

__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t m, uint32_t w) {
    return __vmaxu2(m, w & 0x7FFF7FFFu);   // bit patterns order as magnitudes, NaN last
}
__device__ __forceinline__ uint32_t amax_bits_of(uint32_t m) {
    const uint32_t lo = m & 0xFFFFu, hi = m >> 16;
    return (lo > hi ? lo : hi) << 16;      // bf16 -> fp32 bits
}

// ------------------------------------------------------------------ rows
//
// A lane owns 16 consecutive elements (32 bytes in, 16 bytes of codes out),
// eight lanes a block: the block's amax is three shuffles away, and every
// store of codes fills whole 128-byte lines.  A warp takes kRowU * 512
// elements of one token at a time, all loads issued before the first use.
// k = 0: plain quantisation, row t to row t; k > 0: row t goes to its k
// permuted rows and to row T*k + t, quantised once.  Bound by HBM: 2 bytes
// read an element, 1 + 1/32 written for each copy.  4096 tokens of 4096 to seven
// rows each: 24.3 us, 6.4 TB/s.
constexpr int kRowU = 2;

__global__ void __launch_bounds__(256)
    fp8_rows_kernel(const uint16_t *__restrict__ x, const int32_t *__restrict__ slot_row,
                    long long T, int K, int k, uint8_t *__restrict__ q, float *__restrict__ s) {
    wait_for_kernels_ahead();
    let_kernels_behind_begin();
    const int lane = threadIdx.x & 31;
    const int nb = fp8_blocks(K);
    const int chunks = (K + kRowU * 512 - 1) / (kRowU * 512);
    const long long units = T * chunks;
    const long long nw = (long long)gridDim.x * 8;
    const long long S = k > 0 ? T * k : 0;
    for (long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); i < units; i += nw) {
        const long long t = i / chunks;
        const int c0 = (int)(i - t * chunks) * (kRowU * 512) + lane * 16;
        long long row = t;
        if (k > 0 && lane < k) row = slot_row[t * k + lane];
        uint4 v[kRowU][2];
#pragma unroll
        for (int u = 0; u < kRowU; ++u) {
            const int c = c0 + u * 512;
            v[u][0] = v[u][1] = make_uint4(0, 0, 0, 0);
            if (c < K) {
                const uint4 *p = reinterpret_cast<const uint4 *>(x + t * K + c);
                v[u][0] = __ldg(p);
                v[u][1] = __ldg(p + 1);
            }
        }
        uint4 code[kRowU];
        float sc[kRowU];
#pragma unroll
        for (int u = 0; u < kRowU; ++u) {
            const uint32_t w[8] = {v[u][0].x, v[u][0].y, v[u][0].z, v[u][0].w,
                                   v[u][1].x, v[u][1].y, v[u][1].z, v[u][1].w};
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max_abs_bf16x2(m, w[j]);
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
            const Fp8Scale f = fp8_scale(amax_bits_of(m));
            sc[u] = f.s;
            uint32_t h[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                h[j] = e4m3x2_bf16(w[2 * j], f.r) | (e4m3x2_bf16(w[2 * j + 1], f.r) << 16);
            code[u] = make_uint4(h[0], h[1], h[2], h[3]);
        }
        const int copies = k > 0 ? k + 1 : 1;
        for (int j = 0; j < copies; ++j) {
            long long r = t;
            if (k > 0) {
                r = j < k ? __shfl_sync(0xffffffffu, row, j) : S + t;
                if (j < k && (r < 0 || r >= S)) continue;   // not a routed row
            }
#pragma unroll
            for (int u = 0; u < kRowU; ++u) {
                const int c = c0 + u * 512;
                if (c < K) {
                    *reinterpret_cast<uint4 *>(q + r * K + c) = code[u];
                    if ((lane & 7) == 0) s[r * nb + c / kFp8Block] = sc[u];
                }
            }
        }
    }
}

// --------------------------------------------------------------- tiles
//
// A CTA takes one 128 x 128 tile.  Thread t holds rows 4 (t / 8) .. + 3,
// columns 16 (t % 8) .. + 15: its codes are four 16-byte stores, and 4 x 4
// bytes at a time transpose in registers (byte permutes) into a staging tile
// of the transposed codes, whose 16-byte chunks are exchanged by column group
// so that neither side has a bank conflict.
struct Tile {
    uint4 v[4][2];
};

__device__ __forceinline__ void load_tile(Tile &a, const uint16_t *src, long long pitch, int rows,
                                          int cols) {
    const int r0 = (threadIdx.x >> 3) * 4, c = (threadIdx.x & 7) * 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        a.v[i][0] = a.v[i][1] = make_uint4(0, 0, 0, 0);
        if (r0 + i < rows && c < cols) {
            const uint4 *p = reinterpret_cast<const uint4 *>(src + (r0 + i) * pitch + c);
            a.v[i][0] = __ldg(p);
            if (c + 8 < cols) a.v[i][1] = __ldg(p + 1);
        }
    }
}

__device__ __forceinline__ uint32_t tile_word(const Tile &a, int i, int j) {
    const uint4 &v = a.v[i][j >> 2];
    return (j & 3) == 0 ? v.x : (j & 3) == 1 ? v.y : (j & 3) == 2 ? v.z : v.w;
}

// Word (4 rows) `rg` of transposed row `col` in the staging tile.
__device__ __forceinline__ int stage_word(int col, int rg) {
    return col * 32 + (rg ^ (((col >> 4) & 7) << 2));
}

// h[i]: four codes (columns c4 .. c4 + 3) of row i -> four words, one a column.
__device__ __forceinline__ void stage_4x4(uint32_t *stage, int col, int rg, const uint32_t (&h)[4]) {
    const uint32_t a = __byte_perm(h[0], h[1], 0x5140), b = __byte_perm(h[2], h[3], 0x5140);
    const uint32_t c = __byte_perm(h[0], h[1], 0x7362), d = __byte_perm(h[2], h[3], 0x7362);
    stage[stage_word(col + 0, rg)] = __byte_perm(a, b, 0x5410);
    stage[stage_word(col + 1, rg)] = __byte_perm(a, b, 0x7632);
    stage[stage_word(col + 2, rg)] = __byte_perm(c, d, 0x5410);
    stage[stage_word(col + 3, rg)] = __byte_perm(c, d, 0x7632);
}

__device__ __forceinline__ uint4 staged_chunk(const uint32_t *stage, int col, int chunk) {
    return *reinterpret_cast<const uint4 *>(stage + stage_word(col, chunk * 4));
}

// Weights [G, N, K] -> q [G, N, K], s [G, N/128, K/128] and, when qt is given,
// qt [G, K, N], st [G, K/128, N/128] (the same codes and scales, transposed).
__global__ void __launch_bounds__(256)
    fp8_weights_kernel(const uint16_t *__restrict__ src, int N, int K, uint8_t *__restrict__ q,
                       float *__restrict__ s, uint8_t *__restrict__ qt, float *__restrict__ st) {
    __shared__ __align__(16) uint32_t stage[128 * 32];
    __shared__ uint32_t part[8];
    wait_for_kernels_ahead();
    let_kernels_behind_begin();
    const int nbn = fp8_blocks(N), nbk = fp8_blocks(K);
    const int bk = blockIdx.x % nbk;
    const long long rest = blockIdx.x / nbk;
    const int bn = (int)(rest % nbn);
    const long long g = rest / nbn;
    const int t = threadIdx.x, r0 = (t >> 3) * 4, c0 = (t & 7) * 16;
    const int rows = min(128, N - bn * 128), cols = min(128, K - bk * 128);
    const long long at = (g * N + bn * 128LL) * K + bk * 128;
    Tile a;
    load_tile(a, src + at, K, rows, cols);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max_abs_bf16x2(m, tile_word(a, i, j));
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((t & 31) == 0) part[t >> 5] = m;
    __syncthreads();
    m = part[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) m = __vmaxu2(m, part[i]);
    const Fp8Scale f = fp8_scale(amax_bits_of(m));
    if (t == 0) {
        s[(g * nbn + bn) * nbk + bk] = f.s;
        if (st) st[(g * nbk + bk) * nbn + bn] = f.s;
    }
    uint32_t code[4][4];
#pragma unroll
    for (int c4 = 0; c4 < 4; ++c4) {
        uint32_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            code[i][c4] = h[i] = e4m3x2_bf16(tile_word(a, i, 2 * c4), f.r) |
                                 (e4m3x2_bf16(tile_word(a, i, 2 * c4 + 1), f.r) << 16);
        if (qt) stage_4x4(stage, c0 + 4 * c4, t >> 3, h);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (r0 + i < rows && c0 < cols)
            *reinterpret_cast<uint4 *>(q + at + (long long)(r0 + i) * K + c0) =
                make_uint4(code[i][0], code[i][1], code[i][2], code[i][3]);
    if (!qt) return;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int col = (t >> 3) + 32 * j, chunk = t & 7;
        if (col < cols && chunk * 16 < rows)
            *reinterpret_cast<uint4 *>(qt + (g * K + bk * 128LL + col) * N + bn * 128 +
                                       chunk * 16) = staged_chunk(stage, col, chunk);
    }
}

// Weight-gradient operands: the rows of each group in blocks of 128 from the
// group's first row (the last block filled with zeros), every column of a
// block one scale block.  Block b of all groups together ("chunk") is written
// transposed: code (c, r) at (b C + c) 128 + r, scale (b, c) at b C + c, so
// that a matmul stage is one contiguous run of rows of 128 codes.  Bound by HBM in
// principle; 6789 rows of 4096 in 9 groups take 19.5 us (4.3 TB/s: 2.6 rounds of CTAs,
// each of which loads once and then stores).  Both operands in one launch measured
// 243 us for the whole gradient against 234: the second launch begins during the first.
// first[g] is the group's first chunk (fp8_chunks_kernel); blockIdx.y = chunk.
__global__ void __launch_bounds__(256)
    fp8_columns_kernel(const uint16_t *__restrict__ src, const int32_t *__restrict__ offsets,
                       const int32_t *__restrict__ first, int G, int max_rows, int C,
                       uint8_t *__restrict__ qt, float *__restrict__ st) {
    __shared__ __align__(16) uint32_t stage[128 * 32];
    __shared__ __align__(16) uint32_t part[8][64];   // per warp: bf16 pair maxima of 128 columns
    __shared__ __align__(16) float factor[128];
    wait_for_kernels_ahead();
    let_kernels_behind_begin();
    const int b = blockIdx.y;
    if (b >= first[G]) return;
    int lo = 0, hi = G - 1;                          // the chunk's group
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= b) lo = mid; else hi = mid - 1;
    }
    const int row0 = row_offset(offsets[lo], max_rows) + (b - first[lo]) * 128;
    const int rows = min(128, row_offset(offsets[lo + 1], max_rows) - row0);
    const int col0 = blockIdx.x * 128, cols = min(128, C - col0);
    const int t = threadIdx.x, c0 = (t & 7) * 16;
    Tile a;
    load_tile(a, src + (long long)row0 * C + col0, C, rows, cols);
    // column maxima: over the thread's four rows, the warp's 16 (lanes 8 and
    // 16 apart hold the same columns), then the CTA's 128
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max_abs_bf16x2(m, tile_word(a, i, j));
        m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 8));
        m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 16));
        if ((t & 31) < 8) part[t >> 5][(t & 7) * 8 + j] = m;
    }
    __syncthreads();
    if (t < 128) {
        uint32_t m = 0;
#pragma unroll
        for (int w = 0; w < 8; ++w) m = __vmaxu2(m, part[w][t >> 1]);
        const Fp8Scale f = fp8_scale((t & 1) ? (m & 0xFFFF0000u) : (m << 16));
        factor[t] = f.r;
        if (t < cols) st[(long long)b * C + col0 + t] = f.s;
    }
    __syncthreads();
#pragma unroll
    for (int c4 = 0; c4 < 4; ++c4) {
        const float4 r = *reinterpret_cast<const float4 *>(factor + c0 + 4 * c4);
        uint32_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w0 = tile_word(a, i, 2 * c4), w1 = tile_word(a, i, 2 * c4 + 1);
            h[i] = e4m3x4(bf16_lo(w0) * r.x, bf16_hi(w0) * r.y, bf16_lo(w1) * r.z,
                          bf16_hi(w1) * r.w);
        }
        stage_4x4(stage, c0 + 4 * c4, t >> 3, h);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int col = (t >> 3) + 32 * j, chunk = t & 7;
        if (col < cols)
            *reinterpret_cast<uint4 *>(qt + ((long long)b * C + col0 + col) * 128 + chunk * 16) =
                staged_chunk(stage, col, chunk);
    }
}

// first[g]: chunks of 128 rows before group g, first[G] their number, at most max_chunks
// (which offsets that do not descend never exceed).  One warp.
__global__ void fp8_chunks_kernel(const int32_t *__restrict__ offsets, int G, int max_rows,
                                  int max_chunks, int32_t *__restrict__ first, int *status) {
    wait_for_kernels_ahead();
    let_kernels_behind_begin();
    const int lane = threadIdx.x;
    int carry = 0;
    for (int base = 0; base <= G; base += 32) {
        const int g = base + lane;
        int n = 0;
        if (g < G) {
            const int o = row_offset(offsets[g], max_rows);
            const int end = row_offset(offsets[g + 1], max_rows);
            if (o != offsets[g] || end != offsets[g + 1] || end < o)
                record_status(status, MOE_ERR_INVALID_ARG);
            n = max(0, (end - o + 127) >> 7);
        }
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (g <= G) first[g] = min(carry + incl - n, max_chunks);
        carry += __shfl_sync(0xffffffffu, incl, 31);
    }
}

}  // namespace

moe_status launch_fp8_rows(const uint16_t *x, const int32_t *slot_row, long long T, int K, int k,
                           uint8_t *q, float *s, cudaStream_t st) {
    const long long units = T * ((K + kRowU * 512 - 1) / (kRowU * 512));
    const long long want = (units + 7) / 8;
    const long long most = (long long)num_sms() * 64;
    return launch_early(fp8_rows_kernel, dim3((unsigned)(want < most ? want : most)), 256, 0, st, x,
                        slot_row, T, K, k, q, s);
}

moe_status launch_fp8_weights(const uint16_t *src, int G, int N, int K, uint8_t *q, float *s,
                              uint8_t *qt, float *s_t, cudaStream_t st) {
    const long long tiles = (long long)G * fp8_blocks(N) * fp8_blocks(K);
    if (tiles > 0x7FFFFFFFLL) return MOE_ERR_UNSUPPORTED;
    return launch_early(fp8_weights_kernel, dim3((unsigned)tiles), 256, 0, st, src, N, K, q, s, qt,
                        s_t);
}

moe_status launch_fp8_chunks(const int32_t *offsets, int G, int max_rows, int max_chunks,
                             int32_t *first, cudaStream_t st) {
    int *status = device_status_ptr();
    if (!status) return MOE_ERR_CUDA;
    return launch_early(fp8_chunks_kernel, dim3(1), 32, 0, st, offsets, G, max_rows, max_chunks,
                        first, status);
}

moe_status launch_fp8_columns(const uint16_t *src, const int32_t *offsets, const int32_t *first,
                              int G, int max_rows, int max_chunks, int C, uint8_t *qt,
                              float *s_t, cudaStream_t st) {
    const dim3 grid(fp8_blocks(C), max_chunks);
    return launch_early(fp8_columns_kernel, grid, 256, 0, st, src, offsets, first, G, max_rows, C, qt,
                        s_t);
}

}  // namespace moe
