// fp8_thin.cu -- the FP8 matmul of one matrix with 8 rows at most (a token, or a few
// drafted ones, through a dense projection):
//
//   out[r, n] = w_r sum_b sa[r, b] sb[n / 128, b] sum_{k in block b} A[r, k] B[n, k]
//
// Every weight byte is used for a handful of rows, so the kernel is a stream of the
// weights: what bounds it is how soon and how many of their bytes are on their way.  A
// CTA has 16 weight rows; its eight warps take the blocks of 128 along the contraction
// in turn, four at a time, all of whose bytes are requested at once (cp.async, each
// lane for itself: there would not be the registers), and their sums meet in
// shared memory.  Rows are the columns of mma.m16n8k16 and weights its 16 rows: codes
// become f16, which holds each of them exactly, a block's products are summed in fp32,
// and the block's scales are applied to that sum in fp32.  A lane's 16 bytes of a weight
// row and of a token row hold the same 16 places along the contraction; which of them an
// instruction takes together does not matter, so both are used as they lie in memory.
// Measured, calls in a graph, each on other weights than the one before (from HBM): 4096 x
// 4096 with one row 6.1 us (2.7 TB/s, 1.7 us of them what an empty call takes), 16384 x
// 4096 14.4-15.1 us (4.4-4.7 TB/s); on the same weights again, from L2: 5.1 and 10.3 us, 1024 x
// 512 2.0 us.  A call by itself, from the host: 7.0-7.5 us at 4096 x 4096.
#include "fp8_common.cuh"

namespace moe {
namespace {

constexpr int kThinWarps = 8;
constexpr int kThinBlocks = 4;                                     // of a warp at a time
constexpr int kThinSmem = kThinWarps * kThinBlocks * 4 * 512;      // 4 pieces of 16 bytes a lane

struct ThinParams {
    const uint8_t *a, *b;
    const float *sa, *sb;
    const int32_t *offsets;   // [2]
    int max_rows, N, K;
    const float *row_w;       // of rows < w_rows (others 1), or null
    int w_rows;
    uint16_t *out;
    int *status;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__global__ void __launch_bounds__(kThinWarps * 32) fp8_thin_kernel(const ThinParams p) {
    constexpr int U = kThinBlocks;
    extern __shared__ __align__(16) uint8_t stage[];
    __shared__ float sums[kThinWarps][8][17];
    wait_for_kernels_ahead();
    let_kernels_behind_begin();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r4 = lane >> 2, t4 = lane & 3;
    const int n0 = blockIdx.x * 16, K_blocks = fp8_blocks(p.K);
    const uint8_t *w0 = p.b + (size_t)min(n0 + r4, p.N - 1) * p.K;
    const uint8_t *w1 = p.b + (size_t)min(n0 + r4 + 8, p.N - 1) * p.K;
    const float *sb = p.sb + (size_t)(n0 / kFp8Block) * K_blocks;
    // piece j (row r4 or r4 + 8, half of the block) of block u, this lane's
    const uint32_t mine = smem_u32(stage) + warp * (U * 2048) + lane * 16;
    const int row0 = row_offset(p.offsets[0], p.max_rows);
    const int n = row_offset(p.offsets[1], p.max_rows) - row0;
    if (blockIdx.x == 0 && threadIdx.x == 0 && (row0 != p.offsets[0] || row0 + n != p.offsets[1] || n < 0))
        record_status(p.status, MOE_ERR_INVALID_ARG);
    // this lane's row as an operand, and the first of its two rows of sums
    const int c0 = 2 * t4;
    const bool row_ok = r4 < n;
    const uint8_t *xr = p.a + (size_t)(row0 + r4) * p.K;
    const float *sa = p.sa + (size_t)(row0 + c0) * K_blocks;
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};

    for (int kb0 = warp; kb0 < K_blocks; kb0 += kThinWarps * U) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int k = (kb0 + u * kThinWarps) * kFp8Block + c * 64 + t4 * 16;
                if (k < p.K) {
                    cp_async16(mine + u * 2048 + c * 512, w0 + k);
                    cp_async16(mine + u * 2048 + (2 + c) * 512, w1 + k);
                }
            }
        }
        uint4 x[U][2];
        float s[U], s0[U], s1[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int kb = kb0 + u * kThinWarps;
            const bool in = kb < K_blocks;
            s[u] = in ? __ldg(sb + kb) : 0.0f;
            s0[u] = in && c0 < n ? __ldg(sa + kb) : 0.0f;
            s1[u] = in && c0 + 1 < n ? __ldg(sa + K_blocks + kb) : 0.0f;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int k = kb * kFp8Block + c * 64 + t4 * 16;
                x[u][c] = make_uint4(0, 0, 0, 0);
                if (row_ok && k < p.K) x[u][c] = __ldg(reinterpret_cast<const uint4 *>(xr + k));
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");   // each lane reads its own bytes alone
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int kb = kb0 + u * kThinWarps;
            if (kb >= K_blocks) break;
            float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint4 a0 = make_uint4(0, 0, 0, 0), a1 = a0;
                if (kb * kFp8Block + h * 64 + t4 * 16 < p.K) {
                    a0 = ld_shared_v4(mine + u * 2048 + h * 512);
                    a1 = ld_shared_v4(mine + u * 2048 + (2 + h) * 512);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t l0, h0, l1, h1;
                    e4m3x4_f16((&a0.x)[i], l0, h0);
                    e4m3x4_f16((&a1.x)[i], l1, h1);
                    uint32_t bl, bh;
                    e4m3x4_f16((&x[u][h].x)[i], bl, bh);
                    mma_f16(c, l0, l1, h0, h1, bl, bh);
                }
            }
            const float f0 = s0[u] * s[u], f1 = s1[u] * s[u];
            acc[0] = fmaf(c[0], f0, acc[0]);
            acc[1] = fmaf(c[1], f1, acc[1]);
            acc[2] = fmaf(c[2], f0, acc[2]);
            acc[3] = fmaf(c[3], f1, acc[3]);
        }
    }
    sums[warp][c0][r4] = acc[0];
    sums[warp][c0 + 1][r4] = acc[1];
    sums[warp][c0][r4 + 8] = acc[2];
    sums[warp][c0 + 1][r4 + 8] = acc[3];
    __syncthreads();
    for (int o = threadIdx.x; o < n * 8; o += kThinWarps * 32) {
        const int r = o >> 3, c = 2 * (o & 7), row = row0 + r;
        if (n0 + c >= p.N) continue;
        float v0 = 0.0f, v1 = 0.0f;
#pragma unroll
        for (int i = 0; i < kThinWarps; ++i) {
            v0 += sums[i][r][c];
            v1 += sums[i][r][c + 1];
        }
        const float f = p.row_w && row < p.w_rows ? p.row_w[row] : 1.0f;
        *reinterpret_cast<uint32_t *>(p.out + (size_t)row * p.N + n0 + c) =
            pack_bf16x2(f * v0, f * v1);
    }
}

}  // namespace

moe_status launch_fp8_thin(const uint8_t *aq, const float *as, const int32_t *offsets, int max_rows,
                           const uint8_t *bq, const float *bs, const float *row_w, int w_rows,
                           int N, int K, uint16_t *out, cudaStream_t st) {
    int *status = device_status_ptr();
    if (!status) return MOE_ERR_CUDA;
    const ThinParams p = {aq, bq, as, bs, offsets, max_rows, N, K, row_w, w_rows, out, status};
    static bool attr_set[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
    if (dev < 0 || dev >= 64) return MOE_ERR_UNSUPPORTED;
    if (!attr_set[dev]) {
        if (cudaFuncSetAttribute(fp8_thin_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kThinSmem) != cudaSuccess)
            return MOE_ERR_CUDA;
        attr_set[dev] = true;
    }
    return launch_early(fp8_thin_kernel, dim3((unsigned)((N + 15) / 16)), kThinWarps * 32, kThinSmem,
                        st, p);
}

}  // namespace moe
