// gemm_fp8.cu -- FP8 (E4M3) matmuls whose operands carry one fp32 scale per
// block of 128 along the contraction (format: fp8_common.cuh).
//
//   FP8_ROWS   out[r, n] = w_r sum_b sa[r, b] sb[n / 128, b]
//                              sum_{k in block b} A[r, k] B[g][n, k]     bf16
//              rows grouped by expert g; with the transposed weight it is the
//              data gradient
//   FP8_FFN1   the same for the gate and up rows of W13, then the clamped
//              SwiGLU and its quantisation along I (a tile holds the 128 h
//              columns of one scale block)
//   FP8_WGRAD  dW[g][m, n] = sum_b sa[b, m] sb[b, n] sum_{r in block b} A B
//              over the chunks of 128 rows of group g                    fp32
//
// The tensor core sums the products of one block in fp32 (tcgen05.mma
// kind::f8f6f4: E4M3 operands straight from shared memory, accumulator in tensor
// memory); the scales differ from block to block, so each block's sum leaves tensor
// memory, is multiplied by its scales and added to the tile's accumulator in
// registers, in fp32.
//
// What bounds it: a block of a 128 x 256 tile takes the tensor core 512 cycles, the
// reading of its sums by eight warps 320, the copies of its 48 KB of operands out of L2
// 570, each on its own; side by side the three do not slow one another (512, 355, 570).
// What does cost is their order: with two accumulators, each read between its MMAs and
// its next ones, 580 cycles a block without any scales, and the loop below takes 806
// (FFN1 835, WGRAD with a product for the column scales 1080), measured as the
// difference of long and short contractions.  At that rate the products of a long run of
// blocks go at 2.0 PFLOP/s, half of what the tensor core does on FP8 without block
// scales.  The rest is what a tile costs outside its loop:
// the first operands of the next tile and two blocks of products run during it, then
// the tensor core waits.  So the output leaves through shared memory by TMA stores that
// run during the next tile (ROWS: 1500 cycles a tile, 3000 straight from the registers),
// the next tile's place and scales are found before it, and the weight gradient, whose
// loops are short (a group of 900 rows has 7 blocks) and whose fp32 output is 128 KB a
// tile, takes 4000 cycles for it, a third of its time: the same warps accumulate and
// store, and the output crosses shared memory twice (2048 cycles).
//
// Measured (time of the call): 12345 rows in 33 uneven groups, 4096 x 2048 weights: 114-118
// us, 1.8 PFLOP/s; expert FFN of 32768 rows over 33 groups, d = 4096, I = 2048: 794-823 us,
// 2.0-2.1 PFLOP/s; of 777 rows over 9: 63 us, where the weights alone are 30 us of HBM
// (176 tiles on 152 SMs); weight gradient 4096 x 4096 of 6789 rows in 9 groups: 234 us
// with the quantisation of both operands (39 us), 604 MB of output.
//
// One CTA per SM, persistent, 12 warps: warp 0 TMA producer, warp 1 tensor memory owner
// and MMA issuer, warps 4-11 accumulate (thread = row; two warps per lane quadrant, half
// of the columns each).  Every wait is bounded; on a timeout the CTA records
// MOE_ERR_TIMEOUT, drains its copies and MMAs, frees tensor memory and returns.
#include <cstring>
#include <type_traits>

#include "fp8_common.cuh"
#include "gemm_launch.cuh"

namespace moe {
namespace {

enum Fp8Mode : int { FP8_ROWS = 0, FP8_FFN1 = 1, FP8_WGRAD = 2 };

struct Fp8Params {
    CUtensorMap tmA;   // A codes: [rows, K] (WGRAD [chunks * M, 128]), boxes a_rows x 128
    CUtensorMap tmB;   // B codes: [G * N, K] (WGRAD [chunks * N, 128]), boxes 128 x 256 (FFN1 128)
    CUtensorMap tmO;   // ROWS, WGRAD: output, boxes of 32 rows x 128 bytes
    const int32_t *offsets;   // [G+1] rows of the groups; WGRAD: their chunks
    const float *sa, *sb;
    int G, N, K_blocks, n_tiles;
    int max_rows;             // (not WGRAD)
    int nb_n;                 // scale rows of one group's B
    int a_rows;               // of A's boxes
    int M;                    // WGRAD: output rows
    int I;                    // FFN1
    float clamp;
    const float *row_w;       // ROWS: weight of rows < w_rows (others 1), or null
    int w_rows;
    uint16_t *out;            // ROWS
    uint8_t *hq;              // FFN1: h codes [rows, I] ...
    float *hs;                //       ... and scales [rows, I / 128]
    float *dW;                // WGRAD
    int *status;
    long long wait_limit;
};

constexpr int kF8A = 128 * 128;
constexpr int kF8Epi = 8;                       // epilogue warps
constexpr int kF8Epi0 = 4;                      // the first of them
constexpr int kF8Threads = 32 * (kF8Epi0 + kF8Epi);
constexpr int kF8Bars = 256;
constexpr int kF8Smem = 232448;                 // of a CTA at most
// Scales of a block are overwritten six blocks on: its copy is sent when the MMAs
// of the block three or more before it are done, which began after the sums of the
// block two before that one were read, and with them its scales.
constexpr int kF8Scales = 6;
// 128 bytes of 32 rows on their way out, 128-byte swizzle
constexpr int kF8OutPiece = 32 * 128;

// Registers: the four warps that copy and issue hand most of theirs to the
// eight that hold the accumulators (128 a thread, and 64 in flight from tensor
// memory); 4 x 40 + 8 x 232 is what the block is launched with, 12 x 168.
constexpr int kF8RegsFew = 40, kF8RegsMany = 232;
static_assert(4 * kF8RegsFew + 8 * kF8RegsMany <= 12 * 168, "register split");

template <int MODE, int BN, int ST>
struct F8Shape {
    static constexpr int STAGE = kF8A + BN * 128;
    static constexpr int NACC = BN == 256 ? 2 : 4;   // accumulators in tensor memory
    static constexpr int CW = BN / 2;                // columns of an epilogue warp
    // of them in flight from tensor memory at a time
    static constexpr int CH = MODE == FP8_WGRAD ? 16 : BN < 128 ? CW : 32;
    static constexpr uint32_t IDESC =
        (1u << 4) | ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
    // FFN1: exchange of the largest |h|; WGRAD: ring of both operands' scales
    static constexpr int SIDE =
        MODE == FP8_FFN1 ? 2048 : MODE == FP8_WGRAD ? kF8Scales * (128 + BN) * 4 : 0;
    // pieces of output on their way to memory, for each epilogue warp
    static constexpr int OUTS = MODE == FP8_FFN1 || BN < 128 ? 0 : BN / 128;
    static constexpr int OUT = kF8Epi * OUTS * kF8OutPiece;
    // bytes of a group's offset and first tile
    static constexpr int GROUP = MODE == FP8_WGRAD ? 4 : 8;
    static constexpr int FIXED = ST * STAGE + OUT + SIDE + kF8Bars;
    static constexpr int smem(int G) { return 1024 + FIXED + GROUP * (G + 2); }
};

// One block of 128: D[tmem] = A[smem] B[smem]^T in four steps of K = 32, E4M3
// operands, fp32 accumulator; then both barriers are to hear of its end.  Called by a
// whole warp, which elects the issuing thread here: with uniform control flow around
// it the descriptors stay in uniform registers (inside `if (lane == 0)` the six
// instructions took 400 cycles, time that the tensor core waited for).
// Instruction descriptor: D format [4,6) = 1 (fp32), A and B format 0 (E4M3),
// both K-major, N >> 3 at [17,23), M >> 4 at [24,29).  Matrix descriptors count 16 bytes.
__device__ __forceinline__ void umma_f8_block(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                              uint32_t idesc, uint64_t *bar0, uint64_t *bar1) {
    asm volatile(
        "{\n\t.reg .pred e, f, t;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 f, 0, 0;\n\t"
        "setp.eq.b32 t, 0, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %5, %9, f;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %2, %6, %9, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %3, %7, %9, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %4, %8, %9, t;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%10];\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%11];\n\t}" ::"r"(
            d_tmem),
        "l"(a_desc), "l"(a_desc + 2), "l"(a_desc + 4), "l"(a_desc + 6), "l"(b_desc),
        "l"(b_desc + 2), "l"(b_desc + 4), "l"(b_desc + 6), "r"(idesc), "r"(smem_u32(bar0)),
        "r"(smem_u32(bar1))
        : "memory");
}

// (the same thread, as a warp's election has one outcome)
__device__ __forceinline__ void umma_commit_elected(uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
            smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[32]) { tmem_ld32(taddr, r); }
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// Pairs of fp32 in one instruction.
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(lo), "r"(hi));
    return v;
}
__device__ __forceinline__ uint64_t pair_f(float lo, float hi) {
    return pair(__float_as_uint(lo), __float_as_uint(hi));
}
__device__ __forceinline__ void fma2(uint64_t &acc, uint64_t a, uint64_t b) {
    // volatile: stays between the tensor memory loads that it is meant to cover
    asm volatile("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(a), "l"(b));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float lo_f(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi_f(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }

struct F8Tile {
    int g, nt, row0, rows, kb, k0;   // rows: valid rows from row0; k0: first chunk (WGRAD)
};

// The tiles of a CTA, gridDim.x apart: tile t = q n_tiles + nt.
struct F8Walk {
    int q, nt, dq, dn, n;
    __device__ explicit F8Walk(int n_tiles)
        : q(blockIdx.x / n_tiles), dq(gridDim.x / n_tiles), n(n_tiles) {
        nt = blockIdx.x - q * n;
        dn = gridDim.x - dq * n;
    }
    __device__ void next() {
        q += dq;
        nt += dn;
        if (nt >= n) { nt -= n; ++q; }
    }
};

// Row tile q, column tile nt, found by a whole warp (a ballot over 32 groups at a
// time, from the group of the tile before it: tiles come in order).
template <int MODE>
__device__ __forceinline__ F8Tile f8_tile(const Fp8Params &p, int q, int nt, const int *mt_start,
                                          const int *offs, int from) {
    F8Tile ti;
    ti.nt = nt;
    if constexpr (MODE == FP8_WGRAD) {
        const int mt = (p.M + 127) >> 7;
        ti.g = q / mt;
        ti.row0 = (q - ti.g * mt) * 128;
        ti.rows = min(128, p.M - ti.row0);
        ti.k0 = offs[ti.g];
        ti.kb = offs[ti.g + 1] - ti.k0;
        return ti;
    }
    // the last group that starts at or before row tile q (empty groups start
    // where the next one does)
    int g = from;
    while (true) {
        const int i = g + 1 + (threadIdx.x & 31);
        const unsigned m = __ballot_sync(0xffffffffu, i < p.G && mt_start[min(i, p.G)] <= q);
        g += __popc(m);
        if (m != 0xffffffffu) break;
    }
    ti.g = g;
    ti.row0 = offs[g] + (q - mt_start[g]) * 128;
    ti.rows = min(128, offs[g + 1] - ti.row0);
    ti.kb = p.K_blocks;
    ti.k0 = 0;
    return ti;
}

template <int MODE, int BN, int ST>   // ST: stages of operands in shared memory
__global__ void __launch_bounds__(kF8Threads, 1) fp8_gemm_kernel(const __grid_constant__ Fp8Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    using SH = F8Shape<MODE, BN, ST>;
    constexpr int NACC = SH::NACC, CW = SH::CW, CH = SH::CH;
    uint8_t *out_s = smem + ST * SH::STAGE;   // 1024-aligned
    uint8_t *side = out_s + SH::OUT;
    uint64_t *full = reinterpret_cast<uint64_t *>(side + SH::SIDE);
    uint64_t *empty = full + ST;
    uint64_t *tfull = empty + ST;   // a block's sums are in an accumulator
    uint64_t *tempty = tfull + NACC;          // ... and have been read
    uint64_t *xch = tempty + NACC;            // FFN1: both halves' largest |h| are in `side`
    uint64_t *done = xch + 1;
    uint32_t *tmem_base_s = reinterpret_cast<uint32_t *>(done + 1);
    volatile int *abort_s = reinterpret_cast<volatile int *>(tmem_base_s + 1);
    int *offs = reinterpret_cast<int *>(side + SH::SIDE + kF8Bars);
    int *mt_start = offs + (p.G + 1);

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);   // uniform, to the compiler too
    const int lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < ST; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int a = 0; a < NACC; ++a) {
            mbar_init(&tfull[a], 1);
            mbar_init(&tempty[a], kF8Epi);
        }
        mbar_init(xch, kF8Epi);
        mbar_init(done, 1);
        *abort_s = 0;
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&p.tmA);
        tma_prefetch_desc(&p.tmB);
    }
    if (warp == 1) {
        tmem_alloc(tmem_base_s, NACC * BN);
        tmem_relinquish();
    }
    wait_for_kernels_ahead();
    if (warp == 2) {
        // group offsets and the exclusive prefix of their 128-row tiles
        int carry = 0;
        for (int base = 0; base <= p.G; base += 32) {
            const int g = base + lane;
            int o = 0, mt = 0;
            if constexpr (MODE == FP8_WGRAD) {   // checked where they were made
                if (g <= p.G) offs[g] = p.offsets[g];
            } else {
                bool ok = true;
                if (g <= p.G) {
                    offs[g] = o = row_offset(p.offsets[g], p.max_rows);
                    ok = o == p.offsets[g];
                }
                if (g < p.G) {
                    const int end = row_offset(p.offsets[g + 1], p.max_rows);
                    ok = ok && end >= o;
                    mt = max(0, (end - o + 127) >> 7);
                }
                if (!ok && blockIdx.x == 0) record_status(p.status, MOE_ERR_INVALID_ARG);
            }
            int incl = mt;
#pragma unroll
            for (int sft = 1; sft < 32; sft <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, sft);
                if (lane >= sft) incl += v;
            }
            if (MODE != FP8_WGRAD && g <= p.G) mt_start[g] = carry + incl - mt;
            carry += __shfl_sync(0xffffffffu, incl, 31);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    let_kernels_behind_begin();

    const uint32_t tmem_base = *tmem_base_s;
    const WaitCtl wc{abort_s, p.status, p.wait_limit};
    const int total =
        (MODE == FP8_WGRAD ? p.G * ((p.M + 127) >> 7) : mt_start[p.G]) * p.n_tiles;

    if (warp < kF8Epi0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kF8RegsFew));
    if (warp == 0) {
        uint32_t s = 0, ph = 0, sc = 0;
        uint32_t begun = 0;   // stages with a copy, and its parity
        bool ok = true;
        int g = 0;
        F8Walk at(p.n_tiles);
        for (int t = blockIdx.x; ok && t < total; t += gridDim.x, at.next()) {
            const F8Tile ti = f8_tile<MODE>(p, at.q, at.nt, mt_start, offs, g);
            g = ti.g;
            for (int kb = 0; kb < ti.kb; ++kb) {
                if (!mbar_wait_warp(&empty[s], ph ^ 1u, wc)) { ok = false; break; }
                if (lane == 0) {
                    uint32_t sa_bytes = 0, sb_bytes = 0;
                    if constexpr (MODE == FP8_WGRAD) {
                        sa_bytes = 4 * min(128, p.M - ti.row0);
                        sb_bytes = 4 * min(BN, p.N - ti.nt * BN);
                    }
                    mbar_arrive_expect_tx(&full[s], p.a_rows * 128 + BN * 128 + sa_bytes + sb_bytes);
                    uint8_t *a = smem + s * SH::STAGE;
                    uint8_t *b = a + kF8A;
                    if constexpr (MODE == FP8_WGRAD) {
                        const int c = ti.k0 + kb;
                        tma_load_2d(a, &p.tmA, &full[s], 0, c * p.M + ti.row0);
                        tma_load_2d(b, &p.tmB, &full[s], 0, c * p.N + ti.nt * BN);
                        float *f = reinterpret_cast<float *>(side) + sc * (128 + BN);
                        bulk_load(f, p.sa + (size_t)c * p.M + ti.row0, sa_bytes, &full[s]);
                        bulk_load(f + 128, p.sb + (size_t)c * p.N + ti.nt * BN, sb_bytes,
                                  &full[s]);
                    } else if constexpr (MODE == FP8_FFN1) {
                        const int br = ti.g * 2 * p.I + ti.nt * 128;
                        tma_load_2d(a, &p.tmA, &full[s], kb * 128, ti.row0);
                        tma_load_2d(b, &p.tmB, &full[s], kb * 128, br);
                        tma_load_2d(b + 128 * 128, &p.tmB, &full[s], kb * 128, br + p.I);
                    } else {
                        tma_load_2d(a, &p.tmA, &full[s], kb * 128, ti.row0);
                        tma_load_2d(b, &p.tmB, &full[s], kb * 128, ti.g * p.N + ti.nt * BN);
                    }
                }
                if (++sc == kF8Scales) sc = 0;
                begun = (begun & ~(0x10001u << s)) | (0x10000u << s) | (ph << s);
                if (++s == ST) { s = 0; ph ^= 1u; }
            }
        }
        if (!ok) {
            // drain the copies still in flight before the CTA exits
            for (int i = 0; i < ST; ++i)
                if (begun >> (16 + i) & 1u)
                    mbar_wait_teardown(&full[i], begun >> i & 1u, p.wait_limit);
        }
    } else if (warp == 1) {
        // What it costs from the release of an accumulator to its next MMA is time
        // in which the tensor core has nothing to do.
        const uint64_t ad0 = sdesc_sw128(smem_u32(smem), 16, 1024);
        uint64_t ad = ad0;
        uint32_t s = 0, ph = 0, blk = 0;
        bool ok = true;
        F8Walk at(p.n_tiles);
        for (int t = blockIdx.x; ok && t < total; t += gridDim.x, at.next()) {
            int n = p.K_blocks;
            if constexpr (MODE == FP8_WGRAD) {
                const int g = at.q / ((p.M + 127) >> 7);
                n = __shfl_sync(0xffffffffu, offs[g + 1] - offs[g], 0);
            }
            for (int kb = 0; kb < n; ++kb, ++blk) {
                const uint32_t acc = blk % NACC, aph = (blk / NACC) & 1u;
                // (the operands are there long before the accumulator)
                if (!mbar_wait_warp(&full[s], ph, wc) ||
                    !mbar_wait_warp(&tempty[acc], aph ^ 1u, wc)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                umma_f8_block(tmem_base + acc * BN, ad, ad + kF8A / 16, SH::IDESC, &tfull[acc],
                              &empty[s]);
                ad += SH::STAGE / 16;
                if (++s == ST) { s = 0; ph ^= 1u; ad = ad0; }
            }
        }
        if (!ok) {
            // every MMA this thread issued must finish before TMEM is freed
            umma_commit_elected(done);
            mbar_wait_teardown(done, 0, p.wait_limit);
        }
    }
    } else {
        // ------------------------------------------------ accumulate and finish
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kF8RegsMany));
        const int q = warp & 3;                  // TMEM lane quadrant
        const int part = (warp - kF8Epi0) >> 2;  // its half of the columns
        out_s += (warp - kF8Epi0) * SH::OUTS * kF8OutPiece;
        const int r_local = q * 32 + lane;
        uint32_t blk = 0;
        int it = 0;
        bool ok = true;
        // this thread's columns of a tile: CW from cl0, or for FFN1 64 gate
        // columns from 64 part and the 64 up columns 128 further on
        const int cl0 = MODE == FP8_FFN1 ? 64 * part : CW * part;
        constexpr int kHalf = MODE == FP8_FFN1 ? 128 : CW / 2;   // column step between halves
        // Scales.  Those of WGRAD come with the operands; the others of the next block
        // are loaded a block ahead, a tile's first ones (and its row weight) before the
        // tile before it is written.
        const float *sa = nullptr, *sb0 = nullptr, *sb1 = nullptr;
        bool valid = false;
        float na = 0.0f, nb0 = 0.0f, nb1 = 0.0f, nw = 1.0f;
        auto next_scales = [&](int kb) {
            if (valid) na = __ldg(sa + kb);
            nb0 = __ldg(sb0 + kb);
            if constexpr (MODE == FP8_FFN1) nb1 = __ldg(sb1 + kb);
        };
        uint32_t sc = 0;   // WGRAD: slot of the block's scales
        F8Tile ti{};
        F8Walk at(p.n_tiles);
        auto begin_tile = [&] {
            ti = f8_tile<MODE>(p, at.q, at.nt, mt_start, offs, ti.g);
            at.next();
            valid = r_local < ti.rows;
            const int row = ti.row0 + r_local;
            if constexpr (MODE == FP8_WGRAD) return;
            if constexpr (MODE == FP8_FFN1) {
                sa = p.sa + (size_t)row * p.K_blocks;
                sb0 = p.sb + ((size_t)ti.g * p.nb_n + ti.nt) * p.K_blocks;
                sb1 = sb0 + (size_t)(p.I / 128) * p.K_blocks;
            } else {
                sa = p.sa + (size_t)row * p.K_blocks;
                const int nb = (ti.nt * BN + cl0) / kFp8Block;
                sb0 = p.sb + ((size_t)ti.g * p.nb_n + min(nb, p.nb_n - 1)) * p.K_blocks;
                nw = valid && p.row_w && row < p.w_rows ? __ldg(p.row_w + row) : 1.0f;
            }
            next_scales(0);
        };
        if ((int)blockIdx.x < total) begin_tile();
        for (int t = blockIdx.x; ok && t < total; t += gridDim.x, ++it) {
            uint64_t acc[CW / 2];
#pragma unroll
            for (int j = 0; j < CW / 2; ++j) acc[j] = 0;
            // CH columns at a time, the next ones (also those of the next block) on
            // their way from tensor memory during the products
            constexpr int NCH = CW / CH;
            uint32_t r[2][CH];
            const uint32_t tq = tmem_base + ((uint32_t)(q * 32) << 16) + cl0;
            if (ti.kb > 0) {
                ok = mbar_wait_warp(&tfull[blk % NACC], (blk / NACC) & 1u, wc);
                if (!ok) break;
                tc_fence_after();
                tmem_ld(tq + (blk % NACC) * BN, r[0]);
            }
            // block kb, its first chunk in r[b0]
            auto block = [&](int kb, auto b0c) {
                constexpr int b0 = decltype(b0c)::value;
                const float *cs = reinterpret_cast<const float *>(side) + sc * (128 + BN);
                float f0, f1;
                if constexpr (MODE == FP8_WGRAD) {
                    f0 = f1 = cs[r_local];
                    cs += 128 + cl0;
                    if (++sc == kF8Scales) sc = 0;
                } else {
                    f0 = na * nb0;
                    f1 = na * nb1;
                    if (kb + 1 < ti.kb) next_scales(kb + 1);
                }
                const uint64_t s0 = pair_f(f0, f0);
                const uint64_t s1 = MODE == FP8_FFN1 ? pair_f(f1, f1) : s0;
                float4 f[2][CH / 4];   // WGRAD: column scales of two chunks
                auto load_cs = [&](int c) {
#pragma unroll
                    for (int j = 0; j < CH / 4; ++j)
                        f[c & 1][j] = *reinterpret_cast<const float4 *>(cs + c * CH + 4 * j);
                };
                if constexpr (MODE == FP8_WGRAD) load_cs(0);
                const uint32_t a = blk++ % NACC;
#pragma unroll
                for (int c = 0; c < NCH; ++c) {
                    uint32_t(&now)[CH] = r[(b0 + c) & 1], (&next)[CH] = r[(b0 + c + 1) & 1];
                    tmem_wait_ld();
                    if (c < NCH - 1) {
                        constexpr int kPer = MODE == FP8_FFN1 ? NCH / 2 : NCH;   // to kHalf
                        tmem_ld(tq + a * BN + (c + 1) / kPer * kHalf + (c + 1) % kPer * CH, next);
                        if constexpr (MODE == FP8_WGRAD) load_cs(c + 1);
                    } else {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&tempty[a]);
                        if (kb + 1 < ti.kb) {
                            ok = mbar_wait_warp(&tfull[blk % NACC], (blk / NACC) & 1u, wc);
                            if (!ok) return;
                            tc_fence_after();
                            tmem_ld(tq + (blk % NACC) * BN, next);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < CH / 2; j += 2) {
                        uint64_t v0 = pair(now[2 * j], now[2 * j + 1]);
                        uint64_t v1 = pair(now[2 * j + 2], now[2 * j + 3]);
                        if constexpr (MODE == FP8_WGRAD) {
                            const float4 s = f[c & 1][j / 2];
                            v0 = mul2(v0, pair_f(s.x, s.y));
                            v1 = mul2(v1, pair_f(s.z, s.w));
                        }
                        const uint64_t s = MODE == FP8_FFN1 && c >= NCH / 2 ? s1 : s0;
                        fma2(acc[c * (CH / 2) + j], v0, s);
                        fma2(acc[c * (CH / 2) + j + 1], v1, s);
                    }
                }
            };
            for (int kb = 0; ok && kb < ti.kb;) {
                block(kb++, std::integral_constant<int, 0>());
                if (NCH % 2 == 1 && ok && kb < ti.kb) block(kb++, std::integral_constant<int, 1>());
            }
            if (!ok) break;
            const F8Tile cur = ti;
            const bool cur_valid = valid;
            const int row = cur.row0 + r_local;
            const float w = nw;
            if (t + (int)gridDim.x < total) begin_tile();
            if constexpr (MODE != FP8_FFN1) {
                // 128 bytes of each row at a time: through shared memory, from where one
                // thread's TMA store takes all 32 rows during the next tile; rows at a
                // group's end that are not 32 straight from the registers
                constexpr int EB = MODE == FP8_ROWS ? 2 : 4;   // bytes of a value
                constexpr int PC = 128 / EB;                   // values of a piece
                const int col0 = cur.nt * BN + cl0;
                const bool whole = SH::OUTS > 0 && q * 32 + 32 <= cur.rows;
                auto sixteen = [&](int i) {   // bytes 16 i .. of this thread's row
                    uint4 v;
                    if constexpr (MODE == FP8_ROWS) {
                        const uint64_t *a = acc + 4 * i;
                        v.x = pack_bf16x2(w * lo_f(a[0]), w * hi_f(a[0]));
                        v.y = pack_bf16x2(w * lo_f(a[1]), w * hi_f(a[1]));
                        v.z = pack_bf16x2(w * lo_f(a[2]), w * hi_f(a[2]));
                        v.w = pack_bf16x2(w * lo_f(a[3]), w * hi_f(a[3]));
                    } else {
                        const uint64_t *a = acc + 2 * i;
                        v = make_uint4((uint32_t)a[0], (uint32_t)(a[0] >> 32), (uint32_t)a[1],
                                       (uint32_t)(a[1] >> 32));
                    }
                    return v;
                };
                const size_t out_row = MODE == FP8_ROWS ? row : (size_t)cur.g * p.M + row;
                if (whole) {
                    constexpr int OUTS = SH::OUTS > 0 ? SH::OUTS : 1;
#pragma unroll
                    for (int s = 0; s < CW / PC; ++s) {
                        uint8_t *o = out_s + s % OUTS * kF8OutPiece;
                        // this buffer's last store has been read
                        if (lane == 0) bulk_wait_group_read<OUTS - 1>();
                        __syncwarp();
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            *reinterpret_cast<uint4 *>(o + lane * 128 + ((j ^ (lane & 7)) << 4)) =
                                sixteen(8 * s + j);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            if (col0 + PC * s < p.N)
                                tma_store_2d(&p.tmO, o, col0 + PC * s, (int)out_row);
                            bulk_commit_group();   // empty past the last column
                        }
                    }
                } else if (cur_valid) {
                    uint8_t *dst = (MODE == FP8_ROWS ? reinterpret_cast<uint8_t *>(p.out)
                                                     : reinterpret_cast<uint8_t *>(p.dW)) +
                                   (out_row * p.N + col0) * EB;
#pragma unroll
                    for (int i = 0; i < CW * EB / 16; ++i) {
                        const uint4 v = sixteen(i);
                        if (col0 + i * (16 / EB) < p.N)
                            st_global_v4(dst + 16 * i, v.x, v.y, v.z, v.w);
                    }
                }
            } else {
                // 64 h columns; the other half of the block's 128 is with the
                // warp of the same quadrant and the other part
                uint32_t amax = 0;
                float h[64];
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    h[2 * j] = swiglu_clamped_nan(lo_f(acc[j]), lo_f(acc[32 + j]), p.clamp);
                    h[2 * j + 1] = swiglu_clamped_nan(hi_f(acc[j]), hi_f(acc[32 + j]), p.clamp);
                    amax = max(amax, max(__float_as_uint(h[2 * j]) & 0x7FFFFFFFu,
                                         __float_as_uint(h[2 * j + 1]) & 0x7FFFFFFFu));
                }
                // two buffers in turn: a buffer is rewritten two tiles later,
                // after a barrier that follows its reads
                uint32_t *ex = reinterpret_cast<uint32_t *>(side) + (it & 1) * 256;
                ex[part * 128 + r_local] = amax;
                __syncwarp();
                if (lane == 0) mbar_arrive(xch);
                if (!mbar_wait_warp(xch, (uint32_t)it & 1u, wc)) break;
                amax = max(amax, ex[(part ^ 1) * 128 + r_local]);
                const Fp8Scale f = fp8_scale(amax);
                if (cur_valid) {
                    uint8_t *dst = p.hq + (size_t)row * p.I + cur.nt * 128 + cl0;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float *v = h + 16 * j + 4 * e;
                            w[e] = e4m3x4(v[0] * f.r, v[1] * f.r, v[2] * f.r, v[3] * f.r);
                        }
                        st_global_v4(dst + 16 * j, w[0], w[1], w[2], w[3]);
                    }
                    if (part == 0) p.hs[(size_t)row * (p.I / 128) + cur.nt] = f.s;
                }
            }
        }
    }

    // a thread's last pieces have left shared memory
    if (SH::OUTS > 0 && lane == 0) bulk_wait_group_all();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem_base, NACC * BN);
}

template <int MODE, int BN, int ST>
moe_status launch_fp8(Fp8Params &p, long long max_tiles, cudaStream_t st) {
    auto kern = fp8_gemm_kernel<MODE, BN, ST>;
    static bool attr_set[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
    if (dev < 0 || dev >= 64) return MOE_ERR_UNSUPPORTED;
    if (!attr_set[dev]) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kF8Smem) != cudaSuccess)
            return MOE_ERR_CUDA;
        attr_set[dev] = true;
    }
    static_assert(F8Shape<MODE, BN, ST>::smem(kMaxGroups) <= kF8Smem, "shared memory");
    if (max_tiles <= 0) return MOE_OK;
    p.status = device_status_ptr();
    if (!p.status) return MOE_ERR_CUDA;
    p.wait_limit = kWaitLimitCycles;
    const int grid = max_tiles < num_sms() ? (int)max_tiles : num_sms();
    return launch_early(kern, dim3(grid), kF8Threads, F8Shape<MODE, BN, ST>::smem(p.G), st, p);
}

}  // namespace

// Rows of A's boxes: no more than there are (the MMAs' other rows take whatever the
// stage holds, and what comes of them is not written).
static int box_rows(int max_rows) { return max_rows < 128 ? (max_rows + 7) & ~7 : 128; }

// Column width of a tile: wide ones read fewer operand bytes for a product, narrow
// ones spread over the SMs where there are few.  The least of (rounds of tiles over
// the SMs) x (cycles of a block of 128 along the contraction), the cycles measured with
// one round of tiles.  Widths 256 / 128 / 64 / 32 with 4096 x 4096 weights: 128 rows 17.9
// / 11.7 / 10.3 / 9.4 us, 512 rows 17.6 / 11.9 / 17.5 / 29.0, 1024 rows 18.0 / 20.2 / 32.0 /
// 48.5, 4096 rows 60.3 / 60.7 / 105 / 179; 288 rows in 9 groups, 4096 x 2048 weights: 15.4 /
// 14.9 / 17.2 / 27.8.  (The rule takes the fastest, in the last case the next.)
static int rows_bn(int max_rows, int G, int N) {
    // row tiles: one for each group, or half a tile more than its rows fill
    const int groups = G < max_rows ? G : max_rows;
    const long long filled = (max_rows + 127) / 128 + (groups - 1) / 2;
    const long long rows = filled > groups ? filled : groups;
    int best = 256;
    long long least = -1;
    const int width[4] = {256, 128, 64, 32}, cycles[4] = {850, 520, 384, 320};
    for (int i = 0; i < 4; ++i) {
        const long long tiles = rows * ((N + width[i] - 1) / width[i]);
        const long long cost = (tiles + num_sms() - 1) / num_sms() * cycles[i];
        if (least < 0 || cost < least) {
            least = cost;
            best = width[i];
        }
    }
    return best;
}

moe_status launch_fp8_matmul(const uint8_t *aq, const float *as, const int32_t *offsets, int G,
                             int max_rows, const uint8_t *bq, const float *bs, const float *row_w,
                             int w_rows, int N, int K, uint16_t *out, cudaStream_t st) {
    // A few rows of one matrix (calls in a graph, each on other weights than the one before,
    // from HBM): 6.1 us there against 8.9 here at 4096 x 4096 and one row,
    // 1.9 against 3.1 at 1024 x 512, 7.6 against 25 at 128 x 16384 (few tiles to spread),
    // 14.4 against 13.9 at 16384 x 4096; with 16 rows the products cost it as much as it
    // gains (8.7 against 8.9).
    if (G == 1 && max_rows <= 8)
        return launch_fp8_thin(aq, as, offsets, max_rows, bq, bs, row_w, w_rows, N, K, out, st);
    Fp8Params p;
    std::memset(&p, 0, sizeof p);
    const int BN = rows_bn(max_rows, G, N);
    p.a_rows = box_rows(max_rows);
    if (!encode_tmap_u8_2d(&p.tmA, aq, K, max_rows, K, 128, p.a_rows, 128) ||
        !encode_tmap_u8_2d(&p.tmB, bq, K, (uint64_t)G * N, K, 128, BN, 128) ||
        (BN >= 128 && !encode_tmap_bf16_2d(&p.tmO, out, N, max_rows, 2ULL * N, 64, 32)))
        return MOE_ERR_CUDA;
    p.offsets = offsets;
    p.sa = as;
    p.sb = bs;
    p.G = G;
    p.N = N;
    p.max_rows = max_rows;
    p.K_blocks = fp8_blocks(K);
    p.nb_n = fp8_blocks(N);
    p.n_tiles = (N + BN - 1) / BN;
    p.row_w = row_w;
    p.w_rows = w_rows;
    p.out = out;
    const long long tiles = (long long)row_tile_bound(max_rows, G) * p.n_tiles;
    switch (BN) {
    case 256: return launch_fp8<FP8_ROWS, 256, 3>(p, tiles, st);
    case 128: return launch_fp8<FP8_ROWS, 128, 5>(p, tiles, st);
    case 64: return launch_fp8<FP8_ROWS, 64, 7>(p, tiles, st);
    default: return launch_fp8<FP8_ROWS, 32, 8>(p, tiles, st);
    }
}

moe_status launch_fp8_ffn1(const uint8_t *xq, const float *xs, const int32_t *offsets, int G,
                           int max_rows, const uint8_t *W13q, const float *W13s, int d, int I,
                           float clamp, uint8_t *hq, float *hs, cudaStream_t st) {
    Fp8Params p;
    std::memset(&p, 0, sizeof p);
    p.a_rows = box_rows(max_rows);
    if (!encode_tmap_u8_2d(&p.tmA, xq, d, max_rows, d, 128, p.a_rows, 128) ||
        !encode_tmap_u8_2d(&p.tmB, W13q, d, (uint64_t)G * 2 * I, d, 128, 128, 128))
        return MOE_ERR_CUDA;
    p.offsets = offsets;
    p.sa = xs;
    p.sb = W13s;
    p.G = G;
    p.N = 2 * I;
    p.I = I;
    p.max_rows = max_rows;
    p.K_blocks = d / 128;
    p.nb_n = 2 * I / 128;
    p.n_tiles = I / 128;
    p.clamp = clamp;
    p.hq = hq;
    p.hs = hs;
    return launch_fp8<FP8_FFN1, 256, 4>(p, (long long)row_tile_bound(max_rows, G) * p.n_tiles, st);
}

moe_status launch_fp8_wgrad(const uint8_t *aq, const float *as, const uint8_t *bq, const float *bs,
                            const int32_t *first, int G, int max_chunks, int M, int N, float *dW,
                            cudaStream_t st) {
    constexpr int BN = 256;
    Fp8Params p;
    std::memset(&p, 0, sizeof p);
    p.a_rows = 128;
    if (!encode_tmap_u8_2d(&p.tmA, aq, 128, (uint64_t)max_chunks * M, 128, 128, 128, 128) ||
        !encode_tmap_u8_2d(&p.tmB, bq, 128, (uint64_t)max_chunks * N, 128, 128, BN, 128) ||
        !encode_tmap_f32_2d(&p.tmO, dW, N, (uint64_t)G * M, 4ULL * N, 32, 32))
        return MOE_ERR_CUDA;
    p.offsets = first;
    p.sa = as;
    p.sb = bs;
    p.G = G;
    p.M = M;
    p.N = N;
    p.n_tiles = (N + BN - 1) / BN;
    p.dW = dW;
    return launch_fp8<FP8_WGRAD, BN, 3>(p, (long long)G * ((M + 127) / 128) * p.n_tiles, st);
}

}  // namespace moe
