// gemm_mx4.cu -- grouped matmuls with MXFP4 weights: E2M1 elements, one E8M0 scale for
// each 32 along the contraction (OCP MX v1.0), on the block-scaled tensor-core MMAs.
//
//   ROWS   out[r, n] = w_r A[r] . B[g][n]                                         bf16
//   FFN1   the same for the gate and up rows of W13, then the clamped SwiGLU and its
//          quantisation to MXFP8 along I
//   rows A MXFP4 (kind::mxf4, 64 elements a step) or MXFP8 (kind::mxf8f6f4, 32 elements a
//          step, the weights expanded to a byte each on their way into shared memory)
// ("DeepSeek-V4昇腾训练支持：基于 CANN 平台的TorchTitan-NPU + AutoFuse 极简训练优化实践",
// 性能结果与未来展望: A8W4, MxFP8 and MxFP4 as next steps.)
//
// The tensor cores apply the scales: every product is exact, the sums are fp32.  A stage
// is 128 bytes of each row's codes: 256 elements (4 bits) or 128 (8 bits).  The scales of
// 512 elements of a row are 16 bytes: a warp for each 128 rows of A or B loads them three
// slots of 512 elements ahead, turns them in registers into four blocks of 32 x 16 bytes
// (one for each word of four scales) and writes those to shared memory; the thread that
// issues a stage's MMAs first copies its blocks into tensor memory (tcgen05.cp, which the
// MMAs behind it wait for).  (Rows of 16 bytes by TMA take it about five cycles each: 8192
// rows over 8 groups, 4864 x 4096, 80 us, and 61 without the codes' copies.)
//
// One CTA per SM, persistent, 13 warps: warp 0 TMA producer, warp 1 tensor memory owner
// and MMA issuer, warps 2-4 the scales, warps 5-12 epilogue (thread = row; two warps
// per lane quadrant, half of the columns each).  Where groups hold many rows two CTAs form
// a pair (CL = 2): MMAs of 256 rows, each CTA with its 128 rows of A and half of B in
// shared memory, so that a stage brings 32 KB instead of 48 into each SM; the even CTA
// issues, the scales of all of B are in both.
//
// Tensor memory: two accumulators.  Of 256 columns two and the scales do not fit: the
// second begins where the first still has its last columns (48, or 24 with 8-bit rows), and
// the epilogue reads those first, so that the next tile's MMAs wait for them alone.
//
// Measured, 8192 rows of one group, 4864 x 4096 weights: 52 us with 4-bit rows (6.3 PFLOP/s; the
// MMAs alone 39), 92 with 8-bit ones (3.6; 73 alone): an SM takes in about 64 bytes a cycle, a
// pair's stage is 32 KB (24 with 8-bit rows), and a tile's output costs about a microsecond of
// that.  One row of 4096 x 4096 5.8 us, 33 x 4096 x 2048 weights for a row each 25.4 (HBM needs
// 21.7): an MMA of 128 rows takes about 72 cycles however few its columns are, as long as its
// rows need out of shared memory.  (So the weights as its rows and few token rows as its
// columns was no faster: 9 groups of 86 rows, the FFN 58 us against 44.  Two steps of K to a
// stage where tiles are narrow: 8-bit rows 32 wide 25.5 -> 22.0 us, 128 wide 11.6 -> 11.8,
// 4-bit rows 128 wide 59 -> 70.)
//
// Every wait is bounded; on a timeout the CTA records MOE_ERR_TIMEOUT, drains its copies
// and MMAs, frees tensor memory and returns.
#include <cstring>

#include "fp8_common.cuh"
#include "gemm_launch.cuh"
#include "mx_common.cuh"

namespace moe {
namespace {

enum Mx4Mode : int { MX4_ROWS = 0, MX4_FFN1 = 1 };

struct Mx4Params {
    CUtensorMap tmA;    // A codes, 128 bytes of a row at a time, boxes of a_rows rows
    CUtensorMap tmB;    // B codes, boxes of BN rows (FFN1: BN / 2)
    CUtensorMap tmO;    // ROWS: output, boxes of 32 rows x 32 columns
    const uint8_t *sa, *sb;          // scale rows of A and B, `pitch` bytes each
    int pitch;
    long long b_rows;
    const int32_t *offsets;
    int G, N, blocks, kb, n_tiles;   // blocks of 32 along K; stages of a tile
    int max_rows, a_rows;
    int I;
    float clamp;
    const float *row_w;
    int w_rows;
    uint16_t *out;      // ROWS
    uint8_t *hq, *hsf;  // FFN1: MXFP8 h [rows, I] and its scales
    int h_pitch;
    int *status;
    long long wait_limit;
};

constexpr int kScale0 = 2;                       // scale warps
constexpr int kEpi0 = 5, kEpi = 8;               // epilogue warps
constexpr int kAhead = 3;                        // slots of scales on their way in registers
constexpr int kThreads = 32 * (kEpi0 + kEpi);
constexpr int kCodeA = 128 * 128;
constexpr int kSfRegion = 128 * 16;              // scales of 512 elements of 128 rows
constexpr int kBars = 512;
constexpr int kSmem = 232448;                    // of a CTA at most
constexpr int kWideGroups = 700;                 // whose tables fit beside 256-wide stages
constexpr int kPiece = 32 * 64;                  // 32 rows x 32 bf16 on their way out

template <int MODE, int AB, int BN, int ST, int CL>
struct Shape {
    static constexpr int STAGE = kCodeA + BN / CL * 128;
    static constexpr int WORDS = AB == 4 ? 2 : 1;        // scale words of a row in a stage
    static constexpr int SPS = 4 / WORDS;                // stages of a scale slot
    static constexpr int NB = (BN + 127) / 128;
    static constexpr int SLOT = (1 + NB) * kSfRegion;
    // tensor memory: two accumulators, then two stages' scales
    static constexpr int SFC = WORDS * 4 * (1 + NB);
    static constexpr int SF0 = 512 - 2 * SFC;
    static constexpr int ACC1 = BN == 256 ? SF0 - 256 : BN;   // first column of the second
    static constexpr int OVER = BN == 256 ? 256 - ACC1 : 0;   // columns that they share
    static constexpr bool TMA_OUT = MODE == MX4_ROWS && BN >= 64;
    static constexpr int OUT = TMA_OUT ? kEpi * kPiece : 0;
    static constexpr int TABLES = 8 * ((BN == 256 ? kWideGroups : kMaxGroups) + 2);
    static constexpr int SLOTS = ST * STAGE > 192 * 1024 - 1 ? 2 : 4;   // of scales
    static constexpr int FIXED = ST * STAGE + SLOTS * SLOT + OUT + kBars;
    static constexpr int smem(int G) { return 1024 + FIXED + 8 * (G + 2); }
    static_assert(1024 + FIXED + TABLES <= kSmem, "shared memory");
    static_assert(ACC1 + BN <= SF0 && OVER <= 64, "tensor memory");
    static_assert((2 * ST + 2 * SLOTS + 6) * 8 + 16 <= kBars, "barriers");
    static_assert(CL == 1 || BN == 256, "pairs");
};

struct Tile {
    int g, nt, row0, rows;
};

// The tiles of a CTA (or pair), as far apart as there are of them: tile t = q n_tiles + nt.
struct Walk {
    int q, nt, dq, dn, n;
    __device__ Walk(int n_tiles, int first, int step)
        : q(first / n_tiles), dq(step / n_tiles), n(n_tiles) {
        nt = first - q * n;
        dn = step - dq * n;
    }
    __device__ void next() {
        q += dq;
        nt += dn;
        if (nt >= n) { nt -= n; ++q; }
    }
};

// Row tile q (of CL x 128 rows), found by a whole warp: the last group that starts at or
// before it, 32 groups a ballot from the group of the tile before (empty groups start where
// the next one does).
template <int CL>
__device__ __forceinline__ Tile find_tile(const Mx4Params &p, int q, int nt, const int *mt_start,
                                          const int *offs, int from, int rank) {
    int g = from;
    while (true) {
        const int i = g + 1 + (threadIdx.x & 31);
        const unsigned m = __ballot_sync(0xffffffffu, i < p.G && mt_start[min(i, p.G)] <= q);
        g += __popc(m);
        if (m != 0xffffffffu) break;
    }
    Tile ti;
    ti.g = g;
    ti.nt = nt;
    ti.row0 = offs[g] + ((q - mt_start[g]) * CL + rank) * 128;
    ti.rows = min(128, offs[g + 1] - ti.row0);   // (none: a pair's second half)
    return ti;
}

// tcgen05 instructions of one thread, elected inside each: called by a whole warp in uniform
// control flow, where descriptors and addresses stay in uniform registers.  (Inside a
// branch for the one thread a stage's instructions took the warp up to 400 cycles, as long
// as narrow tiles' MMAs.)  CL = 2: the forms of a pair of CTAs.

// 32 rows of 16 bytes (row j: the scale words of rows j, 32 + j, 64 + j and 96 + j of an
// operand) to four columns of each lane quadrant, as the block-scaled MMAs read them; a pair:
// in both CTAs, each from its own shared memory.  In order with the MMAs of the thread.
template <int CL>
__device__ __forceinline__ void cp_scales(uint32_t taddr, uint64_t desc) {
    if constexpr (CL == 2)
        asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
                     "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr),
                     "l"(desc)
                     : "memory");
    else
        asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
                     "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr),
                     "l"(desc)
                     : "memory");
}

// Descriptor of those 512 bytes (no swizzle, groups of eight rows 128 bytes apart).
__device__ __forceinline__ uint64_t sdesc_scales(uint32_t saddr) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(128u >> 4) << 32) | ((uint64_t)1 << 46);
}

// D[tmem] (+)= (A[smem] * SFA) (B[smem] * SFB)^T, fp32.  AB = 4: E2M1 operands, two elements
// a byte (K = 64, 32 bytes), two E8M0 scales of each row.  AB = 8: E4M3 rows and E2M1
// weights, in shared memory sixteen elements in eight bytes and eight bytes of padding (K =
// 32, 32 bytes), one scale.  Of a pair: M = 256, A's scales of its own rows in each CTA.
#define MOE_MX4_MMA(GROUP, KIND)                                                               \
    asm volatile(                                                                              \
        "{\n\t.reg .pred e, p;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %6, 0;\n\t"      \
        "@e tcgen05.mma.cta_group::" GROUP "." KIND " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::\
            "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(more)                  \
        : "memory")
template <int AB, int CL>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                    uint32_t sfa, uint32_t sfb, uint32_t more) {
    if constexpr (AB == 4 && CL == 2) MOE_MX4_MMA("2", "kind::mxf4.block_scale.scale_vec::2X");
    else if constexpr (AB == 4) MOE_MX4_MMA("1", "kind::mxf4.block_scale.scale_vec::2X");
    else if constexpr (CL == 2) MOE_MX4_MMA("2", "kind::mxf8f6f4.block_scale.scale_vec::1X");
    else MOE_MX4_MMA("1", "kind::mxf8f6f4.block_scale.scale_vec::1X");
}
#undef MOE_MX4_MMA

// The instruction descriptor of a stage's i-th MMA: A / B format [7,10) / [10,13), E2M1 = 1
// where both are packed, E4M3 = 0 and E2M1 = 5 otherwise; N >> 3 at [17,23); scale format
// [23] = 1 (E8M0); M >> 4 at [24,29) (packed: M >> 7 at [27,29)); which scale byte (packed:
// pair of bytes) of each word, B's at [4,6) and A's at [29,31); K-major operands.
template <int AB>
__host__ __device__ constexpr uint32_t mma_desc(int M, int N, int i) {
    const uint32_t byte = AB == 4 ? i % 2 * 2 : i;
    return (byte << 4) | (AB == 4 ? (1u << 7) | (1u << 10) : 5u << 10) |
           ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 4) << 24) | (byte << 29);
}

// Arrives on `bar` (a pair: at the same place in both CTAs) when all before has completed.
template <int CL>
__device__ __forceinline__ void commit(uint64_t *bar) {
    if constexpr (CL == 2)
        asm volatile(
            "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
            "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::"
            "cluster.b64 [%0], %1;\n\t}" ::"r"(smem_u32(bar)),
            "h"((uint16_t)0x3)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
            "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::
                "r"(smem_u32(bar))
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

template <int MODE, int AB, int BN, int ST, int CL>   // ST: stages of codes in shared memory
__global__ void __launch_bounds__(kThreads, 1) mx4_gemm_kernel(const __grid_constant__ Mx4Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    using SH = Shape<MODE, AB, BN, ST, CL>;
    uint8_t *sf = smem + ST * SH::STAGE;
    uint8_t *out_s = sf + SH::SLOTS * SH::SLOT;
    uint64_t *full = reinterpret_cast<uint64_t *>(out_s + SH::OUT);
    uint64_t *empty = full + ST;
    uint64_t *sfready = empty + ST;          // a slot's scales are there
    uint64_t *sfempty = sfready + SH::SLOTS; // ... and copied into tensor memory
    uint64_t *tfull = sfempty + SH::SLOTS;   // [2]
    uint64_t *tempty = tfull + 2;           // [2]
    uint64_t *tover = tempty + 2;           // a tile's shared columns have been read
    uint64_t *done = tover + 1;
    uint32_t *tmem_base_s = reinterpret_cast<uint32_t *>(done + 1);
    volatile int *abort_s = reinterpret_cast<volatile int *>(tmem_base_s + 1);
    int *offs = reinterpret_cast<int *>(out_s + SH::OUT + kBars);
    int *mt_start = offs + (p.G + 1);

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);   // uniform, to the compiler too
    const int lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < ST; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < SH::SLOTS; ++s) {
            mbar_init(&sfready[s], 1 + SH::NB);
            mbar_init(&sfempty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&tfull[a], 1);
            mbar_init(&tempty[a], kEpi * CL);
        }
        mbar_init(tover, kEpi / 2 * CL);
        mbar_init(done, 1);
        *abort_s = 0;
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&p.tmA);
        tma_prefetch_desc(&p.tmB);
    }
    if (warp == 1) {
        if constexpr (CL == 2) {
            tmem_alloc_pair(tmem_base_s, 512);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(tmem_base_s, 512);
            tmem_relinquish();
        }
    }
    wait_for_kernels_ahead();
    if (warp == 2) {
        // group offsets and the exclusive prefix of their row tiles
        int carry = 0;
        for (int base = 0; base <= p.G; base += 32) {
            const int g = base + lane;
            int o = 0, mt = 0;
            bool ok = true;
            if (g <= p.G) {
                offs[g] = o = row_offset(p.offsets[g], p.max_rows);
                ok = o == p.offsets[g];
            }
            if (g < p.G) {
                const int end = row_offset(p.offsets[g + 1], p.max_rows);
                ok = ok && end >= o;
                mt = max(0, (end - o + 128 * CL - 1) / (128 * CL));
            }
            if (!ok && blockIdx.x == 0) record_status(p.status, MOE_ERR_INVALID_ARG);
            int incl = mt;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d) incl += v;
            }
            if (g <= p.G) mt_start[g] = carry + incl - mt;
            carry += __shfl_sync(0xffffffffu, incl, 31);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // a pair's commits and arrivals reach both CTAs' barriers, initialised by now
    if constexpr (CL == 2) cluster_sync_all();
    let_kernels_behind_begin();

    const int rank = CL == 2 ? (int)cluster_ctarank() : 0;
    const int first = blockIdx.x / CL, step = gridDim.x / CL;
    const uint32_t tmem_base = *tmem_base_s;
    const WaitCtl wc{abort_s, p.status, p.wait_limit};
    const long long total = (long long)mt_start[p.G] * p.n_tiles;

    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        uint32_t s = 0, ph = 0;
        uint32_t begun = 0;   // stages with a copy, and its parity
        bool ok = true;
        int g = 0;
        uint32_t j = 0, jph = 0;   // scale slot
        Walk at(p.n_tiles, first, step);
        for (long long t = first; ok && t < total; t += step, at.next()) {
            const Tile ti = find_tile<CL>(p, at.q, at.nt, mt_start, offs, g, rank);
            g = ti.g;
            // B's first row; FFN1: of the gate, whose up row is I further on
            const int br = MODE == MX4_FFN1 ? g * 2 * p.I + ti.nt * (BN / 2) : g * p.N + ti.nt * BN;
            for (int kb = 0; kb < p.kb; ++kb) {
                if (!mbar_wait_warp(&empty[s], ph ^ 1u, wc)) { ok = false; break; }
                // A pair's odd CTA: its scales of a slot are in its shared memory before the
                // slot's first codes are asked for, whose arrival in the even CTA, which
                // issues the pair's MMAs, so tells of both.  (An arrival of its own there,
                // released at cluster scope, takes a warp a microsecond, more than a slot
                // lasts: 12345 rows of 33 groups 66.7 us, by two more warps in turn 56.8, so
                // 55.1; the long FFN 609, 627 and 590.)
                if (CL == 2 && rank == 1 && kb % SH::SPS == 0) {
                    if (!mbar_wait_warp(&sfready[j], jph, wc)) { ok = false; break; }
                    if (++j == SH::SLOTS) { j = 0; jph ^= 1u; }
                }
                if (lane == 0) {
                    uint8_t *a = smem + s * SH::STAGE;
                    uint8_t *b = a + kCodeA;
                    // Coordinates count elements: bytes for packed pairs, 4-bit elements where
                    // the copy expands them (which counts the bytes that it reads).  A pair's
                    // copies all arrive on the even CTA's barrier.
                    if (CL == 1 || rank == 0)
                        mbar_arrive_expect_tx(&full[s], CL * (p.a_rows * 128 +
                                                              BN / CL * (AB == 4 ? 128 : 64)));
                    if (CL == 2 && rank == 1) {
                        const uint32_t bar = dsmem_map(&full[s], 0);
                        tma_load_2d_pairbar(a, &p.tmA, bar, kb * 128, ti.row0);
                        tma_load_2d_pairbar(b, &p.tmB, bar, kb * 128,
                                            br + (MODE == MX4_FFN1 ? p.I : BN / 2));
                    } else {
                        tma_load_2d(a, &p.tmA, &full[s], kb * 128, ti.row0);
                        tma_load_2d(b, &p.tmB, &full[s], kb * 128, br);
                        if constexpr (MODE == MX4_FFN1 && CL == 1)
                            tma_load_2d(b + BN / 2 * 128, &p.tmB, &full[s], kb * 128, br + p.I);
                    }
                }
                begun = (begun & ~(0x10001u << s)) | (0x10000u << s) | (ph << s);
                if (++s == ST) { s = 0; ph ^= 1u; }
            }
        }
        if (!ok) {
            // drain the copies still in flight before the CTA exits
            if (CL == 2 && rank == 1) {
                // (those of codes arrive on the even CTA's barriers, which this one cannot
                // wait on: a copy takes microseconds, this about a millisecond)
                const long long t0 = clock64();
                while (clock64() - t0 < (1LL << 21)) __nanosleep(1000);
            } else {
                for (int i = 0; i < ST; ++i)
                    if (begun >> (16 + i) & 1u)
                        mbar_wait_teardown(&full[i], begun >> i & 1u, p.wait_limit);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer
        const uint64_t ad0 = sdesc_sw128(smem_u32(smem), 16, 1024);
        const uint64_t sd0 = sdesc_scales(smem_u32(sf));
        uint32_t s = 0, ph = 0, j = 0, jph = 0, turn = 0;
        int it = 0;
        bool ok = true;
        for (long long t = first; rank == 0 && ok && t < total; t += step, ++it) {
            if (!mbar_wait_warp(&tempty[it & 1], ((it >> 1) & 1u) ^ 1u, wc) ||
                (SH::OVER > 0 && it > 0 && !mbar_wait_warp(tover, (it - 1) & 1u, wc))) {
                ok = false;
                break;
            }
            const uint32_t d = tmem_base + (it & 1) * SH::ACC1;
            for (int kb = 0; kb < p.kb; ++kb) {
                const int w0 = kb % SH::SPS * SH::WORDS;   // first word of the slot's rows
                if ((w0 == 0 && !mbar_wait_warp(&sfready[j], jph, wc)) ||
                    !(CL == 2 && w0 == 0 ? mbar_wait_cluster_warp(&full[s], ph, wc)
                                         : mbar_wait_warp(&full[s], ph, wc))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const bool last = kb + 1 == p.kb;
                const bool slot_done = last || w0 + SH::WORDS == 4;
                const uint64_t ad = ad0 + s * (SH::STAGE / 16), bd = ad + kCodeA / 16;
                const uint64_t sd = sd0 + j * (SH::SLOT / 16) + w0 * 32;
                const uint32_t sfa = tmem_base + SH::SF0 + turn * SH::SFC;
#pragma unroll
                for (int w = 0; w < SH::WORDS; ++w)
#pragma unroll
                    for (int r = 0; r < 1 + SH::NB; ++r)
                        cp_scales<CL>(sfa + 4 * (w * (1 + SH::NB) + r),
                                      sd + w * 32 + r * (kSfRegion / 16));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t sa = AB == 4 ? sfa + i / 2 * 4 * (1 + SH::NB) : sfa;
                    mma<AB, CL>(d, ad + 2 * i, bd + 2 * i, mma_desc<AB>(128 * CL, BN, i), sa, sa + 4,
                                (kb | i) != 0 ? 1u : 0u);
                }
                commit<CL>(&empty[s]);
                if (slot_done) commit<CL>(&sfempty[j]);
                if (last) commit<CL>(&tfull[it & 1]);
                turn ^= 1u;
                if (slot_done && ++j == SH::SLOTS) { j = 0; jph ^= 1u; }
                if (++s == ST) { s = 0; ph ^= 1u; }
            }
        }
        if (rank == 0 && (CL == 2 || !ok)) {
            // every MMA of this thread must finish before TMEM is freed (a pair's, before
            // either CTA's operands go away)
            commit<CL>(done);
            mbar_wait_teardown(done, 0, p.wait_limit);
        }
    } else if (warp < kEpi0) {
        // ------------------------------------------------ scales
        // Warp m: the region of 128 rows of A (m = 0) or of B.  Row 32 c + l is lane l's
        // v[c]; its word w goes to word c of row l of block w.
        const int m = warp - kScale0;
        uint32_t j = 0, jph = 0;
        Walk at(p.n_tiles, first, step);
        int g = 0, slot = 0;
        const int slots = (p.blocks + 15) / 16;
        long long t = first;
        const uint8_t *src[4];
        // the rows of tile t (rows that are not there: any others, for products that go
        // nowhere)
        auto rows_of_tile = [&] {
            if (t >= total) return;
            const Tile ti = find_tile<CL>(p, at.q, at.nt, mt_start, offs, g, rank);
            g = ti.g;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if (m == 0) {
                    src[c] = p.sa + (size_t)min(ti.row0 + 32 * c + lane, p.max_rows - 1) * p.pitch;
                } else {
                    long long r;
                    if constexpr (MODE == MX4_FFN1) {
                        const int i = (m - 1) * 128 + 32 * c;   // of the tile's B rows
                        r = (long long)g * 2 * p.I + ti.nt * (BN / 2) + i % (BN / 2) +
                            (i >= BN / 2 ? p.I : 0) + lane;
                    } else {
                        r = (long long)g * p.N + ti.nt * BN + (m - 1) * 128 + 32 * c + lane;
                    }
                    src[c] = p.sb + (size_t)min(r, p.b_rows - 1) * p.pitch;
                }
            }
        };
        uint4 v[kAhead][4];
        int at_slot[kAhead];   // slot of the row that v[.] holds, or -1 behind the last tile
        auto load = [&](int i) {
            at_slot[i] = -1;
            if (t >= total) return;
            at_slot[i] = slot;
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (m == 0 || 32 * c < BN)
                    v[i][c] = __ldg(reinterpret_cast<const uint4 *>(src[c]) + slot);
                else
                    v[i][c] = make_uint4(0, 0, 0, 0);
            if (++slot == slots) {
                slot = 0;
                t += step;
                at.next();
                rows_of_tile();
            }
        };
        if (m < 1 + SH::NB) {
            rows_of_tile();
#pragma unroll
            for (int i = 0; i < kAhead; ++i) load(i);
            bool ok = true;
            while (ok) {
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    if (!ok || at_slot[i] < 0) { ok = false; continue; }
                    // scales behind the row's end (its padding may hold anything, a NaN too)
                    // multiply zeros: they become zeros
                    const int left = p.blocks - 16 * at_slot[i];
                    uint32_t mask[4];
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const int n = min(4, max(0, left - 4 * w));
                        mask[w] = n == 4 ? 0xFFFFFFFFu : (1u << (8 * n)) - 1u;
                    }
                    ok = mbar_wait_warp(&sfempty[j], jph ^ 1u, wc);
                    if (!ok) continue;
                    const uint4(&x)[4] = v[i];
                    const uint32_t a = smem_u32(sf + j * SH::SLOT + m * kSfRegion) + lane * 16;
                    st_shared_v4(a, x[0].x & mask[0], x[1].x & mask[0], x[2].x & mask[0],
                                 x[3].x & mask[0]);
                    st_shared_v4(a + 512, x[0].y & mask[1], x[1].y & mask[1], x[2].y & mask[1],
                                 x[3].y & mask[1]);
                    st_shared_v4(a + 1024, x[0].z & mask[2], x[1].z & mask[2], x[2].z & mask[2],
                                 x[3].z & mask[2]);
                    st_shared_v4(a + 1536, x[0].w & mask[3], x[1].w & mask[3], x[2].w & mask[3],
                                 x[3].w & mask[3]);
                    fence_proxy_async_smem();   // the copies into tensor memory read them
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sfready[j]);
                    if (++j == SH::SLOTS) { j = 0; jph ^= 1u; }
                    load(i);
                }
            }
        }
    } else {
        // ------------------------------------------------ epilogue
        const int q = warp & 3;                // TMEM lane quadrant
        const int part = (warp - kEpi0) >> 2;  // its half of the columns
        const int r_local = q * 32 + lane;
        uint8_t *piece = out_s + (warp - kEpi0) * kPiece;
        // Up to 64 columns at a time: CN chunks of CH.  (FFN1: a chunk of gate columns and
        // the up columns that go with it.)
        constexpr int CW = BN / 2;                           // accumulator columns of this warp
        constexpr int CH = CW < 32 ? CW : 32, CN = CW < 64 ? 1 : 2, PH = CW / (CH * CN);
        int it = 0, g = 0;
        Walk at(p.n_tiles, first, step);
        auto arrive = [&](uint64_t *bar) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (rank == 0) mbar_arrive(bar);
                else mbar_arrive_remote_relaxed(dsmem_map(bar, 0));
            }
        };
        for (long long t = first; t < total; t += step, at.next(), ++it) {
            const Tile ti = find_tile<CL>(p, at.q, at.nt, mt_start, offs, g, rank);
            g = ti.g;
            const bool valid = r_local < ti.rows;
            const int row = ti.row0 + r_local;
            float w = 1.0f;
            if (MODE == MX4_ROWS && valid && p.row_w && row < p.w_rows) w = __ldg(p.row_w + row);
            if (!mbar_wait_warp(&tfull[it & 1], (it >> 1) & 1u, wc)) break;
            tc_fence_after();
            const uint32_t tb = tmem_base + ((uint32_t)(q * 32) << 16) + (it & 1) * SH::ACC1;
            // the columns that the next accumulator takes first: the last ones of the first
            // accumulator, the first ones of the second
            const bool down = SH::OVER > 0 && (it & 1) == 0;
#pragma unroll
            for (int i = 0; i < PH; ++i) {
                const int ph = down ? PH - 1 - i : i;
                const int c0 = MODE == MX4_FFN1 ? part * (CW / 2) + ph * CH
                                                : part * CW + ph * CN * CH;
                uint32_t r[CN][CH];
#pragma unroll
                for (int c = 0; c < CN; ++c)
                    tmem_ld(tb + c0 + c * (MODE == MX4_FFN1 ? BN / 2 : CH), r[c]);
                tmem_wait_ld();
                if (SH::OVER > 0 && i == 0 && part == (down ? 1 : 0)) arrive(tover);
                if (i == PH - 1) arrive(&tempty[it & 1]);
                if constexpr (MODE == MX4_FFN1) {
                    if (valid) {
                        float h[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            h[e] = swiglu_clamped_nan(__uint_as_float(r[0][e]),
                                                      __uint_as_float(r[CN - 1][e]), p.clamp);
                        uint32_t wq[8];
                        const uint32_t code = mx_quantize_block(h, wq);
                        const int col = ti.nt * (BN / 2) + c0;
                        uint8_t *dst = p.hq + (size_t)row * p.I + col;
                        st_global_v4(dst, wq[0], wq[1], wq[2], wq[3]);
                        st_global_v4(dst + 16, wq[4], wq[5], wq[6], wq[7]);
                        p.hsf[(size_t)row * p.h_pitch + col / 32] = (uint8_t)code;
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < CN; ++c) {
                        const int col = ti.nt * BN + c0 + c * CH;
                        uint32_t o[CH / 2];
#pragma unroll
                        for (int e = 0; e < CH / 2; ++e)
                            o[e] = pack_bf16x2(w * __uint_as_float(r[c][2 * e]),
                                               w * __uint_as_float(r[c][2 * e + 1]));
                        if (SH::TMA_OUT && q * 32 + 32 <= ti.rows) {
                            // through shared memory, from where one thread's TMA store takes
                            // all 32 rows
                            if (lane == 0) bulk_wait_group_read<0>();   // the last piece has left
                            __syncwarp();
                            const uint32_t sw = (uint32_t)((lane >> 1) & 3);
#pragma unroll
                            for (int e = 0; e < CH / 8; ++e)
                                st_shared_v4(smem_u32(piece) + lane * 64 + (((uint32_t)e ^ sw) << 4),
                                             o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0 && col < p.N) {
                                tma_store_2d(&p.tmO, piece, col, row);
                                bulk_commit_group();
                            }
                        } else if (valid) {
                            uint16_t *dst = p.out + (size_t)row * p.N + col;
#pragma unroll
                            for (int e = 0; e < CH / 8; ++e)
                                if (col + 8 * e < p.N)
                                    st_global_v4(dst + 8 * e, o[4 * e], o[4 * e + 1], o[4 * e + 2],
                                                 o[4 * e + 3]);
                        }
                    }
                }
            }
        }
        // a thread's last pieces have left shared memory
        if (SH::TMA_OUT && lane == 0) bulk_wait_group_all();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if constexpr (CL == 2) {
        // neither CTA leaves while the other may still signal it
        cluster_sync_all();
        if (warp == 1) tmem_dealloc_pair(tmem_base, 512);
        cluster_sync_all();
    } else {
        if (warp == 1) tmem_dealloc(tmem_base, 512);
    }
}

// max_tiles: upper bound of the tiles (of 128 CL rows).
template <int MODE, int AB, int BN, int ST, int CL>
moe_status launch_mx4(Mx4Params &p, long long max_tiles, cudaStream_t st) {
    using SH = Shape<MODE, AB, BN, ST, CL>;
    auto kern = mx4_gemm_kernel<MODE, AB, BN, ST, CL>;
    static int resident[64] = {};   // CTAs or pairs at once
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
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = CL == 1 ? 1 : 2;
    if (!resident[dev]) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) !=
            cudaSuccess)
            return MOE_ERR_CUDA;
        int n = num_sms();
        if (CL == 2 && (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1))
            return MOE_ERR_CUDA;
        resident[dev] = n;
    }
    if (max_tiles <= 0) return MOE_OK;
    p.status = device_status_ptr();
    if (!p.status) return MOE_ERR_CUDA;
    p.wait_limit = kWaitLimitCycles;
    const int n = max_tiles < resident[dev] ? (int)max_tiles : resident[dev];
    cfg.gridDim = dim3(n * CL);
    cfg.dynamicSmemBytes = SH::smem(p.G);
    if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) return MOE_ERR_CUDA;
    return cuda_status(cudaGetLastError());
}

// Rows of A's boxes: no more than there are (the MMAs' other rows take whatever the
// stage holds, and what comes of them is not written).
int box_rows(int max_rows) { return max_rows < 128 ? (max_rows + 7) & ~7 : 128; }

// The tile of a call: wide ones read fewer operand bytes for a product, narrow ones spread
// over the SMs where there are few; pairs of CTAs (256 rows) only where groups hold 256 rows
// on average, as a group's last pair is half empty more often than not.  The least of (rounds
// of tiles over the SMs) x (ns of a stage, measured with many rounds: 8192 x 4096 x 4096 in
// pairs 46 us, and 256 / 128 / 64 / 32 wide 54 / 59 / 95 / 182 with 4-bit rows, 76 and 83 / 106 /
// 162 / 298 with 8-bit ones).  4-bit rows, pairs 256 / 256 / 128 / 64 / 32 wide, us, the rule's
// choice in brackets: 1 row - / 8.6 / 7.0 / 6.6 / [6.2], 512 rows 10.8 / 10.4 / [7.6] / 10.1 / 16.0,
// 1024 rows [11.5] / 11.4 / 11.7 / 17.3 / 26.3, 1280 rows 16.4 / 17.5 / [15.2]; 4096 x 2048 weights of
// 33 groups: 500 rows 29.8 / 26.9 / [25.9] / 30.9 / 47.1, 6000 rows 40.9 / [35.8] / 40.5 / 54.7 / 96, 12345
// rows 55.1 / [52.9] / 61.2 / 87.3 / 158; of 9 groups, 288 rows 12.3 / [10.8] / 9.6 / 11.6 / 16.9 (not
// the fastest).
struct TileChoice {
    int bn;
    bool pair;
};
TileChoice tile_shape(int max_rows, int G, int N, int bits, int narrowest) {
    // row tiles: one for each group, or half a tile more than its rows fill
    const int groups = G < max_rows ? G : max_rows;
    const int width[5] = {256, 256, 128, 64, 32};
    const int ns[2][5] = {{430, 500, 270, 220, 210}, {354, 384, 246, 188, 173}};
    TileChoice best = {narrowest, false};
    long long least = -1;
    for (int i = 0; i < 5 && width[i] >= narrowest; ++i) {
        const bool pair = i == 0;
        const int rows = pair ? 256 : 128, units = pair ? num_sms() / 2 : num_sms();
        if ((pair && max_rows < 256LL * G) || (width[i] == 256 && G > kWideGroups)) continue;
        const long long filled = (max_rows + rows - 1) / rows + (groups - 1) / 2;
        const long long tiles =
            (filled > groups ? filled : groups) * ((N + width[i] - 1) / width[i]);
        const long long cost = (tiles + units - 1) / units * ns[bits == 8][i];
        if (least < 0 || cost < least) {
            least = cost;
            best = {width[i], pair};
        }
    }
    return best;
}

bool encode_operands(Mx4Params &p, int bits, const uint8_t *aq, const uint8_t *asf, int max_rows,
                     const uint8_t *bq, const uint8_t *bsf, uint64_t brows, int b_box, int K) {
    p.sa = asf;
    p.sb = bsf;
    p.pitch = mx_sf_pitch(K);
    p.b_rows = (long long)brows;
    p.max_rows = max_rows;
    p.a_rows = box_rows(max_rows);
    p.blocks = K / 32;
    p.kb = bits == 4 ? (K + 255) / 256 : K / 128;
    const int row = bits == 4 ? K / 2 : K;
    return encode_tmap_u8_2d(&p.tmA, aq, row, max_rows, row, 128, p.a_rows, 128) &&
           (bits == 4 ? encode_tmap_u8_2d(&p.tmB, bq, K / 2, brows, K / 2, 128, b_box, 128)
                      : encode_tmap_u4_expand_2d(&p.tmB, bq, K, brows, b_box));
}

}  // namespace

moe_status launch_mx4_matmul(const uint8_t *aq, const uint8_t *asf, int bits,
                             const int32_t *offsets, int G, int max_rows, const uint8_t *bq,
                             const uint8_t *bsf, const float *row_w, int w_rows, int N, int K,
                             uint16_t *out, cudaStream_t st) {
    Mx4Params p;
    std::memset(&p, 0, sizeof p);
    const TileChoice ts = tile_shape(max_rows, G, N, bits, 32);
    const int BN = ts.bn;
    const int b_box = ts.pair ? 128 : BN;
    if (!encode_operands(p, bits, aq, asf, max_rows, bq, bsf, (uint64_t)G * N, b_box, K) ||
        (BN >= 64 && !encode_tmap_bf16_2d_sw64(&p.tmO, out, N, max_rows, 2ULL * N, 32, 32)))
        return MOE_ERR_CUDA;
    p.offsets = offsets;
    p.G = G;
    p.N = N;
    p.n_tiles = (N + BN - 1) / BN;
    p.row_w = row_w;
    p.w_rows = w_rows;
    p.out = out;
    if (ts.pair) {
        const long long t = (long long)row_pair_bound(max_rows, G) * p.n_tiles;
        return bits == 4 ? launch_mx4<MX4_ROWS, 4, 256, 5, 2>(p, t, st)
                         : launch_mx4<MX4_ROWS, 8, 256, 6, 2>(p, t, st);
    }
    const long long tiles = (long long)row_tile_bound(max_rows, G) * p.n_tiles;
    if (bits == 4) {
        switch (BN) {
        case 256: return launch_mx4<MX4_ROWS, 4, 256, 4, 1>(p, tiles, st);
        case 128: return launch_mx4<MX4_ROWS, 4, 128, 5, 1>(p, tiles, st);
        case 64: return launch_mx4<MX4_ROWS, 4, 64, 7, 1>(p, tiles, st);
        default: return launch_mx4<MX4_ROWS, 4, 32, 8, 1>(p, tiles, st);
        }
    }
    switch (BN) {
    case 256: return launch_mx4<MX4_ROWS, 8, 256, 4, 1>(p, tiles, st);
    case 128: return launch_mx4<MX4_ROWS, 8, 128, 5, 1>(p, tiles, st);
    case 64: return launch_mx4<MX4_ROWS, 8, 64, 7, 1>(p, tiles, st);
    default: return launch_mx4<MX4_ROWS, 8, 32, 8, 1>(p, tiles, st);
    }
}

moe_status launch_mx4_ffn1(const uint8_t *xq, const uint8_t *xsf, const int32_t *offsets, int G,
                           int max_rows, const uint8_t *W13q, const uint8_t *W13sf, int d, int I,
                           float clamp, uint8_t *hq, uint8_t *hsf, cudaStream_t st) {
    Mx4Params p;
    std::memset(&p, 0, sizeof p);
    const TileChoice ts = tile_shape(max_rows, G, 2 * I, 8, 128);
    const int BN = ts.bn;
    if (!encode_operands(p, 8, xq, xsf, max_rows, W13q, W13sf, (uint64_t)G * 2 * I, BN / 2, d))
        return MOE_ERR_CUDA;
    p.offsets = offsets;
    p.G = G;
    p.N = 2 * I;
    p.I = I;
    p.n_tiles = 2 * I / BN;
    p.clamp = clamp;
    p.hq = hq;
    p.hsf = hsf;
    p.h_pitch = mx_sf_pitch(I);
    if (ts.pair)
        return launch_mx4<MX4_FFN1, 8, 256, 6, 2>(
            p, (long long)row_pair_bound(max_rows, G) * p.n_tiles, st);
    const long long tiles = (long long)row_tile_bound(max_rows, G) * p.n_tiles;
    return BN == 256 ? launch_mx4<MX4_FFN1, 8, 256, 4, 1>(p, tiles, st)
                     : launch_mx4<MX4_FFN1, 8, 128, 5, 1>(p, tiles, st);
}

}  // namespace moe
