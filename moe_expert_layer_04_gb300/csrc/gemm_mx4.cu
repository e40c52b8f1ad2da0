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
// 512 elements of a row are 16 bytes; they come by TMA as rows, a warp turns 128 rows of
// them in place into four blocks of 32 x 16 bytes (one for each word of four scales), and
// the thread that issues a stage's MMAs first copies its blocks into tensor memory
// (tcgen05.cp, which the MMAs behind it wait for).
//
// One CTA per SM, persistent, 12 warps: warp 0 TMA producer, warp 1 tensor memory owner
// and MMA issuer, warps 2 and 3 the scales, warps 4-11 epilogue (thread = row; two warps
// per lane quadrant, half of the columns each).  Every wait is bounded; on a timeout the
// CTA records MOE_ERR_TIMEOUT, drains its copies and MMAs, frees tensor memory and returns.
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
    CUtensorMap tmSA;   // scale rows [.., pitch], boxes of 16 bytes x a_rows
    CUtensorMap tmSB;   //                          16 bytes x BN (FFN1: BN / 2)
    CUtensorMap tmO;    // ROWS: output, boxes of 32 rows x 32 columns
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

constexpr int kEpi0 = 4, kEpi = 8;               // epilogue warps
constexpr int kThreads = 32 * (kEpi0 + kEpi);
constexpr int kCodeA = 128 * 128;
constexpr int kSfRegion = 128 * 16;              // scales of 512 elements of 128 rows
constexpr int kSfSlots = 2;
constexpr int kBars = 256;
constexpr int kSmem = 232448;                    // of a CTA at most
constexpr int kWideGroups = 700;                 // whose tables fit beside 256-wide stages
constexpr int kPiece = 32 * 64;                  // 32 rows x 32 bf16 on their way out

// Registers: the four warps that copy and issue hand most of theirs to the eight that
// hold a tile's results (128 a thread); 4 x 40 + 8 x 232 is what 12 x 168 launch with.
constexpr int kRegsFew = 40, kRegsMany = 232;
static_assert(4 * kRegsFew + 8 * kRegsMany <= 12 * 168, "register split");

template <int MODE, int AB, int BN, int ST>
struct Shape {
    static constexpr int STAGE = kCodeA + BN * 128;
    static constexpr int WORDS = AB == 4 ? 2 : 1;        // scale words of a row in a stage
    static constexpr int SPS = 4 / WORDS;                // stages of a scale slot
    static constexpr int NB = (BN + 127) / 128;
    static constexpr int SLOT = (1 + NB) * kSfRegion;
    static constexpr int NACC = BN == 256 ? 1 : 2;
    static constexpr int SF0 = NACC * BN;                // tensor memory: accumulators, then
    static constexpr int SFC = WORDS * 4 * (1 + NB);     // two stages' scales
    static constexpr bool TMA_OUT = MODE == MX4_ROWS && BN >= 64;
    static constexpr int OUT = TMA_OUT ? kEpi * kPiece : 0;
    static constexpr int FIXED = ST * STAGE + kSfSlots * SLOT + OUT + kBars;
    static constexpr int smem(int G) { return 1024 + FIXED + 8 * (G + 2); }
    static_assert(SF0 + 2 * SFC <= 512, "tensor memory");
    static_assert((2 * ST + 2 * kSfSlots + 3 * NACC + 2) * 8 + 16 <= kBars, "barriers");
};

struct Tile {
    int g, nt, row0, rows;
};

// The tiles of a CTA, gridDim.x apart: tile t = q n_tiles + nt.
struct Walk {
    int q, nt, dq, dn, n;
    __device__ explicit Walk(int n_tiles)
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

// Row tile q, found by a whole warp: the last group that starts at or before it, 32 groups
// a ballot from the group of the tile before (empty groups start where the next one does).
__device__ __forceinline__ Tile find_tile(const Mx4Params &p, int q, int nt, const int *mt_start,
                                          const int *offs, int from) {
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
    ti.row0 = offs[g] + (q - mt_start[g]) * 128;
    ti.rows = min(128, offs[g + 1] - ti.row0);
    return ti;
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

template <int MODE, int AB, int BN, int ST>   // ST: stages of codes in shared memory
__global__ void __launch_bounds__(kThreads, 1) mx4_gemm_kernel(const __grid_constant__ Mx4Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    using SH = Shape<MODE, AB, BN, ST>;
    constexpr int NACC = SH::NACC;
    uint8_t *sf = smem + ST * SH::STAGE;
    uint8_t *out_s = sf + kSfSlots * SH::SLOT;
    uint64_t *full = reinterpret_cast<uint64_t *>(out_s + SH::OUT);
    uint64_t *empty = full + ST;
    uint64_t *sffull = empty + ST;          // a slot's scale rows have come
    uint64_t *sfready = sffull + kSfSlots;  // ... and are turned
    uint64_t *sfempty = sfready + kSfSlots; // ... and copied into tensor memory
    uint64_t *tfull = sfempty + kSfSlots;
    uint64_t *tempty = tfull + NACC;
    uint64_t *done = tempty + NACC;
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
        for (int s = 0; s < kSfSlots; ++s) {
            mbar_init(&sffull[s], 1);
            mbar_init(&sfready[s], 2);
            mbar_init(&sfempty[s], 1);
        }
        for (int a = 0; a < NACC; ++a) {
            mbar_init(&tfull[a], 1);
            mbar_init(&tempty[a], kEpi);
        }
        mbar_init(done, 1);
        *abort_s = 0;
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&p.tmA);
        tma_prefetch_desc(&p.tmB);
        tma_prefetch_desc(&p.tmSA);
        tma_prefetch_desc(&p.tmSB);
    }
    if (warp == 1) {
        tmem_alloc(tmem_base_s, 512);
        tmem_relinquish();
    }
    wait_for_kernels_ahead();
    if (warp == 2) {
        // group offsets and the exclusive prefix of their 128-row tiles
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
                mt = max(0, (end - o + 127) >> 7);
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
    let_kernels_behind_begin();

    const uint32_t tmem_base = *tmem_base_s;
    const WaitCtl wc{abort_s, p.status, p.wait_limit};
    const long long total = (long long)mt_start[p.G] * p.n_tiles;

    if (warp < kEpi0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsFew));
    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        uint32_t s = 0, ph = 0, j = 0, jph = 0;
        uint32_t begun = 0, sf_begun = 0;   // stages and slots with a copy, and its parity
        bool ok = true;
        int g = 0;
        Walk at(p.n_tiles);
        for (long long t = blockIdx.x; ok && t < total; t += gridDim.x, at.next()) {
            const Tile ti = find_tile(p, at.q, at.nt, mt_start, offs, g);
            g = ti.g;
            const int br = MODE == MX4_FFN1 ? g * 2 * p.I + ti.nt * (BN / 2) : g * p.N + ti.nt * BN;
            for (int kb = 0; kb < p.kb; ++kb) {
                if (kb % SH::SPS == 0) {
                    if (!mbar_wait_warp(&sfempty[j], jph ^ 1u, wc)) { ok = false; break; }
                    if (lane == 0) {
                        uint8_t *a = sf + j * SH::SLOT;
                        uint8_t *b = a + kSfRegion;
                        const int x = kb / SH::SPS * 16;
                        mbar_arrive_expect_tx(&sffull[j], (p.a_rows + BN) * 16);
                        tma_load_2d(a, &p.tmSA, &sffull[j], x, ti.row0);
                        tma_load_2d(b, &p.tmSB, &sffull[j], x, br);
                        if constexpr (MODE == MX4_FFN1)
                            tma_load_2d(b + BN / 2 * 16, &p.tmSB, &sffull[j], x, br + p.I);
                    }
                    sf_begun = (sf_begun & ~(0x10001u << j)) | (0x10000u << j) | (jph << j);
                    if (++j == kSfSlots) { j = 0; jph ^= 1u; }
                }
                if (!mbar_wait_warp(&empty[s], ph ^ 1u, wc)) { ok = false; break; }
                if (lane == 0) {
                    uint8_t *a = smem + s * SH::STAGE;
                    uint8_t *b = a + kCodeA;
                    // (a copy that expands counts the bytes that it reads)
                    mbar_arrive_expect_tx(&full[s], p.a_rows * 128 + BN * (AB == 4 ? 128 : 64));
                    tma_load_2d(a, &p.tmA, &full[s], kb * 128, ti.row0);
                    // coordinates count elements: bytes for packed pairs, 4-bit elements
                    // where the copy expands them
                    tma_load_2d(b, &p.tmB, &full[s], kb * 128, br);
                    if constexpr (MODE == MX4_FFN1)
                        tma_load_2d(b + BN / 2 * 128, &p.tmB, &full[s], kb * 128, br + p.I);
                }
                begun = (begun & ~(0x10001u << s)) | (0x10000u << s) | (ph << s);
                if (++s == ST) { s = 0; ph ^= 1u; }
            }
        }
        if (!ok) {
            // drain the copies still in flight before the CTA exits
            for (int i = 0; i < ST; ++i)
                if (begun >> (16 + i) & 1u)
                    mbar_wait_teardown(&full[i], begun >> i & 1u, p.wait_limit);
            for (int i = 0; i < kSfSlots; ++i)
                if (sf_begun >> (16 + i) & 1u)
                    mbar_wait_teardown(&sffull[i], sf_begun >> i & 1u, p.wait_limit);
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer
        const uint64_t ad0 = sdesc_sw128(smem_u32(smem), 16, 1024);
        const uint64_t sd0 = sdesc_scales(smem_u32(sf));
        uint32_t s = 0, ph = 0, j = 0, jph = 0, turn = 0;
        int it = 0;
        bool ok = true;
        for (long long t = blockIdx.x; ok && t < total; t += gridDim.x, ++it) {
            const uint32_t acc = it % NACC, aph = (it / NACC) & 1u;
            if (!mbar_wait_warp(&tempty[acc], aph ^ 1u, wc)) { ok = false; break; }
            const uint32_t d = tmem_base + acc * BN;
            for (int kb = 0; kb < p.kb; ++kb) {
                const int w0 = kb % SH::SPS * SH::WORDS;   // first word of the slot's rows
                if (w0 == 0 && !mbar_wait_warp(&sfready[j], jph, wc)) { ok = false; break; }
                if (!mbar_wait_warp(&full[s], ph, wc)) { ok = false; break; }
                tc_fence_after();
                const bool last = kb + 1 == p.kb;
                const bool slot_done = last || w0 + SH::WORDS == 4;
                if (elect_one()) {
                    const uint64_t ad = ad0 + s * (SH::STAGE / 16), bd = ad + kCodeA / 16;
                    const uint64_t sd = sd0 + j * (SH::SLOT / 16) + w0 * 32;
                    const uint32_t sfa = tmem_base + SH::SF0 + turn * SH::SFC;
#pragma unroll
                    for (int w = 0; w < SH::WORDS; ++w) {
#pragma unroll
                        for (int r = 0; r < 1 + SH::NB; ++r)
                            tmem_cp_scales(sfa + w * 4 * (1 + SH::NB) + 4 * r,
                                           sd + w * 32 + r * (kSfRegion / 16));
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t more = (kb | i) != 0 ? 1u : 0u;
                        if constexpr (AB == 4) {
                            const uint32_t a = sfa + i / 2 * 4 * (1 + SH::NB);
                            umma_mxf4(d, ad + 2 * i, bd + 2 * i, idesc_mxf4_f32(128, BN, i % 2 * 2),
                                      a, a + 4, more);
                        } else {
                            umma_mxf8(d, ad + 2 * i, bd + 2 * i, idesc_mxf8_e2m1_f32(128, BN, i),
                                      sfa, sfa + 4, more);
                        }
                    }
                    umma_commit(&empty[s]);
                    if (slot_done) umma_commit(&sfempty[j]);
                    if (last) umma_commit(&tfull[acc]);
                }
                __syncwarp();
                turn ^= 1u;
                if (slot_done && ++j == kSfSlots) { j = 0; jph ^= 1u; }
                if (++s == ST) { s = 0; ph ^= 1u; }
            }
        }
        if (!ok) {
            // every MMA this thread issued must finish before TMEM is freed
            if (elect_one()) umma_commit(done);
            __syncwarp();
            mbar_wait_teardown(done, 0, p.wait_limit);
        }
    } else {
        // ------------------------------------------------ scales
        // Regions of 128 rows x 16 bytes (A, then B), one warp each in turn: word w of row
        // 32 c + l goes to byte 4 c of row l of block w.  In place: every lane has its four
        // rows in registers before the first is written.
        uint32_t j = 0, jph = 0;
        bool ok = true;
        for (long long t = blockIdx.x; ok && t < total; t += gridDim.x) {
            for (int k0 = 0; k0 < p.blocks; k0 += 16) {
                if (!mbar_wait_warp(&sffull[j], jph, wc)) { ok = false; break; }
                // scales behind the row's end (its padding may hold anything, a NaN too)
                // multiply zeros: they become zeros
                const int left = p.blocks - k0;
                uint32_t mask[4];
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const int n = min(4, max(0, left - 4 * w));
                    mask[w] = n == 4 ? 0xFFFFFFFFu : (1u << (8 * n)) - 1u;
                }
#pragma unroll
                for (int r = 0; r < 1 + SH::NB; ++r) {
                    if ((r & 1) != warp - 2) continue;
                    uint8_t *reg = sf + j * SH::SLOT + r * kSfRegion;
                    uint4 v[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        v[c] = *reinterpret_cast<const uint4 *>(reg + (32 * c + lane) * 16);
                    __syncwarp();
                    const uint32_t a = smem_u32(reg) + lane * 16;
                    st_shared_v4(a, v[0].x & mask[0], v[1].x & mask[0], v[2].x & mask[0],
                                 v[3].x & mask[0]);
                    st_shared_v4(a + 512, v[0].y & mask[1], v[1].y & mask[1], v[2].y & mask[1],
                                 v[3].y & mask[1]);
                    st_shared_v4(a + 1024, v[0].z & mask[2], v[1].z & mask[2], v[2].z & mask[2],
                                 v[3].z & mask[2]);
                    st_shared_v4(a + 1536, v[0].w & mask[3], v[1].w & mask[3], v[2].w & mask[3],
                                 v[3].w & mask[3]);
                }
                fence_proxy_async_smem();   // the copies into tensor memory read them
                __syncwarp();
                if (lane == 0) mbar_arrive(&sfready[j]);
                if (++j == kSfSlots) { j = 0; jph ^= 1u; }
            }
        }
    }
    } else {
        // ------------------------------------------------ epilogue
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsMany));
        const int q = warp & 3;                // TMEM lane quadrant
        const int part = (warp - kEpi0) >> 2;  // its half of the columns
        const int r_local = q * 32 + lane;
        uint8_t *piece = out_s + (warp - kEpi0) * kPiece;
        int it = 0, g = 0;
        Walk at(p.n_tiles);
        for (long long t = blockIdx.x; t < total; t += gridDim.x, at.next(), ++it) {
            const Tile ti = find_tile(p, at.q, at.nt, mt_start, offs, g);
            g = ti.g;
            const bool valid = r_local < ti.rows;
            const int row = ti.row0 + r_local;
            float w = 1.0f;
            if (MODE == MX4_ROWS && valid && p.row_w && row < p.w_rows) w = __ldg(p.row_w + row);
            const uint32_t acc = it % NACC, aph = (it / NACC) & 1u;
            if (!mbar_wait_warp(&tfull[acc], aph, wc)) break;
            tc_fence_after();
            const uint32_t tb = tmem_base + ((uint32_t)(q * 32) << 16) + acc * BN;
            auto release = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&tempty[acc]);
            };
            if constexpr (MODE == MX4_FFN1) {
                constexpr int HC = BN / 4;   // h columns of this warp
                uint32_t rg[HC / 32][32], ru[HC / 32][32];
#pragma unroll
                for (int c = 0; c < HC / 32; ++c) {
                    tmem_ld(tb + part * HC + 32 * c, rg[c]);
                    tmem_ld(tb + BN / 2 + part * HC + 32 * c, ru[c]);
                }
                tmem_wait_ld();
                release();
                if (valid) {
#pragma unroll
                    for (int c = 0; c < HC / 32; ++c) {
                        float h[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            h[i] = swiglu_clamped_nan(__uint_as_float(rg[c][i]),
                                                      __uint_as_float(ru[c][i]), p.clamp);
                        uint32_t wq[8];
                        const uint32_t code = mx_quantize_block(h, wq);
                        const int col = ti.nt * (BN / 2) + part * HC + 32 * c;
                        uint8_t *dst = p.hq + (size_t)row * p.I + col;
                        st_global_v4(dst, wq[0], wq[1], wq[2], wq[3]);
                        st_global_v4(dst + 16, wq[4], wq[5], wq[6], wq[7]);
                        p.hsf[(size_t)row * p.h_pitch + col / 32] = (uint8_t)code;
                    }
                }
            } else {
                constexpr int CW = BN / 2, CH = CW < 32 ? CW : 32;   // columns of this warp
                uint32_t o[CW / 2];
#pragma unroll
                for (int c = 0; c < CW / CH; ++c) {
                    uint32_t r[CH];
                    tmem_ld(tb + part * CW + CH * c, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < CH / 2; ++i)
                        o[c * (CH / 2) + i] = pack_bf16x2(w * __uint_as_float(r[2 * i]),
                                                          w * __uint_as_float(r[2 * i + 1]));
                }
                release();
                const int col0 = ti.nt * BN + part * CW;
                if (SH::TMA_OUT && q * 32 + 32 <= ti.rows) {
                    // 32 columns at a time through shared memory, from where one thread's
                    // TMA store takes all 32 rows
#pragma unroll
                    for (int c = 0; c < CW / CH; ++c) {
                        if (lane == 0) bulk_wait_group_read<0>();   // the last piece has left
                        __syncwarp();
                        const uint32_t sw = (uint32_t)((lane >> 1) & 3);
#pragma unroll
                        for (int i = 0; i < CH / 8; ++i)
                            st_shared_v4(smem_u32(piece) + lane * 64 + (((uint32_t)i ^ sw) << 4),
                                         o[c * (CH / 2) + 4 * i], o[c * (CH / 2) + 4 * i + 1],
                                         o[c * (CH / 2) + 4 * i + 2], o[c * (CH / 2) + 4 * i + 3]);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0 && col0 + CH * c < p.N) {
                            tma_store_2d(&p.tmO, piece, col0 + CH * c, row);
                            bulk_commit_group();
                        }
                    }
                } else if (valid) {
                    uint16_t *dst = p.out + (size_t)row * p.N + col0;
#pragma unroll
                    for (int i = 0; i < CW / 8; ++i)
                        if (col0 + 8 * i < p.N)
                            st_global_v4(dst + 8 * i, o[4 * i], o[4 * i + 1], o[4 * i + 2],
                                         o[4 * i + 3]);
                }
            }
        }
        // a thread's last pieces have left shared memory
        if (SH::TMA_OUT && lane == 0) bulk_wait_group_all();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem_base, 512);
}

template <int MODE, int AB, int BN, int ST>
moe_status launch_mx4(Mx4Params &p, long long max_tiles, cudaStream_t st) {
    using SH = Shape<MODE, AB, BN, ST>;
    auto kern = mx4_gemm_kernel<MODE, AB, BN, ST>;
    static bool attr_set[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
    if (dev < 0 || dev >= 64) return MOE_ERR_UNSUPPORTED;
    if (!attr_set[dev]) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) !=
            cudaSuccess)
            return MOE_ERR_CUDA;
        attr_set[dev] = true;
    }
    static_assert(SH::smem(BN == 256 ? kWideGroups : kMaxGroups) <= kSmem, "shared memory");
    if (max_tiles <= 0) return MOE_OK;
    p.status = device_status_ptr();
    if (!p.status) return MOE_ERR_CUDA;
    p.wait_limit = kWaitLimitCycles;
    const int grid = max_tiles < num_sms() ? (int)max_tiles : num_sms();
    return launch_early(kern, dim3(grid), kThreads, SH::smem(p.G), st, p);
}

// Rows of A's boxes: no more than there are (the MMAs' other rows take whatever the
// stage holds, and what comes of them is not written).
int box_rows(int max_rows) { return max_rows < 128 ? (max_rows + 7) & ~7 : 128; }

int rows_bn(int max_rows, int G, int N) {
    const int groups = G < max_rows ? G : max_rows;
    const long long filled = (max_rows + 127) / 128 + (groups - 1) / 2;
    const long long rows = filled > groups ? filled : groups;
    int best = 256;
    long long least = -1;
    const int width[4] = {256, 128, 64, 32}, cycles[4] = {600, 400, 320, 300};
    for (int i = G > kWideGroups ? 1 : 0; i < 4; ++i) {
        const long long tiles = rows * ((N + width[i] - 1) / width[i]);
        const long long cost = (tiles + num_sms() - 1) / num_sms() * cycles[i];
        if (least < 0 || cost < least) {
            least = cost;
            best = width[i];
        }
    }
    return best;
}

bool encode_operands(Mx4Params &p, int bits, const uint8_t *aq, const uint8_t *asf, int max_rows,
                     const uint8_t *bq, const uint8_t *bsf, uint64_t brows, int b_box, int K) {
    const int sfp = mx_sf_pitch(K);
    p.max_rows = max_rows;
    p.a_rows = box_rows(max_rows);
    p.blocks = K / 32;
    p.kb = bits == 4 ? (K + 255) / 256 : K / 128;
    const int row = bits == 4 ? K / 2 : K;
    return encode_tmap_u8_2d(&p.tmA, aq, row, max_rows, row, 128, p.a_rows, 128) &&
           (bits == 4 ? encode_tmap_u8_2d(&p.tmB, bq, K / 2, brows, K / 2, 128, b_box, 128)
                      : encode_tmap_u4_expand_2d(&p.tmB, bq, K, brows, b_box)) &&
           encode_tmap_u8_2d(&p.tmSA, asf, sfp, max_rows, sfp, 16, p.a_rows, 0) &&
           encode_tmap_u8_2d(&p.tmSB, bsf, sfp, brows, sfp, 16, b_box, 0);
}

}  // namespace

moe_status launch_mx4_matmul(const uint8_t *aq, const uint8_t *asf, int bits,
                             const int32_t *offsets, int G, int max_rows, const uint8_t *bq,
                             const uint8_t *bsf, const float *row_w, int w_rows, int N, int K,
                             uint16_t *out, cudaStream_t st) {
    Mx4Params p;
    std::memset(&p, 0, sizeof p);
    const int BN = rows_bn(max_rows, G, N);
    if (!encode_operands(p, bits, aq, asf, max_rows, bq, bsf, (uint64_t)G * N, BN, K) ||
        (BN >= 64 && !encode_tmap_bf16_2d_sw64(&p.tmO, out, N, max_rows, 2ULL * N, 32, 32)))
        return MOE_ERR_CUDA;
    p.offsets = offsets;
    p.G = G;
    p.N = N;
    p.n_tiles = (N + BN - 1) / BN;
    p.row_w = row_w;
    p.w_rows = w_rows;
    p.out = out;
    const long long tiles = (long long)row_tile_bound(max_rows, G) * p.n_tiles;
    if (bits == 4) {
        switch (BN) {
        case 256: return launch_mx4<MX4_ROWS, 4, 256, 4>(p, tiles, st);
        case 128: return launch_mx4<MX4_ROWS, 4, 128, 5>(p, tiles, st);
        case 64: return launch_mx4<MX4_ROWS, 4, 64, 7>(p, tiles, st);
        default: return launch_mx4<MX4_ROWS, 4, 32, 8>(p, tiles, st);
        }
    }
    switch (BN) {
    case 256: return launch_mx4<MX4_ROWS, 8, 256, 4>(p, tiles, st);
    case 128: return launch_mx4<MX4_ROWS, 8, 128, 5>(p, tiles, st);
    case 64: return launch_mx4<MX4_ROWS, 8, 64, 7>(p, tiles, st);
    default: return launch_mx4<MX4_ROWS, 8, 32, 8>(p, tiles, st);
    }
}

moe_status launch_mx4_ffn1(const uint8_t *xq, const uint8_t *xsf, const int32_t *offsets, int G,
                           int max_rows, const uint8_t *W13q, const uint8_t *W13sf, int d, int I,
                           float clamp, uint8_t *hq, uint8_t *hsf, cudaStream_t st) {
    Mx4Params p;
    std::memset(&p, 0, sizeof p);
    const int BN = rows_bn(max_rows, G, 2 * I) == 256 ? 256 : 128;
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
    const long long tiles = (long long)row_tile_bound(max_rows, G) * p.n_tiles;
    return BN == 256 ? launch_mx4<MX4_FFN1, 8, 256, 4>(p, tiles, st)
                     : launch_mx4<MX4_FFN1, 8, 128, 5>(p, tiles, st);
}

}  // namespace moe
