// few.cu -- the whole layer for a few tokens (1 to 32): gate, routing, both
// expert matmuls around the clamped SwiGLU, the shared expert and the combine,
// in two launches.
//
//   logits = x W_g^T (+ offset);  ids, w = top-k or table routing
//   h[r] = silu(min(g, c)) clamp(u, -c, c),  [g|u] = x[t] W13[e]^T
//   y[t] = bf16( h_shared W2[E]^T + sum_j w[t,j] (h[t,j] W2[e_j]^T) )
// ("HyperParallel加速DeepSeek-V4.1多模态1M长序列训练" §2.3 MegaGate and MegaMoE,
// "MindSpore HyperParallel一键开箱DeepSeek-V4.1-Flash" §01 shared expert, at the
// batch sizes of decoding.)
//
// Bound: the weights of the experts that the tokens hit cross HBM once (a few
// rows reuse each of them), so everything else has to hide behind that stream,
// and what cannot hide is the start (launch, gate, routing) and the two places
// where one matmul needs all of the one before it.  The second kernel keeps the
// stream running with a warp for each of the things that wait:
//   1 takes item numbers from the grid's counter, one ahead of the copies
//   1 copies weight rows into a ring in shared memory (two TMA boxes a stage, 32
//     KB), across the boundaries of the phases
//   1 waits for a stage's token operands (a phase's dependence on the one before)
//     and brings them
//  16 multiply, in two groups that take stages, or short tiles, in turn
//   2 add up the multiplying warps' sums, apply the SwiGLU or the routing weight,
//     store and signal
// The work comes as items of 16 weight rows in one order for the whole grid:
//   shared expert's W13 | W13 of the hit experts | shared W2 | their W2
// The first part needs no routing result, so the kernel starts on it while the
// first kernel (gate and routing) still runs (programmatic launch).  An item waits
// only for items before it in the order, all of which running CTAs hold, so the
// kernel needs no particular number of resident CTAs.
//
// Items: 8 gate rows and the matching 8 up rows of W13 (both land in the same
// thread, which applies the SwiGLU), or 2 x 16 rows of W2.  Eight warps split a
// stage's chunks of the contraction, each with mma.m16n8k16 (weights x 8 tokens,
// fp32 sums; at a few rows a weight the matrix pipe is nearly idle, so the 128-row
// tiles of tcgen05 would only add padding); their partial sums meet in shared
// memory in a fixed order.  FP8 weights are expanded to f16 in registers, exactly,
// and each 128-block's sum takes its scale in fp32; the tokens are then f16 as
// well, each scaled by a power of two (a few CTAs of the first kernel).  The second
// matmul's operand h is f16 with FP8 weights (2^-11 of itself; for a clamp whose square
// f16 does not hold, as with bf16 weights), and with bf16 weights the sum of two bf16 terms (2^-16; one term, 2^-8, makes the error of y 1.4 times what
// its own rounding to bf16 leaves).  The terms of up to four rows lie side by side in the
// MMA's eight columns; for more rows the second one is another MMA for the same weights,
// in a loop of its own (inside the first one it cost registers: 32 tokens 1.05 -> 1.16
// ms, so 1.08).  One term measured 58.4 us (so 58.7) for one token, 88 (91) for 23.
// Every sum stays fp32 up to y.  Products of the second matmul go to fp32
// rows per (token, slot); at the end each CTA adds up its share of the columns in
// slot order, so results do not depend on who finishes when.
//
// Measured (time of the call; of the copy bandwidth in brackets), d = 4096, I =
// 2048, 384 experts, top 6: one token 58.9 us (89 %); 32 tokens 1.08 ms with 149 experts
// hit on average (7.0 TB/s of their 7.5 GB); FP8, one token 38.2 us (69 %), 16 tokens 375-390
// us with 87 experts hit (5.7-5.9 TB/s of 2.2 GB).  23 tokens through a table of 97 experts, d
// = 1152, I = 704: 89-92 us with 66 hit (3.6 TB/s).  What holds the last one back is not HBM
// but what a tile of 16 short weight rows costs the multiplying warps whatever it brings
// (waits, the hand-over of sums, a signal).  A token's 38 us: routed 5 us after the
// start, first routed copies after 8, of which the shared W13 hides 4; then the stream
// runs at 5.5-6 TB/s, held back by the copying warp (1.2 us an item of 64 KB) and by the
// time that a stage stays in the ring (2 us on its way, 1.5 until it is read), and two
// dependences.
#include <cfloat>
#include <climits>

#include "fp8_common.cuh"

namespace moe {
namespace {

constexpr int kFewT = 32;              // tokens at most
constexpr int kFewK = 8;               // experts per token at most
constexpr int kFewS = kFewT * kFewK;
constexpr int kFewE = 1024;
constexpr int kGateWarps = 16;
constexpr int kGateSplits = 16;        // at most
constexpr int kMulWarps = 16;
constexpr int kSumWarps = 2;           // each with a buffer of partial sums of its own
constexpr int kCopyWarp = kMulWarps, kActWarp = kMulWarps + 1, kSumWarp0 = kMulWarps + 2;
constexpr int kTicketWarp = kSumWarp0 + kSumWarps;
constexpr int kFewThreads = 32 * (kTicketWarp + 1);
constexpr int kChunk = 128;            // weight bytes of a row that a warp takes
constexpr int kGroups = 2;             // of multiplying warps; they take stages in turn
constexpr int kGroupWarps = kMulWarps / kGroups;
constexpr int kWarpChunks = 2;         // chunks of a stage for one warp
constexpr int kStageChunks = kGroupWarps * kWarpChunks;   // of a row in a stage, at most
constexpr int kFewStage = 16 * kStageChunks * kChunk;   // two boxes of 8 rows
constexpr int kW2Tiles = 2;            // tiles of 16 rows in an item of W2

struct FewParams {
    CUtensorMap tm13, tm2;             // weight bytes: [K / 128 B][rows][128 B], boxes 16 x 8 x 128
    const uint16_t *x, *W_g;
    const float *logit_offset, *bias;
    const uint8_t *is_vision;
    const int32_t *input_ids, *tid2eid;
    int vocab, T, d, E, k, I, hash;
    float scaling, clamp;
    const void *W13, *W2;              // bf16 or E4M3 codes
    const float *W13_s, *W2_s;         // FP8: scales
    uint16_t *y;
    int32_t *ids_out;                  // or null
    float *w_out;                      // or null
    // workspace
    int *counters;   // [0] gate, [1] ticket, [2] exits, [3] f16 tokens, [4] shared h tiles,
                     // [5 + p] those of pass p,
                     // then columns' finished items; zero between calls
    int n_counters;
    float *part;     // [splits, T, E] partial logits
    uint16_t *x16;   // FP8 weights: [T, d] f16 tokens, each scaled by a power of two ...
    float *x16_s;    // ... whose inverse this is [T]
    int h_exp;       // where h is f16, it is times 2^h_exp
    uint64_t *routed;   // [T, k] (expert + 1) << 32 | its weight's bits; zero between calls, so
                        // that a slot's word is its own signal
    uint16_t *h;     // FP8 weights, clamp^2 inside f16: [S + T, I] f16; else [S + T, 2, I],
                     // bf16 terms of h
    float *yp;       // [S + T, d]
    int splits;
    int cps13, cps2;   // chunks of a row in a stage
    int by_tile;       // the groups of multiplying warps take tiles in turn (0: stages)
    int *status;
    long long wait_limit;
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The warp's arrival on a barrier that lets others overwrite what it has loaded from
// shared memory: after the loads have come back, not after they were issued.  `loaded`
// depends on all of this lane's, the vote on every lane's `loaded`, and the address on
// the vote (which is 0, as `zero` is); loads that queue behind stalled ones to global
// memory were seen to read what came after them otherwise.
__device__ __forceinline__ void arrive_after(uint64_t *bar, uint32_t loaded, uint32_t zero,
                                             int lane) {
    const uint32_t none = __any_sync(0xffffffffu, (loaded & zero) != 0);
    __syncwarp();
    if (lane == 0)
        asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar) + none)
                     : "memory");
}

// A stage's two boxes of eight rows and the bytes that `bar` is to count.  With an L2
// policy: the weights pass through L2 once and must not push out what every call uses
// again (the kernels' code, W_g, the token rows).  Called by a whole warp, which elects
// the issuing thread here: with uniform control flow around it the operands stay in
// uniform registers.
__device__ __forceinline__ void copy_stage(void *dst, int half, const CUtensorMap *tm,
                                           uint64_t *bar, int bytes, int r0, int r1, int c0,
                                           uint64_t policy) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%3], %4;\n\t"
        "@e cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%2, {%8, %5, %7}], [%3], %9;\n\t"
        "@e cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%1], [%2, {%8, %6, %7}], [%3], %9;\n\t}" ::"r"(smem_u32(dst)),
        "r"(smem_u32(dst) + half), "l"(reinterpret_cast<uint64_t>(tm)), "r"(smem_u32(bar)),
        "r"(bytes), "r"(r0), "r"(r1), "r"(c0), "r"(0), "l"(policy)
        : "memory");
}

__device__ __forceinline__ int atom_add_acq_rel(int *p, int v) {
    int r;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], %2;" : "=r"(r) : "l"(p), "r"(v) : "memory");
    return r;
}

// A routed slot's word, which says itself that it is there: whoever lists the experts
// needs neither a flag nor the end of the first kernel, each a round trip more.
__device__ __forceinline__ void st_slot(uint64_t *p, uint64_t v) {
    asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(p), "l"(v) : "memory");
}
__device__ __forceinline__ uint64_t ld_slot(const uint64_t *p) {
    uint64_t v;
    asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
    return v;
}
// Bounded like mbar_wait; 0 once the CTA has aborted or the limit ran out.
__device__ __forceinline__ uint64_t wait_slot(const uint64_t *p, const WaitCtl &w) {
    uint64_t v = ld_slot(p);
    const long long t0 = clock64();
    while (v == 0 && !*w.abort) {
        v = ld_slot(p);
        if (clock64() - t0 > w.limit) {
            *w.abort = 1;
            atomicExch(w.status, (int)MOE_ERR_TIMEOUT);
        }
    }
    return v;
}

// ------------------------------------------------------------ gate, routing
//
// A CTA takes 16 experts and one of `splits` parts of the contraction (all SMs
// on the few megabytes of W_g), its warps every sixteenth step of 32; the
// partial logits go to the workspace, and the CTA that finishes last adds
// them in order and routes, a warp per token.  mma fragments straight from
// global memory: a lane's 16 bytes of row l / 4 are eight consecutive k, fed
// as two k-pairs to each of two MMAs; the token operand is read the same way,
// so the order of k inside a step is the same on both sides.
// Scores and weights are rounded once, as moe_route rounds the fp64 values; here the
// values before the rounding are pairs of fp32 (0.2 us for one token and 384 experts),
// as fp64 costs 6 us of latency that nothing hides.
//
// What follows the gate matmul is latency alone, and the routed experts wait for it: so
// all of the last CTA's threads add up the partial logits where they fit its shared
// memory, and the largest key of a round is found by two reductions of the warp over
// keys in the order of unsigned integers.
__device__ __forceinline__ void prefetch_l2(const void *p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}
__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t u = __float_as_uint(v);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// A value as the sum of two fp32 numbers, the second at most half a spacing of the first.
// Sums and products by the error-free transformations of Knuth and Dekker.
struct Pair {
    float h, l;
};
__device__ __forceinline__ Pair two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
// |a| >= |b|
__device__ __forceinline__ Pair fast_two_sum(float a, float b) {
    const float s = __fadd_rn(a, b);
    return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
// c + r p, |c| >= |r p|, to the accuracy of a pair
__device__ __forceinline__ Pair horner(float c, Pair r, Pair p) {
    const float v = __fmul_rn(r.h, p.h);
    const float e = __fmaf_rn(r.l, p.h, __fmaf_rn(r.h, p.l, __fmaf_rn(r.h, p.h, -v)));
    Pair s = fast_two_sum(c, v);
    s.l = __fadd_rn(s.l, e);
    return s;
}
// (a.h + a.l) / (b.h + b.l), one rounding
__device__ __forceinline__ float quotient(Pair a, Pair b) {
    const float q = __fdiv_rn(a.h, b.h);
    const float rest = __fadd_rn(__fmaf_rn(-q, b.h, a.h), __fmaf_rn(-q, b.l, a.l));
    return __fadd_rn(q, __fdiv_rn(rest, b.h));
}

// 1 / (1 + e^-z), rounded to fp32: the nearest value but for 3 of 100000 logits, whose
// neighbour it is (values within 2^-33 of the middle between two).  With e = e^-|z| it
// is 1 / (1 + e) or e / (1 + e).  e = 2^n e^r, r = -|z| - n ln 2 with ln 2 as the sum of
// three numbers of which the first has 12 bits (Cody and Waite), e^r by its series up to
// r^9, the terms up to r^3 in pairs.
__device__ __forceinline__ float sigmoid_rounded(float z) {
    const float t = -fminf(fabsf(z), 110.0f);   // (e^-110 is 0 in fp32; a NaN: below)
    const float n = rintf(t * 1.44269504f);
    const Pair d = {__fmul_rn(n, 3.1946183e-5f), __fmaf_rn(n, 3.1946183e-5f, -__fmul_rn(n, 3.1946183e-5f))};
    Pair r = two_sum(__fmaf_rn(n, -0.693115234375f, t), -d.h);
    r = fast_two_sum(r.h, __fsub_rn(r.l, __fmaf_rn(n, 1.646595e-12f, d.l)));
    float p = 1.0f / 362880.0f;
    p = __fmaf_rn(p, r.h, 1.0f / 40320.0f);
    p = __fmaf_rn(p, r.h, 1.0f / 5040.0f);
    p = __fmaf_rn(p, r.h, 1.0f / 720.0f);
    p = __fmaf_rn(p, r.h, 1.0f / 120.0f);
    p = __fmaf_rn(p, r.h, 1.0f / 24.0f);
    Pair e = fast_two_sum(1.0f / 6.0f, __fmul_rn(r.h, p));
    e.l = __fadd_rn(e.l, -4.967054e-9f);        // 1/6 less its fp32 value
    e = horner(0.5f, r, e);
    e = horner(1.0f, r, e);
    e = horner(1.0f, r, e);
    const int k = (int)n;
    const float f = exp2i(max(k, -100));
    Pair den = fast_two_sum(1.0f, __fmul_rn(e.h, f));
    den.l = __fmaf_rn(e.l, f, den.l);
    float s = quotient(z >= 0.0f ? Pair{1.0f, 0.0f} : e, den);
    if (z < 0.0f) s = s * exp2i(max(k, -126)) * exp2i(min(k + 126, 0));
    return z == z ? s : z;
}

// Token t in f16 (for FP8 weights): times the power of two that brings its
// largest magnitude to [2^14, 2^15), so that bf16's eight bits survive down to
// 2^-31 of that magnitude and lose at most 2^-39 of it below.  By no more than 2^100,
// as the first matmul's sums grow with it and have to stay inside fp32.  One CTA.
__device__ void few_token_f16(const FewParams &p, int t, uint32_t *warp_top) {
    const uint4 *src = reinterpret_cast<const uint4 *>(p.x + (size_t)t * p.d);
    uint32_t m = 0;
    for (int i = threadIdx.x; i < p.d / 8; i += blockDim.x) {
        const uint4 v = __ldg(src + i);
        m = __vmaxu2(m, v.x & 0x7FFF7FFFu);
        m = __vmaxu2(m, v.y & 0x7FFF7FFFu);
        m = __vmaxu2(m, v.z & 0x7FFF7FFFu);
        m = __vmaxu2(m, v.w & 0x7FFF7FFFu);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((threadIdx.x & 31) == 0) warp_top[threadIdx.x >> 5] = m;
    __syncthreads();
    for (int w = 0; w < kGateWarps; ++w) m = __vmaxu2(m, warp_top[w]);
    __syncthreads();
    const uint32_t top = max(m & 0xFFFFu, m >> 16);
    // exponent of the largest; an infinity or NaN among the values stays one
    // under any scale
    const int e = top >= 0x7F80u ? 0 : max((int)(top >> 7) - 127, -86);
    const float f = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
    uint4 *dst = reinterpret_cast<uint4 *>(p.x16 + (size_t)t * p.d);
    for (int i = threadIdx.x; i < p.d / 8; i += blockDim.x) {
        const uint4 v = __ldg(src + i);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t r[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __half2 h = __floats2half2_rn(bf16_lo(w[j]) * f, bf16_hi(w[j]) * f);
            r[j] = *reinterpret_cast<const uint32_t *>(&h);
        }
        dst[i] = make_uint4(r[0], r[1], r[2], r[3]);
    }
    if (threadIdx.x == 0) p.x16_s[t] = __uint_as_float((uint32_t)(127 - 14 + e) << 23);
    __syncthreads();
    if (threadIdx.x == 0) red_release_gpu_add(p.counters + 3, 1);
}

template <int EPL>
__global__ void __launch_bounds__(kGateWarps * 32) few_gate_kernel(const __grid_constant__ FewParams p) {
    // The launch may precede the end of the kernel before it (which hides its
    // latency); nothing is read before that end.  The second kernel may start
    // from here on, never before: it shares the workspace with the call before.
    // (It then needs all of these CTAs to be running, not to have ended.)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if ((int)blockIdx.y >= p.splits) {
        __shared__ uint32_t warp_top[kGateWarps];
        const int n = (gridDim.y - p.splits) * gridDim.x;
        for (int t = (blockIdx.y - p.splits) * gridDim.x + blockIdx.x; t < p.T; t += n)
            few_token_f16(p, t, warp_top);
        return;
    }
    // what the last CTA will read once more, into L2 in the meantime
    if (blockIdx.x == 0 && blockIdx.y == 0) {
        for (int i = threadIdx.x * 32; i < p.E; i += kGateWarps * 32 * 32) {
            if (p.logit_offset) prefetch_l2(p.logit_offset + i);
            if (!p.hash) {
                prefetch_l2(p.bias + i);
                if (p.is_vision) prefetch_l2(p.bias + p.E + i);
            }
        }
        if (p.hash && (int)threadIdx.x < p.T) {
            const int tok = p.input_ids[threadIdx.x];
            if (tok >= 0 && tok < p.vocab) prefetch_l2(p.tid2eid + (size_t)tok * p.k);
        }
    }
    __shared__ float red[kGateWarps][4][32], keys[kGateWarps * 4 * 32];
    __shared__ int s_last;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int e0 = blockIdx.x * 16 + (lane >> 2);
    const int steps = p.d / 32;
    const int lo = (int)((long long)steps * blockIdx.y / p.splits);
    const int hi = (int)((long long)steps * (blockIdx.y + 1) / p.splits);
    const uint16_t *w0 = p.W_g + (size_t)min(e0, p.E - 1) * p.d + (lane & 3) * 8;
    const uint16_t *w1 = p.W_g + (size_t)min(e0 + 8, p.E - 1) * p.d + (lane & 3) * 8;
    for (int t0 = 0; t0 < p.T; t0 += 8) {
        const int tok = t0 + (lane >> 2);
        const uint16_t *xr = p.x + (size_t)min(tok, p.T - 1) * p.d + (lane & 3) * 8;
        float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
        for (int s = lo + warp; s < hi; s += kGateWarps) {
            const uint4 a = __ldg(reinterpret_cast<const uint4 *>(w0 + s * 32));
            const uint4 b = __ldg(reinterpret_cast<const uint4 *>(w1 + s * 32));
            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(xr + s * 32));
            mma_bf16(acc, a.x, b.x, a.y, b.y, v.x, v.y);
            mma_bf16(acc, a.z, b.z, a.w, b.w, v.z, v.w);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) red[warp][i][lane] = acc[i];
        __syncthreads();
        if (threadIdx.x < 128) {
            const int l = threadIdx.x & 31, i = threadIdx.x >> 5;
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < kGateWarps; ++w) v += red[w][i][l];
            const int e = blockIdx.x * 16 + (l >> 2) + (i >> 1) * 8;
            const int t = t0 + (l & 3) * 2 + (i & 1);
            if (e < p.E && t < p.T) p.part[((size_t)blockIdx.y * p.T + t) * p.E + e] = v;
        }
        __syncthreads();
    }
    if (threadIdx.x == 0)
        s_last = atom_add_acq_rel(p.counters, 1) == (int)gridDim.x * p.splits - 1;
    __syncthreads();
    if (!s_last) return;
    float *scores = &red[0][0][0];
    const bool all = !p.hash && p.T * p.E <= kGateWarps * 4 * 32;
    if (all) {
        for (int i = threadIdx.x; i < p.T * p.E; i += kGateWarps * 32) {
            const int t = i / p.E, e = i - t * p.E;
            float z[kGateSplits];
#pragma unroll
            for (int s = 0; s < kGateSplits; ++s)
                z[s] = s < p.splits ? __ldcg(p.part + (size_t)s * p.T * p.E + i) : 0.0f;
            float v = p.logit_offset ? p.logit_offset[e] : 0.0f;
            const float b = p.bias[e + ((p.is_vision && p.is_vision[t]) ? p.E : 0)];
#pragma unroll
            for (int s = 0; s < kGateSplits; ++s) v += z[s];
            v = sigmoid_rounded(v);
            scores[i] = v;
            keys[i] = v + b;
        }
        __syncthreads();
    }
    for (int t = warp; t < p.T; t += kGateWarps) {
        int my_id = 0;
        float my_s = 0.0f;   // lane j < k: expert and score of slot j
        if (p.hash) {
            if (lane < p.k) {
                int tok = p.input_ids[t];
                if (tok < 0 || tok >= p.vocab) {
                    record_status(p.status, MOE_ERR_INVALID_ARG);
                    tok = 0;
                }
                my_id = p.tid2eid[(size_t)tok * p.k + lane];
                if (my_id < 0 || my_id >= p.E) {
                    record_status(p.status, MOE_ERR_INVALID_ARG);
                    my_id = 0;
                }
                float z = 0.0f;
                for (int s = 0; s < p.splits; ++s)
                    z += __ldcg(p.part + ((size_t)s * p.T + t) * p.E + my_id);
                if (p.logit_offset) z += p.logit_offset[my_id];
                my_s = sigmoid_rounded(z);
            }
        } else {
            const float *bt = p.bias + ((p.is_vision && p.is_vision[t]) ? p.E : 0);
            float zv[EPL];
            uint32_t key[EPL];
            if (all) {
#pragma unroll
                for (int i = 0; i < EPL; ++i) {
                    const int e = lane + 32 * i;
                    zv[i] = e < p.E ? scores[t * p.E + e] : 0.0f;
                    key[i] = __float_as_uint(e < p.E ? keys[t * p.E + e] : 0.0f);
                }
            } else {
#pragma unroll
                for (int i = 0; i < EPL; ++i) {
                    const int e = lane + 32 * i;
                    zv[i] = e < p.E && p.logit_offset ? p.logit_offset[e] : 0.0f;
                    key[i] = __float_as_uint(e < p.E ? bt[e] : 0.0f);
                }
                // many loads together: their latency, not their bytes, counts here
                constexpr int U = EPL <= 4 ? 8 : EPL <= 12 ? 4 : 1;
                for (int s0 = 0; s0 < p.splits; s0 += U) {
                    float z[U][EPL];
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int i = 0; i < EPL; ++i) {
                            const int e = lane + 32 * i;
                            z[u][i] = e < p.E && s0 + u < p.splits
                                          ? __ldcg(p.part + ((size_t)(s0 + u) * p.T + t) * p.E + e)
                                          : 0.0f;
                        }
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int i = 0; i < EPL; ++i) zv[i] += z[u][i];
                }
#pragma unroll
                for (int i = 0; i < EPL; ++i) {
                    zv[i] = sigmoid_rounded(zv[i]);
                    key[i] = __float_as_uint(zv[i] + __uint_as_float(key[i]));
                }
            }
            // in the integers' order: no expert 0, a NaN the smallest number
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const float kk = __uint_as_float(key[i]);
                key[i] = lane + 32 * i >= p.E ? 0u : ordered(kk == kk ? kk : -FLT_MAX);
            }
            for (int j = 0; j < p.k; ++j) {
                uint32_t bk = 0u;   // below every key, minus infinity's too
                float bs = 0.0f;
                int be = INT_MAX;
#pragma unroll
                for (int i = 0; i < EPL; ++i) {   // ids grow with i: the first of equals stays
                    if (key[i] > bk) {
                        bk = key[i];
                        bs = zv[i];
                        be = lane + 32 * i;
                    }
                }
                const uint32_t top = __reduce_max_sync(0xffffffffu, bk);
                const int first =
                    (int)__reduce_min_sync(0xffffffffu, bk == top ? (unsigned)be : INT_MAX);
                bs = __shfl_sync(0xffffffffu, bs, first & 31);
                if (be == first) {
#pragma unroll
                    for (int i = 0; i < EPL; ++i)
                        if (lane + 32 * i == first) key[i] = 0u;
                }
                if (lane == j) {   // (there is always one: k <= E)
                    my_id = first;
                    my_s = bs;
                }
            }
        }
        Pair sum = {0.0f, 0.0f};
        for (int j = 0; j < p.k; ++j) {
            const Pair a = two_sum(sum.h, __shfl_sync(0xffffffffu, my_s, j));
            sum = fast_two_sum(a.h, __fadd_rn(a.l, sum.l));
        }
        if (lane < p.k) {
            const size_t o = (size_t)t * p.k + lane;
            // (tiny scores by a power of two, which cancels, so that no product is subnormal)
            const float up = sum.h < 1.0e-20f ? exp2i(100) : 1.0f;
            const float v = my_s * up, num = __fmul_rn(p.scaling, v);
            float w = 0.0f;
            if (sum.h > 0.0f)
                w = quotient({num, __fmaf_rn(p.scaling, v, -num)}, {sum.h * up, sum.l * up});
            st_slot(p.routed + o, (uint64_t)(my_id + 1) << 32 | __float_as_uint(w));
            if (p.ids_out) p.ids_out[o] = my_id;
            if (p.w_out) p.w_out[o] = w;
        }
    }
}

// ------------------------------------------------------------------ experts

// What every role knows about the routing: the hit experts in order, each cut
// into passes of at most 8 NT rows, and the slots (token * k + j) of each.
struct alignas(8) FewPass {
    int e;                             // expert
    int rows;                          // rows | first entry in `slot` << 16
};
struct alignas(8) FewMeta {
    int n_units, n_pass;               // contributions that a column tile waits for; passes
    float w[kFewS];                    // routing weight of each slot
    FewPass pass[kFewS];
    int16_t slot[kFewS];
    int16_t token[kFewS];              // of each entry of `slot`
    // scratch: of each slot, and rows, then first slot of each expert
    int16_t expert[kFewS], rank[kFewS], start[kFewE];
};

// One tile's place in the work, as the copying warp hands it on with each stage.
struct FewTile {
    int tile;      // of 16 weight rows
    int pass;      // -1 the shared expert
    int rows;      // tokens of the pass | first entry in `slot` << 16
    int flags;     // first chunk | kSecond | kLast
};
constexpr int kSecond = 1 << 30;       // W2
constexpr int kLast = 1 << 29;         // the tile's last stage
constexpr int kChunkMask = (1 << 28) - 1;

__device__ __forceinline__ int4 ld_tile(const FewTile *p) {
    const uint4 v = ld_shared_v4(smem_u32(p));
    return make_int4((int)v.x, (int)v.y, (int)v.z, (int)v.w);
}

struct FewItem {
    int pass;
    bool second;
    int tile;
};

// WIDE: FP8 weights and a clamp whose square f16 does not hold
template <bool FP8, int NT, bool WIDE>
struct FewShape {
    static constexpr int STAGES = 5;
    static constexpr int ELT = FP8 ? 1 : 2;
    static constexpr int CHUNK_K = kChunk / ELT;       // contraction of a chunk
    // token operands of a stage: rows of 16 bits an element, pitched so that the
    // rows of a quarter warp's loads meet in no bank; passes of more rows are
    // read from global memory
    static constexpr int ACT_ROWS = FP8 ? 2 : 4;
    static constexpr int TERMS = FP8 && !WIDE ? 1 : 2;   // of h
    static constexpr int ACT_PITCH = 2 * CHUNK_K * kStageChunks + (FP8 ? 16 : 64);
    static constexpr int ACT = ACT_ROWS * ACT_PITCH;
    static constexpr int RED = kSumWarps * kMulWarps * 128 * 4;
    static constexpr int SCALES = FP8 ? 2 * kStageChunks * 4 : 0;
    static constexpr int SMEM = 1024 + STAGES * (kFewStage + ACT + SCALES + 16 /* FewTile */) +
                                RED + 2 * kSumWarps * 16 + (int)sizeof(FewMeta) + 512;
    static_assert(SMEM <= 232448, "shared memory of a CTA");
};

// Item t: shared W13 | W13 of the passes | shared W2 | W2 of the passes, one tile of W13
// or kW2Tiles of W2.  r1, r2: 1 / tiles1, 1 / tiles2 (what rounding leaves wrong is put
// right).  tile < 0: none.
__device__ __forceinline__ FewItem few_item(int t, int tiles1, int tiles2, float r1, float r2,
                                            int n_pass) {
    FewItem it;
    it.second = t >= (n_pass + 1) * tiles1;
    if (it.second) t = (t - (n_pass + 1) * tiles1) * kW2Tiles;
    const int tiles = it.second ? tiles2 : tiles1;
    int q = (int)((float)t * (it.second ? r2 : r1));
    it.tile = t - q * tiles;
    if (it.tile < 0) { --q; it.tile += tiles; }
    if (it.tile >= tiles) { ++q; it.tile -= tiles; }
    it.pass = q - 1;
    if (q > n_pass) it.tile = -1;
    return it;
}

__device__ __forceinline__ void cp_async4(void *dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src)
                 : "memory");
}

// This lane's arrival on `bar` once its cp.async copies have landed (counted in
// the barrier's expected arrivals).
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}

// Weight row of a tile's eight that the MMA's row g takes: rows 0, 4, 1, 5, ...
// The two rows that a quarter warp reads then lie in different halves of the
// swizzled 128 bytes, so that no two of its loads meet in a bank.
__device__ __forceinline__ int few_row(int g) { return (g >> 1) | (g & 1) << 2; }

// The routing as `meta` says it, listed by one warp; the number of passes, or -1 after
// a wait that ran out.  An expert with r rows has ceil(r / (8 NT)) passes, and a pass
// as many units as it has groups of 8 rows.
template <int NT>
__device__ __forceinline__ int few_units(int r, int passes) {
    return passes > 0 ? (passes - 1) * NT + (r - (passes - 1) * 8 * NT + 7) / 8 : 0;
}
template <int NT>
__device__ __forceinline__ void few_passes(FewMeta *meta, int e, int r, int first_row, int first,
                                           int passes) {
    for (int j = 0; j < passes; ++j) {
        const int row = first_row + j * 8 * NT;
        meta->pass[first + j] = {e, min(8 * NT, r - j * 8 * NT) | row << 16};
    }
}

// At most 32 slots, one a lane: a slot's place is the number of slots with a smaller
// expert.  Little code, run once from a cold instruction cache, with the routed experts
// waiting for it.
template <int NT>
__device__ __noinline__ int few_list_short(const FewParams &p, int S, FewMeta *meta, int lane,
                                           const WaitCtl &wc) {
    const uint64_t v = lane < S ? wait_slot(p.routed + lane, wc) : 1;
    if (!__all_sync(0xffffffffu, v != 0)) return -1;
    const int e = lane < S ? (int)(v >> 32) - 1 : INT_MAX;
    const unsigned same = __match_any_sync(0xffffffffu, e), before = same & ((1u << lane) - 1u);
    const int r = __popc(same), passes = (r + 8 * NT - 1) / (8 * NT);
    const bool lead = lane < S && before == 0;
    const int mine = lead ? passes | few_units<NT>(r, passes) << 16 : 0;
    int place = 0, sum = 0, all = 0;
    for (int i = 0; i < S; ++i) {
        const int ei = __shfl_sync(0xffffffffu, e, i), c = __shfl_sync(0xffffffffu, mine, i);
        place += ei < e;
        sum += ei < e ? c : 0;
        all += c;
    }
    if (lane < S) {
        const int at = place + __popc(before);
        meta->slot[at] = (int16_t)lane;
        meta->token[at] = (int16_t)(lane / p.k);
        meta->w[lane] = __uint_as_float((uint32_t)v);
    }
    if (lead) few_passes<NT>(meta, e, r, place, sum & 0xFFFF, passes);
    if (lane == 0) meta->n_units = (all >> 16) + (p.T + 7) / 8;
    __syncwarp();
    return all & 0xFFFF;
}

template <int NT>
__device__ __noinline__ int few_list(const FewParams &p, int S, FewMeta *meta, int lane,
                                     const WaitCtl &wc) {
    for (int e = lane; e < p.E; e += 32) meta->start[e] = 0;
    __syncwarp();
    // slot by slot: its expert, and its rank among the expert's rows
    for (int i0 = 0; i0 < S; i0 += 32) {
        const int i = i0 + lane;
        const uint64_t v = i < S ? wait_slot(p.routed + i, wc) : 1;
        if (!__all_sync(0xffffffffu, v != 0)) return -1;
        const int e = i < S ? (int)(v >> 32) - 1 : -1 - lane;
        const unsigned same = __match_any_sync(0xffffffffu, e), before = same & ((1u << lane) - 1u);
        int rank = 0;
        if (i < S) rank = meta->start[e] + __popc(before);
        __syncwarp();
        if (i < S) {
            if (before == 0) meta->start[e] += __popc(same);
            meta->w[i] = __uint_as_float((uint32_t)v);
            meta->rank[i] = (int16_t)rank;
            meta->expert[i] = (int16_t)e;
        }
        __syncwarp();
    }
    // prefix sums over the experts of passes, slots and units, in one word (each at
    // most kFewS = 256: 10 bits)
    int sum = 0;
    for (int base = 0; base < p.E; base += 32) {
        const int e = base + lane;
        const int r = e < p.E ? meta->start[e] : 0;
        if (!__any_sync(0xffffffffu, r)) continue;
        const int passes = (r + 8 * NT - 1) / (8 * NT);
        const int mine = passes | r << 10 | few_units<NT>(r, passes) << 20;
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        const int excl = sum + incl - mine;
        if (r > 0) {
            meta->start[e] = (int16_t)(excl >> 10 & 1023);
            few_passes<NT>(meta, e, r, excl >> 10 & 1023, excl & 1023, passes);
        }
        sum += __shfl_sync(0xffffffffu, incl, 31);
    }
    __syncwarp();
    for (int i = lane; i < S; i += 32) {
        const int at = meta->start[meta->expert[i]] + meta->rank[i];
        meta->slot[at] = (int16_t)i;
        meta->token[at] = (int16_t)(i / p.k);
    }
    if (lane == 0) meta->n_units = (sum >> 20) + (p.T + 7) / 8;
    __syncwarp();
    return sum & 1023;
}

template <bool FP8, int NT, bool WIDE>
__global__ void __launch_bounds__(kFewThreads, 1) few_experts_kernel(
    const __grid_constant__ FewParams p) {
    using SH = FewShape<FP8, NT, WIDE>;
    constexpr int STAGES = SH::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *acts = ring + STAGES * kFewStage;
    float4 *red = reinterpret_cast<float4 *>(acts + STAGES * SH::ACT);
    FewTile *info = reinterpret_cast<FewTile *>(reinterpret_cast<uint8_t *>(red) + SH::RED);
    // `red`: a buffer of 16 warps' sums for each sum warp; where the groups take tiles
    // in turn, two of 8 for each group and its sum warp
    constexpr int BUFS = 2 * kSumWarps;
    static_assert(kSumWarps == kGroups && kMulWarps == 2 * kGroupWarps, "halves of a buffer");
    FewTile *rinfo = info + STAGES;          // per buffer of `red`; flags: group of 8 rows | kSecond
    float *scales = reinterpret_cast<float *>(rinfo + BUFS);   // FP8: per stage gate, up
    FewMeta *meta =
        reinterpret_cast<FewMeta *>(reinterpret_cast<uint8_t *>(scales) + STAGES * SH::SCALES);
    uint64_t *full = reinterpret_cast<uint64_t *>(meta + 1);
    uint64_t *ifull = full + STAGES;         // `info` of the stage is written
    uint64_t *empty = ifull + STAGES;
    uint64_t *rfull = empty + STAGES;        // a buffer of `red` has every warp's partial sums
    uint64_t *rempty = rfull + BUFS;         // ... and has been read
    uint64_t *qfull = rempty + BUFS;         // an item's number is in `queue`
    uint64_t *qempty = qfull + 1;            // ... and has been taken
    volatile int *queue = reinterpret_cast<volatile int *>(qempty + 1);
    volatile int *abort_s = queue + 1;
    int *last_s = const_cast<int *>(abort_s) + 1;
    volatile int *stop_s = last_s + 1;       // no more items are wanted
    static_assert(sizeof(FewMeta) % 8 == 0, "the barriers behind it are 8-byte aligned");

    // (the warp's number is uniform, to the compiler too)
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 2 + (FP8 ? 32 : 0));
            mbar_init(&ifull[s], 1);
            mbar_init(&empty[s], kMulWarps);
        }
        for (int b = 0; b < BUFS; ++b) {
            mbar_init(&rfull[b], p.by_tile ? kGroupWarps : kMulWarps);
            mbar_init(&rempty[b], 1);
        }
        mbar_init(qfull, 1);
        mbar_init(qempty, 1);
        *abort_s = 0;
        *stop_s = 0;
        fence_barrier_init();
    }
    __syncthreads();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // a next call's first kernel
    const WaitCtl wc{abort_s, p.status, p.wait_limit};
    const uint32_t zero = (uint32_t)p.hash >> 1;   // which the compiler does not know
    const int S = p.T * p.k;
    const int tiles1 = p.I / 8, tiles2 = p.d / 16;
    int *h_done = p.counters + 4;
    int *y_done = h_done + 1 + kFewS;

    if (warp == kCopyWarp) {
        // ------------------------------------------------------------- copy
        // the rows of the items whose numbers it is given.
        uint32_t s = 0, ph = 0;
        uint32_t begun = 0;                // stages that a copy was issued to, and its parity
        const uint64_t policy = policy_evict_first();
        const float rcp1 = 1.0f / (float)tiles1, rcp2 = 1.0f / (float)tiles2;
        bool ok = true;
        int n_pass = -1;
        for (uint32_t n = 0; ok; ++n) {
            if (!mbar_wait_warp(qfull, n & 1u, wc)) break;
            const int t = __shfl_sync(0xffffffffu, *queue, 0);
            // A long list is made ahead by the warp that takes the numbers (which took 4 us
            // off 23 tokens of 5 experts); a short one here, as late as it is needed (made
            // there, one token takes 0.7 us more).
            if (t >= tiles1 && n_pass < 0) {
                n_pass = S <= 32 ? few_list_short<NT>(p, S, meta, lane, wc) : meta->n_pass;
                if (n_pass < 0) break;
            }
            const FewItem it = few_item(t, tiles1, tiles2, rcp1, rcp2, max(n_pass, 0));
            if (lane == 0) {
                if (it.tile < 0) *stop_s = 1;
                mbar_arrive(qempty);
            }
            __syncwarp();
            if (it.tile < 0) {
                if (!mbar_wait_warp(&empty[s], ph ^ 1u, wc)) break;
                if (lane == 0) {
                    info[s].tile = -1;
                    mbar_arrive(&ifull[s]);
                }
                break;
            }
            FewPass ps = {p.E, p.T};
            if (it.pass >= 0) ps = meta->pass[it.pass];
            const int e = ps.e, rows = ps.rows;
            const int K = it.second ? p.I : p.d;
            const int whole = K * SH::ELT / kChunk;   // chunks
            const int chunks = (K * SH::ELT + kChunk - 1) / kChunk;
            const int cps = it.second ? p.cps2 : p.cps13;
            const CUtensorMap *tm = it.second ? &p.tm2 : &p.tm13;
            for (int sub = 0; ok && sub < (it.second ? kW2Tiles : 1); ++sub) {
                // 8 gate rows and the matching 8 up rows, or 16 rows of W2
                const int tile = it.tile + sub;
                const int r0 = it.second ? e * p.d + tile * 16 : e * 2 * p.I + tile * 8;
                const int r1 = r0 + (it.second ? 8 : p.I);
                const float *sc = nullptr;   // FP8: this lane's scale of the first stage
                const int kb = fp8_blocks(K), my_kb = lane & (kStageChunks - 1);
                if constexpr (FP8) {
                    const int row = it.second ? tile * 16
                                              : tile * 8 + (lane >= kStageChunks ? p.I : 0);
                    const int all = it.second ? p.d : 2 * p.I;
                    // (a scale stands for 2^14 weights: their number is an int)
                    sc = (it.second ? p.W2_s : p.W13_s) +
                         (e * fp8_blocks(all) + row / kFp8Block) * kb + my_kb;
                }
                for (int c0 = 0; c0 < chunks; c0 += cps) {
                    if (!mbar_wait_warp(&empty[s], ph ^ 1u, wc)) { ok = false; break; }
                    if (lane == 0) {
                        const int flags = c0 | (it.second ? kSecond : 0) |
                                          (c0 + cps >= chunks ? kLast : 0);
                        *reinterpret_cast<int4 *>(&info[s]) = make_int4(tile, it.pass, rows, flags);
                        mbar_arrive(&ifull[s]);
                        if (c0 >= whole) mbar_arrive(&full[s]);
                    }
                    __syncwarp();
                    if (c0 < whole)
                        copy_stage(ring + s * kFewStage, kFewStage / 2, tm, &full[s],
                                   16 * kChunk * cps, r0, r1, c0, policy);
                    if constexpr (FP8) {
                        if (my_kb < cps && c0 + my_kb < kb)
                            cp_async4(scales + s * 2 * kStageChunks + lane, sc + c0);
                        cp_async_arrive(&full[s]);
                    }
                    begun = (begun & ~(0x10001u << s)) | (0x10000u << s) | (ph << s);
                    if (++s == STAGES) { s = 0; ph ^= 1u; }
                }
            }
        }
        if (*abort_s) {
            // drain the copies still in flight before the CTA exits
            for (int i = 0; i < STAGES; ++i)
                if (begun >> (16 + i) & 1u)
                    mbar_wait_teardown(&full[i], begun >> i & 1u, p.wait_limit);
        }
    } else if (warp == kActWarp) {
        // ------------------------------------------- token operands of a stage
        // Waits until they exist (the tokens in f16 come from the first kernel,
        // a pass's h from the tiles before it) and copies the rows of passes
        // that have few; whoever multiplies waits for nothing else.
        uint32_t s = 0, ph = 0;
        bool have_x = !FP8;
        while (mbar_wait_warp(&ifull[s], ph, wc)) {
            const int4 q = ld_tile(&info[s]);
            if (q.x < 0) break;
            const int n = q.z & 0xFFFF, row0 = q.z >> 16, c0 = q.w & kChunkMask;
            const bool second = q.w & kSecond;
            bool ready = true;
            if (lane == 0) {
                if (second) {
                    // one signal per column tile and group of 8 rows
                    if (c0 == 0)
                        ready = wait_count_geq(h_done + 1 + q.y, tiles1 * ((n + 7) / 8), wc);
                } else if (!have_x) {
                    ready = wait_count_geq(p.counters + 3, p.T, wc);
                }
            }
            have_x = have_x || !second;
            if (!__shfl_sync(0xffffffffu, ready, 0)) break;
            __syncwarp();
            // the copies read what others stored: every lane that issues one needs it
            fence_proxy_async_global();
            const int K = second ? p.I : p.d;
            const int k0 = c0 * SH::CHUNK_K;
            const int cps = second ? p.cps2 : p.cps13;
            const int bytes = 2 * min(cps * SH::CHUNK_K, K - k0);   // none behind the end
            const bool terms = SH::TERMS == 2 && second;   // h: row by row, its two terms
            const int copies = terms ? 2 * n : n;
            const bool copy = copies <= SH::ACT_ROWS && bytes > 0;
            if (lane == 0) {
                if (copy) mbar_arrive_expect_tx(&full[s], copies * bytes);
                else mbar_arrive(&full[s]);
            }
            __syncwarp();
            if (copy && lane < copies) {
                const int r = terms ? lane >> 1 : lane, term = terms ? lane & 1 : 0;
                const int row = q.y < 0    ? (second ? S + r : r)
                                : second ? meta->slot[row0 + r]
                                         : meta->token[row0 + r];
                const uint16_t *src = second ? p.h + ((size_t)row * SH::TERMS + term) * p.I
                                             : (FP8 ? p.x16 : p.x) + (size_t)row * p.d;
                bulk_load(acts + s * SH::ACT + lane * SH::ACT_PITCH, src + k0, bytes, &full[s]);
            }
            if (++s == STAGES) { s = 0; ph ^= 1u; }
        }
    } else if (warp < kMulWarps) {
        // -------------------------------------------------------- multiply
        // Two groups of eight warps take the stages in turn, so that one's waits
        // and loads overlap the other's products; warp w of a group takes two
        // chunks of its stage at most: 16 rows x 128 bytes against the tokens,
        // fragments straight from the row-wise tiles (a lane's 16 bytes are
        // consecutive k, fed as k-pairs to successive MMAs, on both sides alike).
        const int group = warp / kGroupWarps, wl = warp % kGroupWarps;
        // Where a tile is one or two stages long, the groups take tiles in turn instead,
        // and the other group neither writes nor signals anything for it (FP8, 16 tokens
        // 369 -> 356 us; with four stages a tile the ring is too short for it, and
        // stages in turn keep both groups busy).  In either
        // case `role` says which of a tile's stages a group has (0 the first one), so
        // that sums do not depend on which group it is.
        uint32_t s = 0, ph = 0, unit = 0, turn = 0;
        int role = 0;
        auto buffer = [&](uint32_t u) { return (p.by_tile ? 2 * group : 0) + (u & 1u); };
        const int g = lane >> 2, c = lane & 3;
        const int pr = few_row(g);
        float acc[NT][4];
        const uint16_t *act[NT];   // passes of many rows: this lane's token row of each group
        constexpr int NV = FP8 ? 2 : 1;
        while (true) {
            // Every warp goes through every stage in order and releases it, also
            // the other group's: with parity waits, whoever skipped stages could
            // take one lap of the ring for another.
            if (!mbar_wait_warp(&ifull[s], ph, wc)) break;
            const int4 q = ld_tile(&info[s]);
            if (q.x < 0) {
                if (lane == 0) {   // tell the sum warps: each its own, or both
                    for (int b = 0; b < (p.by_tile ? 1 : kSumWarps); ++b, ++unit) {
                        const uint32_t buf = buffer(unit);
                        if (!mbar_wait(&rempty[buf], (unit >> 1 & 1u) ^ 1u, wc)) break;
                        if (wl == 0 && (p.by_tile || group == 0)) rinfo[buf].tile = -1;
                        mbar_arrive(&rfull[buf]);
                    }
                }
                break;
            }
            const int n = q.z & 0xFFFF, row0 = q.z >> 16, c0 = q.w & kChunkMask;
            const bool second = q.w & kSecond;
            const int K = second ? p.I : p.d;
            const int nt = NT == 1 ? 1 : (n + 7) >> 3;
            const bool terms = SH::TERMS == 2 && second;
            const bool in_smem = (terms ? 2 * n : n) <= SH::ACT_ROWS;
            // a row's two terms of h in columns side by side
            const bool beside = terms && n <= 4;
            const int col = beside ? g >> 1 : g, term = beside ? g & 1 : 0;   // row, term
            const bool mine = (turn & (kGroups - 1)) == (uint32_t)group;
            if (c0 == 0) role = mine ? 0 : 1;
            if (!p.by_tile || (q.w & kLast)) ++turn;
            if (c0 == 0 && (mine || !p.by_tile)) {
#pragma unroll
                for (int j = 0; j < NT; ++j) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[j][i] = 0.0f;
                    const int i = j * 8 + col;
                    act[j] = nullptr;
                    if (!in_smem && i < n) {
                        const int row = q.y < 0    ? (second ? S + i : i)
                                        : second ? meta->slot[row0 + i]
                                                 : meta->token[row0 + i];
                        act[j] = second ? p.h + ((size_t)row * SH::TERMS + term) * p.I
                                        : (FP8 ? p.x16 : p.x) + (size_t)row * p.d;
                    }
                }
            }
            const int cps = second ? p.cps2 : p.cps13;
            // this warp's chunks of the stage, which it releases once the last one's
            // weights are in its registers
            // (bf16: counted on from stage to stage and tile to tile, so that what does
            // not divide by eight falls to other warps in turn: 88 -> 85 us for 23 tokens
            // at d = 1152, I = 704; with FP8 weights what it takes to compute shows, 365 ->
            // 377 us for 16 tokens at d = 4096, I = 2048)
            const int w_at = FP8 ? wl : (wl - c0 - 3 * q.x) & (kGroupWarps - 1);
            const int left = min(cps, (K + SH::CHUNK_K - 1) / SH::CHUNK_K - c0) - w_at;
            const int n_ch = !mine || left <= 0 ? 0 : left > kGroupWarps ? 2 : 1;
            static_assert(kWarpChunks == 2, "chunks of a stage for one warp");
            auto release = [&](uint32_t loaded) { arrive_after(&empty[s], loaded, zero, lane); };
            if (mine && !mbar_wait_warp(&full[s], ph, wc)) break;
            if (n_ch == 0) release(0);
#pragma unroll
            for (int ch = 0; ch < kWarpChunks; ++ch) {
                const int cl = w_at + kGroupWarps * ch;   // in the stage
                const int chunk = c0 + cl;              // in the row
                if (ch >= n_ch) break;
                // token operand of the chunk's half h, group j (`at` elements further on)
                auto load_act = [&](int h, int j, uint4 (&v)[NV], int at = 0) {
                    const int kk = (2 * chunk + h) * (SH::CHUNK_K / 2) + c * (SH::CHUNK_K / 8);
#pragma unroll
                    for (int i = 0; i < NV; ++i) {
                        v[i] = make_uint4(0, 0, 0, 0);
                        if (act[j] && kk < K)
                            v[i] = __ldcg(reinterpret_cast<const uint4 *>(act[j] + at + kk) + i);
                    }
                };
                uint4 v0[2][NV];   // group 0
                if (in_smem) {
                    const uint32_t a = smem_u32(acts + s * SH::ACT) + g * SH::ACT_PITCH +
                                       cl * (2 * SH::CHUNK_K) + c * (SH::CHUNK_K / 4);
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int i = 0; i < NV; ++i)
                            v0[h][i] = col < n ? ld_shared_v4(a + h * SH::CHUNK_K + 16 * i)
                                               : make_uint4(0, 0, 0, 0);
                } else {
                    load_act(0, 0, v0[0]);
                    load_act(1, 0, v0[1]);
                }
                // rows pr and pr + 8 of the chunk, 128 bytes each, 16-byte pieces
                // exchanged by row (128-byte swizzle)
                uint4 wq[2][2];   // [half][row pr / pr + 8]
                {
                    const uint32_t a0 =
                        smem_u32(ring + s * kFewStage) + cl * (8 * kChunk) + pr * kChunk;
                    const uint32_t b0 = a0 + kFewStage / 2;
                    const uint32_t first = (uint32_t)(c ^ pr) << 4;
                    wq[0][0] = ld_shared_v4(a0 + first);
                    wq[0][1] = ld_shared_v4(b0 + first);
                    wq[1][0] = ld_shared_v4(a0 + (first ^ 64u));
                    wq[1][1] = ld_shared_v4(b0 + (first ^ 64u));
                }
                float f0 = 1.0f, f1 = 1.0f;
                if constexpr (FP8) {
                    f0 = scales[s * 2 * kStageChunks + cl];
                    f1 = scales[(s * 2 + 1) * kStageChunks + cl];
                }
                if (ch == n_ch - 1) {
                    // something of every load from the stage: of this chunk's, and what
                    // became of the one before
                    uint32_t loaded = wq[0][0].x ^ wq[0][1].x ^ wq[1][0].x ^ wq[1][1].x;
#pragma unroll
                    for (int i = 0; i < NV; ++i) loaded ^= v0[0][i].x ^ v0[1][i].x;
                    if constexpr (FP8) loaded ^= __float_as_uint(f0) ^ __float_as_uint(f1);
                    if (ch > 0)
                        loaded ^= __float_as_uint(acc[0][0]) ^ __float_as_uint(acc[0][2]);
                    release(loaded);
                }
                if constexpr (!FP8) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint4 wa = wq[h][0], wb = wq[h][1];
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            if (j >= nt) break;
                            uint4 v[NV];
                            if (j > 0) load_act(h, j, v);
                            const uint4 b = j > 0 ? v[0] : v0[h][0];
                            mma_bf16(acc[j], wa.x, wb.x, wa.y, wb.y, b.x, b.y);
                            mma_bf16(acc[j], wa.z, wb.z, wa.w, wb.w, b.z, b.w);
                        }
                    }
                    if (terms && !beside) {   // the second terms of h
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint4 wa = wq[h][0], wb = wq[h][1];
#pragma unroll
                            for (int j = 0; j < NT; ++j) {
                                if (j >= nt) break;
                                uint4 v[NV];
                                load_act(h, j, v, p.I);
                                mma_bf16(acc[j], wa.x, wb.x, wa.y, wb.y, v[0].x, v[0].y);
                                mma_bf16(acc[j], wa.z, wb.z, wa.w, wb.w, v[0].z, v[0].w);
                            }
                        }
                    }
                } else {
                    // a contraction that ends inside a chunk: its last 64 codes
                    // are not in the stage (a copied row would run into the next)
                    const bool tail = chunk * 128 + 64 == K;
                    if (tail) {
                        const uint8_t *w = static_cast<const uint8_t *>(second ? p.W2 : p.W13);
                        const int e = q.y < 0 ? p.E : meta->pass[q.y].e;
                        const size_t r = second ? (size_t)e * p.d + q.x * 16 + pr
                                                : (size_t)e * 2 * p.I + q.x * 8 + pr;
                        w += r * K + K - 64 + c * 16;
                        wq[0][0] = __ldg(reinterpret_cast<const uint4 *>(w));
                        wq[0][1] = __ldg(
                            reinterpret_cast<const uint4 *>(w + (size_t)(second ? 8 : p.I) * K));
                        wq[1][0] = wq[1][1] = make_uint4(0, 0, 0, 0);
                        v0[1][0] = v0[1][NV - 1] = make_uint4(0, 0, 0, 0);
                    }
                    // the block of 128, not yet scaled; two sums, so that each
                    // MMA need not wait for the one before it
                    float part[NT][2][4];
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) part[j][0][i] = part[j][1][i] = 0.0f;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t qa[4] = {wq[h][0].x, wq[h][0].y, wq[h][0].z, wq[h][0].w};
                        const uint32_t qb[4] = {wq[h][1].x, wq[h][1].y, wq[h][1].z, wq[h][1].w};
                        uint32_t x0[4], x1[4], y0[4], y1[4];
#pragma unroll
                        for (int m = 0; m < 4; ++m) {
                            e4m3x4_f16(qa[m], x0[m], x1[m]);
                            e4m3x4_f16(qb[m], y0[m], y1[m]);
                            if (WIDE && second) {   // h is bf16: so are they, exactly
                                x0[m] = f16x2_bf16x2(x0[m]);
                                x1[m] = f16x2_bf16x2(x1[m]);
                                y0[m] = f16x2_bf16x2(y0[m]);
                                y1[m] = f16x2_bf16x2(y1[m]);
                            }
                        }
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            if (j >= nt) break;
                            uint4 v[NV];
                            if (j > 0) load_act(h, j, v);
                            const uint4 *b = j > 0 ? v : v0[h];
                            const uint32_t bv[8] = {b[0].x, b[0].y, b[0].z, b[0].w,
                                                    b[NV - 1].x, b[NV - 1].y, b[NV - 1].z,
                                                    b[NV - 1].w};
#pragma unroll
                            for (int m = 0; m < 4; ++m) {
                                if (WIDE && second)
                                    mma_bf16(part[j][m & 1], x0[m], y0[m], x1[m], y1[m], bv[2 * m],
                                             bv[2 * m + 1]);
                                else
                                    mma_f16(part[j][m & 1], x0[m], y0[m], x1[m], y1[m], bv[2 * m],
                                            bv[2 * m + 1]);
                            }
                            if (WIDE && terms && !beside) {   // the second terms of h
                                load_act(h, j, v, p.I);
                                const uint32_t lo[8] = {v[0].x, v[0].y, v[0].z, v[0].w,
                                                        v[NV - 1].x, v[NV - 1].y, v[NV - 1].z,
                                                        v[NV - 1].w};
#pragma unroll
                                for (int m = 0; m < 4; ++m)
                                    mma_bf16(part[j][m & 1], x0[m], y0[m], x1[m], y1[m], lo[2 * m],
                                             lo[2 * m + 1]);
                            }
                        }
                    }
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        acc[j][0] = fmaf(part[j][0][0] + part[j][1][0], f0, acc[j][0]);
                        acc[j][1] = fmaf(part[j][0][1] + part[j][1][1], f0, acc[j][1]);
                        acc[j][2] = fmaf(part[j][0][2] + part[j][1][2], f1, acc[j][2]);
                        acc[j][3] = fmaf(part[j][0][3] + part[j][1][3], f1, acc[j][3]);
                    }
                }
            }
            if (++s == STAGES) { s = 0; ph ^= 1u; }
            if (!(q.w & kLast)) continue;
            if (p.by_tile && !mine) continue;
            // the tile's partial sums, one buffer per group of 8 rows
            bool ok = true;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                if (j >= nt) break;
                const uint32_t buf = buffer(unit);
                ok = mbar_wait_warp(&rempty[buf], (unit >> 1 & 1u) ^ 1u, wc);
                if (!ok) break;
                const int w0 = p.by_tile ? buf * kGroupWarps : buf * kMulWarps + role * kGroupWarps;
                red[(w0 + wl) * 32 + lane] =
                    make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
                if (role == 0 && wl == 0 && lane == 0)
                    *reinterpret_cast<int4 *>(&rinfo[buf]) =
                        make_int4(q.x, q.y, q.z, j | (q.w & kSecond));
                __syncwarp();
                if (lane == 0) mbar_arrive(&rfull[buf]);
                ++unit;
            }
            if (!ok) break;
        }
    } else if (warp == kTicketWarp) {
        // ------------------------------------------------------ item numbers
        // from the grid's counter, one ahead of the copies (two ahead left the CTAs less
        // even at the end: one token 58.0 us, 57.7 so).  A warp of its own: the counter
        // answers after a microsecond, and whoever waits for it does nothing else (a
        // warp's arrivals on barriers wait for its outstanding atomics too).
        int n_pass = -1;
        for (uint32_t n = 0;; ++n) {
            if (!mbar_wait_warp(qempty, (n & 1u) ^ 1u, wc) || *stop_s) break;
            int t = 0;
            if (lane == 0) t = atomicAdd(p.counters + 1, 1);
            t = __shfl_sync(0xffffffffu, t, 0);
            if (S > 32 && t >= tiles1 && n_pass < 0) {
                n_pass = few_list<NT>(p, S, meta, lane, wc);
                if (n_pass < 0) break;
                if (lane == 0) meta->n_pass = n_pass;
            }
            if (lane == 0) {
                *queue = t;
                mbar_arrive(qfull);
            }
            __syncwarp();
        }
    } else {
        // ------------------------------------------- sums over the warps
        const int me = warp - kSumWarp0;
        const int g = few_row(lane >> 2), c = lane & 3;
        for (uint32_t m = 0;; ++m) {
            const uint32_t buf = p.by_tile ? 2 * me + (m & 1u) : me;
            if (!mbar_wait_warp(&rfull[buf], (p.by_tile ? m >> 1 : m) & 1u, wc)) break;
            const int4 q = ld_tile(&rinfo[buf]);
            if (q.x < 0) break;
            const float4 *from = red + buf * (p.by_tile ? kGroupWarps : kMulWarps) * 32 + lane;
            float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int w = 0; w < kMulWarps; ++w) {
                if (w == kGroupWarps && p.by_tile) break;
                const float4 r = from[w * 32];
                v[0] += r.x;
                v[1] += r.y;
                v[2] += r.z;
                v[3] += r.w;
            }
            arrive_after(&rempty[buf], __float_as_uint(v[0]), zero, lane);
            const int n = q.z & 0xFFFF, row0 = q.z >> 16, grp = q.w & kChunkMask;
            const bool second = q.w & kSecond;
            // v[0], v[1]: weight row g, tokens 2c and 2c + 1; v[2], v[3]: row g + 8
            // (or token c's two terms of h)
            const bool beside = SH::TERMS == 2 && second && n <= 4;
            if (beside) {
                v[0] += v[1];
                v[2] += v[3];
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = beside ? c : grp * 8 + 2 * c + i;
                if (r >= n || (beside && i > 0)) continue;
                const int slot = q.y < 0 ? S + r : meta->slot[row0 + r];
                if (second) {
                    const float w = (q.y < 0 ? 1.0f : meta->w[slot]) *
                                    (FP8 ? exp2i(-p.h_exp) : 1.0f);
                    float *o = p.yp + (size_t)slot * p.d + q.x * 16 + g;
                    o[0] = w * v[i];
                    o[8] = w * v[2 + i];
                } else {
                    float up = 1.0f;
                    if constexpr (FP8) up = __ldcg(p.x16_s + (q.y < 0 ? r : meta->token[row0 + r]));
                    const float h = swiglu_clamped_nan(v[i] * up, v[2 + i] * up, p.clamp);
                    const size_t o = (size_t)slot * SH::TERMS * p.I + q.x * 8 + g;
                    if constexpr (SH::TERMS == 1) {
                        p.h[o] = __half_as_ushort(__float2half_rn(h * exp2i(p.h_exp)));
                    } else {
                        const uint32_t top = pack_bf16x2(h, 0.0f) & 0xFFFFu;
                        const float rest = h - bf16_lo(top);   // exact, or not finite
                        p.h[o] = (uint16_t)top;
                        p.h[o + p.I] =
                            isfinite(rest) ? (uint16_t)(pack_bf16x2(rest, 0.0f) & 0xFFFFu) : 0;
                    }
                }
            }
            fence_proxy_async_global();   // copies will read h
            __syncwarp();
            if (lane == 0) red_release_gpu_add(second ? y_done + q.x : h_done + 1 + q.y, 1);
        }
    }

    // The columns of this CTA: every product of a tile's 16 columns is there once
    // all its items have signalled; they are added up in slot order.
    __syncthreads();
    for (int tile = blockIdx.x; tile < tiles2; tile += gridDim.x) {
        if (threadIdx.x == 0) wait_count_geq(y_done + tile, meta->n_units, wc);
        __syncthreads();
        for (int i = threadIdx.x; i < p.T * 16; i += kFewThreads) {
            const int tk = i >> 4, n16 = tile * 16 + (i & 15);
            float v[kFewK + 1];
            v[0] = __ldcg(p.yp + (size_t)(S + tk) * p.d + n16);
#pragma unroll
            for (int j = 0; j < kFewK; ++j)
                v[j + 1] = j < p.k ? __ldcg(p.yp + (size_t)(tk * p.k + j) * p.d + n16) : 0.0f;
            float sum = v[0];
#pragma unroll
            for (int j = 0; j < kFewK; ++j) sum += v[j + 1];
            p.y[(size_t)tk * p.d + n16] = (uint16_t)(pack_bf16x2(sum, 0.0f) & 0xFFFFu);
        }
    }

    // The first kernel stores ids and weights after the slots that say they are there.
    // It has long ended, but only this wait makes its end, and those stores, come before
    // the end of this kernel, which is what whoever runs next on the stream waits for.
    // The last CTA to leave puts every counter and slot back to zero.
    __syncthreads();
    if (threadIdx.x == 0) {
        wait_for_kernels_ahead();
        *last_s = atom_add_acq_rel(p.counters + 2, 1) == (int)gridDim.x - 1;
    }
    __syncthreads();
    if (*last_s) {
        for (int i = threadIdx.x; i < p.n_counters; i += kFewThreads) p.counters[i] = 0;
        for (int i = threadIdx.x; i < S; i += kFewThreads) p.routed[i] = 0;
    }
}

size_t up256(size_t b) { return (b + 255) / 256 * 256; }

struct FewWorkspace {
    int *counters;
    int n_counters;
    float *part;
    uint16_t *x16;
    float *x16_s;
    uint64_t *routed;
    uint16_t *h;
    float *yp;
    size_t bytes;
};

FewWorkspace carve_few(uint8_t *base, int T, int d, int E, int k, int I) {
    FewWorkspace w;
    size_t off = 0;
    auto take = [&](size_t b) {
        uint8_t *q = base + off;
        off += up256(b);
        return q;
    };
    const size_t S = (size_t)T * k;
    w.n_counters = 4 + 1 + kFewS + d / 16;
    w.counters = reinterpret_cast<int *>(take((size_t)w.n_counters * 4));
    w.part = reinterpret_cast<float *>(take((size_t)kGateSplits * T * E * 4));
    w.x16 = reinterpret_cast<uint16_t *>(take((size_t)T * d * 2));
    w.x16_s = reinterpret_cast<float *>(take((size_t)T * 4));
    w.routed = reinterpret_cast<uint64_t *>(take(S * 8));
    w.h = reinterpret_cast<uint16_t *>(take((S + T) * I * 4));   // of two terms, or half of it
    w.yp = reinterpret_cast<float *>(take((S + T) * d * 4));
    w.bytes = off;
    return w;
}

template <bool FP8, int NT, bool WIDE>
moe_status launch_experts(const FewParams &p, cudaStream_t st) {
    using SH = FewShape<FP8, NT, WIDE>;
    auto kern = few_experts_kernel<FP8, NT, WIDE>;
    static bool attr_set[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
    if (dev < 0 || dev >= 64) return MOE_ERR_UNSUPPORTED;
    if (!attr_set[dev]) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SH::SMEM) !=
            cudaSuccess)
            return MOE_ERR_CUDA;
        attr_set[dev] = true;
    }
    const long long items = (long long)(p.T * p.k + 1) * (p.I / 8 + p.d / 16);
    return launch_early(kern, dim3((unsigned)(items < num_sms() ? items : num_sms())), kFewThreads,
                        SH::SMEM, st, p);
}

template <bool FP8, bool WIDE>
moe_status launch_experts_nt(const FewParams &p, cudaStream_t st) {
    // rows of an expert that share one read of its weights: as many groups of
    // 8 as there can be tokens
    if (p.T <= 8) return launch_experts<FP8, 1, WIDE>(p, st);
    if (p.T <= 16) return launch_experts<FP8, 2, WIDE>(p, st);
    return launch_experts<FP8, 4, WIDE>(p, st);
}

}  // namespace

// Rows of `row_bytes` bytes as [row_bytes / 128][rows][128]: a box of 16 x 8 x
// 128 is 16 whole chunks of eight rows, eight rows of a chunk side by side.
// `cps`: chunks of a row in a stage -- the fewest stages, evenly filled.
static bool encode_rows_of_chunks(CUtensorMap *tm, const void *base, uint64_t rows, int row_bytes,
                                  int *cps) {
    const int all = (row_bytes + kChunk - 1) / kChunk;
    const int stages = (all + kStageChunks - 1) / kStageChunks;
    *cps = (all + stages - 1) / stages;
    const int chunks = row_bytes / kChunk;
    return encode_tmap_u8_3d_sw128(tm, base, chunks > 0 ? kChunk : row_bytes, rows,
                                   chunks > 0 ? chunks : 1, row_bytes, kChunk, kChunk, 8, *cps);
}

bool few_supported(int T, int d, int E, int k, int I) {
    return T >= 1 && T <= kFewT && d >= 128 && d % 128 == 0 && I >= 64 && I % 64 == 0 && E >= 1 &&
           E <= kFewE && k >= 1 && k <= kFewK && k <= E && d <= (1 << 20) && I <= (1 << 20);
}

size_t few_workspace_bytes(int T, int d, int E, int k, int I) {
    return carve_few(nullptr, T, d, E, k, I).bytes;
}

moe_status launch_few(const moe_few_args *a, cudaStream_t st) {
    const FewWorkspace w =
        carve_few(static_cast<uint8_t *>(a->ws), a->T, a->d, a->E, a->k, a->I);
    FewParams p{};
    p.x = a->x;
    p.W_g = a->W_g;
    p.logit_offset = a->logit_offset;
    p.bias = a->bias;
    p.is_vision = a->is_vision;
    p.input_ids = a->input_ids;
    p.tid2eid = a->tid2eid;
    p.vocab = a->vocab;
    p.T = a->T;
    p.d = a->d;
    p.E = a->E;
    p.k = a->k;
    p.I = a->I;
    p.hash = a->mode == MOE_ROUTE_HASH;
    p.scaling = a->scaling;
    p.clamp = a->clamp;
    const bool fp8 = a->W13_q != nullptr;
    p.W13 = fp8 ? static_cast<const void *>(a->W13_q) : a->W13;
    p.W2 = fp8 ? static_cast<const void *>(a->W2_q) : a->W2;
    p.W13_s = a->W13_s;
    p.W2_s = a->W2_s;
    p.y = a->y;
    p.ids_out = a->ids;
    p.w_out = a->weights;
    p.counters = w.counters;
    p.n_counters = w.n_counters;
    p.part = w.part;
    p.x16 = w.x16;
    p.x16_s = w.x16_s;
    p.routed = w.routed;
    p.h = w.h;
    p.yp = w.yp;
    p.status = device_status_ptr();
    if (!p.status) return MOE_ERR_CUDA;
    p.wait_limit = kWaitLimitCycles;
    const int elt = fp8 ? 1 : 2;
    if (!encode_rows_of_chunks(&p.tm13, p.W13, (uint64_t)(p.E + 1) * 2 * p.I, p.d * elt,
                               &p.cps13) ||
        !encode_rows_of_chunks(&p.tm2, p.W2, (uint64_t)(p.E + 1) * p.d, p.I * elt, &p.cps2))
        return MOE_ERR_CUDA;
    // tiles of one or two stages: see the multiplying warps
    p.by_tile = p.d * elt <= 2 * p.cps13 * kChunk && p.I * elt <= 2 * p.cps2 * kChunk;
    const int et = (p.E + 15) / 16;
    int splits = num_sms() / et;   // one round: an SM takes one CTA of many experts
    splits = splits < 1 ? 1 : splits > kGateSplits ? kGateSplits : splits;
    if (splits > p.d / 32) splits = p.d / 32;
    p.splits = splits;
    // |h| <= clamp^2: the power of two that keeps it inside f16.  Where none does, h is
    // two bf16 terms as with bf16 weights, and the codes become bf16 too (through fp32:
    // eight more instructions for eight of them).
    const bool wide = !(p.clamp * p.clamp <= 65504.0f);
    p.h_exp = 0;
    while (p.h_exp < 24 && p.clamp * p.clamp * (float)(2 << p.h_exp) <= 65504.0f) ++p.h_exp;
    const dim3 grid(et, splits + (fp8 ? (p.T + et - 1) / et : 0));
    const moe_status s =
        launch_early(p.E <= 128   ? few_gate_kernel<4>
                     : p.E <= 384 ? few_gate_kernel<12>
                                  : few_gate_kernel<32>,
                     grid, kGateWarps * 32, 0, st, p);
    if (s != MOE_OK) return s;
    return !fp8   ? launch_experts_nt<false, false>(p, st)
           : wide ? launch_experts_nt<true, true>(p, st)
                  : launch_experts_nt<true, false>(p, st);
}

}  // namespace moe
