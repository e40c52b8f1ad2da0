// gate_bwd.cu -- a dense gradient at the gate's logits (the balance loss's) into the input's
// and the gate weight's:
//   dX += dz W_g,   dW_g += dz^T x
// Both products run on the tensor cores, as one group of the layer's data-gradient and
// weight-gradient matmuls.  dz is their bf16 operand (off by at most 2^-8 of itself; sums over
// the tokens average that out), padded with zeros to whole tiles of 128 experts; dz W_g is rounded to
// bf16 before it is added.  Measured: 0.87 ms at 65536 tokens, d = 4096, E = 384 (127 us at
// 8192), 1.3 % of the layer's step there; so the sums stay a pass of their own, which
// leaves that backward as it is.
#include "fp8_common.cuh"

namespace moe {
namespace {

int padded(int E) { return (E + 127) / 128 * 128; }

// dz fp32 [T, E] -> bf16 [T, Ep], zeros behind E; the group's offsets.
__global__ void __launch_bounds__(256)
    gate_dz_kernel(const float *__restrict__ dz, int T, int E, int Ep, uint32_t *__restrict__ out,
                   int32_t *__restrict__ offsets) {
    if (blockIdx.x == 0 && threadIdx.x < 2) offsets[threadIdx.x] = threadIdx.x ? T : 0;
    const long long n = (long long)T * (Ep / 2);
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n;
         i += (long long)gridDim.x * blockDim.x) {
        const long long t = i / (Ep / 2);
        const int e = (int)(i - t * (Ep / 2)) * 2;
        const float a = e < E ? __ldg(dz + t * E + e) : 0.0f;
        const float b = e + 1 < E ? __ldg(dz + t * E + e + 1) : 0.0f;
        out[i] = pack_bf16x2(a, b);
    }
}

__global__ void __launch_bounds__(256)
    gate_add_kernel(const uint4 *__restrict__ g, long long n, uint4 *__restrict__ dX) {
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n;
         i += (long long)gridDim.x * blockDim.x) {
        const uint4 a = __ldcs(g + i), b = dX[i];
        const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
        uint32_t s[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            s[j] = pack_bf16x2(bf16_lo(x[j]) + bf16_lo(y[j]), bf16_hi(x[j]) + bf16_hi(y[j]));
        dX[i] = make_uint4(s[0], s[1], s[2], s[3]);
    }
}

__global__ void __launch_bounds__(256)
    gate_addw_kernel(const float4 *__restrict__ g, long long n, float4 *__restrict__ dW) {
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n;
         i += (long long)gridDim.x * blockDim.x) {
        const float4 a = g[i];
        float4 b = dW[i];
        b.x += a.x;
        b.y += a.y;
        b.z += a.z;
        b.w += a.w;
        dW[i] = b;
    }
}

size_t up(size_t b) { return (b + 255) / 256 * 256; }

int blocks_for(long long n) {
    const long long want = (n + 255) / 256, most = (long long)num_sms() * 16;
    return (int)(want < most ? want : most);
}

}  // namespace

size_t gate_bwd_workspace_bytes(int T, int d, int E) {
    const int Ep = padded(E);
    return up((size_t)T * Ep * 2) + up((size_t)T * d * 2) + up((size_t)Ep * d * 4) +
           up(kWgradScratchBytes) + 256;
}

moe_status launch_gate_bwd(const float *dlogits, const uint16_t *x, const uint16_t *W_g, int T,
                           int d, int E, uint16_t *dX, float *dW_g, void *ws, cudaStream_t st) {
    const int Ep = padded(E);
    uint8_t *at = static_cast<uint8_t *>(ws);
    auto take = [&](size_t bytes) {
        uint8_t *p = at;
        at += up(bytes);
        return p;
    };
    uint16_t *dz = reinterpret_cast<uint16_t *>(take((size_t)T * Ep * 2));
    uint16_t *gx = reinterpret_cast<uint16_t *>(take((size_t)T * d * 2));
    float *gw = reinterpret_cast<float *>(take((size_t)Ep * d * 4));
    uint8_t *scratch = take(kWgradScratchBytes);
    int32_t *offsets = reinterpret_cast<int32_t *>(take(8));
    gate_dz_kernel<<<blocks_for((long long)T * (Ep / 2)), 256, 0, st>>>(
        dlogits, T, E, Ep, reinterpret_cast<uint32_t *>(dz), offsets);
    moe_status s = cuda_status(cudaGetLastError());
    if (s == MOE_OK && dX) {
        s = launch_dgrad1(dz, offsets, 1, T, W_g, d, Ep / 2, gx, st, E);
        const long long n = (long long)T * (d / 8);
        if (s == MOE_OK)
            gate_add_kernel<<<blocks_for(n), 256, 0, st>>>(reinterpret_cast<const uint4 *>(gx), n,
                                                           reinterpret_cast<uint4 *>(dX));
        if (s == MOE_OK) s = cuda_status(cudaGetLastError());
    }
    if (s == MOE_OK && dW_g) {
        s = launch_wgrad(dz, Ep, x, d, offsets, 1, T, gw, scratch, st);
        const long long n = (long long)E * (d / 4);
        if (s == MOE_OK)
            gate_addw_kernel<<<blocks_for(n), 256, 0, st>>>(reinterpret_cast<const float4 *>(gw), n,
                                                            reinterpret_cast<float4 *>(dW_g));
        if (s == MOE_OK) s = cuda_status(cudaGetLastError());
    }
    return s;
}

}  // namespace moe
