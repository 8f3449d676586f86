// ndq_lora.cu -- low-rank adapters of many requests beside a shared
// projection: y[m] = base[m] + scale * (x[m] A^T) B^T.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ndq_serve.h"

namespace ndq {
namespace {

__device__ __forceinline__ float bf(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }

// t[m, j] = scale * sum_k x[m, k] A[a, j, k]: a warp per (m, j).
__global__ void __launch_bounds__(256) k_lora_shrink(const LoraParams p) {
    const int64_t wid = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int64_t m = wid / p.rmax, j = wid % p.rmax;
    const uint32_t lane = threadIdx.x & 31u;
    if (m >= p.M) return;
    const int32_t a = p.index[m];
    if (a < 0 || a >= p.nA || j >= p.ranks[a]) return;
    const uint16_t* x = p.x + m * p.K;
    const uint16_t* w = p.a + (static_cast<int64_t>(a) * p.rmax + j) * p.K;
    float s = 0.0f;
    for (int64_t k = lane; k < p.K; k += 32) s = __fmaf_rn(bf(x[k]), bf(w[k]), s);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    if (lane == 0) p.t[m * p.rmax + j] = __fmul_rn(s, p.scales[a]);
}

// y[m, n] = base[m, n] + sum_j t[m, j] B[a, n, j]: a thread per output.
template <bool F32>
__global__ void __launch_bounds__(256) k_lora_expand(const LoraParams p) {
    const int64_t n = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (n >= p.N) return;
    for (int64_t m = blockIdx.y; m < p.M; m += gridDim.y) {
        const int32_t a = p.index[m];
        const int64_t o = m * p.N + n;
        float s = 0.0f;
        if (a >= 0 && a < p.nA) {
            int32_t r = p.ranks[a];
            r = r < p.rmax ? r : static_cast<int32_t>(p.rmax);
            const uint16_t* w = p.b + (static_cast<int64_t>(a) * p.N + n) * p.rmax;
            for (int32_t j = 0; j < r; ++j) s = __fmaf_rn(p.t[m * p.rmax + j], bf(w[j]), s);
        }
        if constexpr (F32)
            static_cast<float*>(p.y)[o] = __fadd_rn(static_cast<const float*>(p.base)[o], s);
        else
            static_cast<__nv_bfloat16*>(p.y)[o] =
                __float2bfloat16_rn(__fadd_rn(bf(static_cast<const uint16_t*>(p.base)[o]), s));
    }
}

}  // namespace

size_t lora_workspace_bytes(int64_t M, int64_t rmax, int64_t) {
    return static_cast<size_t>(M > 0 ? M : 1) * static_cast<size_t>(rmax) * 4u + 16u;
}

int launch_lora(const LoraParams& p, bool out_f32, void* stream) {
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (p.nA > 0)
        k_lora_shrink<<<static_cast<unsigned>((p.M * p.rmax + 7) / 8), 256, 0, st>>>(p);
    const dim3 grid(static_cast<unsigned>((p.N + 255) / 256), static_cast<unsigned>(p.M < 65535 ? p.M : 65535));
    if (out_f32) k_lora_expand<true><<<grid, 256, 0, st>>>(p);
    else k_lora_expand<false><<<grid, 256, 0, st>>>(p);
    return static_cast<int>(cudaGetLastError());
}

}  // namespace ndq
