// ndq_attn_join.cu -- the parts of rows of attention joined (k_attn_join).
//
//     out = sum_k 2^(m_k - M) o_k / sum_k 2^(m_k - M) l_k,   M = max_k m_k
//
// over the parts k that the kernel of the shared prefix and the one of a
// request's own tokens left of a row: values o, maximum m and sum l, 4 (D + 4)
// bytes a part.  A warp takes a row: its lanes read the statistics of 32 parts
// at once, then every part's values together, eight loads under way.  (Joined
// in the kernel of the own tokens, by the last to arrive, rows of short
// requests came one after another on one CTA: 64 requests of 0 to 2000 tokens
// behind 32000, 32 heads, took 91 us there, 48 without the join.)
#include <cuda_runtime.h>

#include "ndq_attn.cuh"

namespace ndq {
namespace {

constexpr int kJoinWarps = 8;

template <int D, bool BF16>
__global__ void __launch_bounds__(kJoinWarps * 32) k_attn_join(const __grid_constant__ PrefixParams p) {
    constexpr int N = D / 32;  // head positions of a lane
    constexpr uint32_t B = 8;
    const uint32_t lane = threadIdx.x & 31u;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kJoinWarps + (threadIdx.x >> 5);
    bool valid = row < p.n_tokens * p.q_heads;
    bool shares = false;
    if (valid) {  // whose row it is, and whether the own rows' kernel left parts of it
        const int32_t t = static_cast<int32_t>(row) / p.q_heads;
        int64_t r = t;
        if (p.q_start) {
            // requests of one length, mostly; else the last that starts at t or before
            r = static_cast<int64_t>(t) * p.n_req / p.n_tokens;
            if (!(p.q_start[r] <= t && t < p.q_start[r + 1])) {
                int64_t a = 0, b = p.n_req;
                while (b - a > 1) {
                    const int64_t m = (a + b) >> 1;
                    if (p.q_start[m] <= t) a = m;
                    else b = m;
                }
                r = a;
            }
        }
        int64_t q0;
        int32_t n, pos;
        attn_request(p, r, q0, n, pos);
        valid = q0 <= t && t < q0 + n && !(p.prompt_rows > 0 && static_cast<int64_t>(n) * p.group >= p.prompt_rows);
        shares = shared_tokens(p, r) > 0;
    }
    attn_pdl_wait();
    if (!valid) return;
    const uint2 own = __ldcg(static_cast<const uint2*>(p.own_records) + row);
    RowParts<D> prefix(p, row);
    if (!shares) prefix.n = 0;
    // (whatever a record holds, no read leaves the parts)
    const uint32_t n_own = own.x + static_cast<uint64_t>(own.y) <= static_cast<uint64_t>(p.own_rows) ? own.y : 0u, n = prefix.n + n_own;
    const float* own_first = p.own_slots + static_cast<uint64_t>(own.x) * (D + 4);
    auto part = [&](uint32_t k) { return k < prefix.n ? prefix.part(k) : own_first + static_cast<uint64_t>(k - prefix.n) * (D + 4); };
    auto stat = [&](uint32_t k) { return __ldcg(reinterpret_cast<const float2*>(part(k) + D)); };

    float M = -INFINITY;
    for (uint32_t k = lane; k < n; k += 32) M = fmaxf(M, stat(k).x);
#pragma unroll
    for (int e = 1; e < 32; e <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, e));
    float L = 0.0f, acc[N];
#pragma unroll
    for (int e = 0; e < N; ++e) acc[e] = 0.0f;
    for (uint32_t k0 = 0; k0 < n; k0 += 32) {
        float f = -1.0f;  // (left out: it saw nothing, or is none)
        if (k0 + lane < n) {
            const float2 x = stat(k0 + lane);
            if (x.x != -INFINITY || x.y != x.y) {
                const float hf = part_root(x.x, M);
                f = hf * hf;
                L = __fmaf_rn(x.y * hf, hf, L);
            }
        }
        const uint32_t here = n - k0 < 32 ? n - k0 : 32;
        for (uint32_t j = 0; j < here; j += B) {
            float v[B][N], w[B];
#pragma unroll
            for (uint32_t i = 0; i < B; ++i) {
                w[i] = __shfl_sync(0xffffffffu, f, static_cast<int>((j + i) & 31u));
                if (j + i >= here || !(w[i] >= 0.0f)) {
                    w[i] = -1.0f;
                    continue;
                }
                const float* src = part(k0 + j + i) + lane * N;
                if constexpr (N == 4) {
                    const float4 x = __ldcg(reinterpret_cast<const float4*>(src));
                    v[i][0] = x.x;
                    v[i][1] = x.y;
                    v[i][2] = x.z;
                    v[i][3] = x.w;
                } else {
                    const float2 x = __ldcg(reinterpret_cast<const float2*>(src));
                    v[i][0] = x.x;
                    v[i][1] = x.y;
                }
            }
#pragma unroll
            for (uint32_t i = 0; i < B; ++i)
                if (w[i] >= 0.0f) {
#pragma unroll
                    for (int e = 0; e < N; ++e) acc[e] = __fmaf_rn(v[i][e], w[i], acc[e]);
                }
        }
    }
#pragma unroll
    for (int e = 1; e < 32; e <<= 1) L += __shfl_xor_sync(0xffffffffu, L, e);
    const float inv = L > 0.0f ? __fdiv_rn(1.0f, L) : (L == L ? 0.0f : L);
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + row * D) + lane * (N / 2);
    if constexpr (N == 4)
        *reinterpret_cast<uint2*>(dst) = make_uint2(narrow2<BF16>(acc[0] * inv, acc[1] * inv), narrow2<BF16>(acc[2] * inv, acc[3] * inv));
    else
        *dst = narrow2<BF16>(acc[0] * inv, acc[1] * inv);
    if (p.lse && lane == 0) p.lse[row] = L > 0.0f ? (M + log2f(L)) * 0.6931471805599453f : (L == L ? -INFINITY : L);
}

template <int D, bool BF16>
int launch_join(const PrefixParams& p, void* stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((p.n_tokens * p.q_heads + kJoinWarps - 1) / kJoinWarps));
    cfg.blockDim = dim3(kJoinWarps * 32);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return static_cast<int>(cudaLaunchKernelEx(&cfg, k_attn_join<D, BF16>, p));
}

}  // namespace

int launch_prefix_join(const PrefixParams& p, int head_dim, bool bf16, void* stream) {
    if (head_dim == 64) return bf16 ? launch_join<64, true>(p, stream) : launch_join<64, false>(p, stream);
    return bf16 ? launch_join<128, true>(p, stream) : launch_join<128, false>(p, stream);
}

}  // namespace ndq
