// ndq_rope.cu -- norms of query and key heads and their rotation by position,
// in one pass:
//
//     z = x / sqrt(mean(x^2) + eps) * weight          (or x, without a weight)
//     (a, b) -> (a cos - b sin, a sin + b cos),  angle = position * inv_freq[i]
//
// for the pairs i of a head's first rot_dim values: (i, i + rot_dim / 2), or
// (2 i, 2 i + 1) when interleaved.  Bound by bytes: every head is read and
// written once.
//
// Work.  A head is taken by L lanes (the power of two at or above D / 16), each
// holding two 16-byte pieces (eight values) whose values pair up with one
// another, so that a rotation needs no exchange and every load and store
// instruction of a group covers whole sectors.  A warp takes one token, or a
// part of its heads when there are few tokens, 32 / L heads at a time; the next
// heads' loads go out before these are computed.
//
// Angles.  A binary32 product position * inv_freq is off by 2^-24 of itself:
// radians, far out.  Here each frequency becomes a fraction of a turn in 64
// bits (its mantissa times 2^64 / (2 pi), in integers), the product with the
// position wraps by itself, and the top 32 bits are the angle to 2^-31 of a
// turn for every position below 2^31.  binary32 holds 24 of them: cosine and sine
// are taken of the top ones and corrected by the rest (a + d: cos a - d sin a,
// sin a + d cos a).  The cosines of a token are computed once a warp: its lane
// groups take different pairs and exchange them.
//
// Measured: 16001 tokens of 40 heads of 128, bfloat16, with norms: 56.4 us, 5.8
// TB/s, 0.86 of the copy bandwidth; 5003 tokens of 72 heads, binary32 in: 48.9 us,
// 5.7 TB/s.  64 tokens: 5.4 us, latency.
#include <cuda_runtime.h>

#include <cstdint>

#include "ndq_attn.cuh"
#include "ndq_device.cuh"
#include "ndq_once.h"
#include "ndq_rope.h"

namespace ndq {
namespace {

constexpr int kRopeWarps = 4;
constexpr int kRopeMaxDim = 256;
constexpr float kRadians = 0x1.921fb6p-30f;  // 2 pi / 2^32
// CTAs of an SM, and of the grid for each SM.  16001 tokens of 40 heads of 128,
// bfloat16: 57.1 us with 6, 61.1 with 5, 65.7 as the compiler would have it (4),
// and 59.5 against 61.1 when no CTA comes after the resident ones.
constexpr int rope_ctas(int in) { return in == 0 ? 5 : 6; }

struct RopeShared {
    uint64_t turn[kRopeMaxDim / 2];  // turns per position, in units of 2^-64
    alignas(16) float w[2][kRopeMaxDim];
};

// inv_freq / (2 pi) modulo 1 in units of 2^-64.  For magnitudes up to 1 the
// error is two units; what lies above grows with the magnitude.  (NaN and
// infinity: some finite frequency.)
__device__ __forceinline__ uint64_t turns(float f) {
    constexpr uint64_t kInv2Pi = 0x28be60db9391054aull;  // floor(2^64 / (2 pi))
    const uint32_t b = __float_as_uint(f);
    const int e = static_cast<int>((b >> 23) & 0xffu);
    const uint64_t m = (b & 0x7fffffu) | (e > 0 ? 0x800000u : 0u);
    const int s = (e > 0 ? e : 1) - 150;  // f = m 2^s
    const uint64_t lo = m * kInv2Pi, hi = __umul64hi(m, kInv2Pi);
    uint64_t t;
    if (s <= -128) t = 0;
    else if (s <= -64) t = hi >> (-s - 64);
    else if (s < 0) t = (hi << (64 + s)) | (lo >> -s);
    else t = s < 64 ? lo << s : 0;
    return (b >> 31) != 0 ? 0 - t : t;
}

template <int IN>
__device__ __forceinline__ void load8(const void* p, int64_t at, uint4* r) {
    if constexpr (IN == 0) {
        const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + at);
        r[0] = q[0];
        r[1] = q[1];
    } else {
        r[0] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
    }
}
template <int IN>
__device__ __forceinline__ void widen8(const uint4* r, float2* v) {
    if constexpr (IN == 0) {
        v[0] = make_float2(__uint_as_float(r[0].x), __uint_as_float(r[0].y));
        v[1] = make_float2(__uint_as_float(r[0].z), __uint_as_float(r[0].w));
        v[2] = make_float2(__uint_as_float(r[1].x), __uint_as_float(r[1].y));
        v[3] = make_float2(__uint_as_float(r[1].z), __uint_as_float(r[1].w));
    } else {
        widen2<IN == 1>(r[0].x, v[0].x, v[0].y);
        widen2<IN == 1>(r[0].y, v[1].x, v[1].y);
        widen2<IN == 1>(r[0].z, v[2].x, v[2].y);
        widen2<IN == 1>(r[0].w, v[3].x, v[3].y);
    }
}

// IN: the inputs' type; BF16: the outputs'; L: lanes of a head.
template <int L, int IN, bool BF16>
__global__ void __launch_bounds__(kRopeWarps * 32, rope_ctas(IN)) k_rope(const __grid_constant__ RopeParams p) {
    constexpr int G = 32 / L;               // heads at a time
    constexpr int R = IN == 0 ? 2 : 1;      // 16-byte words of eight inputs
    constexpr int C = (8 + G - 1) / G;      // cosines that a lane computes
    constexpr int N = IN == 0 ? 1 : 2;      // rounds of heads whose loads are under way
    __shared__ RopeShared S;
    const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31u;
    const int g = static_cast<int>(lane) / L, j = static_cast<int>(lane) % L;
    const int D = p.head_dim, rot = p.rot_dim;
    attn_pdl_wait();  // (the rows are the previous kernel's)
    for (int i = static_cast<int>(tid); i < rot / 2; i += kRopeWarps * 32) S.turn[i] = turns(p.inv_freq[i]);
    for (int i = static_cast<int>(tid); i < D; i += kRopeWarps * 32) {
        S.w[0][i] = p.q_weight ? p.q_weight[i] : 1.0f;
        S.w[1][i] = p.k_weight ? p.k_weight[i] : 1.0f;
    }
    __syncthreads();

    // this lane's pieces: a (values 8 pa ..) and b (8 pb ..)
    const bool live = j < D / 16, turned = j < rot / 16;
    const int pa = !live ? 0 : turned ? j : rot / 8 + 2 * (j - rot / 16);
    const int pb = !live ? 0 : turned ? j + rot / 16 : pa + 1;
    const float inv_dim = 1.0f / static_cast<float>(D);

    const uint32_t parts = static_cast<uint32_t>(p.parts);
    for (uint64_t unit = static_cast<uint64_t>(blockIdx.x) * kRopeWarps + warp; unit < static_cast<uint64_t>(p.n_tokens) * parts;
         unit += static_cast<uint64_t>(gridDim.x) * kRopeWarps) {
        const uint32_t t = parts == 1 ? static_cast<uint32_t>(unit) : static_cast<uint32_t>(unit / parts);
        const uint32_t part = parts == 1 ? 0u : static_cast<uint32_t>(unit % parts);
        const int32_t pos = p.positions[t];
        if (pos < 0) continue;  // padding: left as it was
        // the rotation of this lane's eight pairs
        float2 cs[4], sn[4];
        if (rot > 0) {
            float c1[C], s1[C];
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int i = c * G + g;  // pair i of lane j's eight
                const int pair = p.interleaved ? (i < 4 ? 4 * pa + i : 4 * pb + i - 4) : 8 * pa + i;
                c1[c] = 1.0f;
                s1[c] = 0.0f;
                if (turned && i < 8) {
                    // 32 bits of a turn: the top 25 are the functions' angle (as binary32 exactly),
                    // the other 7, at most 2^-26 of a turn, turn the result by themselves
                    const uint32_t turn = static_cast<uint32_t>((S.turn[pair] * static_cast<uint32_t>(pos)) >> 32);
                    const uint32_t top = (turn + 64u) & ~127u;
                    const float rest = static_cast<float>(static_cast<int32_t>(turn - top)) * kRadians;
                    float sf, cf;
                    sincospif(static_cast<float>(static_cast<int32_t>(top)) * 0x1p-31f, &sf, &cf);
                    c1[c] = __fmaf_rn(-sf, rest, cf);
                    s1[c] = __fmaf_rn(cf, rest, sf);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                cs[i].x = __shfl_sync(0xffffffffu, c1[2 * i / G], (2 * i % G) * L + j);
                cs[i].y = __shfl_sync(0xffffffffu, c1[(2 * i + 1) / G], ((2 * i + 1) % G) * L + j);
                sn[i].x = __shfl_sync(0xffffffffu, s1[2 * i / G], (2 * i % G) * L + j);
                sn[i].y = __shfl_sync(0xffffffffu, s1[(2 * i + 1) / G], ((2 * i + 1) % G) * L + j);
            }
        }
        // heads [h0, h1) of the queries, then of the keys
        auto heads = [&](const void* x, int64_t x_stride, void* y, int64_t y_stride, int h0, int h1, const float* w, bool norm) {
            if (h0 >= h1) return;
            const int64_t xa = static_cast<int64_t>(t) * x_stride, ya = static_cast<int64_t>(t) * y_stride;
            uint4 ra[N][R], rb[N][R];
            auto load = [&](int h, int i) {
                const bool in = live && h < h1;
#pragma unroll
                for (int r = 0; r < R; ++r) ra[i][r] = rb[i][r] = make_uint4(0u, 0u, 0u, 0u);
                if (in) {
                    load8<IN>(x, xa + static_cast<int64_t>(h) * D + 8 * pa, ra[i]);
                    load8<IN>(x, xa + static_cast<int64_t>(h) * D + 8 * pb, rb[i]);
                }
            };
#pragma unroll
            for (int i = 0; i < N; ++i) load(h0 + i * G + g, i);
            auto round = [&](int hb, int i) {
                const int h = hb + g;
                float2 a[4], b[4];
                widen8<IN>(ra[i], a);
                widen8<IN>(rb[i], b);
                if (hb + N * G < h1) load(h + N * G, i);
                if (norm) {
                    auto squares = [&]() {
                        float2 s2 = make_float2(0.0f, 0.0f), s3 = s2;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            s2 = fma2(a[e], a[e], s2);
                            s3 = fma2(b[e], b[e], s3);
                        }
                        float sum = (s2.x + s2.y) + (s3.x + s3.y);
#pragma unroll
                        for (int d = 1; d < L; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                        return sum;
                    };
                    float sum = squares(), eps = p.eps;
                    // Squares that overflow or vanish (rare): the row is scaled by a power of two
                    // first, so that the larger of its largest value and the root of eps (by its
                    // exponent), which decide the norm, comes to [1, 2) (eps beside a vanishing
                    // row, scaled as the row's largest value asks, would be infinite).
                    const bool odd = sum > 0x1p120f || (sum < 0x1p-90f && p.eps < 0x1p-60f);
                    if (__any_sync(0xffffffffu, odd)) {
                        float top = p.eps > 0.0f ? __uint_as_float((((__float_as_uint(p.eps) >> 23) + 127u) >> 1) << 23) : 0.0f;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            top = fmaxf(top, fmaxf(fmaxf(fabsf(a[e].x), fabsf(a[e].y)), fmaxf(fabsf(b[e].x), fabsf(b[e].y))));
#pragma unroll
                        for (int d = 1; d < L; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                        const int ex = static_cast<int>(__float_as_uint(top) >> 23);  // 0: vanishing, 255: infinite
                        if (odd && top > 0.0f && ex < 255) {
                            // by 2^(127 - ex), in two factors that are normal numbers
                            const int up = 127 - (ex > 1 ? ex : 1), u1 = up / 2, u2 = up - u1;
                            const float f1 = __uint_as_float(static_cast<uint32_t>(127 + u1) << 23), f2 = __uint_as_float(static_cast<uint32_t>(127 + u2) << 23);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                a[e] = make_float2(a[e].x * f1 * f2, a[e].y * f1 * f2);
                                b[e] = make_float2(b[e].x * f1 * f2, b[e].y * f1 * f2);
                            }
                            eps = eps * f1 * f2 * f1 * f2;
                        }
                        sum = squares();
                    }
                    const float r = rsqrtf(__fmaf_rn(sum, inv_dim, eps));
                    const float2 rr = make_float2(r, r);
                    const float4* wa = reinterpret_cast<const float4*>(w + 8 * pa);
                    const float4* wb = reinterpret_cast<const float4*>(w + 8 * pb);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float4 f = wa[e], k = wb[e];
                        a[2 * e] = mul2(mul2(a[2 * e], rr), make_float2(f.x, f.y));
                        a[2 * e + 1] = mul2(mul2(a[2 * e + 1], rr), make_float2(f.z, f.w));
                        b[2 * e] = mul2(mul2(b[2 * e], rr), make_float2(k.x, k.y));
                        b[2 * e + 1] = mul2(mul2(b[2 * e + 1], rr), make_float2(k.z, k.w));
                    }
                }
                if (turned) {
                    if (p.interleaved) {
                        auto turn = [](float2& v, float c, float s) {
                            v = make_float2(__fmaf_rn(-v.y, s, v.x * c), __fmaf_rn(v.y, c, v.x * s));
                        };
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            turn(a[e], e & 1 ? cs[e / 2].y : cs[e / 2].x, e & 1 ? sn[e / 2].y : sn[e / 2].x);
                            turn(b[e], e & 1 ? cs[2 + e / 2].y : cs[2 + e / 2].x, e & 1 ? sn[2 + e / 2].y : sn[2 + e / 2].x);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 a0 = a[e], b0 = b[e];
                            a[e] = fma2(make_float2(-b0.x, -b0.y), sn[e], mul2(a0, cs[e]));
                            b[e] = fma2(b0, cs[e], mul2(a0, sn[e]));
                        }
                    }
                }
                if (live && h < h1) {
                    uint16_t* dst = static_cast<uint16_t*>(y) + ya + static_cast<int64_t>(h) * D;
                    *reinterpret_cast<uint4*>(dst + 8 * pa) =
                        make_uint4(narrow2<BF16>(a[0].x, a[0].y), narrow2<BF16>(a[1].x, a[1].y), narrow2<BF16>(a[2].x, a[2].y), narrow2<BF16>(a[3].x, a[3].y));
                    *reinterpret_cast<uint4*>(dst + 8 * pb) =
                        make_uint4(narrow2<BF16>(b[0].x, b[0].y), narrow2<BF16>(b[1].x, b[1].y), narrow2<BF16>(b[2].x, b[2].y), narrow2<BF16>(b[3].x, b[3].y));
                }
            };
            for (int hb = h0; hb < h1; hb += N * G) {
                round(hb, 0);
                if (N >= 2 && hb + G < h1) round(hb + G, N - 1);
            }
        };
        const int H = p.q_heads + p.k_heads;
        const int h0 = static_cast<int>(static_cast<int64_t>(H) * part / parts), h1 = static_cast<int>(static_cast<int64_t>(H) * (part + 1) / parts);
        heads(p.q, p.q_stride, p.q_out, p.q_out_stride, h0 < p.q_heads ? h0 : p.q_heads, h1 < p.q_heads ? h1 : p.q_heads, S.w[0], p.q_weight != nullptr);
        heads(p.k, p.k_stride, p.k_out, p.k_out_stride, h0 > p.q_heads ? h0 - p.q_heads : 0, h1 > p.q_heads ? h1 - p.q_heads : 0, S.w[1], p.k_weight != nullptr);
    }
}

using RopeFn = void (*)(RopeParams);

template <int L>
RopeFn rope_of(int in, bool bf16) {
    switch (in) {
        case 0: return bf16 ? k_rope<L, 0, true> : k_rope<L, 0, false>;
        case 1: return bf16 ? k_rope<L, 1, true> : k_rope<L, 1, false>;
        default: return bf16 ? k_rope<L, 2, true> : k_rope<L, 2, false>;
    }
}

}  // namespace

int launch_rope(RopeParams p, int in, bool bf16, void* stream) {
    static Once sms_of[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return static_cast<int>(e);
    if (dev < 0 || dev >= 64) return static_cast<int>(cudaErrorInvalidDevice);
    int sms = 0;
    const int se = sms_of[dev].get([&](int* n) { return static_cast<int>(cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev)); }, &sms);
    if (se != 0) return se;
    int L = 1;
    while (L * 16 < p.head_dim) L *= 2;
    RopeFn fn = nullptr;
    switch (L) {
        case 1: fn = rope_of<1>(in, bf16); break;
        case 2: fn = rope_of<2>(in, bf16); break;
        case 4: fn = rope_of<4>(in, bf16); break;
        case 8: fn = rope_of<8>(in, bf16); break;
        default: fn = rope_of<16>(in, bf16); break;
    }
    // few tokens: their heads over several warps, one round of a warp's heads to a warp at least
    const int64_t warps = static_cast<int64_t>(sms) * 16, rounds = (p.q_heads + p.k_heads + 32 / L - 1) / (32 / L);
    int64_t parts = warps / p.n_tokens;
    if (parts > rounds) parts = rounds;
    if (parts < 1) parts = 1;
    p.parts = static_cast<int32_t>(parts);
    const int64_t want = (p.n_tokens * parts + kRopeWarps - 1) / kRopeWarps, most = static_cast<int64_t>(sms) * rope_ctas(in);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(want < most ? want : most));
    cfg.blockDim = dim3(kRopeWarps * 32);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void* args[] = {&p};
    return static_cast<int>(cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(fn), args));
}

}  // namespace ndq
