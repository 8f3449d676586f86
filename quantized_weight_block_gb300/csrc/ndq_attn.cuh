// ndq_attn.cuh -- what the attention kernels share: number conversions and
// the reading of a request's lengths.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

#include "ndq_serve.h"

namespace ndq {
namespace {

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void attn_pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void attn_pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Two 16-bit input values to binary32.
template <bool BF16>
__device__ __forceinline__ void widen2(uint32_t w, float& a, float& b) {
    if constexpr (BF16) {
        a = __uint_as_float(w << 16);
        b = __uint_as_float(w & 0xffff0000u);
    } else {
        asm("{\n.reg .f16 l, h;\nmov.b32 {l, h}, %2;\ncvt.f32.f16 %0, l;\ncvt.f32.f16 %1, h;\n}" : "=f"(a), "=f"(b) : "r"(w));
    }
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two outputs, rounded once.
template <bool BF16>
__device__ __forceinline__ uint32_t narrow2(float lo, float hi) {
    if constexpr (BF16) {
        uint32_t r;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    } else {
        return pack_half2(lo, hi);
    }
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Four codes to binary16 pairs (bytes 0, 1) and (2, 3); every code is exact.
template <bool E4M3>
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if constexpr (E4M3) {
        asm("{\n.reg .b16 l, h;\nmov.b32 {l, h}, %2;\ncvt.rn.f16x2.e4m3x2 %0, l;\ncvt.rn.f16x2.e4m3x2 %1, h;\n}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
    } else {
        // c + 128 under the exponent of 1024, then minus 1152
        const uint32_t u = w ^ 0x80808080u;
        const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0x64806480u));
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(0x64806480u));
    }
}

// Bit 7 of every byte that is an E4M3 NaN code (0x7f, 0xff).
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

// The powers of two that bring a row of queries with the largest magnitude
// amax to about 2^10 and back: in binary16 every bfloat16 or binary16 value of
// the row above 2^-24 of the largest is then exact.  (0, infinity, NaN: 1.)
__device__ __forceinline__ void row_scale(float amax, float& up, float& down) {
    const int e = static_cast<int>((__float_as_uint(amax) >> 23) & 0xffu);
    if (e == 0xff || amax == 0.0f) {
        up = down = 1.0f;
        return;
    }
    int s = e - 127 - 10;  // amax in [2^(s + 10), 2^(s + 11))
    s = s < -126 ? -126 : s;
    up = __uint_as_float(static_cast<uint32_t>(127 - s) << 23);
    down = __uint_as_float(static_cast<uint32_t>(127 + s) << 23);
}

// log2 of V's scale and its reciprocal.  A block of scale 0 counts as zeros
// under the smallest scale there is: its weights add to the denominator alone,
// and under a larger one they could raise the maximum so far that binary16
// loses the weights of blocks of small values.  (NaN stays NaN.)
__device__ __forceinline__ void value_scale(float s, float& lg, float& inv) {
    if (s == 0.0f) {
        lg = -100.0f;
        inv = 0x1p100f;
        return;
    }
    const uint32_t b = __float_as_uint(s);
    const float f = s > 0.0f ? __uint_as_float((b & 0x007fffffu) | 0x3f800000u) : s;
    asm("lg2.approx.f32 %0, %1;" : "=f"(lg) : "f"(f));
    lg += s > 0.0f ? static_cast<float>(static_cast<int>(b >> 23) - 127) : 0.0f;
    inv = __fdividef(1.0f, s);
}

// V's scales far apart.  The weights are p = 2^(s + lg - m), the denominator
// sums p / 2^lg.  A token whose p vanishes adds nothing to the values beside
// the largest one's, but with lg far below that one's it may add to the
// denominator: where lg lies more than kScaleSpread below the largest so far,
// 2^(s - m) is taken by itself.  (Elsewhere a p that vanishes, below 2^-126,
// belongs to an s at least 65 below the largest one's.)  Denominators span more
// than 2^126, so one that counts may be large where the factor that it is to be
// scaled by vanishes: it is scaled by halves of the exponent.
constexpr float kScaleSpread = 60.0f;
constexpr int32_t kNoScale = -1000;

// floor(log2(s)) of a scale above 0, else kNoScale.
__device__ __forceinline__ int32_t scale_exponent(float s) {
    return s > 0.0f && s < INFINITY ? static_cast<int32_t>(__float_as_uint(s) >> 23) - 127 : kNoScale;
}

// What of four codes of V a block of scale 0 keeps: E4M3's NaN.
template <bool E4M3>
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {
    if constexpr (E4M3) return w & ((nan_bytes(w) >> 7) * 0xffu);
    else return 0u;
}

// Tokens that the block table has room for (at most 2^30).
__device__ __forceinline__ int32_t table_tokens(const AttnParams& p) { return static_cast<int32_t>(p.width << p.c.bs_log2); }

// Request r's first query row, the number of queries that are computed and the
// position of the first one, kept inside the buffers whatever the device
// arrays hold.  Queries past max_q or n_tokens are left out, and tokens past
// the table are not seen, but both count for the positions: all of a request's
// queries are its last tokens.
__device__ __forceinline__ void attn_request(const AttnParams& p, int64_t r, int64_t& q0, int32_t& n, int32_t& first) {
    int64_t a = r, all = 1, room = 1;
    if (p.q_start) {
        a = p.q_start[r];
        a = a < 0 ? 0 : (a > p.n_tokens ? p.n_tokens : a);
        all = p.q_start[r + 1] - a;
        all = all < 0 ? 0 : all;
        room = p.n_tokens - a < p.max_q ? p.n_tokens - a : p.max_q;
    }
    q0 = a;
    n = static_cast<int32_t>(all < room ? all : room);
    const int64_t len = p.kv_len[r] > 0 ? p.kv_len[r] : 0;
    first = static_cast<int32_t>(len - all > -(1 << 30) ? len - all : -(1 << 30));  // (before 0 in either case)
}

// ---- requests that share prefixes ---------------------------------------------

// What an attention kernel computes: all that its rows see; the shared prefix
// of groups of requests; or the rest, joined with that.
enum AttnMode : int { kAttnAll = 0, kAttnShared = 1, kAttnOwn = 2 };
template <int MODE>
struct AttnArgs {
    using type = PrefixParams;
};
template <>
struct AttnArgs<kAttnAll> {
    using type = AttnParams;
};

// Group g's requests and the tokens that they share: whole blocks, and no
// more than the table has room for.
struct Group {
    int64_t begin, end;
    int32_t tokens;
};
__device__ __forceinline__ Group attn_group(const PrefixParams& p, int64_t g) {
    Group x;
    x.begin = p.group_start[g];
    x.begin = x.begin < 0 ? 0 : (x.begin > p.n_req ? p.n_req : x.begin);
    x.end = p.group_start[g + 1];
    x.end = x.end < x.begin ? x.begin : (x.end > p.n_req ? p.n_req : x.end);
    const int32_t most = table_tokens(p), n = p.prefix_len[g] < most ? p.prefix_len[g] : most;
    x.tokens = n > 0 ? n & ~((1 << p.c.bs_log2) - 1) : 0;
    return x;
}

// The tokens that request r shares with its group.
__device__ __forceinline__ int32_t shared_tokens(const PrefixParams& p, int64_t r) {
    int64_t a = 0, b = p.n_groups;  // the last group that starts at r or before
    while (b - a > 1) {
        const int64_t m = (a + b) >> 1;
        if (p.group_start[m] <= r) a = m;
        else b = m;
    }
    const Group x = attn_group(p, a);
    return x.begin <= r && r < x.end ? x.tokens : 0;
}

// What a part counts for beside the maximum M, as a root (see kScaleSpread).
// A part that saw nothing has 0 for everything, or a NaN that must stay.
__device__ __forceinline__ float part_root(float m, float M) { return m == -INFINITY ? 1.0f : exp2_fast(0.5f * (m - M)); }

// The parts that the prefix's kernel left of one row: a row of a slot holds its
// values, its maximum and its sum, in D + 4 floats.
template <int D>
struct RowParts {
    const float* first;
    uint32_t rows, n;  // rows of a slot, slots

    __device__ __forceinline__ RowParts(const PrefixParams& p, int64_t at) {
        const uint4 x = __ldcg(static_cast<const uint4*>(p.records) + at);
        rows = x.y;
        n = x.z;
        // (whatever a record holds, no read leaves the slots)
        if (rows > kPromptRows || x.w >= rows || n > 2 * kPrefixMaxParts || x.x + static_cast<uint64_t>(n) * rows > static_cast<uint64_t>(p.slot_rows)) n = 0;
        first = p.slots + (static_cast<uint64_t>(x.x) + x.w) * (D + 4);
    }
    __device__ __forceinline__ const float* part(uint32_t k) const { return first + static_cast<uint64_t>(k) * rows * (D + 4); }
    // maximum and sum
    __device__ __forceinline__ float2 stat(uint32_t k) const { return __ldcg(reinterpret_cast<const float2*>(part(k) + D)); }
    // head positions 4 c .. 4 c + 3, by a thread that reads the ones beside them, too
    __device__ __forceinline__ float4 values(uint32_t k, uint32_t c) const { return reinterpret_cast<const float4*>(part(k))[c]; }
    __device__ __forceinline__ float largest(float M) const {
#pragma unroll 4
        for (uint32_t k = 0; k < n; ++k) M = fmaxf(M, stat(k).x);
        return M;
    }
};


}  // namespace
}  // namespace ndq
