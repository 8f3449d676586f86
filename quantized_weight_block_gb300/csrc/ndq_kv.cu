// ndq_kv.cu -- block tables and slot maps from request lengths, and the
// append of new key/value rows to the 8-bit cache.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>

#include "ndq_serve.h"

namespace ndq {
namespace {

// ---------------------------------------------------------------------------
// Block tables and slot maps.
//
// With F(r) the fresh tokens and N(r) = ceil(kv_len / bs) - ceil(cached / bs)
// the blocks request r opens, the token t belongs to the request r with
// sum_{<r} F <= t < sum_{<=r} F, and block b of r is the
// (sum_{<r} N + b - ceil(cached / bs))-th one taken from the free stack.
//
// One launch: a CTA owns kPlanTokens tokens, scans the requests in chunks
// that fit shared memory until it has passed its last token, and finds each
// token's request by bisection in the chunk's prefix sums.  Every CTA repeats
// the scan (8 bytes a request from L2): that costs less than a second launch
// or a chained scan up to tens of thousands of requests.  CTA 0 scans all of
// them and writes the per-request outputs.  Bound by latency: 3.3 us for 64
// requests with a token each, 8.2 us for 2000 with 253 thousand tokens (3 MB
// written) of which the launch is 2.3.
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 256;
constexpr int kPlanPer = 8;                             // requests per thread and chunk
constexpr int kPlanChunk = kPlanThreads * kPlanPer;     // requests per chunk
constexpr int kPlanTokens = kPlanThreads * 4;           // tokens per CTA

// Exclusive prefix of (a, b) over the CTA's threads, and the totals.
__device__ __forceinline__ void scan_pair(uint32_t& a, uint32_t& b, uint32_t& ta, uint32_t& tb, uint2* sh) {
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
    const uint32_t a0 = a, b0 = b;
#pragma unroll
    for (uint32_t d = 1; d < 32; d <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, a, d), y = __shfl_up_sync(0xffffffffu, b, d);
        if (lane >= d) {
            a += x;
            b += y;
        }
    }
    if (lane == 31u) sh[warp] = make_uint2(a, b);
    __syncthreads();
    uint32_t pa = 0, pb = 0;
    ta = tb = 0;
#pragma unroll
    for (uint32_t w = 0; w < kPlanThreads / 32; ++w) {
        if (w == warp) {
            pa = ta;
            pb = tb;
        }
        ta += sh[w].x;
        tb += sh[w].y;
    }
    a += pa - a0;
    b += pb - b0;
}

__global__ void __launch_bounds__(kPlanThreads) k_kv_plan(const PlanParams p) {
    __shared__ uint32_t s_q[kPlanChunk + 1];  // first token of each request of the chunk
    __shared__ uint32_t s_n[kPlanChunk];      // blocks taken before it
    __shared__ uint2 s_w[kPlanThreads / 32];
    const uint32_t tid = threadIdx.x, bl = static_cast<uint32_t>(p.bs_log2), bs = 1u << bl;
    const uint32_t t0 = blockIdx.x * kPlanTokens;
    const uint32_t n_tokens = static_cast<uint32_t>(p.n_tokens);
    const uint32_t t1 = t0 + kPlanTokens < n_tokens ? t0 + kPlanTokens : n_tokens;
    const int32_t count = *p.free_count;
    const bool vec = ((reinterpret_cast<uintptr_t>(p.cached) | reinterpret_cast<uintptr_t>(p.fresh)) & 15u) == 0;
    uint32_t run_q = 0, run_n = 0;
    for (int64_t r0 = 0; r0 < p.n_req && (blockIdx.x == 0 || run_q < t1); r0 += kPlanChunk) {
        const int64_t rt = r0 + static_cast<int64_t>(tid) * kPlanPer;
        uint32_t q[kPlanPer], nb[kPlanPer], kv[kPlanPer], sq = 0, sn = 0;
        int32_t cv[kPlanPer], fv[kPlanPer];
        if (vec && rt + kPlanPer <= p.n_req) {
#pragma unroll
            for (int i = 0; i < kPlanPer; i += 4) {
                *reinterpret_cast<int4*>(cv + i) = *reinterpret_cast<const int4*>(p.cached + rt + i);
                *reinterpret_cast<int4*>(fv + i) = *reinterpret_cast<const int4*>(p.fresh + rt + i);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kPlanPer; ++i) {
                cv[i] = fv[i] = 0;
                if (rt + i < p.n_req) {
                    cv[i] = p.cached[rt + i];
                    fv[i] = p.fresh[rt + i];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kPlanPer; ++i) {
            const int32_t c = cv[i], f = fv[i];
            const uint32_t cu = c > 0 ? static_cast<uint32_t>(c) : 0u, fu = f > 0 ? static_cast<uint32_t>(f) : 0u;
            q[i] = sq;
            nb[i] = sn;
            kv[i] = cu + fu;
            sq += fu;
            sn += ((cu + fu + bs - 1u) >> bl) - ((cu + bs - 1u) >> bl);
        }
        uint32_t tq, tn;
        __syncthreads();  // the previous chunk's tokens are done with s_q, s_n and s_w
        scan_pair(sq, sn, tq, tn, s_w);
#pragma unroll
        for (int i = 0; i < kPlanPer; ++i) {
            const uint32_t j = tid * kPlanPer + i;
            q[i] += run_q + sq;
            s_q[j] = q[i];
            s_n[j] = run_n + sn + nb[i];
            if (blockIdx.x == 0 && rt + i < p.n_req) {
                p.q_start[rt + i] = static_cast<int32_t>(q[i]);
                p.kv_len[rt + i] = static_cast<int32_t>(kv[i]);
            }
        }
        if (tid == 0) s_q[kPlanChunk] = run_q + tq;
        __syncthreads();
        const uint32_t end = run_q + tq;
        if (t0 < end && run_q < t1) {
            constexpr int PT = kPlanTokens / kPlanThreads;  // tokens per thread, looked up side by side
            uint32_t lo[PT] = {}, cu[PT];
#pragma unroll
            for (uint32_t half = kPlanChunk / 2; half > 0; half >>= 1)
#pragma unroll
                for (int i = 0; i < PT; ++i)  // the last request that starts at or before the token
                    if (s_q[lo[i] + half] <= t0 + tid + kPlanThreads * i) lo[i] += half;
#pragma unroll
            for (int i = 0; i < PT; ++i) {
                const uint32_t t = t0 + tid + kPlanThreads * i;
                cu[i] = 0u;
                if (t >= run_q && t < end && t < t1) {
                    const int32_t c = p.cached[r0 + lo[i]];
                    cu[i] = c > 0 ? static_cast<uint32_t>(c) : 0u;
                }
            }
            int32_t id[PT];
#pragma unroll
            for (int i = 0; i < PT; ++i) {
                const uint32_t t = t0 + tid + kPlanThreads * i;
                id[i] = -1;
                if (t >= run_q && t < end && t < t1) {
                    const uint32_t pos = cu[i] + (t - s_q[lo[i]]), blk = pos >> bl, had = (cu[i] + bs - 1u) >> bl;
                    if (blk < p.width) {
                        if (blk >= had) {
                            const uint32_t k = static_cast<uint32_t>(count - 1) - (s_n[lo[i]] + blk - had);
                            if (count > 0 && k < static_cast<uint32_t>(count)) id[i] = p.free_blocks[k];
                        } else {
                            id[i] = p.table[(r0 + lo[i]) * p.width + blk];
                        }
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < PT; ++i) {
                const uint32_t t = t0 + tid + kPlanThreads * i;
                if (t >= run_q && t < end && t < t1) {
                    const uint32_t pos = cu[i] + (t - s_q[lo[i]]), blk = pos >> bl, had = (cu[i] + bs - 1u) >> bl;
                    if (blk >= had && blk < p.width && (pos & (bs - 1u)) == 0u) p.table[(r0 + lo[i]) * p.width + blk] = id[i];
                    p.positions[t] = static_cast<int32_t>(pos);
                    p.slots[t] = id[i] >= 0 ? (static_cast<int64_t>(id[i]) << bl) + (pos & (bs - 1u)) : -1;
                }
            }
        }
        run_q = end;
        run_n += tn;
    }
    for (uint32_t t = t0 + tid; t < t1; t += kPlanThreads)  // padding past the last request's tokens
        if (t >= run_q) {
            p.positions[t] = -1;
            p.slots[t] = -1;
        }
    if (blockIdx.x == 0 && tid == 0) {
        p.q_start[p.n_req] = static_cast<int32_t>(run_q);
        *p.free_left = count - static_cast<int32_t>(run_n);
    }
}

// ---------------------------------------------------------------------------
// Append: quantise new rows into the cache, one scale per block and head.
//
// A run is the adjacent tokens of the call that fall in one block.  Its
// largest magnitude, for one head and one of K and V, gives the scale; then
// its rows are divided by it, rounded and stored.  Bound by reading the rows
// and writing the codes once; a run's rows stay in registers between the two
// sweeps (up to 16 passes of them, more are read again from the cache).
//
// The quotient x / s is not formed: with y a reciprocal of s off by a few
// units, x y (1 - 2^-21) and x y (1 + 2^-21) enclose it, and where both round
// to the same code, that is the code.  Only the others (one in thousands)
// take the division.
//
// Measured: one token of 64 requests, 8 heads of 128: 3.1 us; 8168 tokens of
// nine requests (50 MB moved): 19.5 us, 2.3 TB/s (with the division for every
// value, 39 us).  A CTA's chain of dependent loads is what is left.
// ---------------------------------------------------------------------------
constexpr int kAppendWarps = 4;
constexpr int kAppendHeld = 16;  // passes of rows kept in registers between the two sweeps

template <bool BF16>
__device__ __forceinline__ float2 widen(uint32_t w) {
    if constexpr (BF16)
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    else
        return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// Four values over s, rounded to nearest even and saturated: the codes.
template <bool E4M3>
__device__ __noinline__ uint32_t encode4(float4 v, float s) {
    if (!(s > 0.0f)) return 0u;
    v.x = __fdiv_rn(v.x, s);
    v.y = __fdiv_rn(v.y, s);
    v.z = __fdiv_rn(v.z, s);
    v.w = __fdiv_rn(v.w, s);
    if constexpr (E4M3) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v.x, v.y), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v.z, v.w), __NV_SATFINITE, __NV_E4M3);
        return lo | (hi << 16);
    } else {
        const float f[4] = {v.x, v.y, v.z, v.w};
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float c = fminf(fmaxf(f[i], -127.0f), 127.0f);  // (NaN: -127 here, replaced below)
            const int q = f[i] == f[i] ? __float2int_rn(c) : 0;
            w |= (static_cast<uint32_t>(q) & 0xffu) << (8 * i);
        }
        return w;
    }
}

__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 pair_mul(uint64_t a, uint64_t b) {
    float2 r;
    asm("{\n.reg .b64 m;\nmul.rn.f32x2 m, %2, %3;\nmov.b64 {%0, %1}, m;\n}" : "=f"(r.x), "=f"(r.y) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ void pair_fma(uint64_t a, uint64_t b, uint64_t c, uint32_t& x, uint32_t& y) {
    asm("{\n.reg .b64 m;\nfma.rn.f32x2 m, %2, %3, %4;\nmov.b64 {%0, %1}, m;\n}" : "=r"(x), "=r"(y) : "l"(a), "l"(b), "l"(c));
}
// Four quotients to E4M3 codes.
__device__ __forceinline__ uint32_t round_e4m3(float2 a, float2 b) {
    uint32_t r;
    asm("{\n.reg .b16 l, h;\ncvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\ncvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\nmov.b32 %0, {l, h};\n}"
        : "=r"(r)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}

// encode4 for finite values of at most Q s: the pairs lo and hi enclose 1 / s.
template <bool E4M3>
__device__ __forceinline__ uint32_t encode4_fast(float2 v, float2 w, float s, uint64_t lo, uint64_t hi) {
    const uint64_t pv = pair(v.x, v.y), pw = pair(w.x, w.y);
    if constexpr (E4M3) {
        const uint32_t a = round_e4m3(pair_mul(pv, lo), pair_mul(pw, lo)), b = round_e4m3(pair_mul(pv, hi), pair_mul(pw, hi));
        if (a == b) return a;
    } else {
        // x / s + 1.5 * 2^23, rounded once to nearest even: the low byte is the code (|x / s| < 128)
        const uint64_t big = pair(12582912.0f, 12582912.0f);
        uint32_t a[4], b[4];
        pair_fma(pv, lo, big, a[0], a[1]);
        pair_fma(pw, lo, big, a[2], a[3]);
        pair_fma(pv, hi, big, b[0], b[1]);
        pair_fma(pw, hi, big, b[2], b[3]);
        if (((a[0] ^ b[0]) | (a[1] ^ b[1]) | (a[2] ^ b[2]) | (a[3] ^ b[3])) == 0u)
            return __byte_perm(__byte_perm(a[0], a[1], 0x0040), __byte_perm(a[2], a[3], 0x0040), 0x5410);
    }
    return encode4<E4M3>(make_float4(v.x, v.y, w.x, w.y), s);
}

template <bool E4M3>
__device__ __forceinline__ float4 decode4(uint32_t w) {
    if constexpr (E4M3) {
        const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w & 0xffffu), __NV_E4M3);
        const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> 16), __NV_E4M3);
        const float2 x = __half22float2(__half2(a)), y = __half22float2(__half2(b));
        return make_float4(x.x, x.y, y.x, y.y);
    } else {
        return make_float4(static_cast<float>(static_cast<int8_t>(w)), static_cast<float>(static_cast<int8_t>(w >> 8)),
                           static_cast<float>(static_cast<int8_t>(w >> 16)),
                           static_cast<float>(static_cast<int8_t>(w >> 24)));
    }
}

__device__ __forceinline__ float finite_abs(float x) {
    const float a = fabsf(x);
    return a <= FLT_MAX ? a : 0.0f;
}

// TEAM warps work on a run together.  win (at most 32): the tokens a team
// searches for runs that start among them.
template <int D, bool E4M3, bool BF16, int TEAM>
__global__ void __launch_bounds__(kAppendWarps * 32, TEAM > 1 ? 6 : 4) k_kv_append(const AppendParams p, int win) {
    constexpr int LPR = D / 4;              // lanes per row, four values each
    constexpr int RPP = TEAM * 32 / LPR;    // rows per pass of the team
    constexpr float kQmax = E4M3 ? 448.0f : 127.0f;
    __shared__ uint32_t s_max[kAppendWarps];
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
    const int units = 2 * p.c.heads;
    const int64_t team = TEAM == 1 ? static_cast<int64_t>(blockIdx.x) * kAppendWarps + warp : blockIdx.x;
    const int64_t w0 = team / units * win;
    if (w0 >= p.n_tokens) return;
    const int u = static_cast<int>(team % units), h = u >> 1;
    const bool is_v = u & 1;
    const int bl = p.c.bs_log2, bs = 1 << bl;
    const int64_t limit = p.c.num_blocks << bl;
    const uint16_t* in = (is_v ? p.v : p.k) + static_cast<int64_t>(h) * D;
    const int64_t stride = is_v ? p.v_stride : p.k_stride;
    uint8_t* codes = is_v ? p.c.v : p.c.k;
    float* scales = is_v ? p.c.vs : p.c.ks;
    const int64_t wend = w0 + win < p.n_tokens ? w0 + win : p.n_tokens;
    // which tokens of the window start a run (lane i: token w0 + i)
    bool lead = false;
    int64_t slot = -1;
    if (w0 + lane < wend) {
        slot = p.slots[w0 + lane];
        const int64_t before = w0 + lane > 0 ? p.slots[w0 + lane - 1] : -1;
        lead = slot >= 0 && slot < limit && (before < 0 || (before >> bl) != (slot >> bl));
    }
    uint32_t leads = __ballot_sync(0xffffffffu, lead);
    const uint32_t idx = TEAM == 1 ? lane : threadIdx.x;
    const int row = static_cast<int>(idx / LPR), col = static_cast<int>(idx % LPR) * 4;
    while (leads) {
        const int li = __ffs(leads) - 1;
        leads &= leads - 1;
        const int64_t t0 = w0 + li;
        const int64_t s0 = __shfl_sync(0xffffffffu, slot, li);
        const int64_t blk = s0 >> bl;
        // the first passes of rows, fetched before the run's length is known (all of them are tokens of the call)
        const uint16_t* src = in + t0 * stride + col;
        const int most = p.n_tokens - t0 < bs ? static_cast<int>(p.n_tokens - t0) : bs;
        uint2 held[kAppendHeld];
#pragma unroll
        for (int i = 0; i < kAppendHeld; ++i) {
            const int r = i * RPP + row;
            held[i] = make_uint2(0u, 0u);
            if (r < most) held[i] = *reinterpret_cast<const uint2*>(src + r * stride);
        }
        // the run's length: up to bs tokens of the same block; dense: at adjacent slots, as a plan gives them
        int cnt = 0;
        bool dense = true;
        int64_t ahead[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t t = t0 + 32 * i + lane;
            ahead[i] = 32 * i < bs && t < p.n_tokens ? p.slots[t] : -1;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (32 * i >= bs || cnt < 32 * i) break;
            const uint32_t m = __ballot_sync(0xffffffffu, (ahead[i] >> bl) == blk);
            const int k = m == 0xffffffffu ? 32 : __ffs(~m) - 1;
            dense = dense && __all_sync(0xffffffffu, static_cast<int>(lane) >= k || ahead[i] == s0 + 32 * i + static_cast<int64_t>(lane));
            cnt += k;
        }
        if (cnt > bs) cnt = bs;
        const int n_old = static_cast<int>(s0 & (bs - 1));
        const int64_t unit = blk * p.c.heads + h;
        const float old = n_old > 0 ? scales[unit] : 0.0f;
        // magnitudes compare as 16-bit integers, infinity and NaN above all numbers
        uint32_t top = 0u;
#pragma unroll
        for (int i = 0; i < kAppendHeld; ++i)
            if (i * RPP + row < cnt) top = __vmaxu2(top, __vmaxu2(held[i].x & 0x7fff7fffu, held[i].y & 0x7fff7fffu));
#pragma unroll 4
        for (int r = kAppendHeld * RPP + row; r < cnt; r += RPP) {
            const uint2 w = *reinterpret_cast<const uint2*>(src + r * stride);
            top = __vmaxu2(top, __vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu));
        }
        top = __reduce_max_sync(0xffffffffu, top >> 16 > (top & 0xffffu) ? top >> 16 : top & 0xffffu);
        if constexpr (TEAM > 1) {  // (also: every thread has read the old scale before it is written)
            __syncthreads();
            if (lane == 0) s_max[warp] = top;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < TEAM; ++w) top = s_max[w] > top ? s_max[w] : top;
        }
        const bool odd = top >= (BF16 ? 0x7f80u : 0x7c00u);
        float amax = widen<BF16>(top).x;
        if (odd) {  // the largest finite magnitude, then (rare)
            amax = 0.0f;
            for (int r = 0; r < cnt; ++r)
                for (int d = 0; d < D; d += 2) {
                    const float2 a = widen<BF16>(*reinterpret_cast<const uint32_t*>(in + (t0 + r) * stride + d));
                    amax = fmaxf(amax, fmaxf(finite_abs(a.x), finite_abs(a.y)));
                }
        }
        float fresh = 0.0f;
        if (amax > 0.0f) fresh = fminf(fmaxf(__fdiv_rn(amax, kQmax), 0x1p-100f), 0x1p100f);
        const float s = fmaxf(old, fresh);
        // (a scale cut off at 2^100 leaves values beyond Q s: to be saturated)
        const bool fast = !odd && s > 0.0f && s < 0x1p100f;
        const float y = s > 0.0f ? __fdividef(1.0f, s) : 0.0f;
        const float lo = __fmul_rn(y, 1.0f - 0x1p-21f), hi = __fmul_rn(y, 1.0f + 0x1p-21f);
        const uint64_t lo2 = pair(lo, lo), hi2 = pair(hi, hi);
        uint8_t* out = codes + (unit << bl) * D + col;
        if (old > 0.0f && s > old) {  // the earlier tokens' codes under the grown scale
#pragma unroll 4
            for (int r = row; r < n_old; r += RPP) {
                uint32_t* w = reinterpret_cast<uint32_t*>(out + r * D);
                const bool far = !E4M3 && __vcmpeq4(*w, 0x80808080u) != 0u;  // a code of -128, beyond Q, is to be saturated
                float4 v = decode4<E4M3>(*w);
                v.x = __fmul_rn(v.x, old);
                v.y = __fmul_rn(v.y, old);
                v.z = __fmul_rn(v.z, old);
                v.w = __fmul_rn(v.w, old);
                // (below Q s, or NaN codes, which stay: the short way whatever the new values hold)
                *w = s < 0x1p100f && !far ? encode4_fast<E4M3>(make_float2(v.x, v.y), make_float2(v.z, v.w), s, lo2, hi2) : encode4<E4M3>(v, s);
            }
        }
        auto put = [&](const uint2& w, int r) {
            const float2 a = widen<BF16>(w.x), b = widen<BF16>(w.y);
            const int o = dense ? n_old + r : static_cast<int>(p.slots[t0 + r] & (bs - 1));
            *reinterpret_cast<uint32_t*>(out + o * D) =
                fast ? encode4_fast<E4M3>(a, b, s, lo2, hi2) : encode4<E4M3>(make_float4(a.x, a.y, b.x, b.y), s);
        };
#pragma unroll
        for (int i = 0; i < kAppendHeld; ++i) {
            const int r = i * RPP + row;
            if (r < cnt) put(held[i], r);
        }
#pragma unroll 2
        for (int r = kAppendHeld * RPP + row; r < cnt; r += RPP) put(*reinterpret_cast<const uint2*>(src + r * stride), r);
        __syncwarp();  // every lane has read the old scale
        if (idx == 0) scales[unit] = s;
    }
}

template <int D, bool E4M3>
int append_typed(const AppendParams& p, bool bf16, void* stream) {
    const int64_t units = 2 * static_cast<int64_t>(p.c.heads);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    // A warp per token, head and K or V while all of them are resident at once;
    // beyond, a CTA per 32 tokens, which works on the runs that start there.
    // What decides is the length of the runs, which the host does not know:
    // the number of tokens stands for it.  Measured (INT8, heads of 128, blocks
    // of 64; by warps / by CTAs, us): one token each of 64, 400, 1024 requests,
    // 8 heads: 3.5 / 47, 8.4 / 50, 17 / 68; one prompt of 450 tokens, 8 heads:
    // 24 / 4.8; of 1024, 8 heads: 28 / 8.0; of 3600, one head: 12 / 5.0.  So
    // steps of more than 456 requests at 8 heads, and prompts below as many
    // tokens, take the slower form.
    if (p.n_tokens * units <= 152 * 48) {
        const unsigned grid = static_cast<unsigned>((p.n_tokens * units + kAppendWarps - 1) / kAppendWarps);
        if (bf16) k_kv_append<D, E4M3, true, 1><<<grid, kAppendWarps * 32, 0, st>>>(p, 1);
        else k_kv_append<D, E4M3, false, 1><<<grid, kAppendWarps * 32, 0, st>>>(p, 1);
    } else {
        const int win = p.c.bs_log2 > 4 ? 32 : 16;  // (blocks of 16 would give two or three runs to a window of 32)
        const unsigned grid = static_cast<unsigned>((p.n_tokens + win - 1) / win * units);
        if (bf16) k_kv_append<D, E4M3, true, kAppendWarps><<<grid, kAppendWarps * 32, 0, st>>>(p, win);
        else k_kv_append<D, E4M3, false, kAppendWarps><<<grid, kAppendWarps * 32, 0, st>>>(p, win);
    }
    return static_cast<int>(cudaGetLastError());
}

}  // namespace

int launch_kv_plan(const PlanParams& p, void* stream) {
    const int64_t tiles = (p.n_tokens + kPlanTokens - 1) / kPlanTokens;
    k_kv_plan<<<static_cast<unsigned>(tiles > 0 ? tiles : 1), kPlanThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return static_cast<int>(cudaGetLastError());
}

int launch_kv_append(const AppendParams& p, int head_dim, bool e4m3, bool bf16, void* stream) {
    if (head_dim == 64)
        return e4m3 ? append_typed<64, true>(p, bf16, stream) : append_typed<64, false>(p, bf16, stream);
    return e4m3 ? append_typed<128, true>(p, bf16, stream) : append_typed<128, false>(p, bf16, stream);
}

}  // namespace ndq
