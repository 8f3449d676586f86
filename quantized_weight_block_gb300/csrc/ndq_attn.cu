// ndq_attn.cu -- attention over the 8-bit cache, few rows per request (a
// generation step, a few drafted tokens): k_attn_rows, and the launcher.
//
//     out = softmax(scale * q . (ks kc)) . (vs vc)
//
// A row is one (query token, query head); the rows that share a cache head
// (the tokens of a request times the group's heads) are taken 16 at a time, so
// a code is read once for all of them.  With few rows the operator is bound
// by reading the cache: 2 D bytes a token and head.
//
// Work.  The unit is 128 tokens of one (request, cache head, row tile).  The
// units of all requests, laid end to end, are divided evenly over the CTAs,
// whatever the lengths: a CTA finds its share from the lengths (a block scan
// over the requests) and walks it segment by segment, a segment being its
// part of one row tile.  A row tile that one CTA does not finish leaves a
// partial (maximum, sum, weighted values) in the workspace; the CTA that
// arrives last joins them in CTA order, so the result does not depend on
// timing.
//
// Inside a CTA each warp takes every eighth tile of 16 tokens.  A tile's
// codes come through a ring of asynchronous copies in shared memory that is
// private to the lane which consumes them (the copies only hide latency:
// nothing is exchanged), are widened to binary16 in registers (exact) and go
// through mma.sync m16n8k16: S = Q K^T with the head dimension permuted so
// that a lane's 16-byte copy is its operand, then O += P V with the
// accumulator layout of S as the operand of P.  (With 16 rows the tensor
// cores have next to nothing to do; tcgen05 would want the codes widened
// through shared memory first, four times the traffic of the copy itself.)
//
// Scales.  K's scale multiplies a tile's scores.  V's scale f * 2^e (f in
// [1, 2)) joins the exponent, t = s + e, so that the weights 2^(t - m) f
// which go to binary16 are at most 2 and lose nothing to a V of small scale;
// the denominator sums 2^(t - m) 2^-e.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ndq_attn.cuh"

namespace ndq {
namespace {

constexpr int kRowWarps = 8;
constexpr int kRowThreads = kRowWarps * 32;
constexpr int kRowTile = 16;                       // tokens per warp tile
constexpr int kRowUnit = kRowWarps * kRowTile;     // tokens per unit of work
constexpr int kRowStages = 3;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}

// What a CTA knows of one request.
struct Req {
    int64_t q0;    // its first query row
    int32_t n;     // queries
    int32_t kv;    // tokens
    int32_t lo;    // first token any of its queries sees, a multiple of 16
    int32_t units; // units of one row tile (at least one, so that empty rows are written)
    int32_t tiles; // row tiles per cache head
};

__device__ __forceinline__ Req request(const AttnParams& p, int64_t r) {
    Req x;
    attn_request(p, r, x.q0, x.n, x.kv);
    if (p.prompt_rows > 0 && static_cast<int64_t>(x.n) * p.group >= p.prompt_rows) x.n = 0;  // the other kernel's
    x.lo = 0;
    if (p.window > 0) {
        const int64_t first = static_cast<int64_t>(x.kv) - x.n + 1 - p.window;
        x.lo = first > 0 ? static_cast<int32_t>(first) & ~(kRowTile - 1) : 0;
    }
    x.units = x.kv > x.lo ? (x.kv - x.lo + kRowUnit - 1) / kRowUnit : 1;
    x.tiles = static_cast<int32_t>((static_cast<int64_t>(x.n) * p.group + kAttnRows - 1) / kAttnRows);
    return x;
}

template <int D, bool HALF>
struct RowSmem {
    static constexpr int kRows = HALF ? 8 : 16;
    static constexpr int kStage = 2 * kRowTile * D;                          // one warp's K and V tile
    static constexpr int kRing = kRowWarps * kRowStages * kStage;
    static constexpr int kMerge = kRowWarps * kRows * (D + 4) * 4;           // one partial per warp
    static constexpr int kBytes = kRing > kMerge ? kRing : kMerge;
};

template <int D, bool E4M3, bool BF16, bool HALF>
__global__ void __launch_bounds__(kRowThreads, HALF ? 2 : 1) k_attn_rows(const AttnParams p) {
    using Sm = RowSmem<D, HALF>;
    constexpr int kRows = Sm::kRows;
    constexpr int KS = D / 16;       // k-steps of a score
    constexpr int KC = D / 64;       // 16-byte pieces of a token's K per lane
    constexpr int VB = D / 8;        // bytes of a token's V per lane; n-tiles of a head
    constexpr int OR = HALF ? 2 : 4;
    constexpr uint64_t kSlot = kAttnRows * (D + 2);  // attn_slot_floats(D)
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ uint64_t s_sum[kRowWarps];
    __shared__ int64_t s_r, s_base;
    __shared__ float s_sc[kRowWarps][kRowStages][2];
    __shared__ int32_t s_id[kRowWarps][kRowStages];
    __shared__ float s_m[kRowWarps][kAttnRows], s_l[kRowWarps][kAttnRows];
    __shared__ uint32_t s_last;
    const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31u, g = lane >> 2, t = lane & 3u;
    const int bl = p.c.bs_log2;

    // this CTA's share of the units
    uint64_t mine = 0;
    const int64_t per = (p.n_req + kRowThreads - 1) / kRowThreads;
    for (int64_t i = 0; i < per; ++i) {
        const int64_t r = tid * per + i;
        if (r < p.n_req) {
            const Req x = request(p, r);
            mine += static_cast<uint64_t>(x.tiles) * p.c.heads * x.units;
        }
    }
    uint64_t incl = mine;
#pragma unroll
    for (uint32_t d = 1; d < 32; d <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += y;
    }
    if (lane == 31u) s_sum[warp] = incl;
    __syncthreads();
    uint64_t total = 0, before = incl - mine;
#pragma unroll
    for (uint32_t w = 0; w < kRowWarps; ++w) {
        if (w < warp) before += s_sum[w];
        total += s_sum[w];
    }
    if (total == 0) return;
    const uint64_t ctas = gridDim.x < total ? gridDim.x : total;
    if (blockIdx.x >= ctas) return;
    uint64_t u = total * blockIdx.x / ctas;
    const uint64_t u_end = total * (blockIdx.x + 1) / ctas;
    if (before <= u && u < before + mine) {
        s_r = tid * per;
        s_base = static_cast<int64_t>(before);
    }
    __syncthreads();
    int64_t r = s_r;
    uint64_t base = static_cast<uint64_t>(s_base);  // first unit of request r

    const uint32_t my_ring = smem_u32(ring) + warp * kRowStages * Sm::kStage + lane * 16;
    while (u < u_end) {
        const Req x = request(p, r);
        const uint64_t ru = static_cast<uint64_t>(x.tiles) * p.c.heads * x.units;
        if (u >= base + ru) {
            base += ru;
            ++r;
            continue;
        }
        const uint64_t hj = (u - base) / x.units;
        const int32_t ca = static_cast<int32_t>((u - base) % x.units);
        const int32_t cb = static_cast<int32_t>(x.units - ca < u_end - u ? x.units : ca + (u_end - u));
        const int32_t h = static_cast<int32_t>(hj / x.tiles), j = static_cast<int32_t>(hj % x.tiles);

        // the rows of this tile: row i is (query, head) = divmod(16 j + i, group)
        const int32_t row0 = j * kAttnRows;
        const int32_t rows_left = x.n * p.group - row0;
        const int32_t nrows = rows_left < kAttnRows ? rows_left : kAttnRows;
        uint32_t qf[KS][4];
        float frow[2];
        int32_t see_lo[2], see_hi[2];  // the tokens rows g and g + 8 see
#pragma unroll
        for (int half = 0; half < (HALF ? 1 : 2); ++half) {
            const int32_t i = static_cast<int32_t>(g) + 8 * half;
            const bool ok = i < nrows;
            const int32_t qi = (row0 + (ok ? i : 0)) / p.group, qh = (row0 + (ok ? i : 0)) % p.group;
            const uint16_t* src = p.q + (x.q0 + qi) * p.q_stride + static_cast<int64_t>(h * p.group + qh) * D + t * 16;
            float v[KC * 16];
#pragma unroll
            for (int c = 0; c < KC * 2; ++c) {
                uint4 w = make_uint4(0u, 0u, 0u, 0u);
                if (ok) w = *reinterpret_cast<const uint4*>(src + (c >> 1) * 64 + (c & 1) * 8);
                widen2<BF16>(w.x, v[c * 8 + 0], v[c * 8 + 1]);
                widen2<BF16>(w.y, v[c * 8 + 2], v[c * 8 + 3]);
                widen2<BF16>(w.z, v[c * 8 + 4], v[c * 8 + 5]);
                widen2<BF16>(w.w, v[c * 8 + 6], v[c * 8 + 7]);
            }
            float amax = 0.0f;
#pragma unroll
            for (int c = 0; c < KC * 16; ++c) amax = fmaxf(amax, fabsf(v[c]));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            float up, down;
            row_scale(amax, up, down);
            frow[half] = down * p.scale_log2;
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                qf[s][half] = pack_half2(v[s * 4] * up, v[s * 4 + 1] * up);
                qf[s][half + 2] = pack_half2(v[s * 4 + 2] * up, v[s * 4 + 3] * up);
            }
            const int64_t pos = static_cast<int64_t>(x.kv) - x.n + qi;
            see_hi[half] = ok && pos >= 0 ? static_cast<int32_t>(pos) + 1 : 0;
            see_lo[half] = p.window > 0 && pos + 1 > p.window ? static_cast<int32_t>(pos + 1 - p.window) : 0;
        }
        if constexpr (HALF) {
#pragma unroll
            for (int s = 0; s < KS; ++s) qf[s][1] = qf[s][3] = 0u;
            frow[1] = 0.0f;
            see_lo[1] = see_hi[1] = 0;
        }
        // the tokens some row of the tile sees / every row sees
        const int32_t qa = row0 / p.group, qb = (row0 + nrows - 1) / p.group;
        int64_t any_hi = static_cast<int64_t>(x.kv) - x.n + qb + 1, all_hi = static_cast<int64_t>(x.kv) - x.n + qa + 1;
        int64_t any_lo = 0, all_lo = 0;
        if (p.window > 0) {
            any_lo = all_hi - p.window;
            all_lo = any_hi - p.window;
        }

        float o[VB][OR];
#pragma unroll
        for (int s = 0; s < VB; ++s)
#pragma unroll
            for (int e = 0; e < OR; ++e) o[s][e] = 0.0f;
        float mx[2] = {-INFINITY, -INFINITY}, sum[2] = {0.0f, 0.0f};

        // this warp's tiles: base token x.lo + 16 (8 c + warp), c = ca .. cb - 1
        int32_t tok = x.lo + ca * kRowUnit + static_cast<int32_t>(warp) * kRowTile;
        const int64_t seg_end = static_cast<int64_t>(x.lo) + static_cast<int64_t>(cb) * kRowUnit;
        const int64_t tok_end = seg_end < any_hi ? seg_end : any_hi;
        while (tok + kRowTile <= any_lo && tok < tok_end) tok += kRowUnit;
        const int32_t ntile = tok < tok_end ? static_cast<int32_t>((tok_end - tok + kRowUnit - 1) / kRowUnit) : 0;
        const int32_t* table = p.table + r * p.width;
        const uint64_t head_off = static_cast<uint64_t>(h);

        // tile i of this warp into stage i % kRowStages; its block id was loaded a tile earlier
        auto block_of = [&](int32_t i) -> int32_t {
            if (i >= ntile) return -1;
            const int32_t id = table[(tok + i * kRowUnit) >> bl];
            return id >= 0 && id < p.c.num_blocks ? id : -1;
        };
        auto issue = [&](int32_t i, int32_t id) {
            const uint32_t st = static_cast<uint32_t>(i % kRowStages);
            if (i < ntile && id >= 0) {
                const uint64_t unit = static_cast<uint64_t>(id) * p.c.heads + head_off;
                const uint64_t off = ((unit << bl) + ((tok + i * kRowUnit) & ((1 << bl) - 1))) * D;
                const uint8_t* k = p.c.k + off + t * 16;
                const uint8_t* v = p.c.v + off + g * VB;
                const uint32_t d = my_ring + st * Sm::kStage;
#pragma unroll
                for (int a = 0; a < 2; ++a)
#pragma unroll
                    for (int c = 0; c < KC; ++c) cp_async16(d + (a * KC + c) * 512, k + (a * 8 + g) * D + c * 64);
#pragma unroll
                for (int a = 0; a < 4; ++a) {
                    const uint32_t vt = (a >> 1) * 8 + 2 * t + (a & 1);
                    if constexpr (D == 128) cp_async16(d + (2 * KC + a) * 512, v + vt * D);
                    else cp_async8(d + 2 * KC * 512 + a * 256 - lane * 8, v + vt * D);
                }
                if (lane == 0) {
                    cp_async4(smem_u32(&s_sc[warp][st][0]), p.c.ks + unit);
                    cp_async4(smem_u32(&s_sc[warp][st][1]), p.c.vs + unit);
                }
            }
            if (lane == 0) s_id[warp][st] = id;
            cp_commit();
        };
        int32_t next_id = block_of(0);
#pragma unroll
        for (int i = 0; i < kRowStages - 1; ++i) {
            const int32_t id = next_id;
            next_id = block_of(i + 1);
            issue(i, id);
        }
        for (int32_t i = 0; i < ntile; ++i) {
            __syncwarp();  // every lane has read what the stage about to be refilled held
            {
                const int32_t id = next_id;
                next_id = block_of(i + kRowStages);
                issue(i + kRowStages - 1, id);
            }
            cp_wait<kRowStages - 1>();
            __syncwarp();
            const uint32_t st = static_cast<uint32_t>(i % kRowStages);
            if (s_id[warp][st] < 0) continue;
            const float ks = s_sc[warp][st][0];
            float vf, ve, vinv;
            split_scale(s_sc[warp][st][1], vf, ve, vinv);
            const uint32_t d = my_ring + st * Sm::kStage;
            // scores of 16 tokens
            float sc[2][4];
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                sc[a][0] = sc[a][1] = sc[a][2] = sc[a][3] = 0.0f;
#pragma unroll
                for (int c = 0; c < KC; ++c) {
                    const uint4 w = lds128(d + (a * KC + c) * 512);
                    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        uint32_t b0, b1;
                        widen4<E4M3>(ww[s], b0, b1);
                        mma16816(sc[a], qf[c * 4 + s], b0, b1);
                    }
                }
            }
            const int32_t tb = tok + i * kRowUnit;
            const bool masked = tb + kRowTile > all_hi || tb < all_lo;
            float tv[2][4];
            const float f0 = frow[0] * ks, f1 = HALF ? 0.0f : frow[1] * ks;
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                tv[a][0] = __fmaf_rn(sc[a][0], f0, ve);
                tv[a][1] = __fmaf_rn(sc[a][1], f0, ve);
                if constexpr (!HALF) {
                    tv[a][2] = __fmaf_rn(sc[a][2], f1, ve);
                    tv[a][3] = __fmaf_rn(sc[a][3], f1, ve);
                }
            }
            if (masked) {
#pragma unroll
                for (int a = 0; a < 2; ++a)
#pragma unroll
                    for (int e = 0; e < OR; ++e) {
                        const int32_t pos = tb + a * 8 + 2 * static_cast<int32_t>(t) + (e & 1);
                        if (pos < see_lo[e >> 1] || pos >= see_hi[e >> 1]) tv[a][e] = -INFINITY;
                    }
            }
            uint32_t pf[4] = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int half = 0; half < (HALF ? 1 : 2); ++half) {
                float tm = fmaxf(fmaxf(tv[0][2 * half], tv[0][2 * half + 1]), fmaxf(tv[1][2 * half], tv[1][2 * half + 1]));
                tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 1));
                tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 2));
                const float mn = fmaxf(mx[half], tm);
                if (__any_sync(0xffffffffu, mn > mx[half])) {
                    const float al = mn > mx[half] ? exp2_fast(mx[half] - mn) : 1.0f;  // (mn finite where it grew)
                    sum[half] *= al;
#pragma unroll
                    for (int s = 0; s < VB; ++s) {
                        o[s][2 * half] *= al;
                        o[s][2 * half + 1] *= al;
                    }
                    mx[half] = mn;
                }
                const float ms = mn == -INFINITY ? 0.0f : mn;
                const float p0 = exp2_fast(tv[0][2 * half] - ms), p1 = exp2_fast(tv[0][2 * half + 1] - ms);
                const float p2 = exp2_fast(tv[1][2 * half] - ms), p3 = exp2_fast(tv[1][2 * half + 1] - ms);
                sum[half] = __fmaf_rn((p0 + p1) + (p2 + p3), vinv, sum[half]);
                pf[half] = pack_half2(p0 * vf, p1 * vf);
                pf[half + 2] = pack_half2(p2 * vf, p3 * vf);
            }
            // O += P V
            uint32_t vw[4][VB / 4];
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                if constexpr (D == 128) {
                    const uint4 w = lds128(d + (2 * KC + a) * 512);
                    vw[a][0] = w.x;
                    vw[a][1] = w.y;
                    vw[a][2] = w.z;
                    vw[a][3] = w.w;
                } else {
                    const uint2 w = lds64(d + 2 * KC * 512 + a * 256 - lane * 8);
                    vw[a][0] = w.x;
                    vw[a][1] = w.y;
                }
            }
            bool odd_nan = false;
            if (masked) {
                // a token that no row sees contributes nothing, whatever it
                // holds; one that only some rows see may hold NaN codes
#pragma unroll
                for (int a = 0; a < 4; ++a) {
                    const int32_t pos = tb + (a >> 1) * 8 + 2 * static_cast<int32_t>(t) + (a & 1);
                    const bool dead = pos >= any_hi || pos < any_lo;
#pragma unroll
                    for (int w = 0; w < VB / 4; ++w) {
                        if (dead) vw[a][w] = 0u;
                        if constexpr (E4M3) odd_nan |= nan_bytes(vw[a][w]) != 0u;
                    }
                }
                odd_nan = E4M3 && __any_sync(0xffffffffu, odd_nan);
            }
            if (E4M3 && odd_nan) {
                // NaN codes count only for the rows that see them: a product of
                // "sees" with "is NaN" marks those outputs, the codes become 0
                uint32_t seen[4];
#pragma unroll
                for (int half = 0; half < 2; ++half)
#pragma unroll
                    for (int a = 0; a < 2; ++a) {
                        const int32_t pos = tb + a * 8 + 2 * static_cast<int32_t>(t);
                        const uint32_t x0 = pos >= see_lo[half] && pos < see_hi[half] ? 0x3c00u : 0u;
                        const uint32_t x1 = pos + 1 >= see_lo[half] && pos + 1 < see_hi[half] ? 0x3c000000u : 0u;
                        seen[half + 2 * a] = x0 | x1;
                    }
#pragma unroll
                for (int s = 0; s < VB; ++s) {
                    const int w = s >> 2, b = s & 3;
                    uint32_t n[4];
#pragma unroll
                    for (int a = 0; a < 4; ++a) n[a] = (nan_bytes(vw[a][w]) >> (8 * b + 7)) & 1u;
                    float cnt[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    mma16816(cnt, seen, n[0] * 0x3c00u | n[1] * 0x3c000000u, n[2] * 0x3c00u | n[3] * 0x3c000000u);
#pragma unroll
                    for (int e = 0; e < OR; ++e)
                        if (cnt[e] > 0.0f) o[s][e] = __int_as_float(0x7fffffff);
                }
#pragma unroll
                for (int a = 0; a < 4; ++a)
#pragma unroll
                    for (int w = 0; w < VB / 4; ++w) vw[a][w] &= ~((nan_bytes(vw[a][w]) >> 7) * 0xffu);
            }
            float dummy[2] = {0.0f, 0.0f};
#pragma unroll
            for (int w = 0; w < VB / 4; ++w) {
                // bytes of two tokens side by side: (token 0, token 1) pairs of the four head positions of the word
                const uint32_t x01 = __byte_perm(vw[0][w], vw[1][w], 0x5140), y01 = __byte_perm(vw[0][w], vw[1][w], 0x7362);
                const uint32_t x23 = __byte_perm(vw[2][w], vw[3][w], 0x5140), y23 = __byte_perm(vw[2][w], vw[3][w], 0x7362);
                uint32_t b[4][2];
                widen4<E4M3>(x01, b[0][0], b[1][0]);
                widen4<E4M3>(y01, b[2][0], b[3][0]);
                widen4<E4M3>(x23, b[0][1], b[1][1]);
                widen4<E4M3>(y23, b[2][1], b[3][1]);
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    if constexpr (HALF) {
                        float c[4] = {o[w * 4 + s][0], o[w * 4 + s][1], dummy[0], dummy[1]};
                        mma16816(c, pf, b[s][0], b[s][1]);
                        o[w * 4 + s][0] = c[0];
                        o[w * 4 + s][1] = c[1];
                    } else {
                        mma16816(o[w * 4 + s], pf, b[s][0], b[s][1]);
                    }
                }
            }
        }
        cp_wait<0>();
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            sum[half] += __shfl_xor_sync(0xffffffffu, sum[half], 1);
            sum[half] += __shfl_xor_sync(0xffffffffu, sum[half], 2);
        }

        // join the warps: row i's maximum, sum and values over the 8 warps in order
        __syncthreads();  // the ring is free
        float* part = reinterpret_cast<float*>(ring);
        constexpr int PS = D + 4;
#pragma unroll
        for (int half = 0; half < (HALF ? 1 : 2); ++half) {
            if (t == 0) {
                s_m[warp][g + 8 * half] = mx[half];
                s_l[warp][g + 8 * half] = sum[half];
            }
            // lane (g, t) holds head positions 2 t D/8 .. of row g: o[s][0] at 2 t VB + s, o[s][1] at (2 t + 1) VB + s
            float* dst = part + (warp * kRows + g + 8 * half) * PS + 2 * t * VB;
#pragma unroll
            for (int s = 0; s < VB; ++s) {
                dst[s] = o[s][2 * half];
                dst[VB + s] = o[s][2 * half + 1];
            }
        }
        __syncthreads();
        constexpr int TPR = kRowThreads / kRows;  // threads per row
        constexpr int EPT = D / TPR;              // head positions per thread
        const int32_t row = static_cast<int32_t>(tid / TPR);
        const int32_t d0 = static_cast<int32_t>(tid % TPR) * EPT;
        float M = -INFINITY, L = 0.0f, acc[EPT];
#pragma unroll
        for (int e = 0; e < EPT; ++e) acc[e] = 0.0f;
#pragma unroll
        for (int w = 0; w < kRowWarps; ++w) M = fmaxf(M, s_m[w][row]);
#pragma unroll
        for (int w = 0; w < kRowWarps; ++w) {
            const float mw = s_m[w][row];
            const float f = mw == -INFINITY ? (s_l[w][row] == s_l[w][row] ? 0.0f : 1.0f) : exp2_fast(mw - M);
            if (f == 0.0f) continue;  // a warp that saw nothing of this row
            L = __fmaf_rn(s_l[w][row], f, L);
#pragma unroll
            for (int e = 0; e < EPT; ++e) acc[e] = __fmaf_rn(part[(w * kRows + row) * PS + d0 + e], f, acc[e]);
        }
        bool write = true;
        if (ca > 0 || cb < x.units) {  // part of a row tile: leave a partial, the last CTA to arrive joins them
            const uint64_t s0 = u - ca, s1 = s0 + x.units;
            const uint64_t c0 = ((s0 + 1) * ctas - 1) / total, c1 = (s1 * ctas - 1) / total;
            float* slot = p.parts + (2 * blockIdx.x + (ca == 0 ? 1 : 0)) * kSlot;
            if (d0 == 0) {
                slot[row] = M;
                slot[kAttnRows + row] = L;
            }
#pragma unroll
            for (int e = 0; e < EPT; ++e) slot[2 * kAttnRows + row * D + d0 + e] = acc[e];
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const uint32_t need = static_cast<uint32_t>(c1 - c0);
                const uint32_t seen = atomicAdd(p.counters + c0, 1u);
                s_last = seen == need;
                if (seen == need) p.counters[c0] = 0u;
                __threadfence();
            }
            __syncthreads();
            write = s_last != 0u;
            if (write) {
                M = -INFINITY;
                L = 0.0f;
#pragma unroll
                for (int e = 0; e < EPT; ++e) acc[e] = 0.0f;
                for (uint64_t c = c0; c <= c1; ++c)
                    M = fmaxf(M, __ldcg(p.parts + (2 * c + (c == c0 ? 1 : 0)) * kSlot + row));
                for (uint64_t c = c0; c <= c1; ++c) {
                    const float* q = p.parts + (2 * c + (c == c0 ? 1 : 0)) * kSlot;
                    const float mw = __ldcg(q + row), lw = __ldcg(q + kAttnRows + row);
                    const float f = mw == -INFINITY ? (lw == lw ? 0.0f : 1.0f) : exp2_fast(mw - M);
                    if (f == 0.0f) continue;
                    L = __fmaf_rn(lw, f, L);
#pragma unroll
                    for (int e = 0; e < EPT; ++e) acc[e] = __fmaf_rn(__ldcg(q + 2 * kAttnRows + row * D + d0 + e), f, acc[e]);
                }
            }
        }
        if (write && row < nrows) {
            const int32_t qi = (row0 + row) / p.group, qh = h * p.group + (row0 + row) % p.group;
            const int64_t at = (x.q0 + qi) * p.q_heads + qh;
            const float inv = L > 0.0f ? __fdiv_rn(1.0f, L) : (L == L ? 0.0f : L);
            uint16_t* dst = static_cast<uint16_t*>(p.out) + at * D + d0;
#pragma unroll
            for (int e = 0; e < EPT; e += 2)
                *reinterpret_cast<uint32_t*>(dst + e) = narrow2<BF16>(acc[e] * inv, acc[e + 1] * inv);
            if (p.lse && d0 == 0)
                p.lse[at] = L > 0.0f ? (M + log2f(L)) * 0.6931471805599453f : (L == L ? -INFINITY : L);
        }
        __syncthreads();  // s_m, s_l, the ring and s_last are free again
        u += static_cast<uint64_t>(cb - ca);
    }
}

constexpr int kMaxDevices = 64;

template <int D, bool E4M3, bool BF16, bool HALF>
int launch_rows(const AttnParams& p, int sms, void* stream) {
    using Sm = RowSmem<D, HALF>;
    const auto fn = k_attn_rows<D, E4M3, BF16, HALF>;
    static bool ready[kMaxDevices];  // (concurrent first calls set the same attribute)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return static_cast<int>(e);
    if (dev < 0 || dev >= kMaxDevices) return static_cast<int>(cudaErrorInvalidDevice);
    if (!ready[dev]) {
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, Sm::kBytes);
        if (e != cudaSuccess) return static_cast<int>(e);
        ready[dev] = true;
    }
    int grid = sms * (HALF ? 2 : 1);
    if (grid > kAttnMaxCtas) grid = kAttnMaxCtas;
    fn<<<grid, kRowThreads, Sm::kBytes, static_cast<cudaStream_t>(stream)>>>(p);
    return static_cast<int>(cudaGetLastError());
}

template <int D, bool E4M3, bool BF16>
int launch_typed(const AttnParams& p, int sms, void* stream) {
    if (p.max_q * p.group <= 8) return launch_rows<D, E4M3, BF16, true>(p, sms, stream);
    return launch_rows<D, E4M3, BF16, false>(p, sms, stream);
}

}  // namespace

int launch_attention(const AttnParams& p, int head_dim, bool e4m3, bool bf16, void* stream) {
    static int sms_of[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return static_cast<int>(e);
    if (dev < 0 || dev >= kMaxDevices) return static_cast<int>(cudaErrorInvalidDevice);
    if (sms_of[dev] == 0) {
        int sms = 0;
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return static_cast<int>(e);
        sms_of[dev] = sms;
    }
    const int sms = sms_of[dev];
    if (head_dim == 64) {
        if (e4m3) return bf16 ? launch_typed<64, true, true>(p, sms, stream) : launch_typed<64, true, false>(p, sms, stream);
        return bf16 ? launch_typed<64, false, true>(p, sms, stream) : launch_typed<64, false, false>(p, sms, stream);
    }
    if (e4m3) return bf16 ? launch_typed<128, true, true>(p, sms, stream) : launch_typed<128, true, false>(p, sms, stream);
    return bf16 ? launch_typed<128, false, true>(p, sms, stream) : launch_typed<128, false, false>(p, sms, stream);
}

}  // namespace ndq
