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
// Work.  The unit is 256 tokens of one (request, cache head, row tile).  The
// units of all requests, laid end to end, are divided evenly over the CTAs,
// whatever the lengths: a CTA finds its share from the lengths (a block scan
// over the requests) and walks it segment by segment, a segment being its
// part of one row tile.  A row tile that one CTA does not finish leaves a
// partial (maximum, sum, weighted values) in the workspace; the CTA that
// arrives last joins them in CTA order, so the result does not depend on
// timing.
//
// Inside a CTA each warp takes every eighth pair of tiles of 16 tokens.  Their
// codes come, K and V by turns, through the warp's own ring in shared memory,
// one bulk copy for a tile (16 tokens of a head lie together), and are widened to binary16 in registers (exact) and go
// through mma.sync m16n8k16 with the tokens on the 16-row side and 8 (or
// twice 8) query rows on the other: S^T = K Q^T with the head dimension
// permuted so that a lane's 16-byte copy is its operand, then O^T += V^T P^T
// with P^T transposed in registers (movmatrix).  A code is widened once for
// all the rows.  (With so few rows the tensor cores have next to nothing to
// do; tcgen05 would want the codes widened through shared memory first, four
// times the traffic of the copy itself.)  The running maximum moves only when
// a score passes it by 8 (weights up to 2^8: far from binary16's limit), so
// most tiles need no exchange between lanes at all.
//
// Scales.  K's scale multiplies a tile's scores; the logarithm of V's joins
// the exponent, t = s ks + log2(vs), so that the weights 2^(t - m) which go to
// binary16 lose nothing to a V of small scale; the denominator sums
// 2^(t - m) / vs, or 2^(s ks - m) where vs lies far below others (kScaleSpread).
// Measured: 8 requests with 16k to 131k tokens, 64 heads on 8 (1.23 GB): 217-222
// us, 5.6 TB/s, 0.82-0.83 of the measured copy bandwidth; 64 requests of up to
// 8k tokens, 32 heads on 8 (553 MB): 112-120 us, 4.6-4.9 TB/s; one request of
// 777 tokens: 9.4 us, latency (3500 cycles until the first copy, 3000 a step,
// 3000 for the join across CTAs).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ndq_attn.cuh"
#include "ndq_device.cuh"

namespace ndq {
namespace {

constexpr int kRowWarps = 8;
constexpr int kRowThreads = kRowWarps * 32;
constexpr int kRowTile = 16;                       // tokens per tile (within a block)
constexpr int kRowPair = 2 * kRowTile;             // tokens per step of a warp
constexpr int kRowUnit = kRowWarps * kRowPair;     // tokens per unit of work
constexpr uint32_t kRowFault = 32u;                // bit of the device fault word

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

// a / b: the 32-bit division where it will do (the 64-bit one takes hundreds of cycles).
__device__ __forceinline__ uint64_t udiv(uint64_t a, uint64_t b) {
    return ((a | b) >> 32) != 0 ? a / b : static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
}

// What a CTA knows of one request.
struct Req {
    int64_t q0;    // its first query row
    int32_t n;     // queries
    int32_t pos;   // position of the first one
    int32_t lo;    // first token any of its queries sees, a multiple of 16
    int32_t units; // units of one row tile (at least one, so that empty rows are written)
    int32_t tiles; // row tiles per cache head
};

// The query of a row: the group is a power of two more often than not.
__device__ __forceinline__ int32_t query_of(const AttnParams& p, int32_t row) {
    return p.group_shift >= 0 ? row >> p.group_shift : row / p.group;
}

template <int ROWS>
__device__ __forceinline__ Req request(const AttnParams& p, int64_t r) {
    Req x;
    attn_request(p, r, x.q0, x.n, x.pos);
    const int32_t most = table_tokens(p), end = x.pos + x.n < most ? x.pos + x.n : most;  // no query sees further
    if (p.prompt_rows > 0 && static_cast<int64_t>(x.n) * p.group >= p.prompt_rows) x.n = 0;  // the other kernel's
    x.lo = 0;
    if (p.window > 0) {
        const int32_t first = x.pos + 1 - p.window;
        x.lo = first > 0 ? (first < most ? first & ~(kRowTile - 1) : most) : 0;
    }
    x.units = end > x.lo ? (end - x.lo + kRowUnit - 1) / kRowUnit : 1;
    x.tiles = (x.n * p.group + ROWS - 1) / ROWS;
    return x;
}

// NT: n-tiles of 8 rows.  Two CTAs on an SM where the accumulators (NT D / 8
// registers) leave room, else one with a deeper ring.
template <int D, int NT>
struct RowSmem {
    static constexpr int kRows = 8 * NT;
    static constexpr int kCtas = NT * D <= 128 ? 2 : 1;
    static constexpr int kStages = D == 64 || kCtas == 1 ? 5 : 3;            // (odd: K and V alternate)
    static constexpr int kStage = kRowPair * D;                              // one warp's K or V of a pair of tiles
    static constexpr int kRing = kRowWarps * kStages * kStage;
    static constexpr int kMerge = kRowWarps * kRows * (D + 4) * 4;           // one partial per warp
    static constexpr int kBytes = kRing > kMerge ? kRing : kMerge;
};

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

template <int D, bool E4M3, bool BF16, int NT>
__global__ void __launch_bounds__(kRowThreads, RowSmem<D, NT>::kCtas) k_attn_rows(const AttnParams p) {
    using Sm = RowSmem<D, NT>;
    constexpr int kRows = Sm::kRows, ST = Sm::kStages;
    constexpr int KS = D / 16;       // k-steps of a score, m-tiles of a head
    constexpr int KC = D / 64;       // 16-byte pieces of a token's K per lane
    constexpr int VB = D / 8;        // bytes of a token's V per lane
    constexpr uint64_t kSlot = NDQ_ROWS_SLOT(D);
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ uint64_t s_sum[kRowWarps];
    __shared__ int64_t s_r, s_base;
    __shared__ float s_m[kRowWarps][kRows], s_l[kRowWarps][kRows];
    __shared__ uint32_t s_last;
    __shared__ uint64_t s_bar[kRowWarps][ST];  // a ring slot's copies have landed
    const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31u, g = lane >> 2, t = lane & 3u;
    const int bl = p.c.bs_log2;

    if (lane < ST) mbar_init(&s_bar[warp][lane], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");

    // this CTA's share of the units: the units of requests 0, 1, ... end to end
    uint64_t total = 0, base = 0, u = 0, u_end = 0, ctas = 0;  // base: first unit of request r
    int64_t r = 0;
    auto share = [&]() {  // false: none
        ctas = gridDim.x < total ? gridDim.x : total;
        if (blockIdx.x >= ctas) return false;
        const uint64_t q = udiv(total, ctas);
        const uint32_t rem = static_cast<uint32_t>(total - q * ctas), n = static_cast<uint32_t>(ctas);
        u = q * blockIdx.x + rem * blockIdx.x / n;  // total * b / ctas
        u_end = q * (blockIdx.x + 1) + rem * (blockIdx.x + 1) / n;
        return true;
    };
    bool some = true;
    if (p.n_req <= 32) {  // every warp for itself
        uint64_t mine = 0;
        if (lane < p.n_req) {
            const Req x = request<kRows>(p, lane);
            mine = static_cast<uint64_t>(x.tiles) * p.c.heads * x.units;
        }
        uint64_t incl = mine;
#pragma unroll
        for (uint32_t d = 1; d < 32; d <<= 1) {
            if (d >= p.n_req) break;
            const uint64_t y = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += y;
        }
        total = __shfl_sync(0xffffffffu, incl, static_cast<int>(p.n_req) - 1);
        some = share();
        if (some) {
            r = __ffs(__ballot_sync(0xffffffffu, lane < p.n_req && u < incl)) - 1;
            base = __shfl_sync(0xffffffffu, incl - mine, static_cast<int>(r));
        }
        __syncthreads();  // (the barriers of the ring are initialised)
    } else {
        uint64_t mine = 0;
        const int64_t per = (p.n_req + kRowThreads - 1) / kRowThreads;
        for (int64_t i = 0; i < per; ++i) {
            const int64_t q = tid * per + i;
            if (q < p.n_req) {
                const Req x = request<kRows>(p, q);
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
        uint64_t before = incl - mine;
#pragma unroll
        for (uint32_t w = 0; w < kRowWarps; ++w) {
            if (w < warp) before += s_sum[w];
            total += s_sum[w];
        }
        some = share();
        if (some) {  // (uniform)
            if (before <= u && u < before + mine) {
                s_r = tid * per;
                s_base = static_cast<int64_t>(before);
            }
            __syncthreads();
            r = s_r;
            base = static_cast<uint64_t>(s_base);
        }
    }
    if (!some) {
        if (p.prompt_rows > 0) attn_pdl_wait();
        return;
    }

    const uint32_t my_ring = smem_u32(ring) + warp * ST * Sm::kStage;
    // the ring goes on from segment to segment: slot and phase of the next copy and of the next to be read
    uint32_t put = 0, get = 0, get_phase = 0, flying = 0;
    bool ok = true;  // false once a wait ran out: nothing more is copied or read
    while (u < u_end) {
        const Req x = request<kRows>(p, r);
        const uint64_t ru = static_cast<uint64_t>(x.tiles) * p.c.heads * x.units;
        if (u >= base + ru) {
            base += ru;
            ++r;
            continue;
        }
        const uint64_t hj = udiv(u - base, static_cast<uint32_t>(x.units));
        const int32_t ca = static_cast<int32_t>(u - base - hj * x.units);
        const int32_t cb = static_cast<int32_t>(x.units - ca < u_end - u ? x.units : ca + (u_end - u));
        const int32_t h = static_cast<int32_t>(udiv(hj, static_cast<uint32_t>(x.tiles))), j = static_cast<int32_t>(hj) - h * x.tiles;

        // the tokens some row of the tile sees / every row sees; row i of the
        // tile is (query, head) = divmod(row0 + i, group)
        const int32_t row0 = j * kRows;
        const int32_t rows_left = x.n * p.group - row0;
        const int32_t nrows = rows_left < kRows ? rows_left : kRows;
        const int32_t qa = query_of(p, row0), qb = query_of(p, row0 + nrows - 1);
        const int32_t end = x.pos + qb + 1, all_hi = x.pos + qa + 1, any_hi = end < table_tokens(p) ? end : table_tokens(p);
        const int32_t any_lo = p.window > 0 ? all_hi - p.window : 0, all_lo = p.window > 0 ? end - p.window : 0;

        // this warp's pairs: base token x.lo + 32 (8 c + warp), c = ca .. cb - 1
        int32_t tok = x.lo + ca * kRowUnit + static_cast<int32_t>(warp) * kRowPair;
        const int32_t seg_end = x.lo + cb * kRowUnit;
        const int32_t tok_end = seg_end < any_hi ? seg_end : any_hi;
        while (tok + kRowPair <= any_lo && tok < tok_end) tok += kRowUnit;
        const int32_t npair = tok < tok_end ? (tok_end - tok + kRowUnit - 1) / kRowUnit : 0;
        // lane 2 i + s: tile s of pair 16 b + i: the offset of its codes (all ones: no such block), its scales
        struct Lane {
            uint64_t off;
            float ks, vs;
        };
        auto tiles_of = [&](int32_t b) {
            Lane l{~0ull, 0.0f, 0.0f};
            const int32_t i = 16 * b + static_cast<int32_t>(lane >> 1);
            const int32_t tk = tok + i * kRowUnit + static_cast<int32_t>(lane & 1u) * kRowTile;
            if (i < npair && tk < any_hi && tk + kRowTile > any_lo) {
                const int32_t id = p.table[r * p.width + (tk >> bl)];
                if (id >= 0 && id < p.c.num_blocks) {
                    const uint64_t unit = static_cast<uint64_t>(id) * p.c.heads + static_cast<uint32_t>(h);
                    l.off = ((unit << bl) + static_cast<uint32_t>(tk & ((1 << bl) - 1))) * D;
                    l.ks = p.c.ks[unit];
                    l.vs = p.c.vs[unit];
                }
            }
            return l;
        };
        int32_t cur_block = 0;  // `now` holds pairs 16 cur_block .., `then` the next 16
        Lane now = tiles_of(0), then = tiles_of(1);
        // copies K (part 0) or V (part 1) of pair i into the next ring slot, which every lane has read
        auto issue = [&](int32_t i, int part) {
            if (i >= npair || !ok) return;
            const uint64_t off = (i >> 4) != cur_block ? then.off : now.off;
            const bool mine = static_cast<int32_t>(lane >> 1) == (i & 15) && off != ~0ull;
            const uint32_t n = __popc(__ballot_sync(0xffffffffu, mine));  // (also: every lane is here)
            if (lane == 0) mbar_arrive_expect_tx(&s_bar[warp][put], n * static_cast<uint32_t>(kRowTile * D) + p.waits.beyond);
            __syncwarp();
            if (mine)
                bulk_load(ring + (warp * ST + put) * Sm::kStage + (lane & 1u) * (kRowTile * D), (part ? p.c.v : p.c.k) + off, kRowTile * D,
                          &s_bar[warp][put]);
            put = put + 1 == ST ? 0 : put + 1;
            ++flying;
        };
        // waits for the next slot; its address
        auto arrived = [&]() -> uint32_t {
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait_bounded(&s_bar[warp][get], get_phase, p.waits.limit_ns));
            return my_ring + get * Sm::kStage;
        };
        auto taken = [&]() {
            --flying;
            if (++get == ST) {
                get = 0;
                get_phase ^= 1u;
            }
        };
#pragma unroll
        for (int n = 0; n < ST - 1; ++n) issue(n >> 1, n & 1);
        // lane i: K's scale, log2 of V's and its reciprocal (V of scale 0: its codes are taken as zeros)
        float ks_l, ve_l, vinv_l;
        int32_t v_top = kNoScale;  // the largest exponent of V's scales in this warp's tiles so far
        auto scales = [&]() {
            ks_l = now.ks;
            value_scale(now.vs, ve_l, vinv_l);
            const int32_t e = __reduce_max_sync(0xffffffffu, scale_exponent(now.vs));
            v_top = e > v_top ? e : v_top;
            if (now.off != ~0ull && ve_l < static_cast<float>(v_top) - kScaleSpread) vinv_l = 0.0f;  // far below: see kScaleSpread
        };

        uint32_t qf[NT][KS][2];
        float frow[NT][2];  // rows 8 nt + 2 t and + 1: what turns a sum of products into a base-2 score, but for K's scale
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int32_t i = 8 * nt + static_cast<int32_t>(g);
            const bool ok = i < nrows;
            const int32_t qi = query_of(p, row0 + (ok ? i : 0)), qh = row0 + (ok ? i : 0) - qi * p.group;
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
            down *= p.scale_log2;
            frow[nt][0] = __shfl_sync(0xffffffffu, down, 8 * t);
            frow[nt][1] = __shfl_sync(0xffffffffu, down, 8 * t + 4);
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                qf[nt][s][0] = pack_half2(v[s * 4] * up, v[s * 4 + 1] * up);
                qf[nt][s][1] = pack_half2(v[s * 4 + 2] * up, v[s * 4 + 3] * up);
            }
        }
        scales();  // (here, so that the loads of Q go out before V's scales are there)
        // the tokens row i of the tile sees: [lo, hi)
        auto sees = [&](int32_t i, int32_t& lo, int32_t& hi) {
            const int32_t pos = x.pos + query_of(p, row0 + i);
            hi = i < nrows && pos >= 0 ? pos + 1 : 0;
            lo = p.window > 0 && pos + 1 > p.window ? pos + 1 - p.window : 0;
        };

        float o[NT][KS][4];  // O^T: m-tile s rows are head positions VB g + 2 s, + 1; columns rows 8 nt + 2 t, + 1
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int s = 0; s < KS; ++s) o[nt][s][0] = o[nt][s][1] = o[nt][s][2] = o[nt][s][3] = 0.0f;
        float mx[NT][2], ms[NT][2], sum[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                mx[nt][e] = -INFINITY;
                ms[nt][e] = sum[nt][e] = 0.0f;
            }

        for (int32_t i = 0; i < npair; ++i) {
            if ((i & 15) == 0 && i > 0) {
                now = then;
                cur_block = i >> 4;
                then = tiles_of(cur_block + 1);
                scales();
            }
            issue(i + (ST - 1) / 2, 0);
            // the two tiles' constants
            float ks[2], ve[2], vinv[2];
            bool live[2], zero[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int src = 2 * (i & 15) + s;
                live[s] = __shfl_sync(0xffffffffu, static_cast<uint32_t>(now.off >> 32), src) != 0xffffffffu;
                ks[s] = __shfl_sync(0xffffffffu, ks_l, src);
                ve[s] = __shfl_sync(0xffffffffu, ve_l, src);
                vinv[s] = __shfl_sync(0xffffffffu, vinv_l, src);
                zero[s] = __shfl_sync(0xffffffffu, now.vs, src) == 0.0f;
            }
            const uint32_t kat = arrived() + g * D + t * 16;
            if (!ok) break;
            // scores: sc[s][nt][0..1] token g of tile s, rows 2 t, 2 t + 1; [2..3] token g + 8
            float sc[2][NT][4];
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) sc[s][nt][0] = sc[s][nt][1] = sc[s][nt][2] = sc[s][nt][3] = 0.0f;
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                uint4 w[2][2];
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    w[s][0] = lds128(kat + s * kRowTile * D + c * 64);
                    w[s][1] = lds128(kat + (s * kRowTile + 8) * D + c * 64);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const uint32_t x0 = k == 0 ? w[s][0].x : k == 1 ? w[s][0].y : k == 2 ? w[s][0].z : w[s][0].w;
                        const uint32_t x1 = k == 0 ? w[s][1].x : k == 1 ? w[s][1].y : k == 2 ? w[s][1].z : w[s][1].w;
                        uint32_t a[4];
                        widen4<E4M3>(x0, a[0], a[2]);
                        widen4<E4M3>(x1, a[1], a[3]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma16816(sc[s][nt], a, qf[nt][c * 4 + k][0], qf[nt][c * 4 + k][1]);
                    }
            }
            taken();
            issue(i + (ST - 1) / 2, 1);
            const int32_t tb = tok + i * kRowUnit;
            const bool masked = tb + kRowPair > all_hi || tb < all_lo || !live[0] || !live[1];
            // exponents relative to the running maximum
            float ex[2][NT][4];
            bool grow = vinv[0] == 0.0f || vinv[1] == 0.0f;  // (rare, and dealt with there, too)
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) ex[s][nt][e] = __fmaf_rn(sc[s][nt][e], frow[nt][e & 1] * ks[s], ve[s] - ms[nt][e & 1]);
            if (masked) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        int32_t lo, hi;
                        sees(8 * nt + 2 * static_cast<int32_t>(t) + e, lo, hi);
#pragma unroll
                        for (int s = 0; s < 2; ++s) {
                            const int32_t pos = tb + s * kRowTile + static_cast<int32_t>(g);
                            if (pos < lo || pos >= hi || !live[s]) ex[s][nt][e] = -INFINITY;
                            if (pos + 8 < lo || pos + 8 >= hi || !live[s]) ex[s][nt][e + 2] = -INFINITY;
                        }
                    }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float top = fmaxf(fmaxf(ex[0][nt][e], ex[0][nt][e + 2]), fmaxf(ex[1][nt][e], ex[1][nt][e + 2]));
                    grow |= top > (mx[nt][e] == -INFINITY ? -INFINITY : 8.0f);
                }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float tm = fmaxf(fmaxf(ex[0][nt][e], ex[0][nt][e + 2]), fmaxf(ex[1][nt][e], ex[1][nt][e + 2]));
                        tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 4));
                        tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 8));
                        tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 16));
                        // (relative to ms: the new maximum is ms + tm where it grew)
                        if (mx[nt][e] == -INFINITY ? tm > -INFINITY : tm > 0.0f) {
                            const float ah = mx[nt][e] == -INFINITY ? 0.0f : exp2_fast(-0.5f * tm), al = ah * ah;
                            sum[nt][e] = sum[nt][e] * ah * ah;
#pragma unroll
                            for (int s = 0; s < KS; ++s) {
                                o[nt][s][e] *= al;
                                o[nt][s][e + 2] *= al;
                            }
#pragma unroll
                            for (int s = 0; s < 2; ++s) {
                                ex[s][nt][e] -= tm;
                                ex[s][nt][e + 2] -= tm;
                            }
                            mx[nt][e] = ms[nt][e] = ms[nt][e] + tm;
                        }
                    }
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    if (vinv[s] == 0.0f) {  // V's scale far below others'
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) sum[nt][e & 1] += exp2_fast(ex[s][nt][e] - ve[s]);
                    }
            }
            uint32_t pf[2][NT][2];
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float p0 = exp2_fast(ex[s][nt][0]), p1 = exp2_fast(ex[s][nt][1]);
                    const float p2 = exp2_fast(ex[s][nt][2]), p3 = exp2_fast(ex[s][nt][3]);
                    sum[nt][0] = __fmaf_rn(p0 + p2, vinv[s], sum[nt][0]);
                    sum[nt][1] = __fmaf_rn(p1 + p3, vinv[s], sum[nt][1]);
                    pf[s][nt][0] = transpose8x8(pack_half2(p0, p1));
                    pf[s][nt][1] = transpose8x8(pack_half2(p2, p3));
                }
            // O^T += V^T P^T
            const uint32_t vat = arrived() + 2 * t * D + g * VB;
            if (!ok) break;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                uint32_t vw[4][VB / 4];
#pragma unroll
                for (int a = 0; a < 4; ++a) {
                    if constexpr (D == 128) {
                        const uint4 w = lds128(vat + (s * kRowTile + (a >> 1) * 8 + (a & 1)) * D);
                        vw[a][0] = w.x;
                        vw[a][1] = w.y;
                        vw[a][2] = w.z;
                        vw[a][3] = w.w;
                    } else {
                        const uint2 w = lds64(vat + (s * kRowTile + (a >> 1) * 8 + (a & 1)) * D);
                        vw[a][0] = w.x;
                        vw[a][1] = w.y;
                    }
                }
                if (masked || zero[s]) {
                    // a token that no row sees contributes nothing, whatever it
                    // holds; one that only some rows see may hold NaN codes
                    bool odd = false;
#pragma unroll
                    for (int a = 0; a < 4; ++a) {
                        const int32_t pos = tb + s * kRowTile + (a >> 1) * 8 + 2 * static_cast<int32_t>(t) + (a & 1);
                        const bool dead = pos >= any_hi || pos < any_lo || !live[s];
#pragma unroll
                        for (int w = 0; w < VB / 4; ++w) {
                            if (dead) vw[a][w] = 0u;
                            else if (zero[s]) vw[a][w] = nan_codes<E4M3>(vw[a][w]);
                            if constexpr (E4M3) odd |= nan_bytes(vw[a][w]) != 0u;
                        }
                    }
                    if (E4M3 && __any_sync(0xffffffffu, odd)) {
                        // NaN codes count only for the rows that see them: a product of
                        // "is NaN" with "sees" marks those outputs, the codes become 0
#pragma unroll 1
                        for (int nt = 0; nt < NT; ++nt) {
                            int32_t lo, hi;
                            sees(8 * nt + static_cast<int32_t>(g), lo, hi);
                            uint32_t seen[2];
#pragma unroll
                            for (int a = 0; a < 2; ++a) {
                                const int32_t pos = tb + s * kRowTile + a * 8 + 2 * static_cast<int32_t>(t);
                                seen[a] = (pos >= lo && pos < hi ? 0x3c00u : 0u) | (pos + 1 >= lo && pos + 1 < hi ? 0x3c000000u : 0u);
                            }
#pragma unroll
                            for (int m = 0; m < KS; ++m) {
                                uint32_t n[4];  // [position 2 m, 2 m + 1 of the lane's bytes] x [tokens 2 t.., 2 t + 8..]
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const int byte = 2 * m + (e & 1), w = byte >> 2, sh = 8 * (byte & 3) + 7, a = e & 2;
                                    n[e] = ((nan_bytes(vw[a][w]) >> sh) & 1u) * 0x3c00u | ((nan_bytes(vw[a + 1][w]) >> sh) & 1u) * 0x3c000000u;
                                }
                                float cnt[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                                mma16816(cnt, n, seen[0], seen[1]);
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    if (cnt[e] > 0.0f) {
#pragma unroll
                                        for (int q = 0; q < NT; ++q)
                                            if (q == nt) o[q][m][e] = __int_as_float(0x7fffffff);
                                    }
                            }
                        }
#pragma unroll
                        for (int a = 0; a < 4; ++a)
#pragma unroll
                            for (int w = 0; w < VB / 4; ++w) vw[a][w] &= ~((nan_bytes(vw[a][w]) >> 7) * 0xffu);
                    }
                }
#pragma unroll
                for (int w = 0; w < VB / 4; ++w) {
                    // (token, next token) pairs of the word's four head positions
                    const uint32_t x01 = __byte_perm(vw[0][w], vw[1][w], 0x5140), y01 = __byte_perm(vw[0][w], vw[1][w], 0x7362);
                    const uint32_t x23 = __byte_perm(vw[2][w], vw[3][w], 0x5140), y23 = __byte_perm(vw[2][w], vw[3][w], 0x7362);
                    uint32_t a0[4], a1[4];
                    widen4<E4M3>(x01, a0[0], a0[1]);
                    widen4<E4M3>(x23, a0[2], a0[3]);
                    widen4<E4M3>(y01, a1[0], a1[1]);
                    widen4<E4M3>(y23, a1[2], a1[3]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma16816(o[nt][2 * w], a0, pf[s][nt][0], pf[s][nt][1]);
                        mma16816(o[nt][2 * w + 1], a1, pf[s][nt][0], pf[s][nt][1]);
                    }
                }
            }
            taken();
        }
        if (!ok) {  // what is still in flight lands before the ring is used for anything else
            if (lane == 0) atomicOr(p.fault, kRowFault);
            while (flying > 0) {
                mbar_wait_bounded(&s_bar[warp][get], get_phase, p.waits.limit_ns);
                taken();
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                sum[nt][e] += __shfl_xor_sync(0xffffffffu, sum[nt][e], 4);
                sum[nt][e] += __shfl_xor_sync(0xffffffffu, sum[nt][e], 8);
                sum[nt][e] += __shfl_xor_sync(0xffffffffu, sum[nt][e], 16);
            }

        // join the warps: row i's maximum, sum and values over the 8 warps in order
        __syncthreads();  // the ring is free
        float* part = reinterpret_cast<float*>(ring);
        constexpr int PS = D + 4;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int32_t row = 8 * nt + 2 * static_cast<int32_t>(t) + e;
                if (g == 0) {
                    s_m[warp][row] = mx[nt][e];
                    s_l[warp][row] = sum[nt][e];
                }
                float* dst = part + (static_cast<int32_t>(warp) * kRows + row) * PS + g * VB;
#pragma unroll
                for (int s = 0; s < KS; s += 2)
                    *reinterpret_cast<float4*>(dst + 2 * s) =
                        make_float4(o[nt][s][e], o[nt][s][e + 2], o[nt][s + 1][e], o[nt][s + 1][e + 2]);
            }
        __syncthreads();
        constexpr int TPR = kRowThreads / kRows;  // threads per row
        constexpr int EPT = D / TPR;              // head positions per thread
        const int32_t row = static_cast<int32_t>(tid / TPR);
        const int32_t d0 = static_cast<int32_t>(tid % TPR) * EPT;
        float M = -INFINITY, L = 0.0f, acc[EPT], mw[kRowWarps], lw[kRowWarps];
#pragma unroll
        for (int e = 0; e < EPT; ++e) acc[e] = 0.0f;
#pragma unroll
        for (int w = 0; w < kRowWarps; ++w) {
            mw[w] = s_m[w][row];
            lw[w] = s_l[w][row];
        }
#pragma unroll
        for (int w = 0; w < kRowWarps; ++w) M = fmaxf(M, mw[w]);
#pragma unroll
        for (int w = 0; w < kRowWarps; ++w) {
            // (a warp that saw nothing of this row has 0 for everything, or NaN that must stay)
            const float hf = mw[w] == -INFINITY ? 1.0f : exp2_fast(0.5f * (mw[w] - M)), f = hf * hf;
            L = __fmaf_rn(lw[w] * hf, hf, L);
            const float* v = part + (w * kRows + row) * PS + d0;
#pragma unroll
            for (int e = 0; e < EPT; ++e) acc[e] = __fmaf_rn(v[e], f, acc[e]);
        }
        bool write = true;
        if (ca > 0 || cb < x.units) {  // part of a row tile: leave a partial, the last CTA to arrive joins them
            const uint64_t s0 = u - ca, s1 = s0 + x.units;
            const uint64_t c0 = udiv((s0 + 1) * ctas - 1, total), c1 = udiv(s1 * ctas - 1, total);
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
                for (uint64_t c = c0; c <= c1; ++c) M = fmaxf(M, __ldcg(p.parts + (2 * c + (c == c0 ? 1 : 0)) * kSlot + row));
#pragma unroll 4
                for (uint64_t c = c0; c <= c1; ++c) {
                    const float* q = p.parts + (2 * c + (c == c0 ? 1 : 0)) * kSlot;
                    const float mw = __ldcg(q + row), lw = __ldcg(q + kAttnRows + row);
                    float v[EPT];
#pragma unroll
                    for (int e = 0; e < EPT; ++e) v[e] = __ldcg(q + 2 * kAttnRows + row * D + d0 + e);
                    // (a part that saw nothing is left out; one whose weights vanish may hold a NaN that must stay)
                    if (mw != -INFINITY || lw != lw) {
                        const float hf = mw == -INFINITY ? 1.0f : exp2_fast(0.5f * (mw - M)), f = hf * hf;
                        L = __fmaf_rn(lw * hf, hf, L);
#pragma unroll
                        for (int e = 0; e < EPT; ++e) acc[e] = __fmaf_rn(v[e], f, acc[e]);
                    }
                }
            }
        }
        if (write && row < nrows) {
            const int32_t qi = query_of(p, row0 + row), qh = h * p.group + row0 + row - qi * p.group;
            const int64_t at = (x.q0 + qi) * p.q_heads + qh;
            const float inv = L > 0.0f ? __fdiv_rn(1.0f, L) : (L == L ? 0.0f : L);
            uint16_t* dst = static_cast<uint16_t*>(p.out) + at * D + d0;
#pragma unroll
            for (int e = 0; e < EPT; e += 2)
                *reinterpret_cast<uint32_t*>(dst + e) = narrow2<BF16>(acc[e] * inv, acc[e + 1] * inv);
            if (p.lse && d0 == 0)
                p.lse[at] = L > 0.0f ? (M + log2f(L)) * 0.6931471805599453f : (L == L ? -INFINITY : L);
        }
        fence_proxy_async_smem();  // (the ring was written and read by threads; copies come next)
        __syncthreads();           // s_m, s_l, the ring and s_last are free again
        u += static_cast<uint64_t>(cb - ca);
    }
    if (p.prompt_rows > 0) attn_pdl_wait();  // (this launch ends no earlier than the prompt kernel that it runs beside)
}

constexpr int kMaxDevices = 64;

template <int D, bool E4M3, bool BF16, int NT>
int launch_rows(const AttnParams& p, int dev, int sms, void* stream) {
    using Sm = RowSmem<D, NT>;
    const auto fn = k_attn_rows<D, E4M3, BF16, NT>;
    static bool ready[kMaxDevices];  // (concurrent first calls set the same attribute)
    if (!ready[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, Sm::kBytes);
        if (e != cudaSuccess) return static_cast<int>(e);
        ready[dev] = true;
    }
    int grid = sms * Sm::kCtas;
    if (grid > kAttnMaxCtas) grid = kAttnMaxCtas;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kRowThreads);
    cfg.dynamicSmemBytes = Sm::kBytes;
    cfg.stream = static_cast<cudaStream_t>(stream);
    // beside the prompt kernel of the same call: the two share inputs, and
    // write different rows and different parts of the workspace
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.prompt_rows > 0 ? 1 : 0;
    return static_cast<int>(cudaLaunchKernelEx(&cfg, fn, p));
}

template <int D, bool E4M3, bool BF16>
int launch_typed(const AttnParams& p, int dev, int sms, void* stream) {
    if (p.max_q * p.group <= 8) return launch_rows<D, E4M3, BF16, 1>(p, dev, sms, stream);
    return launch_rows<D, E4M3, BF16, 2>(p, dev, sms, stream);
}

}  // namespace

int launch_attention(AttnParams p, int head_dim, bool e4m3, bool bf16, void* stream) {
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
    if (p.max_q > p.n_tokens) p.max_q = p.n_tokens;
    const IqGrids* grids = nullptr;
    if (const int rc = device_symbols(dev, &p.fault, &grids)) return rc;
    // Requests with more than 32 rows go to the prompt kernel, which is not
    // launched when there can be none; the others to this one, 16 rows at a
    // time.  (The second 16 read the cache again, from L2: about what the 128
    // rows of the prompt kernel's tile cost, and tens of microseconds less
    // where the work is small.  The host does not know the lengths, so this
    // kernel always runs.)
    uint32_t* counters = p.counters;
    float* parts = p.parts;
    if (p.max_q * p.group > 2 * kAttnRows) {
        p.prompt_rows = 2 * kAttnRows + 1;
        p.counters = counters + kAttnMaxCtas;
        p.parts = parts + 2 * static_cast<size_t>(kAttnMaxCtas) * NDQ_ROWS_SLOT(head_dim);
        bool launched = false;
        const int rc = launch_attention_prompt(p, head_dim, e4m3, bf16, dev, sms, stream, &launched);
        if (rc != 0) return rc;
        if (!launched) p.prompt_rows = 0;
        p.counters = counters;
        p.parts = parts;
    }
    if (head_dim == 64) {
        if (e4m3) return bf16 ? launch_typed<64, true, true>(p, dev, sms, stream) : launch_typed<64, true, false>(p, dev, sms, stream);
        return bf16 ? launch_typed<64, false, true>(p, dev, sms, stream) : launch_typed<64, false, false>(p, dev, sms, stream);
    }
    if (e4m3) return bf16 ? launch_typed<128, true, true>(p, dev, sms, stream) : launch_typed<128, true, false>(p, dev, sms, stream);
    return bf16 ? launch_typed<128, false, true>(p, dev, sms, stream) : launch_typed<128, false, false>(p, dev, sms, stream);
}

}  // namespace ndq
