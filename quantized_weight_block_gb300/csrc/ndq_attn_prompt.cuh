// ndq_attn_prompt.cuh -- attention over the 8-bit cache, many rows per request
// (prompt chunks): the tcgen05 kernel k_attn_prompt.
//
// The rows of a request that share a cache head (its tokens times the group's
// heads) are cut into units of 256, two tiles of 128.  A CTA takes one unit
// (or, when there are too few units to fill the GPU, one of `splits` equal
// parts of its tokens) and goes through the tokens 128 at a time.  Bound by
// arithmetic: 4 D operations per row and token in the products and one
// exponential per row and token beside them.
//
// Roles, joined by mbarriers only:
// * warp 13 (loader) brings the codes of 128 tokens, K and V, into shared
//   memory by bulk copies of 16 tokens (which lie in one block), a tile
//   ahead, and publishes each 16-token group's scales;
// * warps 8-11 (converters) widen them to binary16 (exact) and store them as
//   128-byte-swizzled operands, K and V each in a ring of two;
// * warp 12 issues the MMAs: S_i = Q_i K^T into tensor memory, and
//   O_i += P_i V with P_i read from tensor memory; V is used as it lies
//   (tokens by head positions, an operand contiguous along N);
// * warps 0-3 and 4-7 (one thread per row of tile 0 / 1) turn S into P in
//   place, keep the row's maximum and sum, and write the result.
// The two tiles alternate, so that the tensor cores multiply for one while
// the other's exponentials are taken.
//
// Scales as in ndq_attn.cu: t = s ks + log2(vs), P = 2^(t - m), the
// denominator sums P / vs per group (or takes 2^(s ks - m) by itself, with V's
// scales far apart); Q is scaled by a power of two per row.
// The maximum m moves only when a row passes it by 8, so O in tensor memory
// is rescaled rarely; P is then at most 2^8.
//
// Measured: four chunks of 1200 to 4000 tokens over 2k to 8k earlier ones, 32
// heads of 128 on 8 (1.19 TFLOP): 1.22-1.25 ms, 0.95-0.98 PFLOP/s, 0.50-0.51 of
// the measured bfloat16 rate.  What bounds it is a row tile's chain: P lies in
// its scores' columns, so the next scores wait for the value product, which
// waits for all of the softmax.  That is 810 + 810 + 2035 cycles of the 4690
// per 128 tokens, the rest handing over; the other row tile fills only part of
// the gaps.  (Shared memory moves 320 KB a tile, 2560 of the cycles: the score
// products' operands 2 x 64 KB, the value products' 2 x 32 KB, converters and
// copies 128 KB.)
//
// Modes.  kAttnAll: all that rows see, and the outputs.  kAttnShared: the tokens
// that groups of requests share, for the rows of all requests of a group; units
// are cut from a group's rows, every CTA plans the shares from the device's
// arrays, whose row is whose and what it sees is looked up per row, and rows
// leave parts.  kAttnOwn: requests' own tokens, joined with those parts.
// Measured (kAttnShared, 256 rows a unit, 250 tiles, 8 heads; 88 CTAs of 22 or 23
// tiles, the other SMs left to the own tokens): 75 us with cold caches, 25600
// cycles before the first scores, 7400 for the first tile, 4400 for each other
// and 10000 for the parts' way out (135 KB a CTA).
//
// What a tile's rows do not all see is masked per element.  Tokens that no
// row of the CTA sees enter as zeros; a NaN code of V that only some rows see
// is taken out of the product and put into those rows at the end.

#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "ndq_attn.cuh"
#include "ndq_mma.cuh"

namespace ndq {
namespace {

constexpr int kPrConv = 4;                      // converter warps
constexpr int kPrConvWarp = 8;
constexpr int kPrMmaWarp = kPrConvWarp + kPrConv;
constexpr int kPrLoadWarp = kPrMmaWarp + 1;
constexpr int kPrRaw = 2;                       // staged tiles of codes: one of K, one of V
constexpr int kPrCst = 8;                       // tiles of group constants
constexpr int kPrThreads = 512;                 // four warpgroups; warps 14 and 15 idle
// Registers per thread after the split by warpgroup: launched with 128 each,
// 256 * 176 + 128 * 96 + 128 * 64 = 512 * 128.
constexpr int kPrLaunchRegs = 128;
constexpr int kPrTokens = 128;                  // tokens of a K / V tile
constexpr int kPrGroups = kPrTokens / 16;
constexpr float kStepCycles = 4400.0f, kFixedCycles = 30000.0f;  // (kAttnShared) of a tile, and before and after them
constexpr uint32_t kPrFault = 8u;               // bit of the device fault word

struct PrShared {
    uint64_t rawfull[2 * kPrRaw], rawfree[2 * kPrRaw];  // (the second half: see `dual`)
    uint64_t kfull[2], kfree[2], vfull[2], vfree[2];
    uint64_t sfull[2], pfull[2], odone[2];
    float4 cst[kPrCst][kPrGroups];  // per group: K's scale, log2 of V's scale, 1 / V's scale (0: far below others'), 0 for V of scale 0
    uint32_t gap[kPrCst];           // a block of the tile is missing, or V's scale far below others'
    uint32_t tmem;
    uint32_t fault;
    uint32_t nan;   // V has NaN codes in a tile that some rows see only part of
    uint32_t last;
    int64_t r, base;
    uint64_t sum[kPrThreads / 32];
    // the shared prefix (kAttnShared): the group, what of it this CTA takes, and what its rows see
    uint64_t tot[kPrThreads / 32];
    int64_t slot;
    uint32_t parts;
    int32_t lo_min, lo_max, hi_min, hi_max;
};

static_assert(sizeof(PrShared) <= 2048, "beside seven tiles of 32 KB");

template <int D>
struct PrSmem {
    static constexpr uint32_t kTile = kPrTokens * D * 2;  // K, V or Q tile
    static constexpr uint32_t kBytes = 1024 + 7 * kTile + sizeof(PrShared);  // 2 Q, 2 K, 2 V, 2 tiles of codes
};

// MN-major operand (N contiguous, 128-byte swizzle): 64 columns of N 128 rows
// apart in memory (`lead` bytes to the next 64), 8 rows of K 1024 bytes apart.
__device__ __forceinline__ uint64_t sdesc_mn(uint32_t saddr, uint32_t lead) {
    uint64_t d = static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(lead >> 4) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}

// D[tmem] (+)= A[tmem] B: A is binary16 pairs, 8 columns per k-step of 16.
__device__ __forceinline__ void mma_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t bd, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(tmem_d),
        "r"(tmem_a), "l"(bd), "r"(idesc), "r"(acc));
}

// 32 consecutive columns of this thread's lane.
__device__ __forceinline__ void tmem_ld32(uint32_t a, uint32_t* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(a));
}
__device__ __forceinline__ void tmem_ld16(uint32_t a, uint32_t* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(a));
}
__device__ __forceinline__ void tmem_st32(uint32_t a, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(v[0]),
        "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
        "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]),
        "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]),
        "r"(v[29]), "r"(v[30]), "r"(v[31]), "r"(a)
        : "memory");
}
// The wait for the loads before it names their registers, so that nothing that
// uses them can be moved ahead of it.
__device__ __forceinline__ void tmem_wait_ld32(uint32_t* v) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]), "+r"(v[8]),
                   "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]), "+r"(v[16]),
                   "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]), "+r"(v[24]),
                   "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]), "+r"(v[30]), "+r"(v[31])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tmem_wait_ld16(uint32_t* v) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]), "+r"(v[8]),
                   "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
                 :
                 : "memory");
}

// Barriers by number: every thread of the roles that meet there, and no other.
template <int ID, int THREADS>
__device__ __forceinline__ void meet() { asm volatile("barrier.cta.sync %0, %1;" ::"n"(ID), "n"(THREADS) : "memory"); }
constexpr int kMeetAll = 1, kMeetEnd = 2, kMeetRows = 3, kMeetQ = 4;

template <int N>
__device__ __forceinline__ void regs_more() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_less() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t pair_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t pair_add(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// A request's units of 256 rows (0: left to the other kernel).
__device__ __forceinline__ int64_t prompt_tiles(const AttnParams& p, int64_t r, int64_t& q0, int32_t& n, int32_t& pos0) {
    attn_request(p, r, q0, n, pos0);
    const int64_t rows = static_cast<int64_t>(n) * p.group;
    return rows < p.prompt_rows ? 0 : (rows + kPromptRows - 1) / kPromptRows;
}

// (kAttnShared) A group's rows in units of 256 and the tiles of its prefix.
struct SharedUnits {
    int64_t q0;      // its first query
    int64_t rows;    // of all its queries, for one cache head
    int64_t units;   // of all cache heads
    int32_t tiles;   // of 128 tokens
};
__device__ __forceinline__ SharedUnits shared_units(const PrefixParams& p, const Group& g) {
    SharedUnits x;
    int64_t a = g.begin, b = g.end;
    if (p.q_start) {
        a = p.q_start[g.begin];
        a = a < 0 ? 0 : (a > p.n_tokens ? p.n_tokens : a);
        b = p.q_start[g.end];
        b = b < a ? a : (b > p.n_tokens ? p.n_tokens : b);
    }
    x.q0 = a;
    x.rows = g.tokens > 0 ? (b - a) * p.group : 0;
    x.units = (x.rows + kPromptRows - 1) / kPromptRows * p.c.heads;
    x.tiles = (g.tokens + kPrTokens - 1) / kPrTokens;
    return x;
}
// The sum over the block's threads before this one, and of all of them.
__device__ __forceinline__ uint64_t block_scan(uint64_t mine, uint64_t* warps, uint64_t& total) {
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
    uint64_t incl = mine;
#pragma unroll
    for (uint32_t d = 1; d < 32; d <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += y;
    }
    if (lane == 31u) warps[warp] = incl;
    __syncthreads();
    uint64_t before = incl - mine;
    total = 0;
    for (uint32_t w = 0; w < kPrThreads / 32; ++w) {
        if (w < warp) before += warps[w];
        total += warps[w];
    }
    return before;
}

template <int D, bool E4M3, bool BF16, int MODE = kAttnAll>
__global__ void __launch_bounds__(kPrThreads, 1) k_attn_prompt(const __grid_constant__ typename AttnArgs<MODE>::type p) {
    using Sm = PrSmem<D>;
    constexpr uint32_t kTile = Sm::kTile;
    constexpr uint32_t kAtom = kPrTokens * 128;  // 64 head positions of a tile's 128 rows
    constexpr uint32_t kO = 256;                 // tensor-memory columns: S0, S1 at 0, 128; O0, O1 at 256, 256 + D
    extern __shared__ __align__(1024) uint8_t pr_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(pr_raw) + 1023u) & ~uintptr_t(1023));
    uint8_t* sK = base;
    uint8_t* sV = base + 2 * kTile;
    uint8_t* sRaw = base + 4 * kTile;
    uint8_t* sQ = base + 5 * kTile;
    PrShared& S = *reinterpret_cast<PrShared*>(base + 7 * kTile);
    const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31u;
    const int bl = p.c.bs_log2;
    attn_pdl_launch();  // (the kernel for the other requests may start)
    if (tid == 32 * kPrMmaWarp) {  // (beside the loads below)
        for (int i = 0; i < 2 * kPrRaw; ++i) {
            mbar_init(&S.rawfull[i], 1);
            mbar_init(&S.rawfree[i], kPrConv);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&S.vfull[i], kPrConv);
            mbar_init(&S.vfree[i], 1);
            mbar_init(&S.kfull[i], kPrConv);
            mbar_init(&S.kfree[i], 1);
            mbar_init(&S.sfull[i], 1);
            mbar_init(&S.odone[i], 1);
            mbar_init(&S.pfull[i], 4);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        S.fault = 0u;
        S.nan = 0u;
        S.last = 0u;
        S.lo_min = S.hi_min = INT32_MAX;
        S.lo_max = S.hi_max = 0;
    }

    // which unit: blockIdx.x counts (unit, split), units ordered by request,
    // then row tile (the last, longest, first), then head
    const uint64_t unit = blockIdx.x / static_cast<uint32_t>(p.splits);
    const uint32_t split = blockIdx.x % static_cast<uint32_t>(p.splits);
    int64_t slot_row = 0;  // (kAttnShared) this CTA's slot, and the parts of its unit
    uint32_t parts = 1, part = 0;
    // (kAttnShared) At most 128 rows: both row tiles are these rows, and take
    // the tokens' tiles by turns, each leaving a part.  (One row tile alone
    // waits for its own chain of products and softmax.)  There is one Q, and the
    // other's memory holds a second pair of tiles of codes: one pair was
    // brought, widened and given back in 3000 cycles, more than half of what the
    // two row tiles then take.
    bool dual = false;
    if constexpr (MODE == kAttnShared) {
        // Every CTA counts the groups' units and tiles, from these how many
        // tiles a CTA is to take, and then finds its unit and part.
        // (A unit of 128 rows or fewer goes through its tiles two at a time, see
        // `dual`: they count half.)
        uint64_t chunk = 1, sms = static_cast<uint64_t>(p.sms);
        auto steps_of = [&](const SharedUnits& x) { return static_cast<uint32_t>(x.rows <= kPromptRows / 2 ? (x.tiles + 1) / 2 : x.tiles); };
        auto parts_of = [&](const SharedUnits& x) {
            const uint32_t steps = steps_of(x);
            const uint64_t n = chunk >= steps ? 1 : (steps + static_cast<uint32_t>(chunk) - 1) / static_cast<uint32_t>(chunk);
            return static_cast<int64_t>(n > kPrefixMaxParts ? kPrefixMaxParts : n);
        };
        auto set_chunk = [&](uint64_t units, uint64_t work) {
            // CTAs beyond one per unit number at most work / chunk, no more than the SMs
            const uint64_t spare = units + sms / 4 < sms ? sms - units : (sms + 3) / 4;
            chunk = (work >> 32) != 0 ? (work + spare - 1) / spare : static_cast<uint32_t>(work + spare - 1) / static_cast<uint32_t>(spare);
            chunk = chunk < kPrefixMinTiles ? kPrefixMinTiles : chunk;
        };
        auto ctas_of = [&](const SharedUnits& x) { return static_cast<uint64_t>(x.units * parts_of(x)); };
        auto slots_of = [&](const SharedUnits& x) {  // (few rows leave two rows each, see `dual`)
            const int64_t last = x.rows % kPromptRows;
            return static_cast<uint64_t>((x.rows + (last <= kPromptRows / 2 ? last : 0)) * p.c.heads * parts_of(x));
        };
        auto mine = [&](int64_t g, uint64_t c, uint64_t n, int64_t parts_here) {
            S.r = g;
            S.base = static_cast<int64_t>(blockIdx.x - c);
            S.slot = static_cast<int64_t>(n);
            S.parts = static_cast<uint32_t>(parts_here);
        };
        if (p.n_groups <= 32) {  // every warp for itself
            // All requests' tokens but the shared ones, for which the kernel after
            // this one reads the cache meanwhile, on the SMs that are left to it.
            uint64_t own = 0;
            for (int64_t r = tid; r < p.n_req; r += kPrThreads) own += static_cast<uint32_t>(p.kv_len[r] > 0 ? p.kv_len[r] : 0);
            SharedUnits x{};
            Group g{};
            if (lane < p.n_groups) {
                g = attn_group(p, lane);
                x = shared_units(p, g);
            }
            uint64_t units = static_cast<uint64_t>(x.units), work = units * steps_of(x);
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) own += __shfl_xor_sync(0xffffffffu, own, d);
            if (lane == 0) S.tot[warp] = own;
            __syncthreads();
            own = lane < kPrThreads / 32 ? S.tot[lane] : 0;
            uint64_t common = lane < p.n_groups ? static_cast<uint64_t>(g.end - g.begin) * static_cast<uint32_t>(g.tokens) : 0;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) {
                own += __shfl_xor_sync(0xffffffffu, own, d);
                common += __shfl_xor_sync(0xffffffffu, common, d);
            }
            own = own > common ? own - common : 0;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                if (d >= p.n_groups) break;
                units += __shfl_xor_sync(0xffffffffu, units, d);
                work += __shfl_xor_sync(0xffffffffu, work, d);
            }
            units = __shfl_sync(0xffffffffu, units, 0);
            work = __shfl_sync(0xffffffffu, work, 0);
            {
                // SMs in proportion: kStepCycles a tile and, beside it, D / 10 a
                // token and row tile of the own ones (20 bytes a cycle and SM)
                const float row_tiles = fmaxf(1.0f, static_cast<float>(p.n_tokens * p.group) / static_cast<float>(p.n_req * kAttnRows));
                const float here = kFixedCycles * static_cast<float>(p.sms) * 0.5f + static_cast<float>(work) * kStepCycles;
                const float there = static_cast<float>(own) * static_cast<float>(p.c.heads) * row_tiles * (D / 10.0f);
                const uint32_t want = static_cast<uint32_t>(static_cast<float>(p.sms) * here / (here + there)) + 1u;
                sms = want < p.sms / 2u ? p.sms / 2u : (want < static_cast<uint32_t>(p.sms) ? want : static_cast<uint32_t>(p.sms));
            }
            set_chunk(units, work);
            // the smallest chunk whose CTAs still are one wave
            if (p.n_groups == 1) {
                const uint32_t ctas = units < sms ? static_cast<uint32_t>(sms) / static_cast<uint32_t>(units > 0 ? units : 1) : 1u, steps = __shfl_sync(0xffffffffu, steps_of(x), 0);
                chunk = (steps + ctas - 1) / ctas;
                chunk = chunk < kPrefixMinTiles ? kPrefixMinTiles : chunk;
            } else if (units < sms && (work >> 31) == 0) {
                uint32_t lo = static_cast<uint32_t>(work) / static_cast<uint32_t>(sms), hi = static_cast<uint32_t>(chunk);  // lo: too small, hi: will do
                lo = lo < kPrefixMinTiles - 1 ? static_cast<uint32_t>(kPrefixMinTiles) - 1 : lo;
                while (lo + 1 < hi) {
                    const uint32_t mid = (lo + hi) >> 1;
                    chunk = mid;
                    const uint64_t c = x.units > 0 ? ctas_of(x) : 0;
                    if (__reduce_add_sync(0xffffffffu, static_cast<uint32_t>(c < sms ? c : sms + 1)) <= sms) hi = mid;
                    else lo = mid;
                }
                chunk = hi;
            }
            const uint64_t ctas = x.units > 0 ? ctas_of(x) : 0, rows = x.units > 0 ? slots_of(x) : 0;
            uint64_t ci = ctas, ri = rows;
#pragma unroll
            for (uint32_t d = 1; d < 32; d <<= 1) {
                if (d >= p.n_groups) break;
                const uint64_t a = __shfl_up_sync(0xffffffffu, ci, d), b = __shfl_up_sync(0xffffffffu, ri, d);
                if (lane >= d) {
                    ci += a;
                    ri += b;
                }
            }
            const uint32_t here = __ballot_sync(0xffffffffu, blockIdx.x < ci && blockIdx.x >= ci - ctas);
            const uint64_t all_rows = __shfl_sync(0xffffffffu, ri, static_cast<int>(p.n_groups) - 1);
            if (here == 0u || all_rows > static_cast<uint64_t>(p.slot_rows)) return;  // (the latter never)
            if (warp == 0 && lane == static_cast<uint32_t>(__ffs(here)) - 1u) mine(lane, ci - ctas, ri - rows, parts_of(x));
        } else {
            const int64_t per = (p.n_groups + kPrThreads - 1) / kPrThreads;
            uint64_t units = 0, work = 0, all_units = 0, all_work = 0;
            for (int64_t i = 0; i < per; ++i) {
                const int64_t g = tid * per + i;
                if (g < p.n_groups) {
                    const SharedUnits x = shared_units(p, attn_group(p, g));
                    units += static_cast<uint64_t>(x.units);
                    work += static_cast<uint64_t>(x.units) * steps_of(x);
                }
            }
            block_scan(units, S.sum, all_units);
            block_scan(work, S.tot, all_work);
            set_chunk(all_units, all_work);
            uint64_t ctas = 0, rows = 0, all_ctas = 0, all_rows = 0;
            for (int64_t i = 0; i < per; ++i) {
                const int64_t g = tid * per + i;
                if (g < p.n_groups) {
                    const SharedUnits x = shared_units(p, attn_group(p, g));
                    ctas += ctas_of(x);
                    rows += slots_of(x);
                }
            }
            __syncthreads();  // (the sums above are read)
            const uint64_t ctas_before = block_scan(ctas, S.sum, all_ctas), rows_before = block_scan(rows, S.tot, all_rows);
            if (blockIdx.x >= all_ctas || all_rows > static_cast<uint64_t>(p.slot_rows)) return;
            if (ctas_before <= blockIdx.x && blockIdx.x < ctas_before + ctas) {
                uint64_t c = ctas_before, n = rows_before;
                int64_t g = tid * per;
                SharedUnits x = shared_units(p, attn_group(p, g));
                while (blockIdx.x >= c + ctas_of(x)) {
                    c += ctas_of(x);
                    n += slots_of(x);
                    x = shared_units(p, attn_group(p, ++g));
                }
                mine(g, c, n, parts_of(x));
            }
        }
    } else {
        const int64_t per = (p.n_req + kPrThreads - 1) / kPrThreads;
        int64_t q0;
        int32_t n, pos0;
        uint64_t mine = 0;
        for (int64_t i = 0; i < per; ++i) {
            const int64_t r = tid * per + i;
            if (r < p.n_req) mine += static_cast<uint64_t>(prompt_tiles(p, r, q0, n, pos0)) * p.c.heads;
        }
        uint64_t incl = mine;
#pragma unroll
        for (uint32_t d = 1; d < 32; d <<= 1) {
            const uint64_t y = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += y;
        }
        if (lane == 31u) S.sum[warp] = incl;
        __syncthreads();
        uint64_t total = 0, before = incl - mine;
        for (uint32_t w = 0; w < kPrThreads / 32; ++w) {
            if (w < warp) before += S.sum[w];
            total += S.sum[w];
        }
        if (unit >= total) {
            if (MODE == kAttnOwn) attn_pdl_wait();
            return;
        }
        if (before <= unit && unit < before + mine) {
            S.r = tid * per;
            S.base = static_cast<int64_t>(before);
        }
    }
    if (warp == kPrMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&S.tmem)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    __syncthreads();
    int64_t r = S.r, q0 = 0;
    int32_t n = 0, pos0 = 0;  // queries and the position of the first
    int32_t h, row0, nrows;
    int32_t own = 0;         // the first token that is not of a shared prefix, or (kAttnShared) the prefix's tokens
    int64_t group_end = 0;   // (kAttnShared) the end of the group's requests
    if constexpr (MODE == kAttnShared) {
        // r: the group's first request, q0 and n: the queries of all of them
        const Group g = attn_group(p, S.r);
        const SharedUnits x = shared_units(p, g);
        r = g.begin;
        group_end = g.end;
        q0 = x.q0;
        n = static_cast<int32_t>(x.rows / p.group);
        own = g.tokens;
        parts = S.parts;
        const int64_t u = S.base / parts;
        part = static_cast<uint32_t>(S.base - u * parts);
        const int64_t tile = u / p.c.heads;
        h = static_cast<int32_t>(u - tile * p.c.heads);
        row0 = static_cast<int32_t>(tile) * kPromptRows;
        const int64_t rows_left = x.rows - row0;
        nrows = static_cast<int32_t>(rows_left < kPromptRows ? rows_left : kPromptRows);
        dual = nrows <= kPromptRows / 2;
        const int64_t left = dual ? 2 * nrows : nrows;  // rows that a CTA of this unit leaves
        slot_row = S.slot + (tile * kPromptRows * p.c.heads + h * left) * parts + part * left;
    } else {
        uint64_t left = unit - static_cast<uint64_t>(S.base);
        int64_t tiles = prompt_tiles(p, r, q0, n, pos0);
        while (left >= static_cast<uint64_t>(tiles) * p.c.heads) {
            left -= static_cast<uint64_t>(tiles) * p.c.heads;
            ++r;
            tiles = prompt_tiles(p, r, q0, n, pos0);
        }
        h = static_cast<int32_t>(left % p.c.heads);
        row0 = static_cast<int32_t>(tiles - 1 - left / p.c.heads) * kPromptRows;
        const int32_t rows_left = n * p.group - row0;
        nrows = rows_left < kPromptRows ? rows_left : kPromptRows;
        if constexpr (MODE == kAttnOwn) own = shared_tokens(p, r);
    }
    const int32_t nact = nrows > 128 || dual ? 2 : 1;  // row tiles in use
    // tokens that some row / every row of the CTA sees
    const int32_t first_pos = pos0 + row0 / p.group, last_pos = pos0 + (row0 + nrows - 1) / p.group;
    const int32_t most = table_tokens(p);
    int32_t any_hi = last_pos < most ? last_pos + 1 : most, cta_hi = first_pos + 1;
    int32_t any_lo = p.window > 0 && first_pos + 1 > p.window ? first_pos + 1 - p.window : 0;
    int32_t cta_lo = p.window > 0 ? last_pos + 1 - p.window : 0;
    if constexpr (MODE == kAttnOwn) {
        any_lo = any_lo > own ? any_lo : own;
        cta_lo = cta_lo > own ? cta_lo : own;
    }
    int32_t nt = 0, tok0 = 0;  // this CTA's tiles, and the first token of them
    if constexpr (MODE != kAttnShared) {
        const int32_t lo16 = any_lo & ~15;
        const int32_t all_tiles = any_hi > lo16 ? (any_hi - lo16 + kPrTokens - 1) / kPrTokens : 0;
        const int32_t j0 = all_tiles * static_cast<int32_t>(split) / p.splits;
        nt = all_tiles * static_cast<int32_t>(split + 1) / p.splits - j0;
        tok0 = lo16 + j0 * kPrTokens;
    } else {  // (with a window, see below)
        const int32_t tiles = (own + kPrTokens - 1) / kPrTokens;
        const int32_t j0 = tiles * static_cast<int32_t>(part) / static_cast<int32_t>(parts);
        nt = tiles * static_cast<int32_t>(part + 1) / static_cast<int32_t>(parts) - j0;
        tok0 = j0 * kPrTokens;
        any_lo = 0;
        any_hi = own;
    }

    // Q: one row per softmax thread, scaled, as a 128-byte-swizzled operand
    const uint32_t wg = warp >> 2, wrow = tid & 127u;
    float frow = 0.0f;
    int32_t see_lo = 0, see_hi = 0;
    int32_t at = 0;  // index of the row's output (n_tokens * q_heads is below 2^31)
    bool has_row = false;
    // without a window the loader has all that it needs: it goes ahead
    const bool ahead = MODE == kAttnShared && p.window == 0;
    if (MODE == kAttnShared && warp < kPrConvWarp) {
        // The rows' loads first, by D / 8 lanes a row (a thread that read its
        // own row would fetch every line by sixteenths); whose they are and
        // where they sit meanwhile.
        constexpr int LPR = D / 8, RPI = 32 / LPR;  // lanes per row, rows per load
        const int32_t i = static_cast<int32_t>(dual ? wrow : wg * 128u + wrow);
        const int32_t mine = row0 + (i < nrows ? i : 0);
        const int32_t qi = mine / p.group, qh = h * p.group + mine % p.group;
        at = static_cast<int32_t>((q0 + qi) * p.q_heads) + qh;
        const int64_t off = (q0 + qi) * p.q_stride + static_cast<int64_t>(qh) * D;
        uint4 x[32 / RPI];
#pragma unroll
        for (int c = 0; c < 32 / RPI; ++c) {
            const int64_t o = __shfl_sync(0xffffffffu, off, c * RPI + static_cast<int>(lane) / LPR);
            x[c] = *reinterpret_cast<const uint4*>(p.q + o + (lane % LPR) * 8);
        }
        has_row = i < nrows;
        int32_t pos = 0;
        if (has_row) {
            const int64_t t = q0 + qi;
            int64_t rq = t, a0 = t;
            int32_t an = 1;
            if (p.q_start) {
                // requests of one length, mostly; else the last that starts at t or before
                const int32_t reqs = static_cast<int32_t>(group_end - r);
                rq = r + qi / ((n + reqs - 1) / reqs);
                if (!(p.q_start[rq] <= t && t < p.q_start[rq + 1])) {
                    int64_t a = r, b = group_end;
                    while (b - a > 1) {
                        const int64_t m = (a + b) >> 1;
                        if (p.q_start[m] <= t) a = m;
                        else b = m;
                    }
                    rq = a;
                }
            }
            attn_request(p, rq, a0, an, pos);
            has_row = a0 <= t && t < a0 + an;
            pos += static_cast<int32_t>(t - a0);
        }
        see_hi = has_row && pos >= 0 ? (pos < most ? pos + 1 : most) : 0;
        see_hi = see_hi < own ? see_hi : own;
        see_lo = p.window > 0 && pos + 1 > p.window ? pos + 1 - p.window : 0;
        const uint32_t rows_here = __ballot_sync(0xffffffffu, has_row);
        uint8_t* dst = sQ + wg * kTile;
        const uint32_t piece = lane % LPR;
#pragma unroll
        for (int c = 0; c < 32 / RPI; ++c) {
            const uint32_t rl = c * RPI + lane / LPR;  // the row among the warp's 32
            const bool in = (rows_here >> rl & 1u) != 0u;
            const uint32_t ww[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
            float f[8], amax = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                widen2<BF16>(in ? ww[e] : 0u, f[2 * e], f[2 * e + 1]);
                amax = max3(amax, fabsf(f[2 * e]), fabsf(f[2 * e + 1]));
            }
#pragma unroll
            for (int e = 1; e < LPR; e <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, e));
            float up, down;
            row_scale(amax, up, down);
            if (p.scale_log2 < 0.0f) {  // (a negative scale goes into Q: K's scale then keeps the order of scores)
                up = -up;
                down = -down;
            }
            // (the row's owner, lane rl, is served by the lanes of its row)
            const float fr = __shfl_sync(0xffffffffu, down * p.scale_log2, (static_cast<int>(lane) % RPI) * LPR);
            if (lane / RPI == static_cast<uint32_t>(c)) frow = fr;
            if (!(dual && wg == 1))
                *reinterpret_cast<uint4*>(dst + (piece >> 3) * kAtom + sw128(32u * (warp & 3u) + rl, piece & 7u)) =
                make_uint4(pack_half2(f[0] * up, f[1] * up), pack_half2(f[2] * up, f[3] * up), pack_half2(f[4] * up, f[5] * up),
                           pack_half2(f[6] * up, f[7] * up));
        }
        const int32_t l0 = __reduce_min_sync(0xffffffffu, has_row ? see_lo : INT32_MAX), l1 = __reduce_max_sync(0xffffffffu, has_row ? see_lo : 0);
        const int32_t h0 = __reduce_min_sync(0xffffffffu, has_row ? see_hi : INT32_MAX), h1 = __reduce_max_sync(0xffffffffu, see_hi);
        if (lane == 0) {
            atomicMin(&S.lo_min, l0);
            atomicMax(&S.lo_max, l1);
            atomicMin(&S.hi_min, h0);
            atomicMax(&S.hi_max, h1);
        }
        fence_proxy_async_smem();
    }
    if (MODE != kAttnShared && warp < kPrConvWarp) {
        const int32_t i = static_cast<int32_t>(wg * 128u + wrow);
        has_row = i < nrows;
        const int32_t qi = (row0 + (has_row ? i : 0)) / p.group, qh = h * p.group + (row0 + (has_row ? i : 0)) % p.group;
        at = static_cast<int32_t>((q0 + qi) * p.q_heads) + qh;
        const uint4* src = reinterpret_cast<const uint4*>(p.q + (q0 + qi) * p.q_stride + static_cast<int64_t>(qh) * D);
        float amax = 0.0f;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
            const uint4 w = has_row ? src[c] : make_uint4(0u, 0u, 0u, 0u);
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float a, b;
                widen2<BF16>(ww[e], a, b);
                amax = max3(amax, fabsf(a), fabsf(b));
            }
        }
        float up, down;
        row_scale(amax, up, down);
        if (p.scale_log2 < 0.0f) {  // (a negative scale goes into Q: K's scale then keeps the order of scores)
            up = -up;
            down = -down;
        }
        frow = down * p.scale_log2;
        uint8_t* dst = sQ + wg * kTile;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
            const uint4 w = has_row ? src[c] : make_uint4(0u, 0u, 0u, 0u);
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float a, b;
                widen2<BF16>(ww[e], a, b);
                o[e] = pack_half2(a * up, b * up);
            }
            *reinterpret_cast<uint4*>(dst + (c >> 3) * kAtom + sw128(wrow, c & 7)) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        const int32_t pos = pos0 + qi;
        see_hi = has_row && pos >= 0 ? (pos < most ? pos + 1 : most) : 0;
        see_lo = p.window > 0 && pos + 1 > p.window ? pos + 1 - p.window : 0;
        if constexpr (MODE == kAttnOwn) see_lo = see_lo > own ? see_lo : own;
        fence_proxy_async_smem();
    }
    tc_fence_before();
    if (!ahead) __syncthreads();
    else if (warp <= kPrMmaWarp) meet<kMeetQ, (kPrMmaWarp + 1) * 32>();
    tc_fence_after();
    const uint32_t tmem = S.tmem;
    if constexpr (MODE == kAttnShared) {
        // the rows are of many requests: what they see is known now (the
        // loader that went ahead brings the tiles of all of the prefix)
        if (!ahead || warp <= kPrMmaWarp) {
            any_lo = S.lo_min;
            cta_lo = S.lo_max;
            any_hi = S.hi_max;
            cta_hi = S.hi_min;
        }
        if (!ahead) {  // tiles before and behind the windows are left out
            int32_t j0 = tok0 / kPrTokens, j1 = j0 + nt;
            const int32_t first = any_lo / kPrTokens, end = (any_hi + kPrTokens - 1) / kPrTokens;
            j0 = j0 > first ? j0 : first;
            j1 = j1 < end ? j1 : end;
            nt = any_hi > any_lo && j1 > j0 ? j1 - j0 : 0;
            tok0 = j0 * kPrTokens;
        }
    }
    float mx = -INFINITY, sum = 0.0f;
    // the codes of tile j, K (0) or V (1): their barrier, how often it has come round, and their place
    const int32_t raws = MODE == kAttnShared && dual ? 2 : 1;
    auto raw_bar = [&](int32_t j, uint32_t half) { return half + 2u * static_cast<uint32_t>(raws == 2 ? j & 1 : 0); };
    auto raw_turn = [&](int32_t j) { return raws == 2 ? j >> 1 : j; };
    auto raw_at = [&](int32_t j, uint32_t half) { return (raws == 2 && (j & 1) ? sQ + kTile : sRaw) + half * (kTile / 2); };

    if (warp >= kPrConvWarp && warp < kPrMmaWarp) {
        // ---- converters: groups cw and cw + 4 of every tile
        regs_less<96>();
        constexpr int LPR = D / 8, RPI = 32 / LPR, ITS = 16 / RPI;  // lanes per row, rows per load, loads per group
        const uint32_t cw = warp - kPrConvWarp;
        const uint32_t lrow = lane / LPR, piece = lane % LPR;
        bool ok = true;
        // one tile of codes to an operand; rows outside what the CTA sees, and groups of weight 0, as zeros
        auto convert = [&](const uint8_t* raw, uint8_t* tile, int32_t j, bool is_v) {
            const int32_t tb = tok0 + j * kPrTokens;
            const bool part = tb + kPrTokens > cta_hi || tb < cta_lo;  // some rows see only part of this tile
            uint2 x[2][ITS];  // (all loads before the first store: the compiler must assume that they alias)
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int i = 0; i < ITS; ++i)
                    x[q][i] = *reinterpret_cast<const uint2*>(raw + ((cw + 4 * q) * 16 + i * RPI + lrow) * D + piece * 8);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const float4 c = S.cst[j % kPrCst][cw + 4 * q];
                if (c.y == -INFINITY) {
#pragma unroll
                    for (int i = 0; i < ITS; ++i) x[q][i] = make_uint2(0u, 0u);
                } else if (is_v && c.w == 0.0f) {
#pragma unroll
                    for (int i = 0; i < ITS; ++i) x[q][i] = make_uint2(nan_codes<E4M3>(x[q][i].x), nan_codes<E4M3>(x[q][i].y));
                }
            }
            if (part) {
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int i = 0; i < ITS; ++i) {
                        const int32_t tk = tb + static_cast<int32_t>((cw + 4 * q) * 16 + i * RPI + lrow);
                        if (tk >= any_hi || tk < any_lo) x[q][i] = make_uint2(0u, 0u);
                        if (E4M3 && is_v) {  // NaN codes that only some rows see: see the end of the kernel
                            const uint32_t nx = nan_bytes(x[q][i].x), ny = nan_bytes(x[q][i].y);
                            if ((nx | ny) != 0u) S.nan = 1u;
                            x[q][i].x &= ~((nx >> 7) * 0xffu);
                            x[q][i].y &= ~((ny >> 7) * 0xffu);
                        }
                    }
            }
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int i = 0; i < ITS; ++i) {
                    uint4 o;
                    widen4<E4M3>(x[q][i].x, o.x, o.y);
                    widen4<E4M3>(x[q][i].y, o.z, o.w);
                    *reinterpret_cast<uint4*>(tile + (piece >> 3) * kAtom + sw128((cw + 4 * q) * 16 + i * RPI + lrow, piece & 7u)) = o;
                }
            fence_proxy_async_smem();
            __syncwarp();
        };
        auto wait = [&](uint64_t* b, int32_t parity) { return __all_sync(0xffffffffu, mbar_wait_bounded(b, static_cast<uint32_t>(parity & 1), p.waits.limit_ns)); };
        for (int32_t j = 0; j < nt; ++j) {
            const uint32_t st = static_cast<uint32_t>(j & 1);
            ok = wait(&S.rawfull[raw_bar(j, 0)], raw_turn(j)) && (j < 2 || wait(&S.kfree[st], (j >> 1) - 1));
            if (!ok) break;
            convert(raw_at(j, 0), sK + st * kTile, j, false);
            if (lane == 0) {
                mbar_arrive(&S.kfull[st]);
                mbar_arrive(&S.rawfree[raw_bar(j, 0)]);
            }
            ok = wait(&S.rawfull[raw_bar(j, 1)], raw_turn(j)) && (j < 2 || wait(&S.vfree[st], (j >> 1) - 1));
            if (!ok) break;
            convert(raw_at(j, 1), sV + st * kTile, j, true);
            if (lane == 0) {
                mbar_arrive(&S.vfull[st]);
                mbar_arrive(&S.rawfree[raw_bar(j, 1)]);
            }
        }
        if (!ok && lane == 0) atomicOr(&S.fault, 1u);
        tc_fence_before();
        meet<kMeetAll, kPrThreads>();
        return;
    }
    if (warp >= kPrMmaWarp) {
        regs_less<64>();
        if (warp == kPrLoadWarp) {
            // ---- loader: lane 8 i + g holds group g of tile 4 b + i
            const int32_t* table = p.table + r * p.width;
            const uint32_t gl = lane & 7u;
            auto ids_of = [&](int32_t b) -> int32_t {
                const int32_t j = 4 * b + static_cast<int32_t>(lane >> 3);
                const int32_t tk = tok0 + j * kPrTokens + static_cast<int32_t>(gl) * 16;
                if (j >= nt || tk >= any_hi) return -1;
                const int32_t id = table[tk >> bl];
                return id >= 0 && id < p.c.num_blocks ? id : -1;
            };
            bool ok = true;
            int32_t ids = -1, ids_next = ids_of(0), issued = 0;
            int32_t v_top = kNoScale;  // the largest exponent of V's scales so far
            uint64_t off = 0;
            float4 c = make_float4(0.0f, -INFINITY, 0.0f, 0.0f);
            for (int32_t j = 0; j < nt && ok; ++j) {
                if ((j & 3) == 0) {
                    ids = ids_next;
                    ids_next = ids_of((j >> 2) + 1);
                    c = make_float4(0.0f, -INFINITY, 0.0f, 0.0f);  // a missing block: weight 0
                    float vs = 0.0f;
                    if (ids >= 0) {
                        const uint64_t u = static_cast<uint64_t>(ids) * p.c.heads + static_cast<uint32_t>(h);
                        const int32_t tk = tok0 + (j + static_cast<int32_t>(lane >> 3)) * kPrTokens + static_cast<int32_t>(gl) * 16;
                        off = ((u << bl) + (static_cast<uint32_t>(tk) & ((1u << bl) - 1u))) * D;
                        vs = p.c.vs[u];
                        float lg, inv;
                        value_scale(vs, lg, inv);
                        c = make_float4(p.c.ks[u], lg, inv, vs == 0.0f ? 0.0f : 1.0f);
                    }
                    const int32_t e = __reduce_max_sync(0xffffffffu, scale_exponent(vs));
                    v_top = e > v_top ? e : v_top;
                    if (c.y < static_cast<float>(v_top) - kScaleSpread) c.z = 0.0f;  // far below: see kScaleSpread
                }
                const bool mine = static_cast<int32_t>(lane >> 3) == (j & 3);
                const uint32_t n16 = __popc(__ballot_sync(0xffffffffu, mine && ids >= 0));
                const bool far = __any_sync(0xffffffffu, mine && ids >= 0 && c.z == 0.0f);
                for (int32_t half = 0; half < 2; ++half) {  // K, V
                    const uint32_t rs = raw_bar(j, static_cast<uint32_t>(half));
                    if (j >= raws) ok = __all_sync(0xffffffffu, mbar_wait_bounded(&S.rawfree[rs], static_cast<uint32_t>((raw_turn(j) - 1) & 1), p.waits.limit_ns));
                    if (!ok) break;
                    if (half == 0 && mine) S.cst[j % kPrCst][gl] = c;
                    if (half == 0 && lane == 0) S.gap[j % kPrCst] = n16 < kPrGroups || far ? 1u : 0u;
                    __syncwarp();
                    if (lane == 0) mbar_arrive_expect_tx(&S.rawfull[rs], n16 * 16u * D + p.waits.beyond);
                    __syncwarp();
                    if (mine && ids >= 0)
                        bulk_load(raw_at(j, static_cast<uint32_t>(half)) + gl * 16u * D, (half ? p.c.v : p.c.k) + off, 16u * D, &S.rawfull[rs]);
                    ++issued;
                }
            }
            if (!ok) {  // its own copies in flight land before the block ends
                if (lane == 0) atomicOr(&S.fault, 1u);
                for (int32_t i = issued > kPrRaw * raws ? issued - kPrRaw * raws : 0; i < issued; ++i)
                    mbar_wait_bounded(&S.rawfull[raw_bar(i >> 1, static_cast<uint32_t>(i & 1))], static_cast<uint32_t>(raw_turn(i >> 1) & 1), p.waits.limit_ns);
            }
            meet<kMeetAll, kPrThreads>();
            return;
        }
        if (warp != kPrMmaWarp) {  // (only there to make the warpgroup whole)
            meet<kMeetAll, kPrThreads>();
            return;
        }
        // ---- MMA issue
        constexpr uint32_t kIdQ = (1u << 4) | ((kPrTokens >> 3) << 17) | ((128u >> 4) << 24);
        constexpr uint32_t kIdP = (1u << 4) | (1u << 16) | ((static_cast<uint32_t>(D) >> 3) << 17) | ((128u >> 4) << 24);
        // descriptors of the first stages: the address field counts 16 bytes, and
        // no operand crosses its 2^14 (shared memory ends at 2^18 bytes)
        const uint64_t dq = mma_sdesc(smem_addr(sQ)), dk = mma_sdesc(smem_addr(sK)), dv = sdesc_mn(smem_addr(sV), kAtom);
        bool ok = true;
        int32_t issued[2] = {0, 0};  // PV products of each row tile
        int32_t scored[2] = {0, 0};  // score products of each row tile
        auto wait = [&](uint64_t* b, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait_bounded(b, parity, p.waits.limit_ns)); };
        auto scores = [&](int32_t i, int32_t j) {  // S_i = Q_i K_j^T
            const uint64_t a0 = dq + (MODE == kAttnShared && dual ? 0u : static_cast<uint32_t>(i) * (kTile >> 4)), b0 = dk + static_cast<uint32_t>(j & 1) * (kTile >> 4);
            if (elect_one()) {
#pragma unroll
                for (uint32_t s = 0; s < D / 16; ++s)
                    mma_bf16(tmem + 128u * i, a0 + (((s >> 2) * kAtom + (s & 3u) * 32u) >> 4),
                             b0 + (((s >> 2) * kAtom + (s & 3u) * 32u) >> 4), kIdQ, s > 0 ? 1u : 0u);
                mma_commit(&S.sfull[i]);
                if (i == nact - 1 || dual) mma_commit(&S.kfree[j & 1]);
            }
            __syncwarp();
            ++scored[i];
        };
        auto values = [&](int32_t i, int32_t j) {  // O_i += P_i V_j
            const uint64_t b0 = dv + static_cast<uint32_t>(j & 1) * (kTile >> 4);
            const bool more = issued[i] > 0;
            if (elect_one()) {
#pragma unroll
                for (uint32_t s = 0; s < kPrTokens / 16; ++s)
                    mma_ts(tmem + kO + D * i, tmem + 128u * i + 8u * s, b0 + s * (2048u >> 4), kIdP, more || s > 0 ? 1u : 0u);
                mma_commit(&S.odone[i]);
                if (i == nact - 1 || dual) mma_commit(&S.vfree[j & 1]);
            }
            __syncwarp();
            ++issued[i];
        };
        if (MODE == kAttnShared && dual) {  // tile j is row tile j & 1's, in the stage j & 1 of K and V
            for (int32_t j = 0; j < 2 && j < nt && ok; ++j) {
                ok = wait(&S.kfull[j], 0u);
                if (!ok) break;
                tc_fence_after();
                scores(j, j);
            }
            for (int32_t j = 0; j < nt && ok; ++j) {
                const uint32_t turn = static_cast<uint32_t>((j >> 1) & 1);
                ok = wait(&S.vfull[j & 1], turn) && wait(&S.pfull[j & 1], turn);
                if (!ok) break;
                tc_fence_after();
                values(j & 1, j);
                if (j + 2 < nt) {
                    ok = wait(&S.kfull[j & 1], turn ^ 1u);
                    if (!ok) break;
                    tc_fence_after();
                    scores(j & 1, j + 2);
                }
            }
        } else if (nt > 0) {
            ok = wait(&S.kfull[0], 0u);
            if (ok) {
                tc_fence_after();
                for (int32_t i = 0; i < nact; ++i) scores(i, 0);
            }
        }
        for (int32_t j = 0; j < nt && ok && !dual; ++j) {
            ok = wait(&S.vfull[j & 1], static_cast<uint32_t>((j >> 1) & 1));
            for (int32_t i = 0; i < nact && ok; ++i) {
                ok = wait(&S.pfull[i], static_cast<uint32_t>(j & 1));
                if (!ok) break;
                tc_fence_after();
                values(i, j);
                if (j + 1 < nt) {
                    if (i == 0) {
                        ok = wait(&S.kfull[(j + 1) & 1], static_cast<uint32_t>(((j + 1) >> 1) & 1));
                        if (!ok) break;
                        tc_fence_after();
                    }
                    scores(i, j + 1);
                }
            }
        }
        // no MMA may still run when tensor memory is given back
        for (int32_t i = 0; i < 2; ++i) {
            if (scored[i] > 0) ok = wait(&S.sfull[i], static_cast<uint32_t>((scored[i] - 1) & 1)) && ok;
            if (issued[i] > 0) ok = wait(&S.odone[i], static_cast<uint32_t>((issued[i] - 1) & 1)) && ok;
        }
        if (!ok && lane == 0) {
            atomicOr(&S.fault, 1u);
            atomicOr(p.fault, kPrFault);
        }
        tc_fence_before();
        meet<kMeetAll, kPrThreads>();
        meet<kMeetEnd, 256 + 32>();  // the rows are read out of tensor memory
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
        return;
    }
    regs_more<176>();
    if (static_cast<int32_t>(wg) < nact) {
        // ---- softmax: one row per thread
        const uint32_t tS = tmem + 128u * wg + ((32u * (warp & 3u)) << 16), tO = tmem + kO + D * wg + ((32u * (warp & 3u)) << 16);
        const int32_t wrow0 = row0 + 128 * static_cast<int32_t>(wg);
        const int32_t wrows = nrows - 128 * static_cast<int32_t>(wg) < 128 ? nrows - 128 * static_cast<int32_t>(wg) : 128;
        int32_t all_hi = pos0 + wrow0 / p.group + 1;
        int32_t all_lo = p.window > 0 ? pos0 + (wrow0 + wrows - 1) / p.group + 1 - p.window : 0;
        if constexpr (MODE == kAttnOwn) all_lo = all_lo > own ? all_lo : own;
        if constexpr (MODE == kAttnShared) {
            all_hi = cta_hi;
            all_lo = cta_lo;
        }
        float ms = 0.0f;
        bool ok = true;
        const int32_t turns = dual ? (nt + 1 - static_cast<int32_t>(wg)) >> 1 : nt;  // tiles of this row tile
        uint32_t w[kPrTokens / 2];  // the row's weights of the tile, in pairs
        // The weights relative to ms (and less), their sum and the largest exponent.
        auto weigh = [&](auto mask, auto again, bool read, float less, const float4* cst, int32_t tb, float& ts, float& top) {
            constexpr bool kMasked = decltype(mask)::value, kAgain = decltype(again)::value;
            uint32_t v[2][16];
            ts = 0.0f;
            float tops[2] = {-INFINITY, -INFINITY};
            if (MODE == kAttnAll || read) tmem_ld16(tS, v[0]);
#pragma unroll
            for (int q = 0; q < kPrGroups; ++q) {  // a group of 16 tokens; the next one's scores load meanwhile
                if (MODE == kAttnAll || read) {
                    tmem_wait_ld16(v[q & 1]);
                    if (q + 1 < kPrGroups) tmem_ld16(tS + 16 * (q + 1), v[(q + 1) & 1]);
                }
                const uint32_t* x = v[q & 1];
                const float4 k = cst[q];
                const uint64_t f2 = pair(frow * k.x, frow * k.x), c2 = pair(k.y - ms, k.y - ms);
                const int32_t pos = tb + 16 * q;
                float y[16];
#pragma unroll
                for (int e = 0; e < 16; e += 2)
                    unpair(pair_fma(pair(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), f2, c2), y[e], y[e + 1]);
                if constexpr (kMasked) {
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (pos + e < see_lo || pos + e >= see_hi || k.y == -INFINITY) y[e] = -INFINITY;
                }
                if constexpr (kAgain) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) y[e] -= less;
                }
#pragma unroll
                for (int e = 0; e < 16; e += 2) tops[(e >> 1) & 1] = max3(tops[(e >> 1) & 1], y[e], y[e + 1]);
                if constexpr (kMasked) {
                    if (k.z == 0.0f) {  // (rare: V's scale far below others', or a missing block)
                        const float up = k.y == -INFINITY ? 0.0f : k.y;
#pragma unroll
                        for (int e = 0; e < 16; ++e) ts += exp2_fast(y[e] - up);
                    }
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) y[e] = exp2_fast(y[e]);
                uint64_t s2[2] = {pair(y[0], y[1]), pair(y[2], y[3])};
#pragma unroll
                for (int e = 4; e < 16; e += 2) s2[(e >> 1) & 1] = pair_add(s2[(e >> 1) & 1], pair(y[e], y[e + 1]));
#pragma unroll
                for (int e = 0; e < 16; e += 2) w[8 * q + e / 2] = pack_half2(y[e], y[e + 1]);
                float a, b;
                unpair(pair_add(s2[0], s2[1]), a, b);
                ts = __fmaf_rn(a + b, k.z, ts);
            }
            top = fmaxf(tops[0], tops[1]);
        };
        // The first tile's maximum, in a small loop: without it the weights
        // would be taken twice there.
        auto first_top = [&](const float4* cst, int32_t tb) {
            float top = -INFINITY;
#pragma unroll 1
            for (int q = 0; q < kPrGroups; ++q) {
                uint32_t v[16];
                tmem_ld16(tS + 16 * q, v);
                tmem_wait_ld16(v);
                const float4 k = cst[q];
                const float f = frow * k.x;
                const int32_t pos = tb + 16 * q;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float y = __fmaf_rn(__uint_as_float(v[e]), f, k.y);
                    if (pos + e >= see_lo && pos + e < see_hi) top = fmaxf(top, y);
                }
            }
            return top;
        };
        // Pass -1 takes weights of nothing, while the first codes are on their
        // way: it brings the code of the loop, 9 KB, to the SM, which cost 14000
        // cycles of the first tile (33000 on all SMs at once).
        for (int32_t n = MODE != kAttnAll && nt > 0 ? -1 : 0; n < turns; ++n) {
            const int32_t j = MODE == kAttnShared && dual && n >= 0 ? 2 * n + static_cast<int32_t>(wg) : n;  // the tile
            bool masked = false;
            int32_t tb = 0;
            if (MODE == kAttnAll || n >= 0) {
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(&S.sfull[wg], static_cast<uint32_t>(n & 1), p.waits.limit_ns));
                if (!ok) break;
                tc_fence_after();
                tb = tok0 + j * kPrTokens;
                masked = tb + kPrTokens > all_hi || tb < all_lo || S.gap[j % kPrCst] != 0u;
                if (MODE != kAttnAll && __any_sync(0xffffffffu, mx == -INFINITY && see_lo < tb + kPrTokens && see_hi > tb)) {
                    const float top = first_top(S.cst[j % kPrCst], tb);
                    if (mx == -INFINITY) ms = top > -INFINITY && top < INFINITY ? top : 0.0f;
                }
            }
            const float4* cst = S.cst[MODE == kAttnAll || n >= 0 ? j % kPrCst : 0];
            float ts, top;
            if (masked) weigh(std::true_type{}, std::false_type{}, n >= 0, 0.0f, cst, tb, ts, top);
            else weigh(std::false_type{}, std::false_type{}, n >= 0, 0.0f, cst, tb, ts, top);
            if (MODE != kAttnAll && n < 0) continue;
            bool grow = top > (mx == -INFINITY ? -INFINITY : 8.0f);
            if constexpr (MODE != kAttnAll) {
                if (mx == -INFINITY && top >= -8.0f && top <= 8.0f) {  // ms is the maximum, but for roundings
                    mx = ms;
                    grow = false;
                }
            }
            // a row passed its maximum by 8: always in the first tile that it sees (or where that is not known before), rarely later
            if (__any_sync(0xffffffffu, grow)) {
                const float ah = !grow ? 1.0f : (mx == -INFINITY ? 0.0f : exp2_fast(-0.5f * top)), al = ah * ah;
                if (n > 0) {  // O moves to the new maximum once the product before this one is done with it
                    ok = __all_sync(0xffffffffu, mbar_wait_bounded(&S.odone[wg], static_cast<uint32_t>((n - 1) & 1), p.waits.limit_ns));
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t v[32];
                        tmem_ld32(tO + 32 * c, v);
                        tmem_wait_ld32(v);
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * al);
                        tmem_st32(tO + 32 * c, v);
                    }
                    tmem_wait_st();
                }
                sum = sum * ah * ah;
                // the same exponents less the growth, so that the largest is 0 whatever ms + top is rounded to
                const float less = grow ? top : 0.0f;
                weigh(std::true_type{}, std::true_type{}, true, less, cst, tb, ts, top);
                if (grow) mx = ms = ms + less;
            }
            sum += ts;
            tmem_st32(tS, w);
            tmem_st32(tS + 32, w + 32);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.pfull[wg]);
        }
        if (ok && turns > 0) {
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(&S.odone[wg], static_cast<uint32_t>((turns - 1) & 1), p.waits.limit_ns));
            tc_fence_after();
        }
        if (!ok && lane == 0) atomicOr(&S.fault, 1u);
    }
    tc_fence_before();
    meet<kMeetAll, kPrThreads>();
    tc_fence_after();
    const bool fault = S.fault != 0u;
    if (fault && tid == 0) atomicOr(p.fault, kPrFault);
    if constexpr (MODE == kAttnOwn) attn_pdl_wait();  // the prefix's parts are there

    if (!fault && static_cast<int32_t>(wg) < nact) {
        const uint32_t tO = tmem + kO + D * wg + ((32u * (warp & 3u)) << 16);
        // head positions that this row sees as NaN although the product left them out
        uint32_t bad[D / 32] = {};
        if (E4M3 && S.nan != 0u) {
            const int32_t* table = p.table + r * p.width;
            for (int32_t j = 0; j < nt; ++j) {
                const int32_t tb = tok0 + j * kPrTokens;
                if (tb + kPrTokens <= cta_hi && tb >= cta_lo) continue;
                const int32_t a = tb > see_lo ? tb : see_lo, b = tb + kPrTokens < see_hi ? tb + kPrTokens : see_hi;
                for (int32_t tk = a; tk < b; ++tk) {
                    const int32_t id = table[tk >> bl];
                    if (id < 0 || id >= p.c.num_blocks) continue;
                    const uint64_t u = static_cast<uint64_t>(id) * p.c.heads + static_cast<uint32_t>(h);
                    const uint32_t* v = reinterpret_cast<const uint32_t*>(
                        p.c.v + ((u << bl) + (static_cast<uint32_t>(tk) & ((1u << bl) - 1u))) * D);
#pragma unroll
                    for (int w = 0; w < D / 4; ++w) {
                        const uint32_t x = nan_bytes(v[w]) >> 7;
                        bad[w / 8] |= ((x & 1u) | (x >> 7 & 2u) | (x >> 14 & 4u) | (x >> 21 & 8u)) << (4 * (w % 8));
                    }
                }
            }
        }
        // where the row's part goes, if it is one
        const bool leaves = MODE == kAttnShared || p.splits > 1;
        const uint32_t prow = wg * 128u + wrow;
        float* slot = p.parts + static_cast<uint64_t>(blockIdx.x) * NDQ_PROMPT_SLOT(D);
        float4* staged = reinterpret_cast<float4*>(base) + prow * (D / 4 + 1);  // (kAttnShared) the row on its way to its slot
        if constexpr (MODE == kAttnShared) {
            staged[D / 4] = make_float4(mx, sum, 0.0f, 0.0f);
            if (part == 0 && has_row && !(dual && wg == 1))
                static_cast<uint4*>(p.records)[at] =
                    make_uint4(static_cast<uint32_t>(slot_row), static_cast<uint32_t>(nrows), dual ? 2 * parts : parts, prow);
        } else if (leaves) {
            slot[prow] = mx;
            slot[kPromptRows + prow] = sum;
        }
        // what the prefix adds to the row, if this kernel finishes it
        constexpr bool kJoin = MODE == kAttnOwn;
        const bool join = kJoin && own > 0 && !leaves && has_row;
        float inv, self = 1.0f;
        if constexpr (kJoin) {
            if (join) {
                const RowParts<D> rp(p, at);
                const float top = rp.largest(mx), hs = part_root(mx, top);
                mx = top;
                self = hs * hs;
                sum = sum * hs * hs;
                for (uint32_t k = 0; k < rp.n; ++k) {
                    const float2 x = rp.stat(k);
                    if (x.x == -INFINITY && x.y == x.y) continue;
                    const float hf = part_root(x.x, top);
                    sum = __fmaf_rn(x.y * hf, hf, sum);
                }
            }
        }
        inv = sum > 0.0f ? __fdiv_rn(1.0f, sum) : (sum == sum ? 0.0f : sum);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
            uint32_t v[32];
            if (nt > (dual ? static_cast<int32_t>(wg) : 0)) {
                tmem_ld32(tO + 32 * c, v);
                tmem_wait_ld32(v);
            } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = 0u;
            }
            if (E4M3 && S.nan != 0u) {
                uint32_t bc = 0u;
#pragma unroll
                for (int q = 0; q < D / 32; ++q)
                    if (q == c) bc = bad[q];
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if (bc >> e & 1u) v[e] = 0x7fffffffu;
            }
            if constexpr (kJoin) {
                if (join) {
                    const RowParts<D> rp(p, at);
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * self);
                    for (uint32_t k = 0; k < rp.n; ++k) {
                        const float2 st = rp.stat(k);
                        if (st.x == -INFINITY && st.y == st.y) continue;
                        const float hf = part_root(st.x, mx), f = hf * hf;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float4 x = rp.values(k, static_cast<uint32_t>(8 * c + e));
                            v[4 * e] = __float_as_uint(__fmaf_rn(x.x, f, __uint_as_float(v[4 * e])));
                            v[4 * e + 1] = __float_as_uint(__fmaf_rn(x.y, f, __uint_as_float(v[4 * e + 1])));
                            v[4 * e + 2] = __float_as_uint(__fmaf_rn(x.z, f, __uint_as_float(v[4 * e + 2])));
                            v[4 * e + 3] = __float_as_uint(__fmaf_rn(x.w, f, __uint_as_float(v[4 * e + 3])));
                        }
                    }
                }
            }
            if constexpr (MODE == kAttnShared) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    staged[8 * c + e] = make_float4(__uint_as_float(v[4 * e]), __uint_as_float(v[4 * e + 1]), __uint_as_float(v[4 * e + 2]),
                                                    __uint_as_float(v[4 * e + 3]));
            } else if (leaves) {
                float4* d = reinterpret_cast<float4*>(slot + 2 * kPromptRows);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    d[(8 * c + e) * kPromptRows + prow] = make_float4(__uint_as_float(v[4 * e]), __uint_as_float(v[4 * e + 1]),
                                                                     __uint_as_float(v[4 * e + 2]), __uint_as_float(v[4 * e + 3]));
            } else if (!leaves && has_row) {
                uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + static_cast<int64_t>(at) * D + 32 * c);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t o[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        // (a row that saw nothing gives 0, whatever the product left)
                        o[q] = sum == 0.0f ? 0u : narrow2<BF16>(__uint_as_float(v[8 * e + 2 * q]) * inv, __uint_as_float(v[8 * e + 2 * q + 1]) * inv);
                    dst[e] = make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
        }
        if constexpr (MODE == kAttnShared) {
            // the warp's rows, one bulk store (K's, V's and the codes' memory is free: every product is done)
            fence_proxy_async_smem();
            __syncwarp();
            const uint32_t first = 32 * (dual ? warp & 3u : warp);  // the first of them among the unit's rows
            const int32_t mine = nrows - static_cast<int32_t>(first);
            if (lane == 0 && mine > 0) {
                bulk_store(p.slots + (slot_row + (dual ? wg * nrows : 0) + first) * (D + 4), reinterpret_cast<float4*>(base) + 32 * warp * (D / 4 + 1),
                           static_cast<uint32_t>(mine < 32 ? mine : 32) * (D + 4) * 4u);
                bulk_commit();
                bulk_wait_all();
            }
        }
        if (!leaves && p.lse && has_row)
            p.lse[at] = sum > 0.0f ? (mx + log2f(sum)) * 0.6931471805599453f : (sum == sum ? -INFINITY : sum);
    }
    tc_fence_before();
    meet<kMeetEnd, 256 + 32>();
    if (MODE != kAttnShared && p.splits > 1) {
        // the last part of the unit to arrive joins them in order
        __threadfence();
        meet<kMeetRows, 256>();
        if (tid == 0) {
            const uint32_t seen = atomicAdd(p.counters + unit, 1u);
            S.last = seen == static_cast<uint32_t>(p.splits - 1);
            if (S.last) p.counters[unit] = 0u;
            __threadfence();
        }
        meet<kMeetRows, 256>();
        if (S.last && !fault) {  // a thread per row and 8 head positions
            const float* first = p.parts + unit * static_cast<uint64_t>(p.splits) * NDQ_PROMPT_SLOT(D);
            for (int32_t i = static_cast<int32_t>(tid); i < nrows * (D / 8); i += 256) {
                const int32_t prow = i % nrows, c = i / nrows;
                float M = -INFINITY, L = 0.0f;
#pragma unroll
                for (int s = 0; s < kPromptMaxSplits; ++s)
                    if (s < p.splits) M = fmaxf(M, __ldcg(first + s * NDQ_PROMPT_SLOT(D) + prow));
                float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f), b = a;
#pragma unroll 4
                for (int s = 0; s < kPromptMaxSplits; ++s) {
                    if (s >= p.splits) break;
                    const float4* q = reinterpret_cast<const float4*>(first + s * NDQ_PROMPT_SLOT(D) + 2 * kPromptRows);
                    const float4 x = __ldcg(q + (2 * c) * kPromptRows + prow), y = __ldcg(q + (2 * c + 1) * kPromptRows + prow);
                    const float mm = __ldcg(first + s * NDQ_PROMPT_SLOT(D) + prow), ll = __ldcg(first + s * NDQ_PROMPT_SLOT(D) + kPromptRows + prow);
                    // (a part that saw nothing is left out; one whose weights vanish may hold a NaN that must stay)
                    if (mm == -INFINITY && ll == ll) continue;
                    const float hf = mm == -INFINITY ? 1.0f : exp2_fast(0.5f * (mm - M)), f = hf * hf;
                    L = __fmaf_rn(ll * hf, hf, L);
                    a.x = __fmaf_rn(x.x, f, a.x);
                    a.y = __fmaf_rn(x.y, f, a.y);
                    a.z = __fmaf_rn(x.z, f, a.z);
                    a.w = __fmaf_rn(x.w, f, a.w);
                    b.x = __fmaf_rn(y.x, f, b.x);
                    b.y = __fmaf_rn(y.y, f, b.y);
                    b.z = __fmaf_rn(y.z, f, b.z);
                    b.w = __fmaf_rn(y.w, f, b.w);
                }
                const int32_t to = static_cast<int32_t>((q0 + (row0 + prow) / p.group) * p.q_heads) + h * p.group + (row0 + prow) % p.group;
                if constexpr (MODE == kAttnOwn) {
                    if (own > 0) {  // the prefix's parts after them
                        const RowParts<D> rp(p, to);
                        const float top = rp.largest(M), hs = part_root(M, top), fs = hs * hs;
                        M = top;
                        L = L * hs * hs;
                        a = make_float4(a.x * fs, a.y * fs, a.z * fs, a.w * fs);
                        b = make_float4(b.x * fs, b.y * fs, b.z * fs, b.w * fs);
                        for (uint32_t k = 0; k < rp.n; ++k) {
                            const float2 st = rp.stat(k);
                            if (st.x == -INFINITY && st.y == st.y) continue;
                            const float hf = part_root(st.x, M), f = hf * hf;
                            const float4 x = rp.values(k, static_cast<uint32_t>(2 * c)), y = rp.values(k, static_cast<uint32_t>(2 * c + 1));
                            L = __fmaf_rn(st.y * hf, hf, L);
                            a = make_float4(__fmaf_rn(x.x, f, a.x), __fmaf_rn(x.y, f, a.y), __fmaf_rn(x.z, f, a.z), __fmaf_rn(x.w, f, a.w));
                            b = make_float4(__fmaf_rn(y.x, f, b.x), __fmaf_rn(y.y, f, b.y), __fmaf_rn(y.z, f, b.z), __fmaf_rn(y.w, f, b.w));
                        }
                    }
                }
                const float inv = L > 0.0f ? __fdiv_rn(1.0f, L) : (L == L ? 0.0f : L);
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + static_cast<int64_t>(to) * D + 8 * c) =
                    make_uint4(narrow2<BF16>(a.x * inv, a.y * inv), narrow2<BF16>(a.z * inv, a.w * inv),
                               narrow2<BF16>(b.x * inv, b.y * inv), narrow2<BF16>(b.z * inv, b.w * inv));
                if (p.lse && c == 0) p.lse[to] = L > 0.0f ? (M + log2f(L)) * 0.6931471805599453f : (L == L ? -INFINITY : L);
            }
        }
    }
}

// ---- launching ---------------------------------------------------------------

template <int D, bool E4M3, bool BF16, int MODE>
int launch_prompt(const typename AttnArgs<MODE>::type& p, unsigned grid, int dev, void* stream) {
    const auto fn = k_attn_prompt<D, E4M3, BF16, MODE>;
    static bool ready[64];  // (concurrent first calls set the same attribute)
    if (!ready[dev]) {
        const cudaError_t e =
            cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(PrSmem<D>::kBytes));
        if (e != cudaSuccess) return static_cast<int>(e);
        // the register split draws on what the block is launched with
        cudaFuncAttributes attr;
        const cudaError_t e2 = cudaFuncGetAttributes(&attr, fn);
        if (e2 != cudaSuccess) return static_cast<int>(e2);
        if (attr.numRegs != kPrLaunchRegs) return static_cast<int>(cudaErrorInvalidKernelImage);
        ready[dev] = true;
    }
    if constexpr (MODE != kAttnOwn) {
        fn<<<grid, kPrThreads, PrSmem<D>::kBytes, static_cast<cudaStream_t>(stream)>>>(p);
        return static_cast<int>(cudaGetLastError());
    } else {  // beside the kernel of the shared prefixes, which it waits for at the end
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(grid);
        cfg.blockDim = dim3(kPrThreads);
        cfg.dynamicSmemBytes = PrSmem<D>::kBytes;
        cfg.stream = static_cast<cudaStream_t>(stream);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        return static_cast<int>(cudaLaunchKernelEx(&cfg, fn, p));
    }
}

template <int MODE>
int launch_prompt_of(const typename AttnArgs<MODE>::type& p, int head_dim, bool e4m3, bool bf16, unsigned grid, int dev, void* stream) {
    if (head_dim == 64) {
        if (e4m3) return bf16 ? launch_prompt<64, true, true, MODE>(p, grid, dev, stream) : launch_prompt<64, true, false, MODE>(p, grid, dev, stream);
        return bf16 ? launch_prompt<64, false, true, MODE>(p, grid, dev, stream) : launch_prompt<64, false, false, MODE>(p, grid, dev, stream);
    }
    if (e4m3) return bf16 ? launch_prompt<128, true, true, MODE>(p, grid, dev, stream) : launch_prompt<128, true, false, MODE>(p, grid, dev, stream);
    return bf16 ? launch_prompt<128, false, true, MODE>(p, grid, dev, stream) : launch_prompt<128, false, false, MODE>(p, grid, dev, stream);
}

// CTAs of a launch over requests' own rows (kAttnAll, kAttnOwn), with
// p.splits set: 0 when no request can have enough rows, -1 when too many.
inline int64_t prompt_grid(AttnParams& p, int sms) {
    // units at most: a request's last unit may be partial, and has at least prompt_rows rows
    const int64_t rows = p.n_tokens * p.group;
    const int64_t reqs = rows / p.prompt_rows < p.n_req ? rows / p.prompt_rows : p.n_req;
    const int64_t units = (rows / kPromptRows + reqs) * p.c.heads;
    if (units == 0) return 0;
    // too few units to fill the GPU: split their tokens, four tiles to a part at least
    const int64_t most = (p.width << p.c.bs_log2) / (4 * 128);
    int64_t splits = (sms < kPromptMaxParts ? sms : kPromptMaxParts) / units;
    if (splits > kPromptMaxSplits) splits = kPromptMaxSplits;
    if (splits > most) splits = most;
    if (splits < 1) splits = 1;
    p.splits = static_cast<int32_t>(splits);
    return units * splits > INT32_MAX ? -1 : units * splits;
}

}  // namespace
}  // namespace ndq
