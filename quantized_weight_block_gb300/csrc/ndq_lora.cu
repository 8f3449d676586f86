// ndq_lora.cu -- low-rank adapters of many requests beside a shared
// projection:
//
//     t[m, j] = scale[a] * sum_k x[m, k] A[a, j, k]          (shrink, j < rank)
//     y[m, n] = base[m, n] + sum_j t[m, j] B[a, n, j]        (expand),  a = index[m]
//
// Two kernels, t in binary32 in the workspace; the second is launched
// programmatically behind the first and reads what does not depend on it
// before it waits.  There are two pairs:
//
// * few rows (k_lora_shrink_rows, k_lora_expand_rows): bound by the latency
//   of one pass over the adapters' weights.  A CTA takes one row and
//   kShrinkJ ranks over all of K; a thread of the expansion one or more
//   outputs.
// * many rows (k_lora_shrink_tile, k_lora_expand_tile): tiles of 64 and 32
//   rows on the tensor cores (mma.sync m16n8k16: the operator is bound by reading x
//   and base and writing y, and its products need a fraction of even that
//   rate).  A tile goes through the adapters of its rows one by one, with the
//   other adapters' rows as zeros, so any row order is right and adjacent
//   rows of one adapter cost one pass.  x and the weights are bfloat16, so
//   the shrink's products are exact; t enters the expansion as a sum of
//   bfloat16 parts: three for a binary32 result (2^-24 of t is left), two
//   for a bfloat16 one (2^-16, under the result's own rounding of 2^-9).
//   The expansion's weights are loaded from global memory in the order of the
//   fragments: the k-index is permuted so that a lane's 16-byte load is its
//   part of two k-steps, the output columns so that a lane holds 8 adjacent
//   ones.
//
// Any other alignment (K or max_rank not a multiple of 8, buffers off 16
// bytes) takes the few-row kernels with scalar loads.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ndq_serve.h"

namespace ndq {
namespace {

constexpr int kShrinkJ = 4;          // ranks per CTA of k_lora_shrink_rows
constexpr int kLoraThreads = 256;
constexpr int kLoraWarps = kLoraThreads / 32;
constexpr int kTileRows = 32;        // rows of a tensor-core tile
constexpr int kMaxSplit = 8;         // K splits of k_lora_shrink_tile at most

__device__ __forceinline__ float bf(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ int32_t rank_of(const LoraParams& p, int32_t a) {
    if (a < 0 || a >= p.nA) return 0;
    const int32_t r = p.ranks[a];
    return r < 0 ? 0 : (r < p.rmax ? r : static_cast<int32_t>(p.rmax));
}

__device__ __forceinline__ float dot8(const uint4& x, const uint4& w, float s) {
    s = __fmaf_rn(bf_lo(x.x), bf_lo(w.x), s);
    s = __fmaf_rn(bf_hi(x.x), bf_hi(w.x), s);
    s = __fmaf_rn(bf_lo(x.y), bf_lo(w.y), s);
    s = __fmaf_rn(bf_hi(x.y), bf_hi(w.y), s);
    s = __fmaf_rn(bf_lo(x.z), bf_lo(w.z), s);
    s = __fmaf_rn(bf_hi(x.z), bf_hi(w.z), s);
    s = __fmaf_rn(bf_lo(x.w), bf_lo(w.w), s);
    return __fmaf_rn(bf_hi(x.w), bf_hi(w.w), s);
}

// ---- few rows ----------------------------------------------------------------

// One row and kShrinkJ ranks; the CTA's threads split K.
template <bool VEC>
__global__ void __launch_bounds__(kLoraThreads) k_lora_shrink_rows(const LoraParams p) {
    __shared__ float s_part[kLoraWarps][kShrinkJ];
    pdl_launch();
    const int32_t groups = static_cast<int32_t>((p.rmax + kShrinkJ - 1) / kShrinkJ);
    const int64_t m = blockIdx.x / groups;
    const int32_t j0 = static_cast<int32_t>(blockIdx.x % groups) * kShrinkJ;
    const int32_t a = p.index[m];
    if (a < 0 || a >= p.nA) return;
    const uint16_t* x = p.x + m * p.K;
    const uint16_t* w = p.a + (static_cast<int64_t>(a) * p.rmax + j0) * p.K;
    const int32_t have = static_cast<int32_t>(p.rmax) - j0 < kShrinkJ ? static_cast<int32_t>(p.rmax) - j0 : kShrinkJ;
    const int32_t nj = rank_of(p, a) - j0;  // (the weights are fetched before it is known: rows beyond the rank exist)
    float s[kShrinkJ] = {};
    if constexpr (VEC) {
        const int64_t K8 = p.K >> 3;
#pragma unroll 2
        for (int64_t i = threadIdx.x; i < K8; i += kLoraThreads) {
            const uint4 xv = reinterpret_cast<const uint4*>(x)[i];
            uint4 wv[kShrinkJ];
#pragma unroll
            for (int j = 0; j < kShrinkJ; ++j)
                wv[j] = j < have ? __ldg(reinterpret_cast<const uint4*>(w + j * p.K) + i) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int j = 0; j < kShrinkJ; ++j) s[j] = dot8(xv, wv[j], s[j]);
        }
    } else {
        for (int64_t k = threadIdx.x; k < p.K; k += kLoraThreads) {
            const float xv = bf(x[k]);
#pragma unroll
            for (int j = 0; j < kShrinkJ; ++j)
                if (j < nj) s[j] = __fmaf_rn(xv, bf(w[j * p.K + k]), s[j]);
        }
    }
    if (nj <= 0) return;
#pragma unroll
    for (int j = 0; j < kShrinkJ; ++j)
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s[j] = __fadd_rn(s[j], __shfl_xor_sync(0xffffffffu, s[j], d));
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
    if (lane == 0) {
#pragma unroll
        for (int j = 0; j < kShrinkJ; ++j) s_part[warp][j] = s[j];
    }
    __syncthreads();
    if (threadIdx.x < kShrinkJ && static_cast<int32_t>(threadIdx.x) < nj) {
        float v = 0.0f;
#pragma unroll
        for (int q = 0; q < kLoraWarps; ++q) v = __fadd_rn(v, s_part[q][threadIdx.x]);
        p.t[m * p.rmax + j0 + threadIdx.x] = __fmul_rn(v, p.scales[a]);
    }
}

// An output per thread; the weights of the first 16 ranks and base are
// fetched before the wait for t.
template <bool F32, bool VEC>
__global__ void __launch_bounds__(kLoraThreads) k_lora_expand_rows(const LoraParams p) {
    const int64_t n = static_cast<int64_t>(blockIdx.x) * kLoraThreads + threadIdx.x;
    const bool in = n < p.N;
    bool waited = false;
    for (int64_t m = blockIdx.y; m < p.M; m += gridDim.y) {
        const int32_t a = p.index[m];
        const bool has = a >= 0 && a < p.nA;
        const int64_t o = m * p.N + n;
        const uint16_t* w = p.b + (static_cast<int64_t>(has ? a : 0) * p.N + n) * p.rmax;
        const float* t = p.t + m * p.rmax;
        float b = 0.0f, s = 0.0f;
        if (in) {
            if constexpr (F32) b = static_cast<const float*>(p.base)[o];
            else b = bf(static_cast<const uint16_t*>(p.base)[o]);
        }
        if constexpr (VEC) {
            uint4 v[2] = {};  // 16 ranks of the output's weights, fetched beside the adapter's rank
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (in && has && 8 * i < p.rmax) v[i] = __ldg(reinterpret_cast<const uint4*>(w) + i);
            const int32_t r = rank_of(p, a);
            if (!waited) pdl_wait();
            waited = true;
            for (int32_t j0 = 0; j0 < r; j0 += 16) {
                float4 tv[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    tv[i] = j0 + 4 * i < r ? __ldcg(reinterpret_cast<const float4*>(t + j0) + i) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                uint4 u[2] = {v[0], v[1]};
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (in && j0 + 16 + 8 * i < r) v[i] = __ldg(reinterpret_cast<const uint4*>(w + j0 + 16) + i);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t c[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
                    const float f[8] = {tv[2 * i].x, tv[2 * i].y, tv[2 * i].z, tv[2 * i].w,
                                        tv[2 * i + 1].x, tv[2 * i + 1].y, tv[2 * i + 1].z, tv[2 * i + 1].w};
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float wv = (e & 1) ? bf_hi(c[e >> 1]) : bf_lo(c[e >> 1]);
                        if (j0 + 8 * i + e < r) s = __fmaf_rn(f[e], wv, s);  // (t and weights beyond the rank are not defined)
                    }
                }
            }
        } else {
            const int32_t r = rank_of(p, a);
            if (!waited) pdl_wait();
            waited = true;
            if (in)
                for (int32_t j = 0; j < r; ++j) s = __fmaf_rn(__ldcg(t + j), bf(w[j]), s);
        }
        if (in) {
            if constexpr (F32) static_cast<float*>(p.y)[o] = __fadd_rn(b, s);
            else static_cast<__nv_bfloat16*>(p.y)[o] = __float2bfloat16_rn(__fadd_rn(b, s));
        }
    }
    if (!waited) pdl_wait();
}

// ---- many rows -----------------------------------------------------------------

__device__ __forceinline__ void mma_bf16_16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// The next adapter of a tile after `prev` (rows' adapters in s_a; lanes are
// rows), or INT32_MAX: ascending, so each comes once.
__device__ __forceinline__ int32_t next_adapter(int32_t mine, int32_t prev) {
    int32_t c = mine > prev ? mine : INT32_MAX;
    return __reduce_min_sync(0xffffffffu, c);
}

// Sums t over a K split: CTA (tile of 64 rows, split), NT = max_rank / 8 rounded
// up.  x and the adapter's rows of A come through a ring of asynchronous
// copies in shared memory, 64 of K a stage, 16-byte pieces exchanged by row
// so that ldmatrix reads without conflicts.  Warp w takes rows 16 (w % 4)
// and half w / 4 of each stage; the halves are added at the end.
constexpr int kShrinkRows = 64;
constexpr int kShrinkK = 64;
template <int NT>
struct ShrinkSmem {
    static constexpr int kStages = NT <= 8 ? 6 : 4;
    static constexpr int kStage = (kShrinkRows + NT * 8) * kShrinkK * 2;
    static constexpr int kBytes = kStages * kStage;  // (at least the 64 x NT * 8 sums at the end)
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t* r, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

template <int NT>
__global__ void __launch_bounds__(kLoraThreads, 2) k_lora_shrink_tile(const LoraParams p, int splits) {
    using Sm = ShrinkSmem<NT>;
    constexpr int ST = Sm::kStages;
    extern __shared__ __align__(128) uint8_t s_ring[];
    __shared__ int32_t s_a[kShrinkRows];
    pdl_launch();
    const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31u, g = lane >> 2, t = lane & 3u;
    const int64_t m0 = static_cast<int64_t>(blockIdx.x) * kShrinkRows;
    const int32_t split = static_cast<int32_t>(blockIdx.y);
    if (tid < kShrinkRows) {
        int32_t a = -1;
        if (m0 + tid < p.M) {
            a = p.index[m0 + tid];
            if (a >= p.nA) a = -1;
        }
        s_a[tid] = a;
    }
    __syncthreads();
    const int32_t mine0 = s_a[lane], mine1 = s_a[lane + 32];
    auto next = [&](int32_t prev) {  // the tile's adapters in ascending order
        const int32_t c0 = mine0 > prev ? mine0 : INT32_MAX, c1 = mine1 > prev ? mine1 : INT32_MAX;
        return __reduce_min_sync(0xffffffffu, c0 < c1 ? c0 : c1);
    };
    const int32_t steps = static_cast<int32_t>((p.K + kShrinkK - 1) / kShrinkK);
    const int32_t st0 = static_cast<int32_t>(static_cast<int64_t>(steps) * split / splits);
    const int32_t n = static_cast<int32_t>(static_cast<int64_t>(steps) * (split + 1) / splits) - st0;
    const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(s_ring));
    const uint32_t piece = tid & 7u, crow = tid >> 3;  // this thread copies piece `piece` of rows crow, crow + 32, ...
    const uint32_t mrow = 16u * (warp & 3u), khalf = warp >> 2;
    for (int32_t a = next(-1); a != INT32_MAX; a = next(a)) {
        const int32_t r = rank_of(p, a);
        if (r == 0) continue;
        const bool live0 = s_a[crow] == a, live1 = s_a[crow + 32] == a;
        const uint16_t* x = p.x + (m0 + crow) * p.K + piece * 8;
        const uint16_t* w = p.a + (static_cast<int64_t>(a) * p.rmax + crow) * p.K + piece * 8;
        auto issue = [&](int32_t i) {
            if (i < n) {
                const int64_t k = static_cast<int64_t>(st0 + i) * kShrinkK;
                const bool in = k + piece * 8 < p.K;  // (K is a multiple of 8)
                const uint32_t d = ring + static_cast<uint32_t>(i % ST) * Sm::kStage + crow * 128u + ((piece ^ (crow & 7u)) << 4);
                cp_async16(d, live0 && in ? x + k : p.x, live0 && in ? 16u : 0u);
                cp_async16(d + 32u * 128u, live1 && in ? x + 32 * p.K + k : p.x, live1 && in ? 16u : 0u);
#pragma unroll
                for (int q = 0; q < (NT + 3) / 4; ++q) {
                    const int32_t j = static_cast<int32_t>(crow) + 32 * q;
                    if (j < NT * 8) {
                        const bool ok = in && j < r;
                        cp_async16(d + (kShrinkRows + 32u * q) * 128u, ok ? w + static_cast<int64_t>(32 * q) * p.K + k : p.a, ok ? 16u : 0u);
                    }
                }
            }
            cp_commit();
        };
        float acc[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.0f;
        __syncthreads();  // the ring and the previous adapter's sums are free
#pragma unroll
        for (int i = 0; i < ST - 1; ++i) issue(i);
        for (int32_t i = 0; i < n; ++i) {
            cp_wait<ST - 2>();
            __syncthreads();  // stage i is there, and every warp is done with stage i - 1
            issue(i + ST - 1);
            const uint32_t sx = ring + static_cast<uint32_t>(i % ST) * Sm::kStage, sw = sx + kShrinkRows * 128u;
#pragma unroll
            for (uint32_t ks = 0; ks < 2; ++ks) {
                const uint32_t u0 = 4u * khalf + 2u * ks;  // the k-step's first piece
                uint32_t af[4];
                const uint32_t ar = mrow + (lane & 15u);
                ldmatrix4(af, sx + ar * 128u + (((u0 + (lane >> 4)) ^ (ar & 7u)) << 4));
#pragma unroll
                for (int j = 0; j < NT; j += 2) {
                    uint32_t bfr[4];
                    // matrices: ranks 8 j.., pieces u0, u0 + 1; ranks 8 (j + 1).., the same
                    const uint32_t br = 8u * j + ((lane >> 4) << 3) + (lane & 7u);
                    const uint32_t row = NT == 1 ? (lane & 7u) : br;
                    ldmatrix4(bfr, sw + row * 128u + (((u0 + ((lane >> 3) & 1u)) ^ (row & 7u)) << 4));
                    mma_bf16_16816(acc[j], af, bfr[0], bfr[1]);
                    if (NT > 1) mma_bf16_16816(acc[j + (NT > 1 ? 1 : 0)], af, bfr[2], bfr[3]);
                }
            }
        }
        cp_wait<0>();
        __syncthreads();
        float* sums = reinterpret_cast<float*>(s_ring);  // [64][NT * 8]: the second half of K
        if (khalf == 1) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) sums[(mrow + g + 8 * (e >> 1)) * (NT * 8) + 8 * j + 2 * t + (e & 1)] = acc[j][e];
        }
        __syncthreads();
        if (khalf == 0) {
            const float sc = p.scales[a];
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t row = mrow + g + 8 * (e >> 1);
                    const int32_t c = 8 * j + 2 * static_cast<int32_t>(t) + (e & 1);
                    if (c < r && s_a[row] == a)
                        p.t[(static_cast<int64_t>(split) * p.M + m0 + row) * p.rmax + c] =
                            __fmul_rn(__fadd_rn(acc[j][e], sums[row * (NT * 8) + c]), sc);
                }
        }
    }
}

// y of 32 rows by `chunks` x 256 columns: each warp 32 adjacent columns at a
// time.  t's parts are laid out as A fragments in shared memory.  The usual
// tile (one adapter, VEC, all 32 columns inside) fetches base and weights
// `stages` chunks ahead through asynchronous copies private to the lane that
// consumes them; loaded into registers chunk by chunk the same tiles took
// twice the time, waiting.
__host__ __device__ constexpr int expand_parts(bool f32) { return f32 ? 3 : 2; }
__host__ __device__ constexpr int expand_t_bytes(bool f32, int rmax) { return (rmax + 31) / 32 * expand_parts(f32) * 4 * 32 * 16; }
__host__ __device__ constexpr int expand_stage_bytes(bool f32, int rmax) {  // of one warp: base 4 rows, weights 4 pieces per 32 ranks
    return 32 * 16 * ((f32 ? 8 : 4) + 4 * ((rmax + 31) / 32));
}

template <bool F32, bool VEC>
__global__ void __launch_bounds__(kLoraThreads, 2) k_lora_expand_tile(const LoraParams p, int splits, int chunks, int groups, int stages) {
    constexpr int PARTS = expand_parts(F32);
    constexpr int BW = F32 ? 8 : 4;  // words of base per lane and row
    constexpr int BP = F32 ? 8 : 4;  // 16-byte pieces of base per lane
    extern __shared__ __align__(16) uint8_t s_raw[];
    uint4* s_t = reinterpret_cast<uint4*>(s_raw);  // [k-step pair][part][half of the rows][k-step][lane]
    __shared__ int32_t s_a[kTileRows];
    const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31u, g = lane >> 2, t = lane & 3u;
    const int64_t m0 = static_cast<int64_t>(blockIdx.x / groups) * kTileRows;
    int32_t mine = -1;
    if (m0 + lane < p.M) {
        mine = p.index[m0 + lane];
        if (mine < 0 || mine >= p.nA) mine = -1;
    }
    if (warp == 0) s_a[lane] = mine;
    const int64_t cbase = (static_cast<int64_t>(blockIdx.x % groups) * chunks * kLoraWarps + warp) * 32;
    const int32_t first = next_adapter(mine, -1);
    const bool one = first == INT32_MAX || next_adapter(mine, first) == INT32_MAX;  // a single adapter: lay t out once
    pdl_wait();
    __syncthreads();
    // lays adapter a's t out: rows of other adapters and ranks beyond r as zeros
    auto lay = [&](int32_t a, int32_t r) {
        const int32_t pairs = (r + 31) / 32;
        for (int32_t i = static_cast<int32_t>(tid); i < pairs * 2 * 2 * 32; i += kLoraThreads) {
            const int32_t ln = i & 31, ks = (i >> 5) & 1, half = (i >> 6) & 1, pr = i >> 7;
            const int32_t gg = ln >> 2, tt = ln & 3;
            // the splits' sums, in order; all loads go out before the first addition
            const int32_t j = 32 * pr + 8 * tt + 4 * ks;
            float v[2][4] = {};
            float4 ld[2][kMaxSplit];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int32_t row = 16 * half + gg + 8 * e;
                const bool ok = s_a[row] == a && j < r;
                const float* src = p.t + (m0 + row) * p.rmax + j;
#pragma unroll
                for (int q = 0; q < kMaxSplit; ++q)
                    ld[e][q] = ok && q < splits ? __ldcg(reinterpret_cast<const float4*>(src + static_cast<int64_t>(q) * p.M * p.rmax))
                                                : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int q = 0; q < kMaxSplit; ++q) {
                    v[e][0] = __fadd_rn(v[e][0], ld[e][q].x);
                    v[e][1] = __fadd_rn(v[e][1], ld[e][q].y);
                    v[e][2] = __fadd_rn(v[e][2], ld[e][q].z);
                    v[e][3] = __fadd_rn(v[e][3], ld[e][q].w);
                }
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (j + c >= r) v[e][c] = 0.0f;  // (t beyond the rank is not written)
            }
#pragma unroll
            for (int part = 0; part < PARTS; ++part) {
                uint4 f;
                f.x = pack_bf16(v[0][0], v[0][1]);
                f.y = pack_bf16(v[1][0], v[1][1]);
                f.z = pack_bf16(v[0][2], v[0][3]);
                f.w = pack_bf16(v[1][2], v[1][3]);
                s_t[(((pr * PARTS + part) * 2 + half) * 2 + ks) * 32 + ln] = f;
                v[0][0] = __fsub_rn(v[0][0], bf_lo(f.x));
                v[0][1] = __fsub_rn(v[0][1], bf_hi(f.x));
                v[1][0] = __fsub_rn(v[1][0], bf_lo(f.y));
                v[1][1] = __fsub_rn(v[1][1], bf_hi(f.y));
                v[0][2] = __fsub_rn(v[0][2], bf_lo(f.z));
                v[0][3] = __fsub_rn(v[0][3], bf_hi(f.z));
                v[1][2] = __fsub_rn(v[1][2], bf_lo(f.w));
                v[1][3] = __fsub_rn(v[1][3], bf_hi(f.w));
            }
        }
    };
    const int32_t first_rank = first != INT32_MAX ? rank_of(p, first) : 0;
    if (one && first != INT32_MAX) {
        lay(first, first_rank);
        __syncthreads();
    }
    int c0 = 0;  // chunks done by the ring
    if constexpr (VEC) {
        int full = 0;  // chunks of this warp with all their columns inside
        while (full < chunks && cbase + static_cast<int64_t>(full) * kLoraWarps * 32 + 32 <= p.N) ++full;
        if (one && first_rank > 0 && stages > 1) {
            c0 = full;
            const int32_t r = first_rank, pairs = (r + 31) / 32;
            const uint32_t stage = static_cast<uint32_t>(expand_stage_bytes(F32, static_cast<int>(p.rmax)));
            const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(s_raw)) +
                                  static_cast<uint32_t>(expand_t_bytes(F32, static_cast<int>(p.rmax))) +
                                  warp * static_cast<uint32_t>(stages) * stage + lane * 16u;
            const size_t el = F32 ? 4 : 2;
            const uint8_t* bsrc = static_cast<const uint8_t*>(p.base) + ((m0 + g) * p.N + cbase + 8 * t) * el;
            const uint16_t* wsrc = p.b + (static_cast<int64_t>(first) * p.N + cbase + 8 * (g >> 1) + (g & 1u)) * p.rmax + 8 * t;
            const uint32_t wbytes[4] = {8u * t < static_cast<uint32_t>(r) ? 16u : 0u, 32u + 8u * t < static_cast<uint32_t>(r) ? 16u : 0u,
                                        64u + 8u * t < static_cast<uint32_t>(r) ? 16u : 0u, 96u + 8u * t < static_cast<uint32_t>(r) ? 16u : 0u};
            auto issue = [&](int c) {
                if (c < full) {
                    uint32_t d = ring + static_cast<uint32_t>(c % stages) * stage;
                    const uint8_t* b = bsrc + static_cast<int64_t>(c) * (kLoraWarps * 32) * el;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const bool in = m0 + g + 8 * i < p.M;
                        const uint8_t* row = b + 8 * i * p.N * el;
#pragma unroll
                        for (int q = 0; q < BP / 4; ++q, d += 512u)
                            cp_async16(d, in ? row + 16 * q : static_cast<const uint8_t*>(p.base), in ? 16u : 0u);
                    }
                    const uint16_t* w = wsrc + static_cast<int64_t>(c) * (kLoraWarps * 32) * p.rmax;
#pragma unroll
                    for (int pr = 0; pr < 4; ++pr)
                        if (pr < pairs) {
#pragma unroll
                            for (int e = 0; e < 4; ++e, d += 512u)
                                cp_async16(d, wbytes[pr] ? w + 2 * e * p.rmax + 32 * pr : p.b, wbytes[pr]);
                        }
                }
                cp_commit();
            };
            for (int c = 0; c < stages - 1; ++c) issue(c);
            for (int c = 0; c < full; ++c) {
                issue(c + stages - 1);
                if (stages == 4) cp_wait<3>();
                else if (stages == 3) cp_wait<2>();
                else cp_wait<1>();
                const uint8_t* st = s_raw + expand_t_bytes(F32, static_cast<int>(p.rmax)) +
                                    (warp * static_cast<uint32_t>(stages) + static_cast<uint32_t>(c % stages)) * stage + lane * 16u;
                float acc[2][4][4] = {};
#pragma unroll 1
                for (int32_t pr = 0; pr < pairs; ++pr) {
                    uint4 wv[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) wv[e] = *reinterpret_cast<const uint4*>(st + (BP + 4 * pr + e) * 512);
                    const int32_t left = r - 32 * pr - 8 * static_cast<int32_t>(t);
                    if (left > 0 && left < 8) {  // beyond the adapter's rank: not 0 * garbage
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            wv[e].x = left >= 2 ? wv[e].x : wv[e].x & 0xffffu;
                            wv[e].y = left >= 4 ? wv[e].y : (left >= 3 ? wv[e].y & 0xffffu : 0u);
                            wv[e].z = left >= 6 ? wv[e].z : (left >= 5 ? wv[e].z & 0xffffu : 0u);
                            wv[e].w = left >= 7 ? wv[e].w & 0xffffu : 0u;
                        }
                    }
                    const uint4* f = s_t + pr * (PARTS * 128) + lane;
#pragma unroll
                    for (int part = 0; part < PARTS; ++part)
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const uint4 f0 = f[(part * 2 + half) * 64], f1 = f[(part * 2 + half) * 64 + 32];
                            const uint32_t a0[4] = {f0.x, f0.y, f0.z, f0.w}, a1[4] = {f1.x, f1.y, f1.z, f1.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) mma_bf16_16816(acc[half][e], a0, wv[e].x, wv[e].y);
#pragma unroll
                            for (int e = 0; e < 4; ++e) mma_bf16_16816(acc[half][e], a1, wv[e].z, wv[e].w);
                        }
                }
                uint8_t* yb = static_cast<uint8_t*>(p.y) + ((m0 + g) * p.N + cbase + static_cast<int64_t>(c) * (kLoraWarps * 32) + 8 * t) * el;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (m0 + g + 8 * i >= p.M) continue;
                    uint8_t* y = yb + 8 * i * p.N * el;
                    const int half = i >> 1, k = 2 * (i & 1);
                    if constexpr (F32) {
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            float4 v = *reinterpret_cast<const float4*>(st + (2 * i + q) * 512);
                            v.x = __fadd_rn(v.x, acc[half][2 * q][k]);
                            v.y = __fadd_rn(v.y, acc[half][2 * q][k + 1]);
                            v.z = __fadd_rn(v.z, acc[half][2 * q + 1][k]);
                            v.w = __fadd_rn(v.w, acc[half][2 * q + 1][k + 1]);
                            *reinterpret_cast<float4*>(y + 16 * q) = v;
                        }
                    } else {
                        uint4 v = *reinterpret_cast<const uint4*>(st + i * 512);
                        uint32_t* u = &v.x;
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            u[q] = pack_bf16(__fadd_rn(bf_lo(u[q]), acc[half][q][k]), __fadd_rn(bf_hi(u[q]), acc[half][q][k + 1]));
                        *reinterpret_cast<uint4*>(y) = v;
                    }
                }
            }
            cp_wait<0>();
        }
    }
    for (int c = c0; c < chunks; ++c) {
        const int64_t n0 = cbase + static_cast<int64_t>(c) * kLoraWarps * 32;
        if (one && n0 >= p.N) break;
        // this lane's outputs: rows g + 8 i, columns n0 + 8 t + 0 .. 7 (n-tile e: columns 2 e, 2 e + 1)
        const int64_t nl = n0 + 8 * t;
        uint32_t bw[4][BW];  // base
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t m = m0 + g + 8 * i;
#pragma unroll
            for (int q = 0; q < BW; ++q) bw[i][q] = 0u;
            if (m < p.M) {
                const int64_t o = m * p.N + nl;
                if constexpr (F32) {
                    const uint32_t* b = static_cast<const uint32_t*>(p.base) + o;
                    if constexpr (VEC) {
#pragma unroll
                        for (int q = 0; q < 8; q += 4)
                            if (nl + q < p.N) *reinterpret_cast<uint4*>(&bw[i][q]) = *reinterpret_cast<const uint4*>(b + q);
                    } else {
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            if (nl + q < p.N) bw[i][q] = b[q];
                    }
                } else {
                    const uint16_t* b = static_cast<const uint16_t*>(p.base) + o;
                    if constexpr (VEC) {
                        if (nl < p.N) *reinterpret_cast<uint4*>(&bw[i][0]) = *reinterpret_cast<const uint4*>(b);
                    } else {
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            if (nl + q < p.N) bw[i][q / 2] |= static_cast<uint32_t>(b[q]) << (16 * (q & 1));
                    }
                }
            }
        }
        float acc[2][4][4] = {};
        // adds adapter a's part (its t laid out): column of B's fragment n-tile e, index g: n0 + 8 (g / 2) + 2 e + g % 2
        auto add = [&](int32_t a, int32_t r) {
            const int64_t n = n0 + 8 * (g >> 1) + (g & 1u);
            const uint16_t* w = p.b + (static_cast<int64_t>(a) * p.N + n) * p.rmax + 8 * t;
            const bool whole = n0 + 32 <= p.N;
            for (int32_t pr = 0; 32 * pr < r; ++pr) {
                uint4 wv[4];
                if (whole && 32 * pr + 32 <= r) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) wv[e] = __ldg(reinterpret_cast<const uint4*>(w + 2 * e * p.rmax + 32 * pr));
                } else {
                    const int32_t left = r - 32 * pr - 8 * static_cast<int32_t>(t);  // ranks of this lane's piece
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        wv[e] = make_uint4(0u, 0u, 0u, 0u);
                        if (n + 2 * e < p.N && left > 0) {
                            wv[e] = __ldg(reinterpret_cast<const uint4*>(w + 2 * e * p.rmax + 32 * pr));
                            if (left < 8) {  // beyond the adapter's rank: not 0 * garbage
                                wv[e].x = left >= 2 ? wv[e].x : wv[e].x & 0xffffu;
                                wv[e].y = left >= 4 ? wv[e].y : (left >= 3 ? wv[e].y & 0xffffu : 0u);
                                wv[e].z = left >= 6 ? wv[e].z : (left >= 5 ? wv[e].z & 0xffffu : 0u);
                                wv[e].w = left >= 7 ? wv[e].w & 0xffffu : 0u;
                            }
                        }
                    }
                }
                const uint4* f = s_t + pr * (PARTS * 128) + lane;
#pragma unroll
                for (int part = 0; part < PARTS; ++part)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const uint4 f0 = f[(part * 2 + half) * 64], f1 = f[(part * 2 + half) * 64 + 32];
                        const uint32_t a0[4] = {f0.x, f0.y, f0.z, f0.w}, a1[4] = {f1.x, f1.y, f1.z, f1.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) mma_bf16_16816(acc[half][e], a0, wv[e].x, wv[e].y);
#pragma unroll
                        for (int e = 0; e < 4; ++e) mma_bf16_16816(acc[half][e], a1, wv[e].z, wv[e].w);
                    }
            }
        };
        if (one) {
            if (first_rank > 0) add(first, first_rank);
        } else {
            for (int32_t a = first; a != INT32_MAX; a = next_adapter(mine, a)) {
                const int32_t r = rank_of(p, a);
                __syncthreads();
                lay(a, r);
                __syncthreads();
                add(a, r);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t m = m0 + g + 8 * i;
            if (m >= p.M) continue;
            const int64_t o = m * p.N + nl;
            const int half = i >> 1, c0 = 2 * (i & 1);
            if constexpr (F32) {
                float* y = static_cast<float*>(p.y) + o;
                float v[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] = __fadd_rn(__uint_as_float(bw[i][q]), acc[half][q >> 1][c0 + (q & 1)]);
                if constexpr (VEC) {
#pragma unroll
                    for (int q = 0; q < 8; q += 4)
                        if (nl + q < p.N) *reinterpret_cast<float4*>(y + q) = make_float4(v[q], v[q + 1], v[q + 2], v[q + 3]);
                } else {
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        if (nl + q < p.N) y[q] = v[q];
                }
            } else {
                uint16_t* y = static_cast<uint16_t*>(p.y) + o;
                uint32_t v[4];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    v[q] = pack_bf16(__fadd_rn(bf_lo(bw[i][q]), acc[half][q][c0]), __fadd_rn(bf_hi(bw[i][q]), acc[half][q][c0 + 1]));
                if constexpr (VEC) {
                    if (nl < p.N) *reinterpret_cast<uint4*>(y) = make_uint4(v[0], v[1], v[2], v[3]);
                } else {
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        if (nl + q < p.N) y[q] = static_cast<uint16_t>(v[q / 2] >> (16 * (q & 1)));
                }
            }
        }
    }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Rows from which the tensor-core tiles are taken (rule: where a 32-row tile
// is worth its pass over the adapters of its rows).
constexpr int64_t kTileMinRows = 96;

// K splits: enough CTAs for two on each SM, at least 512 of K each.
int shrink_splits(int64_t M, int64_t K) {
    const int64_t tiles = (M + kShrinkRows - 1) / kShrinkRows;
    int64_t s = (2 * 152 + tiles - 1) / tiles;
    if (s > K / 512) s = K / 512;
    if (s > kMaxSplit) s = kMaxSplit;
    return s < 1 ? 1 : static_cast<int>(s);
}

cudaLaunchConfig_t behind(cudaLaunchAttribute* attr, dim3 grid, size_t smem, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kLoraThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

cudaError_t expand_ready() {
    static bool ready[64];  // (concurrent first calls set the same attributes)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (ready[dev]) return cudaSuccess;
    for (const void* fn : {reinterpret_cast<const void*>(k_lora_expand_tile<true, true>), reinterpret_cast<const void*>(k_lora_expand_tile<true, false>),
                           reinterpret_cast<const void*>(k_lora_expand_tile<false, true>), reinterpret_cast<const void*>(k_lora_expand_tile<false, false>)}) {
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024);
        if (e != cudaSuccess) return e;
    }
    ready[dev] = true;
    return cudaSuccess;
}

template <int NT>
cudaError_t shrink_tile(const LoraParams& p, int splits, cudaStream_t st) {
    constexpr int smem = ShrinkSmem<NT>::kBytes;
    static bool ready[64];  // (concurrent first calls set the same attribute)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!ready[dev]) {
        e = cudaFuncSetAttribute(k_lora_shrink_tile<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        ready[dev] = true;
    }
    const dim3 grid(static_cast<unsigned>((p.M + kShrinkRows - 1) / kShrinkRows), static_cast<unsigned>(splits));
    k_lora_shrink_tile<NT><<<grid, kLoraThreads, smem, st>>>(p, splits);
    return cudaGetLastError();
}

}  // namespace

// Room for any M' <= M: M' * splits is at most 8 M' and, splits being
// (304 + tiles - 1) / tiles, at most 64 (304 + tiles).
size_t lora_workspace_bytes(int64_t M, int64_t rmax, int64_t K) {
    if (M < 1) M = 1;
    int64_t s = K / 512 < kMaxSplit ? K / 512 : kMaxSplit;
    if (s < 1) s = 1;
    const int64_t bound = kShrinkRows * (2 * 152 + (M + kShrinkRows - 1) / kShrinkRows);
    const int64_t rows = M * s < bound || bound < M ? M * s : bound;
    return static_cast<size_t>(rows) * static_cast<size_t>(rmax) * 4u + 16u;
}

int launch_lora(const LoraParams& p, bool out_f32, void* stream) {
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool vec_a = p.K % 8 == 0 && aligned16(p.x) && aligned16(p.a);
    const bool vec_b = p.rmax % 8 == 0 && aligned16(p.b);
    cudaLaunchAttribute attr[1];
    if (p.M >= kTileMinRows && vec_a && vec_b && p.nA > 0) {
        const int splits = shrink_splits(p.M, p.K);
        cudaError_t e;
        if (p.rmax <= 8) e = shrink_tile<1>(p, splits, st);
        else if (p.rmax <= 16) e = shrink_tile<2>(p, splits, st);
        else if (p.rmax <= 32) e = shrink_tile<4>(p, splits, st);
        else if (p.rmax <= 64) e = shrink_tile<8>(p, splits, st);
        else e = shrink_tile<16>(p, splits, st);
        if (e != cudaSuccess) return static_cast<int>(e);
        const bool vec_y = p.N % (out_f32 ? 4 : 8) == 0 && aligned16(p.base) && aligned16(p.y);
        const int64_t tiles = (p.M + kTileRows - 1) / kTileRows, cols = (p.N + kLoraWarps * 32 - 1) / (kLoraWarps * 32);
        // the ring: as many stages (2 to 4) as fit two CTAs on an SM, or else one
        const int rm = static_cast<int>(p.rmax), tb = expand_t_bytes(out_f32, rm), sb = expand_stage_bytes(out_f32, rm) * kLoraWarps;
        int stages = 4, per_sm = 2;
        while (stages > 2 && tb + stages * sb > 110 * 1024) --stages;
        if (tb + stages * sb > 110 * 1024) {
            per_sm = 1;
            stages = 4;
            while (stages > 2 && tb + stages * sb > 220 * 1024) --stages;
        }
        const size_t smem = static_cast<size_t>(tb + stages * sb);
        // column chunks per CTA: t is laid out once for all of them, as long as there are CTAs for three rounds
        int64_t chunks = tiles * cols / (3 * 152 * per_sm);
        chunks = chunks < 1 ? 1 : (chunks > 16 ? 16 : chunks);
        const int64_t groups = (cols + chunks - 1) / chunks;
        e = expand_ready();
        if (e != cudaSuccess) return static_cast<int>(e);
        cudaLaunchConfig_t cfg = behind(attr, dim3(static_cast<unsigned>(tiles * groups)), smem, st);
        const int ch = static_cast<int>(chunks), cg = static_cast<int>(groups);
        if (out_f32) e = vec_y ? cudaLaunchKernelEx(&cfg, k_lora_expand_tile<true, true>, p, splits, ch, cg, stages)
                               : cudaLaunchKernelEx(&cfg, k_lora_expand_tile<true, false>, p, splits, ch, cg, stages);
        else e = vec_y ? cudaLaunchKernelEx(&cfg, k_lora_expand_tile<false, true>, p, splits, ch, cg, stages)
                       : cudaLaunchKernelEx(&cfg, k_lora_expand_tile<false, false>, p, splits, ch, cg, stages);
        return static_cast<int>(e);
    }
    if (p.nA > 0) {
        const int64_t groups = (p.rmax + kShrinkJ - 1) / kShrinkJ;
        const unsigned grid = static_cast<unsigned>(p.M * groups);  // (the host keeps M * max_rank below 2^31)
        if (vec_a) k_lora_shrink_rows<true><<<grid, kLoraThreads, 0, st>>>(p);
        else k_lora_shrink_rows<false><<<grid, kLoraThreads, 0, st>>>(p);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return static_cast<int>(e);
    }
    const dim3 grid(static_cast<unsigned>((p.N + kLoraThreads - 1) / kLoraThreads),
                    static_cast<unsigned>(p.M < 65535 ? p.M : 65535));
    cudaLaunchConfig_t cfg = behind(attr, grid, 0, st);
    if (p.nA == 0) cfg.numAttrs = 0;  // nothing of this call to run behind
    cudaError_t e;
    if (out_f32) e = vec_b ? cudaLaunchKernelEx(&cfg, k_lora_expand_rows<true, true>, p)
                           : cudaLaunchKernelEx(&cfg, k_lora_expand_rows<true, false>, p);
    else e = vec_b ? cudaLaunchKernelEx(&cfg, k_lora_expand_rows<false, true>, p)
                   : cudaLaunchKernelEx(&cfg, k_lora_expand_rows<false, false>, p);
    return static_cast<int>(e);
}

}  // namespace ndq
