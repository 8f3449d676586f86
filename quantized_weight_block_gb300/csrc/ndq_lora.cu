// ndq_lora.cu -- low-rank adapters of many requests beside a shared
// projection:
//
//     t[m, j] = scale[a] * sum_k x[m, k] A[a, j, k]          (shrink, j < rank)
//     y[m, n] = base[m, n] + sum_j t[m, j] B[a, n, j]        (expand),  a = index[m]
//
// t in binary32.  There are two ways:
//
// * few rows (k_lora_rows): bound by the latency of one pass over the
//   adapters' weights.  One launch, a cluster of CTAs to a row: each sums some
//   of the ranks over all of K, and after an exchange of t through distributed
//   shared memory expands some of the columns.
// * many rows (k_lora_shrink_tile, k_lora_expand_tile; t in the workspace, the
//   second launched programmatically behind the first): tiles of 64 rows on
//   the tensor cores (mma.sync m16n8k16: the operator is bound by reading x
//   and base and writing y, and its products need a fraction of even that
//   rate).  A tile goes through the adapters of its rows one by one, with the
//   other adapters' rows as zeros, so any row order is right and adjacent
//   rows of one adapter cost one pass.  x and the weights are bfloat16, so
//   the shrink's products are exact; t enters the expansion as a sum of
//   bfloat16 parts: three for a binary32 result (2^-24 of t is left), two
//   for a bfloat16 one (2^-16, under the result's own rounding of 2^-9).
//   In the expansion the k-index is permuted so that a lane's 16 bytes are
//   its part of two k-steps, the output columns so that a lane holds 8
//   adjacent ones.
//
// Any other alignment (K or max_rank not a multiple of 8, buffers off 16
// bytes) takes the few-row kernel with scalar loads.
//
// Measured: 61 rows, 48 adapters of rank 16, K = N = 4096: 5.8 us (8.1-8.9 us a
// call from Python); 5003 rows of six requests, rank 64, K = 4096, N = 14336,
// bfloat16: 123-128 us, 28 for the shrink and 98 for the expansion (288 MB: 2.9
// TB/s; its mma.sync products alone are 46 us of every SM's time).

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cooperative_groups.h>
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cstdint>
#include <type_traits>

#include "ndq_device.cuh"
#include "ndq_serve.h"

namespace ndq {
namespace {

constexpr int kRowCtas = 8;          // CTAs to a row there
constexpr int kLoraThreads = 256;
constexpr int kLoraWarps = kLoraThreads / 32;
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

// One row to a cluster of kRowCtas CTAs.  CTA c sums the ranks J c .. J c + J - 1,
// J (c + 8) .. of t, its threads splitting K; the CTAs read each other's t
// through distributed shared memory; then each expands its columns, the first
// of which (weights of 16 ranks and base) it fetched at the start.
template <bool F32, bool VEC_A, bool VEC_B, int J>
__global__ void __cluster_dims__(kRowCtas, 1, 1) __launch_bounds__(kLoraThreads, 4) k_lora_rows(const LoraParams p) {
    namespace cg = cooperative_groups;
    __shared__ float s_part[kLoraWarps][J];
    __shared__ float s_t[128];               // this CTA's ranks, at their index
    __shared__ __align__(16) float s_all[128];
    cg::cluster_group cluster = cg::this_cluster();
    const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5, c = cluster.block_rank();
    const int64_t step = static_cast<int64_t>(kRowCtas) * kLoraThreads;
    for (int64_t m = blockIdx.x / kRowCtas; m < p.M; m += gridDim.x / kRowCtas) {
        const int32_t a = p.index[m];
        const bool has = a >= 0 && a < p.nA;
        const int64_t n0 = static_cast<int64_t>(c) * kLoraThreads + tid;
        auto base_at = [&](int64_t n) -> float {
            if constexpr (F32) return static_cast<const float*>(p.base)[m * p.N + n];
            else return bf(static_cast<const uint16_t*>(p.base)[m * p.N + n]);
        };
        const uint16_t* wb = p.b + static_cast<int64_t>(has ? a : 0) * p.N * p.rmax;
        float b0 = 0.0f;
        uint4 v0[2] = {};
        if (n0 < p.N) {
            b0 = base_at(n0);
            if constexpr (VEC_B) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (has && 8 * i < p.rmax) v0[i] = __ldg(reinterpret_cast<const uint4*>(wb + n0 * p.rmax) + i);
            }
        }
        // (weights are fetched before the rank is known: the rows beyond it exist)
        const int32_t r = rank_of(p, a);
        const uint16_t* x = p.x + m * p.K;
        for (int32_t j0 = static_cast<int32_t>(c) * J; has && j0 < p.rmax; j0 += kRowCtas * J) {
            const uint16_t* w = p.a + (static_cast<int64_t>(a) * p.rmax + j0) * p.K;
            const int32_t nj = static_cast<int32_t>(p.rmax) - j0 < J ? static_cast<int32_t>(p.rmax) - j0 : J;
            float s[J] = {};
            if constexpr (VEC_A) {
                const int64_t K8 = p.K >> 3;
#pragma unroll 2
                for (int64_t i = tid; i < K8; i += kLoraThreads) {
                    const uint4 xv = __ldg(reinterpret_cast<const uint4*>(x) + i);
                    uint4 wv[J];
#pragma unroll
                    for (int j = 0; j < J; ++j)
                        wv[j] = j < nj ? __ldg(reinterpret_cast<const uint4*>(w + j * p.K) + i) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                    for (int j = 0; j < J; ++j) s[j] = dot8(xv, wv[j], s[j]);
                }
            } else {
                for (int64_t k = tid; k < p.K; k += kLoraThreads) {
                    const float xv = bf(x[k]);
#pragma unroll
                    for (int j = 0; j < J; ++j)
                        if (j < nj) s[j] = __fmaf_rn(xv, bf(w[j * p.K + k]), s[j]);
                }
            }
            if (j0 >= r) break;  // (uniform; later groups are beyond the rank too)
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) s[j] = __fadd_rn(s[j], __shfl_xor_sync(0xffffffffu, s[j], d));
            if (lane == 0) {
#pragma unroll
                for (int j = 0; j < J; ++j) s_part[warp][j] = s[j];
            }
            __syncthreads();
            if (tid < J) {
                float v = 0.0f;
#pragma unroll
                for (int q = 0; q < kLoraWarps; ++q) v = __fadd_rn(v, s_part[q][tid]);
                s_t[j0 + tid] = __fmul_rn(v, p.scales[a]);
            }
            __syncthreads();
        }
        cluster.sync();  // every CTA's t is in its shared memory
        if (static_cast<int32_t>(tid) < r)
            s_all[tid] = cluster.map_shared_rank(s_t, (tid / J) % kRowCtas)[tid];
        else if (tid < 128)
            s_all[tid] = 0.0f;
        cluster.sync();  // and read by all of them
        for (int64_t n = n0; n < p.N; n += step) {
            float s = 0.0f;
            const uint16_t* w = wb + n * p.rmax;
            if constexpr (VEC_B) {
                for (int32_t j0 = 0; j0 < r; j0 += 16) {
                    uint4 v[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (n == n0 && j0 == 0) v[i] = v0[i];
                        else v[i] = j0 + 8 * i < r ? __ldg(reinterpret_cast<const uint4*>(w + j0) + i) : make_uint4(0u, 0u, 0u, 0u);
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t q[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const int32_t j = j0 + 8 * i + e;
                            const float wv = (e & 1) ? bf_hi(q[e >> 1]) : bf_lo(q[e >> 1]);
                            if (j < r) s = __fmaf_rn(s_all[j], wv, s);  // (weights beyond the rank are not defined)
                        }
                    }
                }
            } else {
                for (int32_t j = 0; j < r; ++j) s = __fmaf_rn(s_all[j], bf(w[j]), s);
            }
            const float y = __fadd_rn(n == n0 ? b0 : base_at(n), s);
            if constexpr (F32) static_cast<float*>(p.y)[m * p.N + n] = y;
            else static_cast<__nv_bfloat16*>(p.y)[m * p.N + n] = __float2bfloat16_rn(y);
        }
        __syncthreads();  // s_all is read
    }
}

// ---- many rows -----------------------------------------------------------------

__device__ __forceinline__ void mma_bf16_16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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
    // (blockIdx.z of gridDim.z: every gridDim.z-th of the tile's adapters)
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
    uint32_t turn = 0;
    for (int32_t a = next(-1); a != INT32_MAX; a = next(a)) {
        if (turn++ % gridDim.z != blockIdx.z) continue;
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

// Expansion of tiles of 64 rows, 256 columns (128 for wide binary32 cases) at a
// time.  t's parts are laid out once a tile as A fragments in shared memory.
// Warp 16 brings base (one tensor copy of the tile's rows; a bulk copy per row
// took 80 cycles each to issue, 16-byte loads scattered over the rows read HBM
// at 2 TB/s) and the adapter's weights (one piece of memory) into a ring; warps 0-15, 2 row halves by 8 column groups,
// multiply, add and store.  A CTA's part of a tile is gone through once for
// each adapter of its rows (and once for rows without one), with those rows
// alone; so the order of (tile, columns) is divided over the CTAs by weight, a
// tile counting as often as the adapter changes along its rows.  (blockIdx.y of
// gridDim.y takes every gridDim.y-th of a tile's adapters.)  Without
// VEC (N or a buffer off the 16-byte grid) base and weights are loaded directly.
constexpr int kExpandRows = 64;
constexpr int kExpandWarps = 16;
constexpr int kExpandThreads = (kExpandWarps + 1) * 32;
constexpr int kExpandStages = 4;  // at most
constexpr int kExpandTiles = 2048;  // tiles whose weights are counted
constexpr uint32_t kLoraFault = 16u;  // bit of the device fault word

__host__ __device__ constexpr int expand_parts(bool f32) { return f32 ? 3 : 2; }
__host__ __device__ constexpr int expand_t_bytes(bool f32, int rmax) { return (rmax + 31) / 32 * expand_parts(f32) * 8 * 32 * 16; }
__host__ __device__ constexpr int expand_stage_bytes(bool f32, int rmax, int cols) {
    return kExpandRows * cols * (f32 ? 4 : 2) + cols * rmax * 2;
}

// What a bfloat16 part leaves of v: at most 2^119.  The bounds are for infinite
// parts, of which nothing is left: a finite rest (of NaN, too) keeps them what they are.
__device__ __forceinline__ float rest(float v, float part) { return fminf(fmaxf(__fsub_rn(v, part), -0x1p119f), 0x1p119f); }

// Splits 8 values of t into PARTS bfloat16 A fragments: rows g (v[0]) and g + 8 (v[1]) of four adjacent ranks.
template <int PARTS>
__device__ __forceinline__ void lay_parts(float (&v)[2][4], uint4* dst, int stride) {
#pragma unroll
    for (int part = 0; part < PARTS; ++part) {
        uint4 f;
        f.x = pack_bf16(v[0][0], v[0][1]);
        f.y = pack_bf16(v[1][0], v[1][1]);
        f.z = pack_bf16(v[0][2], v[0][3]);
        f.w = pack_bf16(v[1][2], v[1][3]);
        dst[part * stride] = f;
        v[0][0] = rest(v[0][0], bf_lo(f.x));
        v[0][1] = rest(v[0][1], bf_hi(f.x));
        v[1][0] = rest(v[1][0], bf_lo(f.y));
        v[1][1] = rest(v[1][1], bf_hi(f.y));
        v[0][2] = rest(v[0][2], bf_lo(f.z));
        v[0][3] = rest(v[0][3], bf_hi(f.z));
        v[1][2] = rest(v[1][2], bf_lo(f.w));
        v[1][3] = rest(v[1][3], bf_hi(f.w));
    }
}

// Ranks beyond the adapter's in a piece of 8 of which `left` (1 .. 7) count: not 0 * garbage.
__device__ __forceinline__ void cut_ranks(uint4& w, int32_t left) {
    w.x = left >= 2 ? w.x : w.x & 0xffffu;
    w.y = left >= 4 ? w.y : (left >= 3 ? w.y & 0xffffu : 0u);
    w.z = left >= 6 ? w.z : (left >= 5 ? w.z & 0xffffu : 0u);
    w.w = left >= 7 ? w.w & 0xffffu : 0u;
}

template <bool F32, bool VEC>
__global__ void __launch_bounds__(kExpandThreads, 1) k_lora_expand_tile(const LoraParams p, const __grid_constant__ CUtensorMap base_map,
                                                                        int splits, int cols, int stages) {
    constexpr int PARTS = expand_parts(F32);
    constexpr int EL = F32 ? 4 : 2;
    extern __shared__ __align__(128) uint8_t s_buf[];
    __shared__ uint64_t s_full[kExpandStages], s_empty[kExpandStages];
    __shared__ int32_t s_a[kExpandRows];
    __shared__ uint32_t s_fault;
    const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31u, g = lane >> 2, t = lane & 3u;
    const int rmax = static_cast<int>(p.rmax);
    const uint32_t tbytes = static_cast<uint32_t>(expand_t_bytes(F32, rmax)), stage = static_cast<uint32_t>(expand_stage_bytes(F32, rmax, cols));
    uint4* s_t = reinterpret_cast<uint4*>(s_buf);  // [k-step pair][part][16 rows][k-step][lane]
    uint8_t* ring = s_buf + tbytes;
    const int64_t tiles = (p.M + kExpandRows - 1) / kExpandRows, per = (p.N + cols - 1) / cols;
    __shared__ uint32_t s_w[kExpandTiles + 1];  // weights of the tiles before each
    __shared__ uint32_t s_run[kExpandWarps];
    const int32_t nw = tiles <= kExpandTiles ? static_cast<int32_t>(tiles) : 0;  // (more: all alike)
    if (warp < kExpandWarps)
        for (int32_t i = static_cast<int32_t>(warp); i < nw; i += kExpandWarps) {
            uint32_t changes = 0;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int64_t m = static_cast<int64_t>(i) * kExpandRows + lane + 32 * q;
                const bool diff = m < p.M && (lane + q) > 0 && p.index[m] != p.index[m - 1];
                changes += __popc(__ballot_sync(0xffffffffu, diff));
            }
            if (lane == 0) s_w[i] = changes + 1u;
        }
    __syncthreads();
    if (warp < kExpandWarps) {  // exclusive prefix sums, kExpandTiles / 512 tiles a thread
        constexpr int TPT = kExpandTiles / (kExpandWarps * 32);
        uint32_t v[TPT], sum = 0;
#pragma unroll
        for (int q = 0; q < TPT; ++q) {
            const int32_t i = static_cast<int32_t>(tid) * TPT + q;
            v[q] = sum;
            sum += i < nw ? s_w[i] : 0u;
        }
        uint32_t incl = sum;
#pragma unroll
        for (uint32_t d = 1; d < 32; d <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += y;
        }
        if (lane == 31u) s_run[warp] = incl;
        asm volatile("barrier.cta.sync 1, %0;" ::"n"(kExpandWarps * 32) : "memory");
        uint32_t before = incl - sum;
        for (uint32_t q = 0; q < warp; ++q) before += s_run[q];
#pragma unroll
        for (int q = 0; q < TPT; ++q) {
            const int32_t i = static_cast<int32_t>(tid) * TPT + q;
            if (i <= nw) s_w[i] = before + v[q];
        }
        if (static_cast<int32_t>(tid) * TPT + TPT == nw) s_w[nw] = before + sum;
    }
    __syncthreads();
    // this CTA's columns: from (tile, chunk) to (tile, chunk), in chunks from the first tile on
    auto place = [&](int64_t b) -> int64_t {
        if (nw == 0) return tiles * per * b / gridDim.x;
        const int64_t u = static_cast<int64_t>(s_w[nw]) * per * b / gridDim.x;  // in weighted chunks
        int32_t lo = 0, hi = nw;
        while (hi - lo > 1) {
            const int32_t mid = (lo + hi) >> 1;
            if (static_cast<int64_t>(s_w[mid]) * per <= u) lo = mid;
            else hi = mid;
        }
        if (u >= static_cast<int64_t>(s_w[nw]) * per) return tiles * per;
        return lo * per + (u - static_cast<int64_t>(s_w[lo]) * per) / (s_w[lo + 1] - s_w[lo]);
    };
    const int64_t w0 = place(blockIdx.x), w1 = place(blockIdx.x + 1);
    if (tid == 0) {
        for (int i = 0; i < stages; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_empty[i], kExpandWarps);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        s_fault = 0u;
    }
    __syncthreads();
    // the adapters of a tile, by lane: rows lane and lane + 32 (-1: none; INT32_MAX: no row)
    auto rows_of = [&](int64_t tile, int32_t (&mine)[2]) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t m = tile * kExpandRows + lane + 32 * i;
            mine[i] = INT32_MAX;
            if (m < p.M) {
                const int32_t a = p.index[m];
                mine[i] = a >= 0 && a < p.nA ? a : -1;
            }
        }
    };
    auto next = [&](const int32_t (&mine)[2], int32_t prev) {  // ascending, INT32_MAX at the end
        const int32_t c0 = mine[0] > prev ? mine[0] : INT32_MAX, c1 = mine[1] > prev ? mine[1] : INT32_MAX;
        return __reduce_min_sync(0xffffffffu, c0 < c1 ? c0 : c1);
    };

    if (warp == kExpandWarps) {
        // ---- loader
        int issued = 0;
        bool ok = true;
        for (int64_t w = w0; VEC && w < w1 && ok;) {
            const int64_t tile = w / per, m0 = tile * kExpandRows;
            const int64_t end = (tile + 1) * per < w1 ? (tile + 1) * per : w1;
            int32_t mine[2];
            rows_of(tile, mine);
            uint32_t turn = 0;
            for (int32_t a = next(mine, -2); a != INT32_MAX && ok; a = next(mine, a)) {
                if (turn++ % gridDim.y != blockIdx.y) continue;
                const bool weights = rank_of(p, a) > 0;
                for (int64_t c = w; c < end; ++c) {
                    const int64_t n0 = c % per * cols;
                    const int st = issued % stages;
                    if (issued >= stages) ok = __all_sync(0xffffffffu, mbar_wait_bounded(&s_empty[st], static_cast<uint32_t>((issued / stages - 1) & 1), p.waits.limit_ns));
                    if (!ok) break;
                    const uint32_t nc = static_cast<uint32_t>(p.N - n0 < cols ? p.N - n0 : cols);
                    const uint32_t wb = weights ? nc * static_cast<uint32_t>(rmax) * 2u : 0u;
                    uint8_t* d = ring + static_cast<uint32_t>(st) * stage;
                    if (lane == 0) {
                        // (all 64 rows, zeros past M and N: those of other adapters are not looked at)
                        mbar_arrive_expect_tx(&s_full[st], kExpandRows * static_cast<uint32_t>(cols) * EL + wb + p.waits.beyond);
                        asm volatile(
                            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::
                                "r"(smem_addr(d)),
                            "l"(reinterpret_cast<uint64_t>(&base_map)), "r"(static_cast<int32_t>(n0)), "r"(static_cast<int32_t>(m0)),
                            "r"(smem_addr(&s_full[st]))
                            : "memory");
                        if (weights)
                            bulk_load(d + kExpandRows * static_cast<uint32_t>(cols) * EL, p.b + (static_cast<int64_t>(a) * p.N + n0) * p.rmax, wb, &s_full[st]);
                    }
                    __syncwarp();
                    ++issued;
                }
            }
            w = end;
        }
        if (!ok) {  // its own copies in flight land before the block ends
            if (lane == 0) {
                atomicOr(&s_fault, 1u);
                atomicOr(p.fault, kLoraFault);
            }
            for (int i = issued > stages ? issued - stages : 0; i < issued; ++i)
                mbar_wait_bounded(&s_full[i % stages], static_cast<uint32_t>((i / stages) & 1), p.waits.limit_ns);
        }
        __syncthreads();
        return;
    }

    // ---- compute: rows 32 rh .. of the tile, columns 32 cg .. of the chunk
    const uint32_t rh = warp >> 3, cg = warp & 7u;
    pdl_wait();
    // lays adapter a's t out: rows of other adapters and ranks beyond r as zeros
    auto lay = [&](int64_t m0, int32_t a, int32_t r) {
        const int32_t pairs = (r + 31) / 32;
        for (int32_t i = static_cast<int32_t>(tid); i < pairs * 4 * 2 * 32; i += kExpandWarps * 32) {
            const int32_t ln = i & 31, ks = (i >> 5) & 1, quarter = (i >> 6) & 3, pr = i >> 8;
            const int32_t gg = ln >> 2, j = 32 * pr + 8 * (ln & 3) + 4 * ks;
            // the splits' sums, in order; all loads go out before the first addition
            float v[2][4] = {};
            float4 ld[2][kMaxSplit];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int32_t row = 16 * quarter + gg + 8 * e;
                const bool in = s_a[row] == a && j < r;
                const float* src = p.t + (m0 + row) * p.rmax + j;
#pragma unroll
                for (int q = 0; q < kMaxSplit; ++q)
                    ld[e][q] = in && q < splits ? __ldcg(reinterpret_cast<const float4*>(src + static_cast<int64_t>(q) * p.M * p.rmax))
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
            lay_parts<PARTS>(v, s_t + (pr * PARTS * 8 + quarter * 2 + ks) * 32 + ln, 8 * 32);
        }
    };
    // one k-step pair: A fragments of this warp's 32 rows times the pieces wv
    auto multiply = [&](float (&acc)[2][4][4], int32_t pr, const uint4 (&wv)[4]) {
        const uint4* f = s_t + (pr * PARTS * 8 + rh * 4) * 32 + lane;
#pragma unroll
        for (int part = 0; part < PARTS; ++part)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const uint4 f0 = f[(part * 8 + half * 2) * 32], f1 = f[(part * 8 + half * 2 + 1) * 32];
                const uint32_t a0[4] = {f0.x, f0.y, f0.z, f0.w}, a1[4] = {f1.x, f1.y, f1.z, f1.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) mma_bf16_16816(acc[half][e], a0, wv[e].x, wv[e].y);
#pragma unroll
                for (int e = 0; e < 4; ++e) mma_bf16_16816(acc[half][e], a1, wv[e].z, wv[e].w);
            }
    };
    auto meet = [&]() { asm volatile("barrier.cta.sync 1, %0;" ::"n"(kExpandWarps * 32) : "memory"); };

    int used = 0;
    bool ok = true;  // (a warp whose wait ran out goes on without working: the others meet it; the loader's wait for it runs out)
    for (int64_t w = w0; w < w1;) {
        const int64_t tile = w / per, m0 = tile * kExpandRows;
        const int64_t end = (tile + 1) * per < w1 ? (tile + 1) * per : w1;
        int32_t mine[2];
        rows_of(tile, mine);
        meet();  // every warp is done with the previous tile
        if (warp == 0) {
            s_a[lane] = mine[0];
            s_a[lane + 32] = mine[1];
        }
        uint32_t turn = 0;
        for (int32_t a = next(mine, -2); a != INT32_MAX; a = next(mine, a)) {
            if (turn++ % gridDim.y != blockIdx.y) continue;
            const int32_t r = rank_of(p, a);
            meet();  // s_a is there, and every warp is done with the previous adapter's t
            lay(m0, a, r);
            meet();
            for (int64_t c = w; c < end; ++c) {
                const int64_t n0 = c % per * cols;
                const int64_t nl = n0 + 32 * cg + 8 * t;  // this lane's 8 columns (n-tile e: columns 2 e, 2 e + 1)
                float acc[2][4][4] = {};
                const uint8_t* sb = nullptr;
                if constexpr (VEC) {
                    const int st = used % stages;
                    ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(&s_full[st], static_cast<uint32_t>((used / stages) & 1), p.waits.limit_ns));
                    sb = ring + static_cast<uint32_t>(st) * stage;
                }
                if (ok && static_cast<int>(32 * cg) < cols) {
                    // column of B's fragment n-tile e, index g: 32 cg + 8 (g / 2) + 2 e + g % 2
                    const int32_t nb = static_cast<int32_t>(32 * cg + 8 * (g >> 1) + (g & 1u));
                    const uint8_t* sw = sb + kExpandRows * cols * EL + (nb * rmax + 8 * static_cast<int>(t)) * 2;
                    const uint16_t* src = p.b + (static_cast<int64_t>(a < 0 ? 0 : a) * p.N + n0 + nb) * p.rmax + 8 * t;
#pragma unroll 1
                    for (int32_t pr = 0; 32 * pr < r; ++pr) {
                        uint4 wv[4];
                        const int32_t left = r - 32 * pr - 8 * static_cast<int32_t>(t);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            wv[e] = make_uint4(0u, 0u, 0u, 0u);
                            if constexpr (VEC) {
                                if (left > 0) wv[e] = *reinterpret_cast<const uint4*>(sw + (2 * e * rmax + 32 * pr) * 2);
                            } else {
                                if (left > 0 && n0 + nb + 2 * e < p.N) wv[e] = __ldg(reinterpret_cast<const uint4*>(src + 2 * e * p.rmax + 32 * pr));
                            }
                            if (left > 0 && left < 8) cut_ranks(wv[e], left);
                        }
                        multiply(acc, pr, wv);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int32_t row = static_cast<int32_t>(32 * rh + g) + 8 * i;
                        if (s_a[row] != a) continue;  // (also rows beyond M)
                        const int half = i >> 1, k = 2 * (i & 1);
                        const int64_t o = (m0 + row) * p.N + nl;
                        if constexpr (!VEC) {
#pragma unroll
                            for (int q = 0; q < 8; ++q) {
                                if (nl + q >= p.N) continue;
                                const float v = acc[half][q >> 1][k + (q & 1)];
                                if constexpr (F32) static_cast<float*>(p.y)[o + q] = __fadd_rn(static_cast<const float*>(p.base)[o + q], v);
                                else static_cast<uint16_t*>(p.y)[o + q] =
                                    static_cast<uint16_t>(pack_bf16(__fadd_rn(bf(static_cast<const uint16_t*>(p.base)[o + q]), v), 0.0f));
                            }
                            continue;
                        }
                        uint8_t* y = static_cast<uint8_t*>(p.y) + o * EL;
                        const uint8_t* b = sb + (row * cols + 32 * static_cast<int>(cg) + 8 * static_cast<int>(t)) * EL;
                        if constexpr (F32) {
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                if (nl + 4 * q >= p.N) continue;
                                float4 v = *reinterpret_cast<const float4*>(b + 16 * q);
                                v.x = __fadd_rn(v.x, acc[half][2 * q][k]);
                                v.y = __fadd_rn(v.y, acc[half][2 * q][k + 1]);
                                v.z = __fadd_rn(v.z, acc[half][2 * q + 1][k]);
                                v.w = __fadd_rn(v.w, acc[half][2 * q + 1][k + 1]);
                                *reinterpret_cast<float4*>(y + 16 * q) = v;
                            }
                        } else if (nl < p.N) {
                            uint4 v = *reinterpret_cast<const uint4*>(b);
                            uint32_t* u = &v.x;
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                u[q] = pack_bf16(__fadd_rn(bf_lo(u[q]), acc[half][q][k]), __fadd_rn(bf_hi(u[q]), acc[half][q][k + 1]));
                            *reinterpret_cast<uint4*>(y) = v;
                        }
                    }
                }
                if constexpr (VEC) {
                    __syncwarp();
                    if (lane == 0 && ok) mbar_arrive(&s_empty[used % stages]);  // (a stage that did not land is not filled again)
                    ++used;
                }
            }
        }
        w = end;
    }
    if (!ok && lane == 0) {
        atomicOr(&s_fault, 1u);
        atomicOr(p.fault, kLoraFault);
    }
    __syncthreads();
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Rows from which the tensor-core tiles are taken.  What decides is the rows of
// an adapter, which the host does not know: the number of rows stands for it.
// Measured (K = 4096, bfloat16; row by row / in tiles, us), at rank 16, N = 4096
// one adapter: 61 rows 6.1 / 10, 128 rows 10 / 10, 512 rows 34 / 14; rows dealt to
// 48 adapters in turn: 61 rows 6.4 / 41, 128 rows 11 / 69, 512 rows 36 / 180.  At
// rank 64, N = 14336 one adapter: 61 rows 45 / 17, 150 rows 101 / 18, 512 rows
// 298 / 24; 48 adapters: 61 rows 47 / 123, 150 rows 120 / 231, 512 rows 342 / 465.
// So many rows of as many adapters take the slower form, and wide projections
// beside fewer than 128 rows of one adapter, too.
constexpr int64_t kTileMinRows = 128;

// K splits: as many CTAs as two on each SM make at most (one more would wait
// for a whole other round), at least 512 of K each.
int shrink_splits(int64_t M, int64_t K) {
    const int64_t tiles = (M + kShrinkRows - 1) / kShrinkRows;
    int64_t s = 2 * 152 / tiles;
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

constexpr int kExpandSmem = 212 * 1024;  // (beside 10 KB of static shared memory)

PFN_cuTensorMapEncodeTiled_v12000 box_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;  // (benign race: same value)
    if (!encode) {
        void* fp = nullptr;
        cudaDriverEntryPointQueryResult q;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fp, 12000, cudaEnableDefault, &q);
        if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || !fp) return nullptr;
        encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fp);
    }
    return encode;
}

cudaError_t expand_ready(int dev) {
    static bool ready[64];  // (concurrent first calls set the same attributes)
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (ready[dev]) return cudaSuccess;
    for (const void* fn : {reinterpret_cast<const void*>(k_lora_expand_tile<true, true>), reinterpret_cast<const void*>(k_lora_expand_tile<true, false>),
                           reinterpret_cast<const void*>(k_lora_expand_tile<false, true>), reinterpret_cast<const void*>(k_lora_expand_tile<false, false>)}) {
        const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kExpandSmem);
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
    // what is left of the GPU goes to a tile's adapters (CTAs beyond their number end at once)
    const int64_t tiles = (p.M + kShrinkRows - 1) / kShrinkRows;
    int64_t z = 2 * 152 / (tiles * splits);
    z = z < 1 ? 1 : (z > 16 ? 16 : z);
    if (z > p.nA) z = p.nA;
    const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(splits), static_cast<unsigned>(z));
    k_lora_shrink_tile<NT><<<grid, kLoraThreads, smem, st>>>(p, splits);
    return cudaGetLastError();
}

}  // namespace

// Room for any M' <= M: M' * splits is at most 8 M' and, splits being 304 / tiles
// or 1, at most 64 (304 + tiles).
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
        // chunks of 256 columns, or of 128 when two stages of 256 do not fit; then up to four stages
        const int rm = static_cast<int>(p.rmax), tb = expand_t_bytes(out_f32, rm);
        const int cols = tb + 2 * expand_stage_bytes(out_f32, rm, 256) <= kExpandSmem ? 256 : 128;
        int stages = kExpandStages;
        while (stages > 1 && tb + stages * expand_stage_bytes(out_f32, rm, cols) > kExpandSmem) --stages;
        const size_t smem = static_cast<size_t>(tb + stages * expand_stage_bytes(out_f32, rm, cols));
        int dev = 0;
        e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return static_cast<int>(e);
        LoraParams q = p;
        const IqGrids* grids = nullptr;
        if (const int rc = device_symbols(dev, &q.fault, &grids)) return rc;
        e = expand_ready(dev);
        if (e != cudaSuccess) return static_cast<int>(e);
        const int64_t work = (p.M + kExpandRows - 1) / kExpandRows * ((p.N + cols - 1) / cols);
        // a small number of tiles: their adapters are dealt to several CTAs (those without one end at once)
        int64_t deal = 2 * 152 / work;
        deal = deal < 1 ? 1 : (deal > 8 ? 8 : deal);
        if (deal > p.nA) deal = p.nA;
        cudaLaunchConfig_t cfg = behind(attr, dim3(static_cast<unsigned>(work < 152 ? work : 152), static_cast<unsigned>(deal)), smem, st);
        cfg.blockDim = dim3(kExpandThreads);
        CUtensorMap map = {};
        if (vec_y) {  // base as [M, N], boxes of 64 rows by `cols`
            const PFN_cuTensorMapEncodeTiled_v12000 encode = box_encoder();
            if (!encode) return static_cast<int>(cudaErrorNotSupported);
            const cuuint64_t gdim[2] = {static_cast<cuuint64_t>(p.N), static_cast<cuuint64_t>(p.M)};
            const cuuint64_t gstride[1] = {static_cast<cuuint64_t>(p.N) * (out_f32 ? 4u : 2u)};
            const cuuint32_t box[2] = {static_cast<cuuint32_t>(cols), kExpandRows}, estride[2] = {1u, 1u};
            if (encode(&map, out_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p.base), gdim,
                       gstride, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
                return static_cast<int>(cudaErrorInvalidValue);
        }
        if (out_f32) e = vec_y ? cudaLaunchKernelEx(&cfg, k_lora_expand_tile<true, true>, q, map, splits, cols, stages)
                               : cudaLaunchKernelEx(&cfg, k_lora_expand_tile<true, false>, q, map, splits, cols, stages);
        else e = vec_y ? cudaLaunchKernelEx(&cfg, k_lora_expand_tile<false, true>, q, map, splits, cols, stages)
                       : cudaLaunchKernelEx(&cfg, k_lora_expand_tile<false, false>, q, map, splits, cols, stages);
        return static_cast<int>(e);
    }
    const int64_t rows = p.M < 65536 ? p.M : 65536;
    const unsigned grid = static_cast<unsigned>(rows * kRowCtas);
    auto go = [&](auto f32, auto va, auto vb) {
        // ranks at a time of a CTA: so many that up to 32 are spread over the whole cluster
        if (p.rmax <= 2 * kRowCtas) k_lora_rows<decltype(f32)::value, decltype(va)::value, decltype(vb)::value, 2><<<grid, kLoraThreads, 0, st>>>(p);
        else k_lora_rows<decltype(f32)::value, decltype(va)::value, decltype(vb)::value, 4><<<grid, kLoraThreads, 0, st>>>(p);
    };
    auto by_b = [&](auto f32, auto va) { vec_b ? go(f32, va, std::true_type{}) : go(f32, va, std::false_type{}); };
    auto by_a = [&](auto f32) { vec_a ? by_b(f32, std::true_type{}) : by_b(f32, std::false_type{}); };
    out_f32 ? by_a(std::true_type{}) : by_a(std::false_type{});
    return static_cast<int>(cudaGetLastError());
}

}  // namespace ndq
