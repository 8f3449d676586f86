// ndq_embed.cuh -- rows of a packed table, decoded and scaled:
//
//     y[t] = scale * W[ids[t]]
//
// W decoded as DequantizePacked decodes it to binary32, one binary32 product
// with the scale, one rounding to the output type.  Bound by bytes: a row's
// payload read and its outputs written (2 or 4 bytes for about half a byte).
//
// Work.  The unit is a segment of 128 chunks of one token's row (2048 elements,
// 1024 of nvfp4), four chunks to a lane; warps take the segments of all tokens in
// turn.  A warp is on its own: it has the 16-byte lines of its next segment on
// their way to shared memory while it decodes this one, and leaves the outputs to
// one bulk store (lanes that store their own 32 bytes fill half sectors, which
// caps the write rate), so that nothing waits for another warp.
//
// Measured: 16001 rows of 4096 values, q4_k to bfloat16: 31.7 us, 5.2 TB/s, 0.77
// of the copy bandwidth; q8_0 36.6 us, 5.4 TB/s; q6_k 37.9 us, 4.8 TB/s; 8000
// rows, q4_0 to binary32: 28.7 us, 5.2 TB/s.  What bounds it is instructions (22 M
// of a warp, 62 % issue) beside the waits that 20 warps an SM leave open (five
// CTAs of 45 KB): with one chunk to a lane it took 49.7 us, with two 36.5 (30 M,
// 68 % issue); divisions in every unit took 54 us before.  More segments on their
// way (three, four) were slower: fewer CTAs fit an SM.  One row: 4.4 us, latency.
#pragma once

#include "ndq_device.cuh"
#include "ndq_embed.h"

namespace ndq {
namespace {

constexpr int kEmbedWarps = 4;
constexpr int kEmbedChunks = 4;  // of a lane, in a segment
constexpr int kEmbedStages = 2;  // packed segments of a warp in shared memory

template <int F>
struct EmbedSeg {
    static constexpr uint32_t kElems = 32u * kEmbedChunks * Fmt<F>::CE;
    static constexpr uint32_t kBytes = kElems / Fmt<F>::B * Fmt<F>::S;
    // a segment from the 16-byte line below its first byte, and what the decoders read beyond it
    static constexpr uint32_t kStage = (kBytes + 15u + 20u + 15u) / 16u * 16u;
    static_assert(kElems % Fmt<F>::B == 0, "whole blocks");
};

template <int F>
__global__ void __launch_bounds__(kEmbedWarps * 32) k_embed(const __grid_constant__ EmbedParams p) {
    using Fm = Fmt<F>;
    using Sg = EmbedSeg<F>;
    constexpr int CE = Fm::CE;
    __shared__ SmemHdr H;  // the decoders' 16-entry tables
    __shared__ __align__(16) uint8_t s_in[kEmbedWarps][kEmbedStages][Sg::kStage];
    __shared__ __align__(16) uint8_t s_out[kEmbedWarps][Sg::kElems * 4];
    __shared__ int64_t s_row[kEmbedWarps][kEmbedStages];     // the staged segments' rows, and where they start in their lines
    __shared__ uint32_t s_phase[kEmbedWarps][kEmbedStages];
    const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31u;
    if (tid < 16) {
        H.lut_iq4[tid] = static_cast<float>(c_iq4[tid]);
        H.lut_v[tid] = static_cast<float>(c_v[tid]);
    }
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");  // (the ids may be the previous kernel's)

    const DevTensor& t = p.w;
    const uint32_t step = gridDim.x * kEmbedWarps;
    // The units' tokens and segments, by steps (a division a unit would cost a third of the decode).
    const uint32_t u0 = blockIdx.x * kEmbedWarps + warp, tk_step = step / p.segs, seg_step = step % p.segs;
    struct Unit {
        uint32_t tk, seg;
    };
    auto next = [&](Unit& n) {
        n.tk += tk_step;
        n.seg += seg_step;
        if (n.seg >= p.segs) {
            n.seg -= p.segs;
            ++n.tk;
        }
    };
    // a unit's row of the table, or -1
    auto row_of = [&](uint32_t tk) -> int64_t {
        if (tk >= p.n_tokens) return -1;
        const int64_t id = p.ids64 ? static_cast<const int64_t*>(p.ids)[tk] : static_cast<const int32_t*>(p.ids)[tk];
        return id >= 0 && static_cast<uint64_t>(id) < p.n_rows ? id : -1;
    };
    // a unit's lines on their way, its row and token for when they are there
    auto fetch = [&](const Unit& n, int64_t id, uint32_t buf) {
        if (id >= 0) {  // (every line holds payload bytes)
            const uint64_t left = p.K - static_cast<uint64_t>(n.seg) * Sg::kElems;
            const uint32_t bytes = left < Sg::kElems ? static_cast<uint32_t>(left) / Fm::B * Fm::S : Sg::kBytes;
            const uint8_t* src = t.x + (static_cast<uint64_t>(id) * p.bpr + static_cast<uint64_t>(n.seg) * (Sg::kElems / Fm::B)) * Fm::S;
            const uint32_t ph = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(src) & 15u);
            const uint32_t lines = (ph + bytes + 15u) >> 4, d = smem_addr(s_in[warp][buf]);
            for (uint32_t i = lane; i < lines; i += 32)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d + 16u * i), "l"(src - ph + 16u * i) : "memory");
            if (lane == 0) s_phase[warp][buf] = ph;
        }
        if (lane == 0) s_row[warp][buf] = id;
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    Unit now{u0 / p.segs, u0 % p.segs}, ahead = now;
    uint32_t buf = 0, half = 0;
    int64_t id = row_of(ahead.tk);
#pragma unroll
    for (int i = 0; i < kEmbedStages - 1; ++i) {
        fetch(ahead, id, i);
        next(ahead);
        id = row_of(ahead.tk);
    }
    Ctx x{&H, nullptr, t.divs, 0, t.blocks_per_div, p.grids, code_count(t), 0, 0};
    for (; now.tk < p.n_tokens; next(now), buf = (buf + 1) % kEmbedStages) {
        fetch(ahead, id, (buf + kEmbedStages - 1) % kEmbedStages);
        next(ahead);
        id = row_of(ahead.tk);  // (for the next turn)
        asm volatile("cp.async.wait_group %0;" ::"n"(kEmbedStages - 1) : "memory");
        __syncwarp();
        const int64_t row = s_row[warp][buf];
        const uint64_t e0 = static_cast<uint64_t>(now.seg) * Sg::kElems, at = static_cast<uint64_t>(now.tk) * p.y_stride;
        const uint32_t el = p.out == KO_F32 ? 4u : 2u;
        x.row0 = static_cast<uint64_t>(row);
        x.col0 = e0;
        x.block0 = static_cast<uint64_t>(row) * p.bpr + static_cast<uint64_t>(now.seg) * (Sg::kElems / Fm::B);
        uint8_t* so = s_out[warp] + half;
        if (p.yvec) {
            // the last bulk store from here has read it (16-bit outputs fill the halves by turns)
            if (lane == 0) {
                if (p.out == KO_F32) bulk_wait_read<0>();
                else bulk_wait_read<1>();
            }
            __syncwarp();
        }
#pragma unroll
        for (int k = 0; k < kEmbedChunks; ++k) {
            const uint32_t c = lane + 32u * k;
            const uint64_t e = e0 + c * CE;
            const bool ok = e < p.K;
            float v[CE];
            if (ok && row >= 0) {
                if (p.aligned)
                    Fm::template chunk<false>(s_in[warp][buf], 0u, c, v, x);
                else
                    Fm::template chunk<true>(s_in[warp][buf], s_phase[warp][buf], c, v, x);
                if (p.scale != 1.0f) {
#pragma unroll
                    for (int i = 0; i < CE; ++i) v[i] = __fmul_rn(v[i], p.scale);
                }
            } else {
#pragma unroll
                for (int i = 0; i < CE; ++i) v[i] = 0.0f;
            }
            if (p.yvec) {
                uint4* o = reinterpret_cast<uint4*>(so + c * CE * el);
                if (p.out == KO_F32) {
#pragma unroll
                    for (int i = 0; i < CE / 4; ++i)
                        o[i] = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                                          __float_as_uint(v[4 * i + 3]));
                } else {
                    uint32_t w[CE / 2];
#pragma unroll
                    for (int i = 0; i < CE / 2; ++i)
                        w[i] = p.out == KO_BF16 ? pack_bf16(v[2 * i], v[2 * i + 1]) : pack_f16(v[2 * i], v[2 * i + 1]);
#pragma unroll
                    for (int i = 0; i < CE / 8; ++i) o[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                }
            } else if (ok) {
                if (p.out == KO_F32) store_chunk<KO_F32, CE>(p.y, at + e, v, false);
                else if (p.out == KO_BF16) store_chunk<KO_BF16, CE>(p.y, at + e, v, false);
                else store_chunk<KO_F16, CE>(p.y, at + e, v, false);
            }
        }
        if (p.yvec) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                const uint64_t left = p.K - e0;
                bulk_store(static_cast<uint8_t*>(p.y) + (at + e0) * el, so, (left < Sg::kElems ? static_cast<uint32_t>(left) : Sg::kElems) * el);
                bulk_commit();
            }
            if (p.out != KO_F32) half ^= Sg::kElems * 2;
        }
        __syncwarp();  // every lane has read the packed segment
    }
    if (lane == 0) bulk_wait_all();
}

}  // namespace

template <int F>
EmbedKernelFn embed_kernel(uint32_t* seg) {
    *seg = EmbedSeg<F>::kElems;
    return k_embed<F>;
}

}  // namespace ndq
