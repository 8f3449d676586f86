// ndq_embed.cuh -- rows of a packed table, decoded and scaled:
//
//     y[t] = scale * W[ids[t]]
//
// W decoded as DequantizePacked decodes it to binary32, one binary32 product
// with the scale, one rounding to the output type.  Bound by bytes: a row's
// payload read and its outputs written (2 or 4 bytes for about half a byte).
//
// Work.  The unit is a segment of 32 chunks of one token's row (512 elements,
// 256 of nvfp4), a chunk to a lane; warps take the segments of all tokens in
// turn.  A warp is on its own: it keeps the 16-byte lines of its next three
// segments on their way to shared memory while it decodes this one, and leaves
// the outputs to one bulk store (lanes that store their own 32 bytes fill half
// sectors, which caps the write rate), so that nothing waits for another warp.
#pragma once

#include "ndq_device.cuh"
#include "ndq_embed.h"

namespace ndq {
namespace {

constexpr int kEmbedWarps = 8;
constexpr int kEmbedStages = 4;  // packed segments of a warp in shared memory

template <int F>
struct EmbedSeg {
    static constexpr uint32_t kElems = 32u * Fmt<F>::CE;
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
    const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31u;
    if (tid < 16) {
        H.lut_iq4[tid] = static_cast<float>(c_iq4[tid]);
        H.lut_v[tid] = static_cast<float>(c_v[tid]);
    }
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");  // (the ids may be the previous kernel's)

    const DevTensor& t = p.w;
    const uint32_t step = gridDim.x * kEmbedWarps;
    // a unit's row of the table, or -1 (the units of a token follow one another)
    auto row_of = [&](uint32_t u) -> int64_t {
        if (u >= p.units) return -1;
        const uint32_t tk = u / p.segs;
        const int64_t id = p.ids64 ? static_cast<const int64_t*>(p.ids)[tk] : static_cast<const int32_t*>(p.ids)[tk];
        return id >= 0 && static_cast<uint64_t>(id) < p.n_rows ? id : -1;
    };
    auto source = [&](uint32_t u, int64_t id) { return t.x + (static_cast<uint64_t>(id) * p.bpr + (u % p.segs) * (Sg::kElems / Fm::B)) * Fm::S; };
    auto fetch = [&](uint32_t u, int64_t id, uint32_t buf) {  // (every line holds payload bytes)
        if (id >= 0) {
            const uint64_t left = p.K - static_cast<uint64_t>(u % p.segs) * Sg::kElems;
            const uint32_t bytes = left < Sg::kElems ? static_cast<uint32_t>(left) / Fm::B * Fm::S : Sg::kBytes;
            const uint8_t* src = source(u, id);
            const uint32_t ph = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(src) & 15u);
            const uint32_t lines = (ph + bytes + 15u) >> 4, d = smem_addr(s_in[warp][buf]);
            for (uint32_t i = lane; i < lines; i += 32)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d + 16u * i), "l"(src - ph + 16u * i) : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    uint32_t u = blockIdx.x * kEmbedWarps + warp, buf = 0, half = 0;
    int64_t id[kEmbedStages];  // rows of this unit and the next ones
#pragma unroll
    for (int i = 0; i < kEmbedStages; ++i) id[i] = row_of(u + i * step);
#pragma unroll
    for (int i = 0; i < kEmbedStages - 1; ++i) fetch(u + i * step, id[i], i);
    Ctx x{&H, nullptr, t.divs, 0, t.blocks_per_div, p.grids, code_count(t), 0, 0};
    for (; u < p.units; u += step, buf = (buf + 1) % kEmbedStages) {
        const int64_t id_after = row_of(u + kEmbedStages * step);
        fetch(u + (kEmbedStages - 1) * step, id[kEmbedStages - 1], (buf + kEmbedStages - 1) % kEmbedStages);
        asm volatile("cp.async.wait_group %0;" ::"n"(kEmbedStages - 1) : "memory");
        __syncwarp();
        const uint32_t seg = u % p.segs;
        const uint64_t e0 = static_cast<uint64_t>(seg) * Sg::kElems, e = e0 + lane * CE;
        const bool ok = e < p.K;
        float v[CE];
        if (ok && id[0] >= 0) {
            x.row0 = static_cast<uint64_t>(id[0]);
            x.col0 = e0;
            x.block0 = static_cast<uint64_t>(id[0]) * p.bpr + seg * (Sg::kElems / Fm::B);
            if (p.aligned)
                Fm::template chunk<false>(s_in[warp][buf], 0u, lane, v, x);
            else
                Fm::template chunk<true>(s_in[warp][buf], static_cast<uint32_t>(reinterpret_cast<uintptr_t>(source(u, id[0])) & 15u),
                                         lane, v, x);
#pragma unroll
            for (int i = 0; i < CE; ++i) v[i] = __fmul_rn(v[i], p.scale);
        } else {
#pragma unroll
            for (int i = 0; i < CE; ++i) v[i] = 0.0f;
        }
        const uint64_t at = static_cast<uint64_t>(u / p.segs) * p.y_stride;
        if (p.yvec) {
            // the last bulk store from here has read it (16-bit outputs fill the halves by turns)
            if (lane == 0) {
                if (p.out == KO_F32) bulk_wait_read<0>();
                else bulk_wait_read<1>();
            }
            __syncwarp();
            uint8_t* so = s_out[warp] + half;
            uint4* o = reinterpret_cast<uint4*>(so + lane * CE * (p.out == KO_F32 ? 4 : 2));
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
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                const uint32_t el = p.out == KO_F32 ? 4u : 2u;
                const uint64_t left = p.K - e0;
                bulk_store(static_cast<uint8_t*>(p.y) + (at + e0) * el, so,
                           (left < Sg::kElems ? static_cast<uint32_t>(left) : Sg::kElems) * el);
                bulk_commit();
            }
            if (p.out != KO_F32) half ^= Sg::kElems * 2;
        } else if (ok) {
            if (p.out == KO_F32) store_chunk<KO_F32, CE>(p.y, at + e, v, false);
            else if (p.out == KO_BF16) store_chunk<KO_BF16, CE>(p.y, at + e, v, false);
            else store_chunk<KO_F16, CE>(p.y, at + e, v, false);
        }
        __syncwarp();  // every lane has read the packed segment
#pragma unroll
        for (int i = 0; i + 1 < kEmbedStages; ++i) id[i] = id[i + 1];
        id[kEmbedStages - 1] = id_after;
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
