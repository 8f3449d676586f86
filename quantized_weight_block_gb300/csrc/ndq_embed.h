// ndq_embed.h -- launch descriptor of the packed embedding lookup, shared by
// the host ABI (ndq_api.cpp) and its kernels.  Not part of the public ABI.
#pragma once

#include "ndq_internal.h"

namespace ndq {

struct EmbedParams {
    DevTensor w;         // the table's payload as a decode descriptor (y unused)
    const void* ids;     // int32 or int64 [n_tokens]
    void* y;             // outputs, rows y_stride elements apart
    uint64_t y_stride;
    uint64_t n_rows;     // rows of the table
    uint64_t K;
    uint64_t bpr;        // payload blocks per row
    uint32_t n_tokens;
    uint32_t units;      // (set by the launcher) segments of all tokens' rows
    uint32_t segs;       // (set by the launcher) segments of a row
    int32_t out;         // KOut: KO_F32, KO_F16 or KO_BF16
    int32_t ids64;
    float scale;
    uint32_t yvec;       // 1: every output segment starts on a 16-byte boundary
    uint32_t aligned;    // (set by the launcher) 1: every packed segment starts on a 16-byte boundary
    const IqGrids* grids;  // (set by the launcher)
};
using EmbedKernelFn = void (*)(EmbedParams);

// Kernels of a family: the first that knows it (nullptr: none), and the
// elements of a segment.
EmbedKernelFn embed_simple(int kfmt, uint32_t* seg);
EmbedKernelFn embed_kquant(int kfmt, uint32_t* seg);
EmbedKernelFn embed_iq(int kfmt, uint32_t* seg);
EmbedKernelFn embed_grouped(int kfmt, uint32_t* seg);

// Launch p.  Returns 0, a CUDA error code, or -1 when there are 2^31 segments or more.
int launch_embed(EmbedParams p, void* stream);

}  // namespace ndq
