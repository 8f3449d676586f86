// ndq_embed.cu -- launcher of the packed embedding lookup.
#include <cuda_runtime.h>

#include "ndq_embed.h"
#include "ndq_once.h"

namespace ndq {

namespace {
Once g_resident[64][KF_COUNT];  // CTAs of a device at once
}  // namespace

int launch_embed(EmbedParams p, void* stream) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return static_cast<int>(e);
    if (dev < 0 || dev >= 64) return static_cast<int>(cudaErrorInvalidDevice);
    unsigned int* fault = nullptr;
    if (const int rc = device_symbols(dev, &fault, &p.grids)) return rc;
    uint32_t seg = 0;
    EmbedKernelFn fn = nullptr;
    for (const auto family : {embed_simple, embed_kquant, embed_iq, embed_grouped})
        if (!fn) fn = family(p.w.fmt, &seg);
    if (!fn) return static_cast<int>(cudaErrorInvalidValue);
    constexpr int kThreadsPerCta = 128;
    int resident = 0;
    const int re = g_resident[dev][p.w.fmt].get(
        [&](int* n) {
            int sms = 0, ctas = 0;
            cudaError_t r = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
            if (r == cudaSuccess) r = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&ctas, fn, kThreadsPerCta, 0);
            *n = sms * (ctas > 0 ? ctas : 1);
            return static_cast<int>(r);
        },
        &resident);
    if (re != 0) return re;
    const uint64_t segs = (p.K + seg - 1) / seg, units = segs * p.n_tokens;
    if (segs > INT32_MAX || units > INT32_MAX) return -1;
    p.segs = static_cast<uint32_t>(segs);
    p.units = static_cast<uint32_t>(units);
    p.aligned = (reinterpret_cast<uintptr_t>(p.w.x) & 15u) == 0 && p.bpr * p.w.S % 16u == 0 && seg / p.w.B * p.w.S % 16u == 0;
    const uint64_t want = (units + 3) / 4, most = static_cast<uint64_t>(resident);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(want < most ? want : most));
    cfg.blockDim = dim3(kThreadsPerCta);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void* args[] = {&p};
    return static_cast<int>(cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(fn), args));
}

}  // namespace ndq
