// ndq_embed.cu -- launcher of the packed embedding lookup.
#include <cuda_runtime.h>

#include "ndq_embed.h"

namespace ndq {

namespace {
struct EmbedDevice {
    int sms = 0;
    int ctas[KF_COUNT] = {};  // per SM (0: not yet asked)
};
EmbedDevice g_embed_dev[64];
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
    EmbedDevice& di = g_embed_dev[dev];
    constexpr int kThreadsPerCta = 128;
    if (di.ctas[p.w.fmt] == 0) {  // (concurrent first calls find the same values)
        int sms = 0, ctas = 0;
        if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return static_cast<int>(e);
        if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&ctas, fn, kThreadsPerCta, 0)) != cudaSuccess) return static_cast<int>(e);
        di.sms = sms;
        di.ctas[p.w.fmt] = ctas > 0 ? ctas : 1;
    }
    const uint64_t segs = (p.K + seg - 1) / seg, units = segs * p.n_tokens;
    if (segs > INT32_MAX || units > INT32_MAX) return -1;
    p.segs = static_cast<uint32_t>(segs);
    p.units = static_cast<uint32_t>(units);
    p.aligned = (reinterpret_cast<uintptr_t>(p.w.x) & 15u) == 0 && p.bpr * p.w.S % 16u == 0 && seg / p.w.B * p.w.S % 16u == 0;
    const uint64_t want = (units + 3) / 4, resident = static_cast<uint64_t>(di.sms) * static_cast<uint64_t>(di.ctas[p.w.fmt]);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(want < resident ? want : resident));
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
