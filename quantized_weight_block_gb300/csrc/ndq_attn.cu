// ndq_attn.cu -- launcher of attention over the 8-bit cache.
#include "ndq_attn_rows.cuh"
#include "ndq_once.h"

namespace ndq {
namespace {

constexpr int kMaxDevices = 64;

}  // namespace

int launch_attention(AttnParams p, int head_dim, bool e4m3, bool bf16, void* stream) {
    static Once sms_of[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return static_cast<int>(e);
    if (dev < 0 || dev >= kMaxDevices) return static_cast<int>(cudaErrorInvalidDevice);
    int sms = 0;
    const int se = sms_of[dev].get([&](int* n) { return static_cast<int>(cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev)); }, &sms);
    if (se != 0) return se;
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
    return launch_rows_of<kAttnAll>(p, head_dim, e4m3, bf16, dev, sms, stream);
}

}  // namespace ndq
