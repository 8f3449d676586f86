// ndq_attn_prefix.cu -- attention of requests that share prefixes: the kernel of
// the shared prefixes, and the launcher of all.
#include "ndq_attn_prompt.cuh"
#include "ndq_once.h"

namespace ndq {

constexpr double kPrefixMinSaved = 128e6;  // bytes of the cache
constexpr int64_t kPrefixMostRows = 128;   // rows of a request and cache head, on average

int launch_prefix_shared(const PrefixParams& p, int head_dim, bool e4m3, bool bf16, int dev, void* stream) {
    // units at most: a group's last one may be partial, and every group in use has a token
    const int64_t groups = p.n_groups < p.n_tokens ? p.n_groups : p.n_tokens;
    const int64_t grid = (p.n_tokens * p.group / kPromptRows + groups) * p.c.heads + kPrefixMaxExtra;
    if (grid > INT32_MAX) return static_cast<int>(cudaErrorInvalidValue);
    return launch_prompt_of<kAttnShared>(p, head_dim, e4m3, bf16, static_cast<unsigned>(grid), dev, stream);
}

int launch_attention_prefix(PrefixParams p, int head_dim, bool e4m3, bool bf16, void* stream) {
    static Once sms_of[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return static_cast<int>(e);
    if (dev < 0 || dev >= 64) return static_cast<int>(cudaErrorInvalidDevice);
    int sms = 0;
    const int se = sms_of[dev].get([&](int* n) { return static_cast<int>(cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev)); }, &sms);
    if (se != 0) return se;
    p.sms = sms < kPrefixMaxExtra ? sms : kPrefixMaxExtra;
    if (p.max_q > p.n_tokens) p.max_q = p.n_tokens;
    const IqGrids* grids = nullptr;
    if (const int rc = device_symbols(dev, &p.fault, &grids)) return rc;
    // Where sharing saves little: what it can save at most (what the host knows
    // are the tables' widths), or requests whose own rows fill the prompt
    // kernel's tiles, so that its products are the work.  Measured in us, shared
    // beside not, of 32 heads of 128 on 8 | 64 of 64 on 8 | 8 of 128 on 8, steps:
    // 16 requests behind 2000 tokens 34 beside 27 | 31 beside 22 | 32 beside 27,
    // behind 4000 (131 | 66 | 131 MB to save at most) 36 beside 35 | 34 beside 27
    // | 34 beside 35, 64 behind 1000 (169 | 85 | 169 MB) 35 beside 40 | 31 beside
    // 33 | 33 beside 40, behind 32000 91 beside 519 | 88 beside 357 | 65 beside
    // 503; eight requests behind 4000, 32 heads of 128 on 8, of 96 rows each 83
    // beside 87, of 256 118 beside 101, of 512 150 beside 102.
    // What the numbers do not tell: the rows are an average (64 single tokens and
    // a chunk of 2048 behind 32000 take 1.92 ms, unshared, and 1.22 ms in two
    // calls), and windows (64 behind 32000: with one of 500 tokens 51 beside 31,
    // of 2048 137 beside 58, of 4096 116 beside 88, of 8192 139 beside 149).
    const int64_t groups = p.n_groups < p.n_req ? p.n_groups : p.n_req;
    const double saved = static_cast<double>(p.n_req - groups) * static_cast<double>(p.width << p.c.bs_log2) * (2.0 * head_dim * p.c.heads);
    if (saved < kPrefixMinSaved || p.n_tokens * p.group >= kPrefixMostRows * p.n_req) return launch_attention(p, head_dim, e4m3, bf16, stream);
    p.splits = 1;
    if (const int rc = launch_prefix_shared(p, head_dim, e4m3, bf16, dev, stream)) return rc;
    // the requests' own tokens, by their rows as in launch_attention
    uint32_t* counters = p.counters;
    float* parts = p.parts;
    if (p.max_q * p.group > 2 * kAttnRows) {
        p.prompt_rows = 2 * kAttnRows + 1;
        p.counters = counters + kAttnMaxCtas;
        p.parts = parts + 2 * static_cast<size_t>(kAttnMaxCtas) * NDQ_ROWS_SLOT(head_dim);
        bool launched = false;
        if (const int rc = launch_prefix_own_prompt(p, head_dim, e4m3, bf16, dev, stream, &launched)) return rc;
        if (!launched) p.prompt_rows = 0;
        p.counters = counters;
        p.parts = parts;
    }
    if (const int rc = launch_prefix_own_rows(p, head_dim, e4m3, bf16, dev, stream)) return rc;
    return launch_prefix_join(p, head_dim, bf16, stream);
}

}  // namespace ndq
