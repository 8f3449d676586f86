// ndq_serve.h -- launch descriptors of the serving operators (block tables,
// 8-bit cache append, attention over that cache, low-rank adapters), shared
// by the host ABI (ndq_serve_api.cpp) and their kernels.  Not part of the
// public ABI.
#pragma once

#include <cstddef>
#include <cstdint>

namespace ndq {

// What the kernels wait with: the limit of a wait, and the bytes that every
// staged copy is waited for beyond those it brings (0; else a requested check
// of the failure path: no copy is ever seen to land).
constexpr uint64_t kWaitNs = 2000000000ull;  // 2 s
struct Waits {
    uint64_t limit_ns = kWaitNs;
    uint32_t beyond = 0;
};

struct PlanParams {
    const int32_t* cached;
    const int32_t* fresh;
    const int32_t* free_blocks;
    const int32_t* free_count;
    int32_t* table;
    int32_t* q_start;
    int32_t* kv_len;
    int32_t* positions;
    int64_t* slots;
    int32_t* free_left;
    int64_t n_req;
    int64_t n_tokens;
    int64_t width;
    int32_t bs_log2;
};
int launch_kv_plan(const PlanParams& p, void* stream);

// The cache as the kernels see it.
struct KvCache {
    uint8_t* k;
    uint8_t* v;
    float* ks;
    float* vs;
    int64_t num_blocks;
    int32_t heads;
    int32_t bs_log2;
};

struct AppendParams {
    KvCache c;
    const uint16_t* k;
    const uint16_t* v;
    int64_t k_stride;
    int64_t v_stride;
    const int64_t* slots;
    int64_t n_tokens;
};
int launch_kv_append(const AppendParams& p, int head_dim, bool e4m3, bool bf16, void* stream);

// The attention workspace: arrival counters (zero between calls), then the
// partial results of the two kernels, which may run side by side.  Few rows:
// CTAs of a launch at most, each leaving up to two partials of 16 rows.
// Prompts: units of 256 rows whose tokens are split over at most one CTA per
// SM in all, each leaving one partial.
constexpr int kAttnMaxCtas = 512;
constexpr int kAttnRows = 16;
constexpr int kPromptRows = 256;
constexpr int kPromptMaxSplits = 16;
constexpr int kPromptMaxParts = 192;  // (units * splits <= SMs when splits > 1)
constexpr size_t kAttnCounterBytes = 4096;
static_assert((kAttnMaxCtas + kPromptMaxParts) * 4 <= kAttnCounterBytes, "counters");
#define NDQ_ROWS_SLOT(D) (static_cast<size_t>(ndq::kAttnRows) * ((D) + 2))     // floats of a partial
#define NDQ_PROMPT_SLOT(D) (static_cast<size_t>(ndq::kPromptRows) * ((D) + 2))
constexpr size_t attn_workspace_bytes(int head_dim) {
    return kAttnCounterBytes + 4u * (2u * kAttnMaxCtas * NDQ_ROWS_SLOT(head_dim) + kPromptMaxParts * NDQ_PROMPT_SLOT(head_dim));
}

struct AttnParams {
    KvCache c;
    const uint16_t* q;
    void* out;
    float* lse;
    const int32_t* table;
    const int32_t* kv_len;
    const int32_t* q_start;  // or nullptr: one query per request
    uint32_t* counters;  // of the kernel that is launched
    float* parts;
    int64_t n_tokens;
    int64_t n_req;
    int64_t q_stride;
    int64_t width;
    int32_t window;  // 0: none (at most 2^30, so positions and windows add up in 32 bits)
    int64_t max_q;
    int32_t q_heads;
    int32_t group;   // query heads per cache head
    int32_t group_shift;  // its logarithm, or -1
    float scale_log2;  // scale * log2(e)
    unsigned int* fault;  // device fault word (set by the launcher)
    Waits waits;
    int32_t splits;       // prompts: CTAs per unit (set by the launcher)
    int32_t prompt_rows;  // > 0: requests with at least this many rows are left to the prompt kernel
};
int launch_attention_prompt(AttnParams p, int head_dim, bool e4m3, bool bf16, int dev, int sms, void* stream,
                            bool* launched);
int launch_attention(AttnParams p, int head_dim, bool e4m3, bool bf16, void* stream);

struct LoraParams {
    const uint16_t* x;
    const uint16_t* a;
    const uint16_t* b;
    const int32_t* ranks;
    const float* scales;
    const int32_t* index;
    const void* base;
    void* y;
    float* t;  // workspace
    int64_t M, K, N, nA, rmax;
    unsigned int* fault;  // device fault word (set by the launcher)
    Waits waits;
};
size_t lora_workspace_bytes(int64_t M, int64_t rmax, int64_t K);
int launch_lora(const LoraParams& p, bool out_f32, void* stream);

}  // namespace ndq
