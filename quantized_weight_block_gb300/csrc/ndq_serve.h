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

// Attention of requests that share prefixes: the prefix of each group of
// requests, read once for the rows of all of them (k_attn_prompt), every
// request's own tokens (k_attn_rows, in parts of one warp each; k_attn_prompt
// for many rows, which finishes those), and the join of the parts of a row
// (k_attn_join).
//
// A part is a row of D + 4 floats: values, maximum, sum.  The prefix's parts
// lie in slots: a unit (256 rows of a group and cache head at most) leaves one
// slot, of a row for each of its own, for each CTA that shares its tokens (two
// where it has 128 rows or fewer).  A row finds them by its record: the first
// slot's offset in rows, the rows of a slot, the slots, the row in the slot.
// The parts of its own tokens follow one another; their record is the first
// one's row and their number.
constexpr int kPrefixMaxParts = 64;   // CTAs of a unit at most
constexpr uint64_t kPrefixMinTiles = 2;  // tiles of 128 tokens of a CTA at least
constexpr int kPrefixMaxExtra = 192;  // CTAs beyond one per unit at most (no more than SMs)
constexpr int64_t prefix_slot_rows(int64_t n_tokens, int64_t q_heads) {
    return 2 * n_tokens * q_heads + static_cast<int64_t>(kPrefixMaxExtra) * kPromptRows;
}
constexpr int64_t prefix_own_rows(int64_t n_tokens, int64_t q_heads) {  // units beyond one a row tile: no more than warps
    return n_tokens * q_heads + static_cast<int64_t>(kAttnMaxCtas) * 8 * kAttnRows;
}
struct PrefixLayout {  // bytes from the workspace's start
    size_t records, own_records, slots, own_slots, bytes;
};
constexpr PrefixLayout prefix_layout(int head_dim, int64_t n_tokens, int64_t q_heads) {
    const size_t rows = static_cast<size_t>(n_tokens * q_heads), row = 4 * static_cast<size_t>(head_dim + 4);
    PrefixLayout x{};
    x.records = (attn_workspace_bytes(head_dim) + 255) / 256 * 256;
    x.own_records = (x.records + 16 * rows + 255) / 256 * 256;
    x.slots = (x.own_records + 8 * rows + 255) / 256 * 256;
    x.own_slots = (x.slots + row * static_cast<size_t>(prefix_slot_rows(n_tokens, q_heads)) + 255) / 256 * 256;
    x.bytes = x.own_slots + row * static_cast<size_t>(prefix_own_rows(n_tokens, q_heads));
    return x;
}
struct PrefixParams : AttnParams {
    const int32_t* group_start;
    const int32_t* prefix_len;
    int64_t n_groups;
    void* records;      // uint4 [n_tokens, q_heads]
    void* own_records;  // uint2 [n_tokens, q_heads]
    float* slots;
    float* own_slots;
    int64_t slot_rows;  // rows that they have room for
    int64_t own_rows;
    int32_t sms;        // (set by the launcher)
};
int launch_attention_prefix(PrefixParams p, int head_dim, bool e4m3, bool bf16, void* stream);
// The kernels' launches (each in its own translation unit).
int launch_prefix_shared(const PrefixParams& p, int head_dim, bool e4m3, bool bf16, int dev, void* stream);
int launch_prefix_own_prompt(PrefixParams p, int head_dim, bool e4m3, bool bf16, int dev, void* stream, bool* launched);
int launch_prefix_own_rows(const PrefixParams& p, int head_dim, bool e4m3, bool bf16, int dev, void* stream);
int launch_prefix_join(const PrefixParams& p, int head_dim, bool bf16, void* stream);

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
