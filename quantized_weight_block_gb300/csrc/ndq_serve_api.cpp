// ndq_serve_api.cpp -- the serving operators' part of the C ABI declared in
// include/ndq.h: host validation and launches.

#include <cmath>
#include <cstdint>

#include "ndq.h"
#include "ndq_serve.h"

namespace {

// A failure-path check requested for this host thread's next call with copies.
thread_local ndq::Waits t_waits;

ndq::Waits take_waits() {
    const ndq::Waits w = t_waits;
    t_waits = ndq::Waits{};
    return w;
}

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

int block_log2(int bs) {
    switch (bs) {
        case 16: return 4;
        case 32: return 5;
        case 64: return 6;
        case 128: return 7;
        default: return -1;
    }
}

int check_cache(const ndq_kv_cache* c, ndq::KvCache* d) {
    if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale) return NDQ_ERR_NULL;
    if (c->code_type != NDQ_FLOAT8E4M3FN && c->code_type != NDQ_INT8) return NDQ_ERR_BAD_DTYPE;
    d->bs_log2 = block_log2(c->block_size);
    if (d->bs_log2 < 0 || (c->head_dim != 64 && c->head_dim != 128) || c->kv_heads < 1 || c->kv_heads > 4096 ||
        c->num_blocks < 1 || c->num_blocks > INT32_MAX)
        return NDQ_ERR_BAD_ARG;
    // the cache's bytes fit a signed 64-bit offset: 2^31 * 2^12 * 2^7 * 2^7 < 2^63
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
        return NDQ_ERR_MISALIGNED;
    d->k = static_cast<uint8_t*>(c->k);
    d->v = static_cast<uint8_t*>(c->v);
    d->ks = c->k_scale;
    d->vs = c->v_scale;
    d->num_blocks = c->num_blocks;
    d->heads = c->kv_heads;
    return NDQ_OK;
}

// A piece of memory, of `bytes` (0: none).
struct Piece {
    const void* p;
    int64_t bytes;
};
bool overlap(const Piece& a, const Piece& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.bytes > 0 && b.bytes > 0 && (x < y ? y - x < static_cast<uintptr_t>(a.bytes) : x - y < static_cast<uintptr_t>(b.bytes));
}

// Rows of dense heads, 16-byte aligned, `stride` elements of 2 bytes apart.
int check_rows(const void* p, int64_t stride, int64_t row) {
    if (stride < row || stride > (int64_t(1) << 40)) return NDQ_ERR_BAD_ARG;
    if (!aligned(p, 16) || stride % 8 != 0) return NDQ_ERR_MISALIGNED;
    return NDQ_OK;
}

}  // namespace

extern "C" {

int ndq_kv_plan(const int32_t* cached, const int32_t* fresh, int64_t n_req, int block_size,
                const int32_t* free_blocks, const int32_t* free_count, int32_t* block_table, int64_t table_width,
                int32_t* q_start, int32_t* kv_len, int32_t* positions, int64_t* slots, int64_t n_tokens,
                int32_t* free_left, void* stream) {
    if (n_req < 0 || n_tokens < 0 || table_width < 0) return NDQ_ERR_NEGATIVE_DIM;
    const int bl = block_log2(block_size);
    if (bl < 0 || n_req > INT32_MAX - 1 || n_tokens > INT32_MAX - 1 || table_width > INT32_MAX - 1)
        return NDQ_ERR_BAD_ARG;
    if (!free_count || !q_start || !free_left) return NDQ_ERR_NULL;
    if (n_req > 0 && (!cached || !fresh || !kv_len || !free_blocks)) return NDQ_ERR_NULL;
    if (n_req > 0 && table_width > 0 && !block_table) return NDQ_ERR_NULL;
    if (n_tokens > 0 && (!positions || !slots)) return NDQ_ERR_NULL;
    if (free_left == free_count) return NDQ_ERR_BAD_ARG;
    if (!aligned(cached, 4) || !aligned(fresh, 4) || !aligned(free_blocks, 4) || !aligned(free_count, 4) ||
        !aligned(block_table, 4) || !aligned(q_start, 4) || !aligned(kv_len, 4) || !aligned(positions, 4) ||
        !aligned(slots, 8) || !aligned(free_left, 4))
        return NDQ_ERR_MISALIGNED;
    // The CTAs read the inputs while others write: an output may be neither an
    // input nor another output.  (Of the stack only the bottom is known here.)
    const int64_t entries = n_req * table_width;  // (below 2^62)
    const Piece out[] = {{block_table, 4 * (entries < INT64_C(1) << 60 ? entries : INT64_C(1) << 60)}, {q_start, 4 * (n_req + 1)},
                         {kv_len, 4 * n_req}, {positions, 4 * n_tokens}, {slots, 8 * n_tokens}, {free_left, 4}};
    const Piece in[] = {{cached, 4 * n_req}, {fresh, 4 * n_req}, {free_blocks, n_req > 0 ? 4 : 0}, {free_count, 4}};
    for (int i = 0; i < 6; ++i) {
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return NDQ_ERR_BAD_ARG;
        for (const Piece& x : in)
            if (overlap(out[i], x)) return NDQ_ERR_BAD_ARG;
    }
    ndq::PlanParams p{};
    p.cached = cached;
    p.fresh = fresh;
    p.free_blocks = free_blocks;
    p.free_count = free_count;
    p.table = block_table;
    p.q_start = q_start;
    p.kv_len = kv_len;
    p.positions = positions;
    p.slots = slots;
    p.free_left = free_left;
    p.n_req = n_req;
    p.n_tokens = n_tokens;
    p.width = table_width;
    p.bs_log2 = bl;
    return ndq::launch_kv_plan(p, stream) == 0 ? NDQ_OK : NDQ_ERR_CUDA;
}

int ndq_kv_append(const ndq_kv_cache* cache, const void* k, const void* v, int in_dtype, int64_t k_stride,
                  int64_t v_stride, const int64_t* slots, int64_t n_tokens, void* stream) {
    ndq::AppendParams p{};
    int rc = check_cache(cache, &p.c);
    if (rc != NDQ_OK) return rc;
    if (n_tokens < 0) return NDQ_ERR_NEGATIVE_DIM;
    if (n_tokens > INT32_MAX || n_tokens > (INT64_C(1) << 33) / cache->kv_heads) return NDQ_ERR_BAD_ARG;  // (the launch's blocks)
    if (in_dtype != NDQ_BFLOAT16 && in_dtype != NDQ_FLOAT16) return NDQ_ERR_BAD_DTYPE;
    if (n_tokens == 0) return NDQ_OK;
    if (!k || !v || !slots) return NDQ_ERR_NULL;
    const int64_t row = static_cast<int64_t>(cache->kv_heads) * cache->head_dim;
    if ((rc = check_rows(k, k_stride, row)) != NDQ_OK || (rc = check_rows(v, v_stride, row)) != NDQ_OK) return rc;
    if (!aligned(slots, 8)) return NDQ_ERR_MISALIGNED;
    p.k = static_cast<const uint16_t*>(k);
    p.v = static_cast<const uint16_t*>(v);
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.slots = slots;
    p.n_tokens = n_tokens;
    return ndq::launch_kv_append(p, cache->head_dim, cache->code_type == NDQ_FLOAT8E4M3FN, in_dtype == NDQ_BFLOAT16,
                                 stream) == 0
               ? NDQ_OK
               : NDQ_ERR_CUDA;
}

size_t ndq_attention_workspace_bytes(int head_dim) {
    return head_dim == 64 || head_dim == 128 ? ndq::attn_workspace_bytes(head_dim) : 0;
}

int ndq_attention_kv8(const ndq_kv_cache* cache, const void* q, int dtype, int64_t n_tokens, int q_heads,
                      int64_t q_stride, const int32_t* block_table, int64_t table_width, const int32_t* kv_len,
                      const int32_t* q_start, int64_t n_req, int64_t max_q, float scale, int64_t window, void* out,
                      float* lse, void* workspace, size_t ws_bytes, void* stream) {
    ndq::AttnParams p{};
    int rc = check_cache(cache, &p.c);
    if (rc != NDQ_OK) return rc;
    if (n_tokens < 0 || n_req < 0 || max_q < 0 || table_width < 0 || window < 0) return NDQ_ERR_NEGATIVE_DIM;
    if (dtype != NDQ_BFLOAT16 && dtype != NDQ_FLOAT16) return NDQ_ERR_BAD_DTYPE;
    if (n_tokens > INT32_MAX / 2 || n_req > INT32_MAX / 2 ||
        table_width > (INT64_C(1) << 30) / cache->block_size)
        return NDQ_ERR_BAD_ARG;
    if (q_heads < 1 || q_heads > 4096 || q_heads % cache->kv_heads != 0 ||
        n_tokens > INT32_MAX / q_heads)
        return NDQ_ERR_BAD_ARG;
    if (!std::isfinite(scale)) return NDQ_ERR_BAD_ARG;
    if (n_tokens == 0 || n_req == 0 || max_q == 0) return NDQ_OK;
    if (!q_start && n_tokens != n_req) return NDQ_ERR_BAD_ARG;
    if (!q || !out || !kv_len || (table_width > 0 && !block_table)) return NDQ_ERR_NULL;
    const int64_t row = static_cast<int64_t>(q_heads) * cache->head_dim;
    if ((rc = check_rows(q, q_stride, row)) != NDQ_OK) return rc;
    if (!aligned(out, 16) || !aligned(lse, 4) || !aligned(block_table, 4) || !aligned(kv_len, 4) ||
        !aligned(q_start, 4))
        return NDQ_ERR_MISALIGNED;
    if (!workspace || !aligned(workspace, 16) || ws_bytes < ndq::attn_workspace_bytes(cache->head_dim))
        return NDQ_ERR_WORKSPACE;
    p.q = static_cast<const uint16_t*>(q);
    p.out = out;
    p.lse = lse;
    p.table = block_table;
    p.kv_len = kv_len;
    p.q_start = q_start;
    p.counters = static_cast<uint32_t*>(workspace);
    p.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + ndq::kAttnCounterBytes);
    p.n_tokens = n_tokens;
    p.n_req = n_req;
    p.q_stride = q_stride;
    p.width = table_width;
    p.window = window > (INT64_C(1) << 30) ? 0 : static_cast<int32_t>(window);  // (no table is that long)
    p.max_q = q_start ? max_q : 1;
    p.q_heads = q_heads;
    p.group = q_heads / cache->kv_heads;
    p.group_shift = -1;
    for (int i = 0; i < 13; ++i)
        if (p.group == 1 << i) p.group_shift = i;
    p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
    p.waits = take_waits();
    return ndq::launch_attention(p, cache->head_dim, cache->code_type == NDQ_FLOAT8E4M3FN, dtype == NDQ_BFLOAT16,
                                 stream) == 0
               ? NDQ_OK
               : NDQ_ERR_CUDA;
}

size_t ndq_lora_workspace_bytes(int64_t M, int64_t max_rank, int64_t K) {
    if (M < 0 || K < 0 || max_rank < 1 || max_rank > 128 || M > INT32_MAX) return 0;
    return ndq::lora_workspace_bytes(M, max_rank, K);
}

int ndq_lora_add(const void* x_bf16, int64_t M, int64_t K, const void* lora_a, const void* lora_b,
                 int64_t n_adapters, int64_t max_rank, int64_t N, const int32_t* ranks, const float* scales,
                 const int32_t* index, const void* base, int dtype, void* y, void* workspace, size_t ws_bytes,
                 void* stream) {
    if (M < 0 || K < 0 || N < 0 || n_adapters < 0) return NDQ_ERR_NEGATIVE_DIM;
    if (dtype != NDQ_FLOAT && dtype != NDQ_BFLOAT16) return NDQ_ERR_BAD_DTYPE;
    if (max_rank < 1 || max_rank > 128 || M > INT32_MAX / 2 || K > INT32_MAX / 2 || N > INT32_MAX / 2 ||
        n_adapters > INT32_MAX / 2 || M > INT32_MAX / max_rank)
        return NDQ_ERR_BAD_ARG;
    if (M == 0 || N == 0) return NDQ_OK;
    if (!base || !y || !index) return NDQ_ERR_NULL;
    if (n_adapters > 0 && (!ranks || !scales || !lora_b || (K > 0 && (!x_bf16 || !lora_a)))) return NDQ_ERR_NULL;
    const uintptr_t el = dtype == NDQ_FLOAT ? 4 : 2;
    if (!aligned(x_bf16, 2) || !aligned(lora_a, 2) || !aligned(lora_b, 2) || !aligned(ranks, 4) ||
        !aligned(scales, 4) || !aligned(index, 4) || !aligned(base, el) || !aligned(y, el))
        return NDQ_ERR_MISALIGNED;
    if (!workspace || !aligned(workspace, 16) || ws_bytes < ndq::lora_workspace_bytes(M, max_rank, K))
        return NDQ_ERR_WORKSPACE;
    ndq::LoraParams p{};
    p.x = static_cast<const uint16_t*>(x_bf16);
    p.a = static_cast<const uint16_t*>(lora_a);
    p.b = static_cast<const uint16_t*>(lora_b);
    p.ranks = ranks;
    p.scales = scales;
    p.index = index;
    p.base = base;
    p.y = y;
    p.t = static_cast<float*>(workspace);
    p.M = M;
    p.K = K;
    p.N = N;
    p.nA = n_adapters;
    p.rmax = max_rank;
    p.waits = take_waits();
    return ndq::launch_lora(p, dtype == NDQ_FLOAT, stream) == 0 ? NDQ_OK : NDQ_ERR_CUDA;
}

int ndq_test_lose_copies(uint32_t wait_limit_us) {
    if (wait_limit_us > 2000000u || (wait_limit_us > 0 && wait_limit_us < 1000u)) return NDQ_ERR_BAD_COUNT;
    t_waits = ndq::Waits{};
    if (wait_limit_us > 0) {
        t_waits.limit_ns = static_cast<uint64_t>(wait_limit_us) * 1000u;
        t_waits.beyond = 16u;
    }
    return NDQ_OK;
}

}  // extern "C"
