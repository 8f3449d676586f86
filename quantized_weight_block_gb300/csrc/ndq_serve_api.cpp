// ndq_serve_api.cpp -- the serving operators' part of the C ABI declared in
// include/ndq.h: host validation and launches.

#include <cmath>
#include <cstdint>

#include "ndq.h"
#include "ndq_overlap.h"
#include "ndq_rope.h"
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

// Rows of dense heads, 16-byte aligned, `stride` elements of 2 bytes apart.
int check_rows(const void* p, int64_t stride, int64_t row) {
    if (stride < row || stride > (int64_t(1) << 40)) return NDQ_ERR_BAD_ARG;
    if (!aligned(p, 16) || stride % 8 != 0) return NDQ_ERR_MISALIGNED;
    return NDQ_OK;
}

// What the attention calls have in common: their checks and the launch
// descriptor, but for the workspace.  empty: there is nothing to compute.
int check_attention(const ndq_kv_cache* cache, const void* q, int dtype, int64_t n_tokens, int q_heads, int64_t q_stride,
                    const int32_t* block_table, int64_t table_width, const int32_t* kv_len, const int32_t* q_start,
                    int64_t n_req, int64_t max_q, float scale, int64_t window, void* out, float* lse, ndq::AttnParams* d,
                    bool* empty) {
    ndq::AttnParams& p = *d;
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
    *empty = n_tokens == 0 || n_req == 0 || max_q == 0;
    if (*empty) return NDQ_OK;
    if (!q_start && n_tokens != n_req) return NDQ_ERR_BAD_ARG;
    if (!q || !out || !kv_len || (table_width > 0 && !block_table)) return NDQ_ERR_NULL;
    const int64_t row = static_cast<int64_t>(q_heads) * cache->head_dim;
    if ((rc = check_rows(q, q_stride, row)) != NDQ_OK) return rc;
    if (!aligned(out, 16) || !aligned(lse, 4) || !aligned(block_table, 4) || !aligned(kv_len, 4) ||
        !aligned(q_start, 4))
        return NDQ_ERR_MISALIGNED;
    p.q = static_cast<const uint16_t*>(q);
    p.out = out;
    p.lse = lse;
    p.table = block_table;
    p.kv_len = kv_len;
    p.q_start = q_start;
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
    const ndq::Rows out[] = {{block_table, 4 * (entries < INT64_C(1) << 60 ? entries : INT64_C(1) << 60)}, {q_start, 4 * (n_req + 1)},
                         {kv_len, 4 * n_req}, {positions, 4 * n_tokens}, {slots, 8 * n_tokens}, {free_left, 4}};
    const ndq::Rows in[] = {{cached, 4 * n_req}, {fresh, 4 * n_req}, {free_blocks, n_req > 0 ? 4 : 0}, {free_count, 4}};
    for (int i = 0; i < 6; ++i) {
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return NDQ_ERR_BAD_ARG;
        for (const ndq::Rows& x : in)
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
    bool empty = false;
    const int rc = check_attention(cache, q, dtype, n_tokens, q_heads, q_stride, block_table, table_width, kv_len, q_start, n_req,
                                   max_q, scale, window, out, lse, &p, &empty);
    if (rc != NDQ_OK || empty) return rc;
    if (!workspace || !aligned(workspace, 16) || ws_bytes < ndq::attn_workspace_bytes(cache->head_dim))
        return NDQ_ERR_WORKSPACE;
    p.counters = static_cast<uint32_t*>(workspace);
    p.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + ndq::kAttnCounterBytes);
    p.waits = take_waits();
    return ndq::launch_attention(p, cache->head_dim, cache->code_type == NDQ_FLOAT8E4M3FN, dtype == NDQ_BFLOAT16,
                                 stream) == 0
               ? NDQ_OK
               : NDQ_ERR_CUDA;
}

size_t ndq_attention_prefix_workspace_bytes(int head_dim, int64_t n_tokens, int q_heads, int kv_heads) {
    if ((head_dim != 64 && head_dim != 128) || n_tokens < 0 || n_tokens > INT32_MAX / 2 || kv_heads < 1 || q_heads < 1 ||
        q_heads > 4096 || q_heads % kv_heads != 0 || n_tokens > INT32_MAX / q_heads)
        return 0;
    return ndq::prefix_layout(head_dim, n_tokens, q_heads).bytes;
}

int ndq_attention_prefix_kv8(const ndq_kv_cache* cache, const void* q, int dtype, int64_t n_tokens, int q_heads,
                             int64_t q_stride, const int32_t* block_table, int64_t table_width, const int32_t* kv_len,
                             const int32_t* q_start, int64_t n_req, int64_t max_q, const int32_t* group_start,
                             const int32_t* prefix_len, int64_t n_groups, float scale, int64_t window, void* out,
                             float* lse, void* workspace, size_t ws_bytes, void* stream) {
    ndq::PrefixParams p{};
    bool empty = false;
    if (n_groups < 0) return NDQ_ERR_NEGATIVE_DIM;
    const int rc = check_attention(cache, q, dtype, n_tokens, q_heads, q_stride, block_table, table_width, kv_len, q_start, n_req,
                                   max_q, scale, window, out, lse, &p, &empty);
    if (rc != NDQ_OK) return rc;
    if (n_groups > INT32_MAX / 2) return NDQ_ERR_BAD_ARG;
    if (empty) return NDQ_OK;
    if (n_groups > 0 && (!group_start || !prefix_len)) return NDQ_ERR_NULL;
    if (!aligned(group_start, 4) || !aligned(prefix_len, 4)) return NDQ_ERR_MISALIGNED;
    const int D = cache->head_dim;
    const ndq::PrefixLayout at = ndq::prefix_layout(D, n_tokens, q_heads);
    if (!workspace || !aligned(workspace, 256) || ws_bytes < at.bytes) return NDQ_ERR_WORKSPACE;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.counters = static_cast<uint32_t*>(workspace);
    p.parts = reinterpret_cast<float*>(ws + ndq::kAttnCounterBytes);
    p.group_start = group_start;
    p.prefix_len = prefix_len;
    p.n_groups = n_groups;
    p.records = ws + at.records;
    p.own_records = ws + at.own_records;
    p.slots = reinterpret_cast<float*>(ws + at.slots);
    p.own_slots = reinterpret_cast<float*>(ws + at.own_slots);
    p.slot_rows = ndq::prefix_slot_rows(n_tokens, q_heads);
    p.own_rows = ndq::prefix_own_rows(n_tokens, q_heads);
    p.waits = take_waits();
    const bool e4m3 = cache->code_type == NDQ_FLOAT8E4M3FN, bf16 = dtype == NDQ_BFLOAT16;
    const int e = n_groups == 0 ? ndq::launch_attention(p, D, e4m3, bf16, stream) : ndq::launch_attention_prefix(p, D, e4m3, bf16, stream);
    return e == 0 ? NDQ_OK : NDQ_ERR_CUDA;
}

int ndq_qk_norm_rope(const void* q, int q_heads, int64_t q_stride, const void* k, int k_heads, int64_t k_stride, int in_dtype,
                     int64_t n_tokens, int head_dim, int rot_dim, int interleaved, const int32_t* positions,
                     const float* inv_freq, const float* q_weight, const float* k_weight, float eps, void* q_out,
                     int64_t q_out_stride, void* k_out, int64_t k_out_stride, int out_dtype, void* stream) {
    if (n_tokens < 0 || q_heads < 0 || k_heads < 0) return NDQ_ERR_NEGATIVE_DIM;
    if ((in_dtype != NDQ_FLOAT && in_dtype != NDQ_BFLOAT16 && in_dtype != NDQ_FLOAT16) ||
        (out_dtype != NDQ_BFLOAT16 && out_dtype != NDQ_FLOAT16))
        return NDQ_ERR_BAD_DTYPE;
    if (n_tokens > INT32_MAX || q_heads > 4096 || k_heads > 4096 || head_dim < 16 || head_dim > 256 || head_dim % 16 != 0 ||
        rot_dim < 0 || rot_dim > head_dim || rot_dim % 16 != 0 || !std::isfinite(eps) || eps < 0.0f ||
        (interleaved != 0 && interleaved != 1))
        return NDQ_ERR_BAD_ARG;
    if (n_tokens == 0 || q_heads + k_heads == 0) return NDQ_OK;
    if (!positions || (rot_dim > 0 && !inv_freq) || (q_heads > 0 && (!q || !q_out)) || (k_heads > 0 && (!k || !k_out)))
        return NDQ_ERR_NULL;
    if (!aligned(positions, 4) || !aligned(inv_freq, 4) || !aligned(q_weight, 4) || !aligned(k_weight, 4))
        return NDQ_ERR_MISALIGNED;
    struct Side {
        const void* x;
        int heads;
        int64_t stride;
        void* y;
        int64_t y_stride;
    };
    const Side sides[] = {{q, q_heads, q_stride, q_out, q_out_stride}, {k, k_heads, k_stride, k_out, k_out_stride}};
    for (const Side& s : sides) {
        if (s.heads == 0) continue;
        const int64_t row = static_cast<int64_t>(s.heads) * head_dim;
        // (rows of 4-byte values are 16-byte aligned every fourth; one rule for all types)
        int rc = check_rows(s.x, s.stride, row);
        if (rc == NDQ_OK) rc = check_rows(s.y, s.y_stride, row);
        if (rc != NDQ_OK) return rc;
        if (s.x == s.y && (in_dtype != out_dtype || s.stride != s.y_stride)) return NDQ_ERR_BAD_ARG;
    }
    // An output may be its own input; otherwise it is read before and after it is
    // written, by different warps.  (Rows that lie between one another's are apart:
    // queries and keys of one fused projection.)
    const int64_t el = in_dtype == NDQ_FLOAT ? 4 : 2;
    ndq::Rows in[2], out[2];
    for (int i = 0; i < 2; ++i) {
        const int64_t row = static_cast<int64_t>(sides[i].heads) * head_dim, n = sides[i].heads > 0 ? n_tokens : 0;
        in[i] = {sides[i].x, row * el, n, sides[i].stride * el};
        out[i] = {sides[i].y, row * 2, n, sides[i].y_stride * 2};
    }
    const ndq::Rows small[] = {{positions, 4 * n_tokens}, {inv_freq, 2 * rot_dim}, {q_weight, q_heads > 0 && q_weight ? 4 * head_dim : 0},
                               {k_weight, k_heads > 0 && k_weight ? 4 * head_dim : 0}};
    if (overlap(out[0], out[1])) return NDQ_ERR_BAD_ARG;
    for (int i = 0; i < 2; ++i) {
        if ((in[i].p != out[i].p && overlap(out[i], in[i])) || overlap(out[i], in[1 - i])) return NDQ_ERR_BAD_ARG;
        for (const ndq::Rows& x : small)
            if (overlap(out[i], x)) return NDQ_ERR_BAD_ARG;
    }
    ndq::RopeParams p{};
    p.q = q;
    p.k = k;
    p.q_out = q_out;
    p.k_out = k_out;
    p.q_weight = q_weight;
    p.k_weight = k_weight;
    p.inv_freq = inv_freq;
    p.positions = positions;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.q_out_stride = q_out_stride;
    p.k_out_stride = k_out_stride;
    p.n_tokens = n_tokens;
    p.q_heads = q_heads;
    p.k_heads = k_heads;
    p.head_dim = head_dim;
    p.rot_dim = rot_dim;
    p.interleaved = interleaved;
    p.eps = eps;
    return ndq::launch_rope(p, in_dtype == NDQ_FLOAT ? 0 : in_dtype == NDQ_BFLOAT16 ? 1 : 2, out_dtype == NDQ_BFLOAT16, stream) == 0
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
