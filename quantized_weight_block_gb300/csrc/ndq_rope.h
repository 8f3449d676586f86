// ndq_rope.h -- launch descriptor of the norm and rotation of heads, shared by
// the host ABI (ndq_serve_api.cpp) and its kernels.  Not part of the public ABI.
#pragma once

#include <cstdint>

namespace ndq {

struct RopeParams {
    const void* q;  // [n_tokens, q_heads, head_dim], rows q_stride elements apart
    const void* k;
    void* q_out;
    void* k_out;
    const float* q_weight;  // or nullptr: no norm
    const float* k_weight;
    const float* inv_freq;  // [rot_dim / 2]
    const int32_t* positions;
    int64_t q_stride;
    int64_t k_stride;
    int64_t q_out_stride;
    int64_t k_out_stride;
    int64_t n_tokens;
    int32_t q_heads;
    int32_t k_heads;
    int32_t head_dim;  // a multiple of 16 up to 256
    int32_t rot_dim;   // a multiple of 16 up to head_dim
    int32_t interleaved;
    int32_t parts;     // (set by the launcher) warps of a token
    float eps;
};
// in: 0 binary32, 1 bfloat16, 2 binary16.  Returns 0 or a CUDA error code.
int launch_rope(RopeParams p, int in, bool bf16, void* stream);

}  // namespace ndq
