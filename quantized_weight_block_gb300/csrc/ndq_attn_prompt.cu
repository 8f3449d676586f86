// ndq_attn_prompt.cu -- launcher of the prompt kernel (ndq_attn_prompt.cuh)
// over all that rows see.
#include "ndq_attn_prompt.cuh"

namespace ndq {

int launch_attention_prompt(AttnParams p, int head_dim, bool e4m3, bool bf16, int dev, int sms, void* stream,
                            bool* launched) {
    const int64_t grid = prompt_grid(p, sms);
    *launched = grid > 0;
    if (grid == 0) return 0;
    if (grid < 0) return static_cast<int>(cudaErrorInvalidValue);
    return launch_prompt_of<kAttnAll>(p, head_dim, e4m3, bf16, static_cast<unsigned>(grid), dev, stream);
}

}  // namespace ndq
