// ndq_attn_prefix_prompt.cu -- launcher of the prompt kernel over requests' own
// tokens, joined with the prefixes that they share.
#include "ndq_attn_prompt.cuh"

namespace ndq {

int launch_prefix_own_prompt(PrefixParams p, int head_dim, bool e4m3, bool bf16, int dev, void* stream, bool* launched) {
    const int64_t grid = prompt_grid(p, p.sms);
    *launched = grid > 0;
    if (grid == 0) return 0;
    if (grid < 0) return static_cast<int>(cudaErrorInvalidValue);
    return launch_prompt_of<kAttnOwn>(p, head_dim, e4m3, bf16, static_cast<unsigned>(grid), dev, stream);
}

}  // namespace ndq
