// ndq_attn_prefix_rows.cu -- launcher of the few-row kernel over requests' own
// tokens, whose parts are joined with those of the prefixes that they share.
#include "ndq_attn_rows.cuh"

namespace ndq {

int launch_prefix_own_rows(const PrefixParams& p, int head_dim, bool e4m3, bool bf16, int dev, void* stream) {
    return launch_rows_of<kAttnOwn>(p, head_dim, e4m3, bf16, dev, p.sms, stream);
}

}  // namespace ndq
