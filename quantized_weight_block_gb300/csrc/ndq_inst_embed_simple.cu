// Packed embedding lookup: the formats of 32-value blocks.
#include "ndq_embed.cuh"

namespace ndq {
EmbedKernelFn embed_simple(int kfmt, uint32_t* seg) {
    switch (kfmt) {
        case KF_Q4_0: return embed_kernel<KF_Q4_0>(seg);
        case KF_Q4_1: return embed_kernel<KF_Q4_1>(seg);
        case KF_Q5_0: return embed_kernel<KF_Q5_0>(seg);
        case KF_Q5_1: return embed_kernel<KF_Q5_1>(seg);
        case KF_Q8_0: return embed_kernel<KF_Q8_0>(seg);
        case KF_Q8_1: return embed_kernel<KF_Q8_1>(seg);
        case KF_IQ4_NL: return embed_kernel<KF_IQ4_NL>(seg);
        case KF_MXFP4: return embed_kernel<KF_MXFP4>(seg);
        default: return nullptr;
    }
}
}  // namespace ndq
