// Packed embedding lookup: the K-quants and the ternary formats.
#include "ndq_embed.cuh"

namespace ndq {
EmbedKernelFn embed_kquant(int kfmt, uint32_t* seg) {
    switch (kfmt) {
        case KF_Q2_K: return embed_kernel<KF_Q2_K>(seg);
        case KF_Q3_K: return embed_kernel<KF_Q3_K>(seg);
        case KF_Q4_K: return embed_kernel<KF_Q4_K>(seg);
        case KF_Q5_K: return embed_kernel<KF_Q5_K>(seg);
        case KF_Q6_K: return embed_kernel<KF_Q6_K>(seg);
        case KF_Q8_K: return embed_kernel<KF_Q8_K>(seg);
        case KF_TQ1_0: return embed_kernel<KF_TQ1_0>(seg);
        case KF_TQ2_0: return embed_kernel<KF_TQ2_0>(seg);
        default: return nullptr;
    }
}
}  // namespace ndq
