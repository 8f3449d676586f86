// Packed embedding lookup: the codebook formats.
#include "ndq_embed.cuh"

namespace ndq {
EmbedKernelFn embed_iq(int kfmt, uint32_t* seg) {
    switch (kfmt) {
        case KF_IQ2_XXS: return embed_kernel<KF_IQ2_XXS>(seg);
        case KF_IQ2_XS: return embed_kernel<KF_IQ2_XS>(seg);
        case KF_IQ2_S: return embed_kernel<KF_IQ2_S>(seg);
        case KF_IQ3_XXS: return embed_kernel<KF_IQ3_XXS>(seg);
        case KF_IQ3_S: return embed_kernel<KF_IQ3_S>(seg);
        case KF_IQ1_S: return embed_kernel<KF_IQ1_S>(seg);
        case KF_IQ1_M: return embed_kernel<KF_IQ1_M>(seg);
        case KF_IQ4_XS: return embed_kernel<KF_IQ4_XS>(seg);
        default: return nullptr;
    }
}
}  // namespace ndq
