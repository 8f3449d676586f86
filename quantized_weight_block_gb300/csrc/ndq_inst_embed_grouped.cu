// Packed embedding lookup: the other gguf formats and the NInfer ones.
#include "ndq_embed.cuh"

namespace ndq {
EmbedKernelFn embed_grouped(int kfmt, uint32_t* seg) {
    switch (kfmt) {
        case KF_GGUF_NVFP4: return embed_kernel<KF_GGUF_NVFP4>(seg);
        case KF_NVFP4: return embed_kernel<KF_NVFP4>(seg);
        case KF_Q4_G64: return embed_kernel<KF_Q4_G64>(seg);
        case KF_Q1_0: return embed_kernel<KF_Q1_0>(seg);
        case KF_Q2_0: return embed_kernel<KF_Q2_0>(seg);
        case KF_Q5_G64: return embed_kernel<KF_Q5_G64>(seg);
        case KF_Q6_G64: return embed_kernel<KF_Q6_G64>(seg);
        case KF_T2_G128: return embed_kernel<KF_T2_G128>(seg);
        case KF_FP8_ROW_BF16: return embed_kernel<KF_FP8_ROW_BF16>(seg);
        case KF_FP8_ROW_FP16: return embed_kernel<KF_FP8_ROW_FP16>(seg);
        default: return nullptr;
    }
}
}  // namespace ndq
