// Instantiations of the attention kernel for one head size (QG_ATTN_D): fp32 activations with
// row tiles of 4, 8, 12 and (64 wide) 16, bf16 with 8 and 16.
#include "attention.cuh"

namespace qg {

#define QG_CAT2(a, b) a##b
#define QG_CAT(a, b) QG_CAT2(a, b)

AttnKernel QG_CAT(attention_lookup_, QG_ATTN_D)(int act, int rows) {
    constexpr int D = QG_ATTN_D;
    if (act == QG_ACT_BF16)
        return rows <= 8 ? attn_kernel<__nv_bfloat16, D, 1, kOne>() : attn_kernel<__nv_bfloat16, D, 2, kOne>();
    if constexpr (D == 64)
        if (rows > 12) return attn_kernel<float, D, 2, kTwice>();
    return rows <= 4 ? attn_kernel<float, D, 1, kSide>() : rows <= 8 ? attn_kernel<float, D, 1, kTwice>()
                                                                    : attn_kernel<float, D, 3, kSide>();
}

}  // namespace qg
