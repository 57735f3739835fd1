// Instantiations of the attention kernel for one head size (QG_ATTN_D): fp32 activations with
// row tiles of 4, 8, 12 and 16, bf16 with 8 and 16.
#include "attention.cuh"

namespace qg {

#define QG_CAT2(a, b) a##b
#define QG_CAT(a, b) QG_CAT2(a, b)

AttnKernel QG_CAT(attention_lookup_, QG_ATTN_D)(int act, int tiles) {
    constexpr int D = QG_ATTN_D;
    if (act == QG_ACT_BF16)
        return tiles == 1 ? attn_kernel<__nv_bfloat16, D, 1, 1>() : attn_kernel<__nv_bfloat16, D, 2, 1>();
    return tiles == 1 ? attn_kernel<float, D, 1, 2>() : tiles == 2 ? attn_kernel<float, D, 2, 2>()
         : tiles == 3 ? attn_kernel<float, D, 3, 2>() : attn_kernel<float, D, 4, 2>();
}

}  // namespace qg
