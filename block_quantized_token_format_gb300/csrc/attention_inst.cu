// Instantiations of the attention kernel for one head size (QG_ATTN_D): fp32 activations with
// 8 or 16 rows per tile, bf16 with 16.
#include "attention.cuh"

namespace qg {

#define QG_CAT2(a, b) a##b
#define QG_CAT(a, b) QG_CAT2(a, b)

AttnKernel QG_CAT(attention_lookup_, QG_ATTN_D)(int act, int rows) {
    constexpr int D = QG_ATTN_D;
    if (act == QG_ACT_BF16) return attn_kernel<__nv_bfloat16, D, 16, 1>();
    return rows == 8 ? attn_kernel<float, D, 8, 2>() : attn_kernel<float, D, 16, 2>();
}

}  // namespace qg
