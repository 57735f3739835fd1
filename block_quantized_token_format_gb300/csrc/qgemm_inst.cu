// Instantiations of the many-token product for one weight format (QG_INST_FMT): bf16
// activations (with one chain of sums and with several) and fp32 ones.
#include "qgemm.cuh"

namespace qg {

#define QG_CAT2(a, b) a##b
#define QG_CAT(a, b) QG_CAT2(a, b)

const void* QG_CAT(qgemm_lookup_fmt, QG_INST_FMT)(bool f32, bool chains) {
    return f32 ? (const void*)&qgemm_kernel<QG_INST_FMT, true, false>
               : chains ? (const void*)&qgemm_kernel<QG_INST_FMT, false, true> : (const void*)&qgemm_kernel<QG_INST_FMT, false, false>;
}

}  // namespace qg
