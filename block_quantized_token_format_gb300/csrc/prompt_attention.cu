#include "qgemv_host.h"
extern "C" {
size_t qg_prompt_attention_workspace_bytes(qg_act, int64_t, int, int, int) { return 256; }
qg_status qg_prompt_attention(qg_act act, const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                              int64_t v_stride, int64_t n_tok, int n_heads, int n_kv_heads, int head_dim, const int32_t* cu_seq,
                              int n_seq, int longest, int window, float scale, void* out, int64_t out_stride, float* lse,
                              void* workspace, size_t workspace_bytes, void* stream) { return QG_EUNSUPPORTED; }
}
