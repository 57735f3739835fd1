// qg_prompt_attention: argument checks, tensor maps, launch.  Formulas and argument rules are in
// include/qgemv.h; the kernels in prompt_attention_bf16.cu and prompt_attention_f32.cu.
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "kv_layout.h"
#include "prompt_attention.cuh"

namespace qg {

namespace {

constexpr int kMostPrompts = 16384, kMostGroup = 128;

// Boxes of `tokens` tokens, `heads` heads and 64 values of [n_tok][n_heads][D], 16-bit.
qg_status encode_heads(CUtensorMap* map, const void* p, int64_t n_tok, int n_heads, int D, int64_t stride, int heads, int tokens) {
    const EncodeTiledFn enc = encode_tiled();
    if (!enc) return QG_ECUDA;
    const cuuint64_t dims[3] = {cuuint64_t(D), cuuint64_t(n_heads), cuuint64_t(n_tok)};
    const cuuint64_t strides[2] = {cuuint64_t(D) * 2, cuuint64_t(stride) * 2};
    const cuuint32_t box[3] = {64, cuuint32_t(heads), cuuint32_t(tokens)};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? QG_OK : QG_ECUDA;
}

// What a call needs of its workspace: with fp32 the staged terms and their powers of two.
struct PromptSpace { size_t q, k, v, qscale, kscale, vscale, total; };
PromptSpace prompt_space(qg_act act, int64_t n_tok, int n_heads, int n_kv, int D) {
    PromptSpace s{};
    if (act == QG_ACT_F32) {
        auto take = [&](size_t bytes) { const size_t at = s.total; s.total = (at + bytes + 255) / 256 * 256; return at; };
        const size_t n = size_t(n_tok);
        s.q = take(n * size_t(n_heads) * size_t(D) * 4);
        s.k = take(n * size_t(n_kv) * size_t(D) * 4);
        s.v = take(n * size_t(n_kv) * size_t(D) * 4);
        s.qscale = take(n * size_t(n_heads) * 4);
        s.kscale = take(n * size_t(n_kv) * 4);
        s.vscale = take(n * size_t(n_kv) * 4);
    }
    s.total = std::max<size_t>(s.total, 256);
    return s;
}

}  // namespace
}  // namespace qg

using namespace qg;

extern "C" {

size_t qg_prompt_attention_workspace_bytes(qg_act act, int64_t n_tok, int n_heads, int n_kv_heads, int head_dim) {
    if ((act != QG_ACT_F32 && act != QG_ACT_BF16) || n_tok < 0 || n_tok > (int64_t(1) << 31) - 1025 || n_kv_heads < 1 ||
        n_heads < 1 || n_heads > 65535 || n_heads % n_kv_heads != 0 || !kv_dim_ok(head_dim))
        return 0;
    return prompt_space(act, n_tok, n_heads, n_kv_heads, head_dim).total;
}

qg_status qg_prompt_attention(qg_act act, const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                              int64_t v_stride, int64_t n_tok, int n_heads, int n_kv_heads, int head_dim, const int32_t* cu_seq,
                              int n_seq, int longest, int window, float scale, void* out, int64_t out_stride, float* lse,
                              void* workspace, size_t workspace_bytes, void* stream) {
    const int64_t most = (int64_t(1) << 31) - 1;
    if (act != QG_ACT_F32 && act != QG_ACT_BF16) return QG_EINVAL;
    if (n_heads < 1 || n_heads > 65535 || n_kv_heads < 1 || n_heads % n_kv_heads != 0 || !kv_dim_ok(head_dim)) return QG_EINVAL;
    if (n_tok < 0 || n_tok > most - 1024 || n_seq < 0 || longest < 1 || window < 0 || !std::isfinite(scale)) return QG_EINVAL;
    const int group = n_heads / n_kv_heads;
    if (n_seq > kMostPrompts || group > kMostGroup) return QG_EUNSUPPORTED;
    const size_t need = qg_prompt_attention_workspace_bytes(act, n_tok, n_heads, n_kv_heads, head_dim);
    if (!workspace || workspace_bytes < need) return QG_EWORKSPACE;
    if (!aligned(workspace, 16)) return QG_EALIGN;
    if (n_tok == 0 || n_seq == 0) return QG_OK;
    if (!q || !k || !v || !out || !cu_seq || out == q || out == k || out == v) return QG_EINVAL;
    const int64_t width = int64_t(n_heads) * head_dim, kv_width = int64_t(n_kv_heads) * head_dim, size = act == QG_ACT_F32 ? 4 : 2;
    if (q_stride < width || out_stride < width || k_stride < kv_width || v_stride < kv_width) return QG_EINVAL;
    if (q_stride > most || out_stride > most || k_stride > most || v_stride > most) return QG_EINVAL;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || q_stride * size % 16 != 0 ||
        k_stride * size % 16 != 0 || v_stride * size % 16 != 0 || out_stride * size % 16 != 0 || !aligned(cu_seq, 4) || !aligned(lse, 4))
        return QG_EALIGN;
    const int tokens = 128 / group;
    const bool f32 = act == QG_ACT_F32;
    const PromptKernel kern = f32 ? prompt_f32(head_dim) : prompt_bf16(head_dim);
    const int64_t items = (n_tok / tokens + n_seq) * n_kv_heads * kern.parts;
    if (items > most - 65536 || (f32 && 2 * n_tok > most)) return QG_EUNSUPPORTED;
    int dev = 0, sms = 0, optin = 0;
    PromptArgs a{};
    qg_status st = device_info(&dev, &sms, &optin, &a.status);
    if (st != QG_OK) return st;
    const int resident = blocks_per_sm(kern.fn, dev, optin, kern.threads, size_t(kern.smem));
    if (resident < 1) return QG_EUNSUPPORTED;
    if (f32) {
        const PromptSpace sp = prompt_space(act, n_tok, n_heads, n_kv_heads, head_dim);
        uint8_t* const ws = static_cast<uint8_t*>(workspace);
        PromptStage p{};
        p.q = static_cast<const float*>(q), p.k = static_cast<const float*>(k), p.v = static_cast<const float*>(v);
        p.q_stride = q_stride, p.k_stride = k_stride, p.v_stride = v_stride;
        p.cu_seq = cu_seq;
        p.q_out = reinterpret_cast<uint16_t*>(ws + sp.q), p.k_out = reinterpret_cast<uint16_t*>(ws + sp.k);
        p.v_out = reinterpret_cast<uint16_t*>(ws + sp.v);
        p.qscale = reinterpret_cast<float*>(ws + sp.qscale), p.kscale = reinterpret_cast<float*>(ws + sp.kscale);
        p.vscale = reinterpret_cast<float*>(ws + sp.vscale);
        p.n_tok = int(n_tok), p.n_seq = n_seq, p.n_heads = n_heads, p.n_kv = n_kv_heads;
        a.qscale = p.qscale, a.kscale = p.kscale, a.vscale = p.vscale;
        st = encode_heads(&a.qmap, p.q_out, 2 * n_tok, n_heads, head_dim, width, group, tokens);
        if (st == QG_OK) st = encode_heads(&a.kmap, p.k_out, 2 * n_tok, n_kv_heads, head_dim, kv_width, 1, kern.tile_keys);
        if (st == QG_OK) st = encode_heads(&a.vmap, p.v_out, 2 * n_tok, n_kv_heads, head_dim, kv_width, 1, kern.tile_keys);
        if (st == QG_OK) st = prompt_stage(head_dim, p, stream);
    } else {
        st = encode_heads(&a.qmap, q, n_tok, n_heads, head_dim, q_stride, group, tokens);
        if (st == QG_OK) st = encode_heads(&a.kmap, k, n_tok, n_kv_heads, head_dim, k_stride, 1, kern.tile_keys);
        if (st == QG_OK) st = encode_heads(&a.vmap, v, n_tok, n_kv_heads, head_dim, v_stride, 1, kern.tile_keys);
    }
    if (st != QG_OK) return st;
    a.v = v;
    a.v_stride = v_stride;
    a.cu_seq = cu_seq;
    a.out = out;
    a.lse = lse;
    a.out_stride = out_stride;
    a.n_tok = int(n_tok);
    a.n_seq = n_seq;
    a.n_heads = n_heads;
    a.n_kv = n_kv_heads;
    a.group = group;
    a.tokens = tokens;
    a.window = window;
    a.asks = items > int64_t(resident) * sms;
    // (bf16, zero: the smallest number instead, which leaves masked scores at -infinity and others, the
    // largest fp32 number among them, below 2^-21.)
    a.c = std::max(std::fabs(scale) * kLog2e, f32 ? 0.0f : FLT_TRUE_MIN);
    a.negate = scale < 0.0f ? 1u << 13 : 0u;
    a.wait_limit = wait_limit();
    a.drain_limit = std::max<uint32_t>(a.wait_limit, 1u << 16);
    a.extra_tx = test_extra_tx();
    void* params[] = {&a};
    return launch_after(kern.fn, int(items), kern.threads, size_t(kern.smem), 1, f32, params, stream);
}

}  // extern "C"
