// C ABI of the attention over the 4-bit cache: validation, row tile and ring depth, launch.
// The operation and every argument rule are documented in include/qgemv.h.
#include <algorithm>
#include <cmath>

#include "attention.cuh"
#include "qgemv_host.h"

namespace qg {

AttnKernel attention_lookup_64(int act, int rows);
AttnKernel attention_lookup_128(int act, int rows);
AttnKernel attention_lookup_256(int act, int rows);

namespace {

AttnKernel lookup(int act, int D, int rows) {
    return D == 64 ? attention_lookup_64(act, rows) : D == 128 ? attention_lookup_128(act, rows)
                                                               : attention_lookup_256(act, rows);
}

// Rows of a tile for `rows` rows of a request and key/value head; a tile is one pass over the
// keys.  Measured on 12 requests of up to 20000 keys, us:
//   bf16: a pass of 16 rows costs 1.6 to 1.8 of 8, so 16, unless that leaves half a tile empty
//     (24 rows: 128 wide 75 with three tiles of 8, 93 with two of 16; 32 rows: 98 and 93).
//   fp32, 128 and 256 wide: a tile of 12 (three of one term beside the other) costs 1.5 of 8 and is
//     the better one where it is enough (12 rows: 54 against 63 with two of 8; 24 rows: 94 and 90; heads
//     of 256: 62 and 67; 102 and 92).  A tile of 16 cost more than two of 8 (70 and 63; 80 and 67).
//   fp32, 64 wide: what a pass costs whatever its rows weighs more: as few passes of up to 16 as it
//     takes, in equal shares (16 rows: 66, with two of 8 86; 24 rows: 103, with three of 8 125).
int row_tile(int act, int D, int64_t rows) {
    const int64_t eights = (rows + 7) / 8, passes = (rows + 15) / 16;
    if (eights == 1) return int(rows);
    if (act == QG_ACT_BF16) return eights % 2 != 0 && eights <= 5 ? 8 : 16;
    if (D == 64) return int((rows + passes - 1) / passes);
    return rows <= 12 ? 12 : 8;
}

// Floats of all partials of a grid of CTAs: two per CTA, one per warp.
size_t partial_floats(const AttnKernel& k, int grid) { return size_t(grid) * size_t(2 + k.warps) * size_t(k.partial); }

}  // namespace
}  // namespace qg

using namespace qg;

extern "C" {

size_t qg_attention_workspace_bytes(int n_heads, int n_kv_heads, int head_dim) {
    if (!kv_dim_ok(head_dim) || n_kv_heads < 1 || n_kv_heads > 65535 || n_heads < 1 || n_heads > 65535 ||
        n_heads % n_kv_heads != 0)
        return 0;
    size_t most = 0;
    for (int act = 0; act < 2; ++act)
        for (int rows = 4; rows <= 16; rows += 4)
            most = std::max(most, partial_floats(lookup(act, head_dim, rows), kAttnGrid));
    return size_t(QG_ATTENTION_ZERO_BYTES) + most * sizeof(float);
}

qg_status qg_attention(const qg_cache* cache, qg_act act, const void* q, int64_t q_stride, int64_t n_tok, int n_heads,
                       const int32_t* table, int64_t table_stride, const int32_t* seq_len, const int32_t* cu_new,
                       int n_req, int max_new, int window, const uint32_t* span_mask, float scale, void* out,
                       int64_t out_stride, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
    qg_status st = kv_check(cache);
    if (st != QG_OK) return st;
    const int D = cache->head_dim, n_kv = cache->n_kv_heads;
    const int64_t most = (int64_t(1) << 31) - 1;
    if (act != QG_ACT_F32 && act != QG_ACT_BF16) return QG_EINVAL;
    if (n_heads < 1 || n_heads > 65535 || n_heads % n_kv != 0 || n_req < 0 || n_tok < 0 || n_tok > most || max_new < 1 ||
        window < 0 || !std::isfinite(scale) || table_stride < 0 || table_stride > most)
        return QG_EINVAL;
    if (n_req > kMaxAttnReq) return QG_EUNSUPPORTED;
    if (!workspace || workspace_bytes < qg_attention_workspace_bytes(n_heads, n_kv, D)) return QG_EWORKSPACE;
    if (!aligned(workspace, 16)) return QG_EALIGN;
    if (n_req == 0 || n_tok == 0) return QG_OK;
    if (!q || !out || !table || !seq_len || !cu_new) return QG_EINVAL;
    const int64_t width = int64_t(n_heads) * D, size = act == QG_ACT_F32 ? 4 : 2;
    if (q_stride < width || out_stride < width) return QG_EINVAL;
    if (!aligned(q, 16) || !aligned(out, 16) || q_stride * size % 16 != 0 || out_stride * size % 16 != 0 ||
        !aligned(table, 4) || !aligned(seq_len, 4) || !aligned(cu_new, 4) || !aligned(span_mask, 4) || !aligned(lse, 4))
        return QG_EALIGN;
    int dev = 0, sms = 0, optin = 0;
    AttnArgs a{};
    st = device_info(&dev, &sms, &optin, &a.status);
    if (st != QG_OK) return st;
    const int group = n_heads / n_kv;
    const int64_t all_rows = int64_t(max_new) * group;
    AttnKernel k{};
    int depth = 0;
    auto fits = [&](int d) { return size_t(k.smem(n_req, d)) + kStaticSmemReserve <= size_t(optin); };
    // The deepest ring (2 to 8 stages per warp) that fits one CTA per SM; a long list of requests
    // may leave room only for fewer rows at a time.
    for (int rows = row_tile(act, D, all_rows); rows >= 1 && depth < 2; rows -= 4) {
        k = lookup(act, D, rows);
        for (depth = 8; depth >= 2 && !fits(depth); --depth) {}
    }
    if (depth < 2) return QG_EUNSUPPORTED;
    const int smem = k.smem(n_req, depth);
    // Records are numbered with 32 bits on the device.
    if (cache->n_pages * n_kv > ((int64_t(1) << 32) - 1) / (cache->page_tokens / kRecordTokens)) return QG_EUNSUPPORTED;
    if (blocks_per_sm(k.fn, dev, optin, 32 * k.warps, size_t(smem)) < 1) return QG_EUNSUPPORTED;
    a.data = static_cast<const uint8_t*>(cache->data);
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.table = table;
    a.seq_len = seq_len;
    a.cu_new = cu_new;
    a.span_mask = span_mask;
    a.tickets = static_cast<uint32_t*>(workspace);
    a.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + QG_ATTENTION_ZERO_BYTES);
    a.q_stride = q_stride;
    a.out_stride = out_stride;
    a.table_stride = table_stride;
    a.n_tok = n_tok;
    a.n_pages = cache->n_pages;
    a.n_req = n_req;
    a.n_heads = n_heads;
    a.n_kv = n_kv;
    a.group = group;
    a.page_records = cache->page_tokens / kRecordTokens;
    a.group_inv = group == 1 ? 0xFFFFFFFFu : uint32_t((uint64_t(1) << 32) / uint32_t(group));
    a.page_inv = a.page_records == 1 ? 0xFFFFFFFFu : uint32_t((uint64_t(1) << 32) / uint32_t(a.page_records));
    a.window = window;
    a.depth = depth;
    a.scale_log2 = float(std::frexp((scale == 0.0f ? 1.0 : std::fabs(double(scale))) * 1.4426950408889634, &a.scale_exp));
    a.scale_sign = scale > 0.0f ? 1.0f : scale < 0.0f ? -1.0f : 0.0f;
    a.wait_limit = wait_limit();
    a.drain_limit = std::max<uint32_t>(a.wait_limit, 1u << 16);
    a.test_extra_tx = test_extra_tx();
    void* params[] = {&a};
    return launch_early(k.fn, std::min(sms, kAttnGrid), 32 * k.warps, size_t(smem), 1, params, stream);
}

}  // extern "C"
