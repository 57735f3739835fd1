// Byte layout of the 4-bit key/value cache, shared by the kernels that write and read it.
//
// The cache is a pool of pages of `page_tokens` tokens (a multiple of 16).  A page holds,
// per key/value head, page_tokens / 16 records; a record holds 16 tokens of one head, keys
// and values, so that a tile of keys and its values is one contiguous piece of memory (one
// bulk copy).  With G = head_dim / 32 blocks per token and head, in sets of I = min(G, 4):
//
//   key codes    [G / I][16 tokens][4 c][I] uint32: nibble j of word (t, c, g) is dim 32 g + 8 c + j
//   key scales   [8 token pairs][G][2 tokens] fp16
//   value codes  [G / I][2 halves][8 r][4 pairs of the half][I][2 tokens] uint16: nibble j of
//                halfword (t, r, g) is dim 32 g + 4 r + j
//   value scales as the key scales
//
// The orders are those in which the lanes of a warp read matrix operands: lane 4 r + c reads
// key r's words of column group c as one 16-byte load (four blocks of the head), and for the
// token pair c the halfwords of row r of both tokens as one 16-byte load, so no lane needs
// another lane's bytes and no load conflicts in shared memory.
#pragma once

#include <cstdint>

#include "../../include/qgemv.h"

namespace qg {

constexpr int kRecordTokens = 16;

__host__ __device__ constexpr int kv_groups(int D) { return D / 32; }
__host__ __device__ constexpr int kv_set(int D) { return kv_groups(D) < 4 ? kv_groups(D) : 4; }
__host__ __device__ constexpr int kv_record_bytes(int D) { return 18 * D; }
__host__ __device__ constexpr int kv_k_scales(int D) { return 8 * D; }
__host__ __device__ constexpr int kv_v_codes(int D) { return 9 * D; }
__host__ __device__ constexpr int kv_v_scales(int D) { return 17 * D; }

// Byte of the key word (token t of the record, column group c, block g), of the value
// halfword (t, r, g) and of a scale (t, g) within their parts.
__host__ __device__ constexpr int kv_key_word(int D, int t, int c, int g) {
    return ((g / kv_set(D) * 16 + t) * 4 + c) * kv_set(D) * 4 + g % kv_set(D) * 4;
}
__host__ __device__ constexpr int kv_value_half(int D, int t, int r, int g) {
    return ((((g / kv_set(D) * 2 + t / 8) * 8 + r) * 4 + t / 2 % 4) * kv_set(D) + g % kv_set(D)) * 4 + t % 2 * 2;
}
__host__ __device__ constexpr int kv_scale(int D, int t, int g) { return ((t / 2) * kv_groups(D) + g) * 4 + t % 2 * 2; }

inline bool kv_dim_ok(int D) { return D == 64 || D == 128 || D == 256; }

// The cache description's own checks (no pointer is read).
inline qg_status kv_check(const qg_cache* c) {
    if (!c || !c->data || !kv_dim_ok(c->head_dim) || c->n_kv_heads < 1 || c->n_kv_heads > 65535 || c->n_pages < 1 ||
        c->n_pages > (int64_t(1) << 31) - 1 || c->page_tokens < 16 || c->page_tokens > 65536 ||
        c->page_tokens % kRecordTokens != 0)
        return QG_EINVAL;
    return (reinterpret_cast<uintptr_t>(c->data) & 15) != 0 ? QG_EALIGN : QG_OK;
}

constexpr unsigned kStatusBadPage = 8u;       // a slot or page outside the cache, or a table row too short
constexpr unsigned kStatusBadLength = 16u;    // lengths, counts or positions that do not fit the call
constexpr unsigned kStatusNoPages = 32u;      // the list of free pages ran out

}  // namespace qg
