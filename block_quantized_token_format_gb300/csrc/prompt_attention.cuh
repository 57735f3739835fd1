// Causal attention of packed prompts (qg_prompt_attention): what the bf16 and the fp32 kernel share.
// Formulas and argument rules are in include/qgemv.h.
//
// An item is 128 rows of the products: T = 128 / group tokens of one prompt times the `group` query
// heads that read one key/value head (row = token * group + head), so short prompts fill rows with
// heads and every key tile serves all of them.  A CTA takes one item, later tokens (more keys) first.
// Items are numbered without a prefix sum: prompt r's begin at slot cu_seq[r] / T + r, which leaves
// room for each prompt's last, partly filled item; a slot beyond a prompt's items has no work.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "umma.cuh"

namespace qg {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr unsigned kPromptBadLength = 16u;       // QG_DEVICE_BAD_LENGTH

struct PromptArgs {
    CUtensorMap qmap, kmap, vmap;
    const void *k, *v;
    long long k_stride, v_stride;
    const int32_t* cu_seq;
    void* out;
    float* lse;
    long long out_stride;
    int n_tok, n_seq, n_heads, n_kv, group, tokens, window;      // tokens: T
    float c;                       // |scale| log2 e
    uint32_t negate;               // of the instruction descriptor, where scale < 0
    const float *kscale, *vscale;  // fp32: powers of two
    unsigned int* status;
    uint32_t wait_limit, drain_limit, extra_tx;
};

// One item's place: prompt's first token and length, first query (of the prompt), key/value head.
struct PromptItem { int seq0, len, t0, head; };

// False: nothing to do.
__device__ __forceinline__ bool prompt_item(const PromptArgs& a, int slot, int head, PromptItem& it) {
    int lo = 0, hi = a.n_seq;                            // the last prompt that begins at or before the slot
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.cu_seq[mid] / a.tokens + mid <= slot) lo = mid; else hi = mid;
    }
    const int from = a.cu_seq[lo], to = a.cu_seq[lo + 1];
    if (from < 0 || to < from || to > a.n_tok) return false;         // (reported by prompt_check)
    const long long t0 = (long long)(slot - (from / a.tokens + lo)) * a.tokens;
    it.seq0 = from;
    it.len = to - from;
    it.t0 = int(min(t0, 0x7FFFFFFFll));
    it.head = head;
    return t0 >= 0 && t0 < it.len;
}
// Entries of cu_seq, checked by one CTA.
__device__ __forceinline__ void prompt_check(const PromptArgs& a) {
    bool bad = false;
    for (int r = int(threadIdx.x); r < a.n_seq; r += int(blockDim.x)) {
        const int from = a.cu_seq[r], to = a.cu_seq[r + 1];
        bad |= from < 0 || to < from || to > a.n_tok;
    }
    if (bad) atomicOr(a.status, kPromptBadLength);
}

// Key tiles of an item: the first key (of the prompt) and their number.
template <int KT> __device__ __forceinline__ void key_range(const PromptArgs& a, const PromptItem& it, int& first, int& tiles) {
    const int last = min(it.t0 + a.tokens, it.len) - 1;
    first = a.window > 0 ? max(0, it.t0 - a.window + 1) : 0;
    tiles = (last - first) / KT + 1;
}
// Whether some row of the item does not see every key of the tile that begins at k0.
template <int KT> __device__ __forceinline__ bool on_edge(const PromptArgs& a, const PromptItem& it, int k0) {
    const int last = min(it.t0 + a.tokens, it.len) - 1;
    return k0 + KT - 1 > it.t0 || (a.window > 0 && k0 < last - a.window + 1);
}

__device__ __forceinline__ float exp2_of(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

struct PromptKernel { const void* fn; int threads, smem, boxes_kt; };

}  // namespace qg
