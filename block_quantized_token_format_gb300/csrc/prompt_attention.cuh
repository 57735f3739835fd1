// Causal attention of packed prompts (qg_prompt_attention): what the bf16 and the fp32 kernel share.
// Formulas and argument rules are in include/qgemv.h.
//
// An item is 128 rows of the products: T = 128 / group tokens of one prompt times the `group` query
// heads that read one key/value head (row = token * group + head), so short prompts fill rows with
// heads and every key tile serves all of them.  Later tokens (more keys) come first.
// Items are numbered without a prefix sum: prompt r's begin at slot cu_seq[r] / T + r, which leaves
// room for each prompt's last, partly filled item; a slot beyond a prompt's items has no work.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "qgemv_host.h"
#include "umma.cuh"

namespace qg {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr unsigned kPromptBadLength = 16u;       // QG_DEVICE_BAD_LENGTH

struct PromptArgs {
    CUtensorMap qmap, kmap, vmap;
    const void* v;
    long long v_stride;
    const int32_t* cu_seq;
    void* out;
    float* lse;
    long long out_stride;
    int n_tok, n_seq, n_heads, n_kv, group, tokens, window;      // tokens: T
    int asks;                      // the grid does not run at once: CTAs take on what others would
    float c;                       // |scale| log2 e
    uint32_t negate;               // of the instruction descriptor, where scale < 0
    const float *qscale, *kscale, *vscale;       // fp32: powers of two, [n_tok][n_heads], [n_tok][n_kv]
    unsigned int* status;
    uint32_t wait_limit, drain_limit, extra_tx;
};

// One item's place: prompt's first token and length, first query (of the prompt), key/value head;
// its first key and number of key tiles.
struct PromptItem { int seq0, len, t0, head, first, tiles; };

// The piece of `per` tokens of a prompt that a slot is; false: nothing to do.  Whole warps.
__device__ __forceinline__ bool prompt_piece(const int32_t* cu_seq, int n_seq, int n_tok, int per, int slot, PromptItem& it) {
    int lo = 0, hi = n_seq;                              // the last prompt that begins at or before the slot,
    const int lane = int(threadIdx.x) & 31;              // 32 probes at a time
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, probe = lo + (lane + 1) * step;
        const bool before = probe < hi && cu_seq[probe] / per + probe <= slot;
        lo += __popc(__ballot_sync(tc::kFullMask, before)) * step;
        hi = min(hi, lo + step);
    }
    const int from = cu_seq[lo], to = cu_seq[lo + 1];
    if (from < 0 || to < from || to > n_tok) return false;           // (reported by prompt_check)
    const long long t0 = (long long)(slot - (from / per + lo)) * per;
    it.seq0 = from;
    it.len = to - from;
    it.t0 = int(min(t0, 0x7FFFFFFFll));
    return t0 >= 0 && t0 < it.len;
}
// Entries of cu_seq, 32 by the warp that has the item `at` (there are as many items as prompts).
__device__ __forceinline__ void prompt_check(const PromptArgs& a, int at) {
    const long long r = (long long)at * 32 + (int(threadIdx.x) & 31);
    if (r >= a.n_seq) return;
    const int from = a.cu_seq[r], to = a.cu_seq[r + 1];
    if (from < 0 || to < from || to > a.n_tok) atomicOr(a.status, kPromptBadLength);
}

// Key tiles of an item: the first key (of the prompt) and their number.  `whole`: tiles begin at
// multiples of KT.
template <int KT> __device__ __forceinline__ void key_range(const PromptArgs& a, PromptItem& it, bool whole) {
    const int last = min(it.t0 + a.tokens, it.len) - 1;
    it.first = a.window > 0 ? max(0, it.t0 - a.window + 1) : 0;
    if (whole) it.first = it.first / KT * KT;
    it.tiles = (last - it.first) / KT + 1;
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

// One row's place in its item.
struct PromptRow { bool there; int tok, pos, low; };     // of the prompt; last and first visible key
__device__ __forceinline__ PromptRow prompt_row(const PromptArgs& a, const PromptItem& it, int row) {
    PromptRow r;
    r.tok = it.t0 + row / a.group;
    r.there = row < a.tokens * a.group && r.tok < it.len;
    r.pos = r.there ? r.tok : -1;
    r.low = r.there && a.window > 0 ? max(0, r.tok - a.window + 1) : 0;
    return r;
}

__device__ __forceinline__ void sts128(uint32_t a, const uint32_t (&y)[4]) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" :: "r"(a), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]) : "memory");
}
__device__ __forceinline__ float4 lds4(uint32_t a) {
    const uint4 w = tc::lds128(a);
    return make_float4(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w));
}
// Halves of a word whose exponents (mask) are all ones get bit 15 and 31.
template <uint32_t MASK> __device__ __forceinline__ uint32_t not_finite(uint32_t w) {
    return ((w & MASK) + (0x80008000u - MASK)) & 0x80008000u;
}
constexpr uint32_t kBf16Exp = 0x7F807F80u, kFp16Exp = 0x7C007C00u;
// Makes zeros of the values of `bytes` at v that are not finite; 128 * SIDES threads, each its own 16
// bytes of every 2048 * SIDES.  True if this thread met one.
template <uint32_t MASK, int SIDES> __device__ __forceinline__ bool clear_not_finite(uint32_t v, int bytes, int tid) {
    v += uint32_t(tid) * 16;
    uint32_t seen = 0;
#pragma unroll 8
    for (int i = 0; i < bytes; i += 2048 * SIDES) {
        const uint4 w = tc::lds128(v + i);
        seen |= not_finite<MASK>(w.x) | not_finite<MASK>(w.y) | not_finite<MASK>(w.z) | not_finite<MASK>(w.w);
    }
    if (!seen) return false;
    for (int i = 0; i < bytes; i += 2048 * SIDES) {
        const uint4 w = tc::lds128(v + i);
        uint32_t y[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int n = 0; n < 4; ++n) y[n] &= ~((not_finite<MASK>(y[n]) >> 15) * 0xFFFFu);
        sts128(v + i, y);
    }
    tc::fence_async();
    return true;
}
// What was left out: adds the values that are not finite, of the keys on edge tiles that the row
// sees, to 32 outputs from `dim` on.
template <int KT, typename T>
__device__ __forceinline__ void add_not_finite(const PromptArgs& a, const PromptItem& it, const PromptRow& r, int dim, int D, float (&y)[32]) {
    for (int j = 0; j < it.tiles; ++j) {
        const int k0 = it.first + j * KT;
        if (!on_edge<KT>(a, it, k0)) continue;
        for (int key = max(k0, r.low); key <= min(k0 + KT - 1, r.pos); ++key) {
            const T* const v = static_cast<const T*>(a.v) + (long long)(it.seq0 + key) * a.v_stride + it.head * D + dim;
#pragma unroll
            for (int n = 0; n < 32; ++n) {
                const float w = float(v[n]);
                if ((__float_as_uint(w) & 0x7F800000u) == 0x7F800000u) y[n] += w;
            }
        }
    }
}

// Stores a row's 32 16-bit values (16 words, this lane's row) from `to` on.  Four neighbouring lanes
// first exchange their quarters, so that a store writes 64 bytes of a row and not 16 of each of 32
// rows: a store takes the memory pipe once per 128-byte line that it touches.
__device__ __forceinline__ void store_rows(uint16_t* to, bool there, const uint32_t (&w)[16], int lane) {
    uint32_t q[4][4];                                    // piece p of the row, later of the rows of the four lanes
#pragma unroll
    for (int p = 0; p < 4; ++p)
#pragma unroll
        for (int n = 0; n < 4; ++n) q[p][n] = w[4 * p + n];
    // Lane i gives piece p and gets piece i of lane p's row: two exchanges, of bit 0 and of bit 1.
#pragma unroll
    for (int m = 1; m < 4; m *= 2) {
        const bool up = (lane & m) != 0;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            if (p & m) continue;
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const uint32_t got = __shfl_xor_sync(tc::kFullMask, up ? q[p][n] : q[p | m][n], m);
                if (up) q[p][n] = got; else q[p | m][n] = got;
            }
        }
    }
    const unsigned long long mine = there ? reinterpret_cast<unsigned long long>(to) : 0ull;
#pragma unroll
    for (int p = 0; p < 4; ++p) {                        // (q[p] is now piece `lane % 4` of the row of lane p of the four)
        const unsigned long long row = __shfl_sync(tc::kFullMask, mine, (lane & ~3) + p);
        if (row) *reinterpret_cast<uint4*>(row + (lane & 3) * 16) = make_uint4(q[p][0], q[p][1], q[p][2], q[p][3]);
    }
}

// Two fp32 values in a register pair, as the packed instructions take them.
__device__ __forceinline__ unsigned long long pair_of(uint32_t lo, uint32_t hi) {
    unsigned long long d;
    asm("mov.b64 %0, {%1,%2};" : "=l"(d) : "r"(lo), "r"(hi));
    return d;
}
__device__ __forceinline__ float2 values_of(unsigned long long p) {
    float2 v;
    asm("mov.b64 {%0,%1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(p));
    return v;
}
__device__ __forceinline__ unsigned long long pair_of(float x) { return pair_of(__float_as_uint(x), __float_as_uint(x)); }
__device__ __forceinline__ unsigned long long pair_fma(unsigned long long a, unsigned long long b, unsigned long long c) {
    unsigned long long d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ unsigned long long pair_add(unsigned long long a, unsigned long long b) {
    unsigned long long d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
// The largest of N scores (NaN counts as none).
template <int N> __device__ __forceinline__ float largest(const uint32_t (&x)[N]) {
    float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < N; i += 8)
#pragma unroll
        for (int n = 0; n < 4; ++n)
            asm("max.f32 %0, %0, %1, %2;" : "+f"(m[n]) : "f"(__uint_as_float(x[i + 2 * n])), "f"(__uint_as_float(x[i + 2 * n + 1])));
    return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}
// The SIDES warps that share 32 rows meet (`rows`: which of the four).  One whose wait has given up
// leaves instead, so that the others, if they are in meet(), go on; they then find `dead` and leave too.
template <int SIDES> __device__ __forceinline__ bool meet(int rows, const volatile uint32_t& dead) {
    if (__any_sync(tc::kFullMask, dead != 0)) return false;
    asm volatile("bar.sync %0, %1;" :: "r"(rows + 1), "n"(32 * SIDES) : "memory");
    return true;
}
template <int SIDES> __device__ __forceinline__ void leave(int rows) {
    asm volatile("bar.arrive %0, %1;" :: "r"(rows + 1), "n"(32 * SIDES) : "memory");
}
// The largest of the row's lanes' maxima, and the sum of their sums (in the same order in each).
template <int SIDES> __device__ __forceinline__ float largest_of(const float* shared, int row) {
    float m = shared[row];
#pragma unroll
    for (int s = 1; s < SIDES; ++s) m = fmaxf(m, shared[s * 128 + row]);
    return m;
}
template <int SIDES> __device__ __forceinline__ float sum_of_lanes(const float* shared, int row) {
    float m = shared[row];
#pragma unroll
    for (int s = 1; s < SIDES; ++s) m += shared[s * 128 + row];
    return m;
}

struct PromptKernel { const void* fn; int threads, smem, tile_keys, parts; };       // parts: CTAs of an item
PromptKernel prompt_bf16(int D);
PromptKernel prompt_f32(int D);

// fp32: queries, keys and values as two fp16 terms each, with their powers of two.
struct PromptStage {
    const float *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    const int32_t* cu_seq;
    uint16_t *q_out, *k_out, *v_out;
    float *qscale, *kscale, *vscale;
    int n_tok, n_seq, n_heads, n_kv;
};
qg_status prompt_stage(int D, const PromptStage& p, void* stream);

}  // namespace qg
