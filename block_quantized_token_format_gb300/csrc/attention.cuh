// Attention of new tokens over the paged 4-bit key/value cache (qg_attention): the kernel.
//
//     s_k = scale * q . key_k,   out = sum_k softmax(s)_k value_k,   lse = log sum_k exp(s_k)
//
// Work.  A row is one (new token, query head); the rows of a request that read the same
// key/value head are cut into tiles of ROWS, and an item is one (request, key/value head, row
// tile) with its visible keys in units of 32.  All items' units form one sequence, dealt in
// equal contiguous parts to the CTAs and, within a CTA, to its warps: a batch of any lengths
// loads every SM alike, and a single long request is split over all of them.  Each warp runs
// its part alone, with a running maximum and sum per row; parts of an item are joined in
// order, first the warps' within the CTA, then the CTAs' by the last of them to finish (a
// ticket; no CTA ever waits on another), so results do not change from run to run.
//
// Memory.  A unit's keys and values are two records of the cache, each one bulk copy into the
// warp's own ring (mbarrier-counted, bounded waits), so the bytes in flight are set by shared
// memory and every byte is read from HBM once per row tile.  Page numbers are fetched a batch
// of 16 units ahead of their copies.
//
// Arithmetic.  The tensor cores' m16n8k16 (fp16 in, fp32 out) is the right size here: a
// decode step has 1 to 32 rows per key/value head, far below the 64 or 128 rows of a tcgen05
// tile, and operands that come out of nibbles in registers would have to go back through
// shared memory for it.  Every operand is exact:
//  * scores: a key's codes enter as they are, as the fp16 subnormals code * 2^-20 (a shift and
//    a mask per two codes, no arithmetic); the sum starts at -8 * sum(q) of its block, and the
//    block's scale multiplies the fp32 result. (Four bits lower, code * 2^-24, would save
//    half the shifts, but the tensor core aligns products by their exponent fields, and a
//    subnormal that far down loses 6 bits of the sum: measured 9 ulps against 0.17.) A query is
//    scaled by a power of two to [2^14, 2^15) and split into two fp16 terms (22 bits; one term
//    is exact for bf16 queries).
//  * outputs: a value is (16 + code) * d - 24 * d in one fp16 FMA, which is exact because
//    d has 8 significant bits; probabilities are two fp16 terms (one for bf16 outputs), scaled
//    by 2^7 relative to a reference that follows the running maximum within 2^8, so that the
//    outputs are rescaled rarely and no probability that counts becomes subnormal.
// With at most 8 rows the two terms are the two halves of one 16-row operand (PACKED: the low
// terms would-be padding rows, no extra work); with 16 rows they are two products into one
// accumulator.
#pragma once

#include <cuda_bf16.h>

#include "kv_layout.h"
#include "qgemv_kernels.cuh"

namespace qg {

constexpr int kUnit = 32;                 // keys per unit: two records
constexpr int kMaxAttnReq = 4096;
constexpr int kAttnGrid = 160;             // most CTAs of a launch (one per SM; the workspace is sized by it)
static_assert(kAttnGrid * 4 <= QG_ATTENTION_ZERO_BYTES, "one ticket per CTA");
constexpr float kProbShift = 7.0f;        // probabilities are scaled by 2^7 ...
constexpr float kRefSlack = 8.0f;         // ... and the reference follows the maximum within 2^8: below 2^15
constexpr uint32_t kNoItem = 0xFFFFFFFFu;

struct AttnArgs {
    const uint8_t* data;
    const void* q;
    void* out;
    float* lse;
    const int32_t *table, *seq_len, *cu_new;
    const uint32_t* span_mask;
    uint32_t* tickets;         // [grid], zero on entry and on exit
    float* partial;            // [grid][2] CTA partials, then [grid][warps] warp partials
    unsigned int* status;
    long long q_stride, out_stride, table_stride, n_tok, n_pages;
    int n_req, n_heads, n_kv, group, page_records, window, depth;
    float scale_log2;          // scale * log2(e) * 2^20 (the codes' exponent)
    uint32_t wait_limit, drain_limit, test_extra_tx;
};

template <int D, int ROWS, int TERMS> struct AttnShape {
    static constexpr bool kPacked = ROWS == 8;
    static_assert(ROWS == 16 || (ROWS == 8 && TERMS == 2), "8 rows hold both terms in one operand");
#ifndef QG_W
#define QG_W 12
#endif
    static constexpr int kWarps = D == 256 && ROWS == 16 && TERMS == 2 ? 6 : D == 256 ? 8 : QG_W;
    static constexpr int kRec = kv_record_bytes(D);
    static constexpr int kStage = 2 * kRec;
    static constexpr int kQMats = kPacked ? 1 : TERMS;
    static constexpr int kQBytes = kQMats * (D / 16) * 512;          // queries in operand order
    static constexpr int kInitBytes = kv_groups(D) * 16 * 4;         // -8 * sum(q) per block and row
    static constexpr int kPartial = ROWS * (D + 2);                  // floats: [ROWS][D], m[ROWS], l[ROWS]
};

// Shared memory: prefix of units per request, the warps' records of unfinished items, then
// per warp its barriers, queries and ring.
struct AttnSmem { int meta_off, warp_off, bar_off, q_off, init_off, ring_off, warp_bytes, total; };
template <int D, int ROWS, int TERMS> __host__ __device__ inline AttnSmem attn_smem(int n_req, int depth) {
    using S = AttnShape<D, ROWS, TERMS>;
    AttnSmem p;
    p.meta_off = ((n_req + 1) * 4 + 7) / 8 * 8;
    p.warp_off = (p.meta_off + (4 * S::kWarps + 1) * 4 + 127) / 128 * 128;
    p.ring_off = 0;
    p.q_off = depth * S::kStage;
    p.init_off = p.q_off + S::kQBytes;
    p.bar_off = p.init_off + S::kInitBytes;
    p.warp_bytes = (p.bar_off + depth * 8 + 127) / 128 * 128;
    p.total = p.warp_off + S::kWarps * p.warp_bytes;
    return p;
}

// ------------------------------------------------------------------------------ PTX helpers

__device__ __forceinline__ void bulk_load(uint32_t dst, uint64_t src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 :: "r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}
// d = a b + {c0, c0, c1, c1}: an accumulator of its own, so that a start value costs no moves.
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1, float c0, float c1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%11,%11};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint4& a, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ f2_t f2_add(f2_t a, f2_t b) {
    f2_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f2_t f2_mul(f2_t a, f2_t b) {
    f2_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f2_t f2_of(float x, float y) { return f2_pack(__float_as_uint(x), __float_as_uint(y)); }
__device__ __forceinline__ float2 f2_get(f2_t a) {
    float2 r;
    asm("mov.b64 {%0,%1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
    return r;
}
__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 bits_h2(uint32_t b) { return *reinterpret_cast<__half2*>(&b); }
__device__ __forceinline__ f2_t f2_of_h2(uint32_t b) {
    const float2 f = __half22float2(bits_h2(b));
    return f2_of(f.x, f.y);
}
// A pair as its fp16 rounding and the fp16 rounding of what that leaves.
__device__ __forceinline__ void split_pair(float x, float y, uint32_t& hi, uint32_t& lo) {
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    hi = h2_bits(h);
    lo = h2_bits(__floats2half2_rn(x - f.x, y - f.y));
}
template <int N> __device__ __forceinline__ void lds_words(uint32_t a, uint32_t* w) {
    if constexpr (N == 4) {
        const uint4 v = lds128(a);
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else {
        static_assert(N == 2, "two or four blocks of a set");
        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(a));
    }
}
__device__ __forceinline__ void load8(const float* p, float* x) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* x) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void store4(float* p, float a, float b, float c, float d) {
    *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, float a, float b, float c, float d) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(a, b), hi = __floats2bfloat162_rn(c, d);
    uint2 v;
    v.x = *reinterpret_cast<const uint32_t*>(&lo);
    v.y = *reinterpret_cast<const uint32_t*>(&hi);
    *reinterpret_cast<uint2*>(p) = v;
}

// ------------------------------------------------------------------------------ work

// A request's share of the work: its visible keys in units (from the first one a window
// leaves) and its row tiles; 0 units for a request that does not fit the call.
struct Request {
    int seq, first_tok, fresh, first_unit, units, tiles;
};
template <int ROWS> __device__ __forceinline__ Request request_of(const AttnArgs& a, int r, bool& bad_len, bool& bad_page) {
    Request q;
    q.seq = a.seq_len[r];
    q.first_tok = a.cu_new[r];
    const int end = a.cu_new[r + 1];
    q.fresh = end - q.first_tok;
    q.units = q.first_unit = q.tiles = 0;
    const bool ok = q.seq >= 0 && q.first_tok >= 0 && end >= q.first_tok && end <= a.n_tok &&
                    !(a.span_mask && q.fresh > 32);
    bad_len |= !ok;
    const long long records = ((long long)q.seq + kRecordTokens - 1) / kRecordTokens;
    const bool fits = records <= a.table_stride * a.page_records;
    bad_page |= ok && !fits;
    if (!ok || !fits || q.fresh == 0) { q.fresh = 0; return q; }
    if (a.window > 0) q.first_unit = max(0, q.seq - q.fresh + 1 - a.window) / kUnit;
    q.units = max(1, int(((long long)q.seq + kUnit - 1) / kUnit) - q.first_unit);
    q.tiles = int(((long long)q.fresh * a.group + ROWS - 1) / ROWS);
    return q;
}

// An item, decoded from a unit's place in the sequence.
struct Item {
    Request rq;
    int r, head, tile, unit;       // unit: within the item
    uint32_t start;                // the item's first unit in the sequence: its identity
};
template <int ROWS> __device__ __forceinline__ Item item_at(const AttnArgs& a, const uint32_t* cum, int r, uint32_t u) {
    bool x = false, y = false;
    Item it;
    it.r = r;
    it.rq = request_of<ROWS>(a, r, x, y);
    const uint32_t rem = u - cum[r], n = rem / uint32_t(it.rq.units);
    it.unit = int(rem - n * uint32_t(it.rq.units));
    it.head = int(n / uint32_t(it.rq.tiles));
    it.tile = int(n - uint32_t(it.head) * uint32_t(it.rq.tiles));
    it.start = u - uint32_t(it.unit);
    return it;
}
// The request whose units hold u, searched from request r on (units only grow).
__device__ __forceinline__ int find_request(const uint32_t* cum, int lo, int n_req, uint32_t u) {
    int hi = n_req;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cum[mid] <= u) lo = mid; else hi = mid;
    }
    return lo;
}

// What a row may see: keys in (low, pos], of its request's new tokens those in bits.
struct Sight {
    int pos, low, begin;
    uint32_t bits;
    __device__ __forceinline__ bool sees(int key) const {
        return key <= pos && key > low && (key < begin || ((bits >> ((key - begin) & 31)) & 1u));
    }
};

// Row i of an item's tile: its token and head, or token -1.
template <int ROWS> __device__ __forceinline__ void row_of(const AttnArgs& a, const Item& it, int row, int& j, int& head) {
    const int i = it.tile * ROWS + row;
    j = i / a.group;
    head = it.head * a.group + (i - j * a.group);
    if (j >= it.rq.fresh) j = -1;
}

// ------------------------------------------------------------------------------ kernel

template <typename T, int D, int ROWS, int TERMS>
__global__ void __launch_bounds__(32 * AttnShape<D, ROWS, TERMS>::kWarps, 1) attention_kernel(const AttnArgs a) {
    using S = AttnShape<D, ROWS, TERMS>;
    constexpr int W = S::kWarps, NG = kv_groups(D), GI = kv_set(D), NS = NG / GI;
    constexpr bool PACKED = S::kPacked;
    extern __shared__ __align__(128) uint8_t smem[];
    uint32_t* const cum = reinterpret_cast<uint32_t*>(smem);
    const AttnSmem lay = attn_smem<D, ROWS, TERMS>(a.n_req, a.depth);
    unsigned long long* const wsum = reinterpret_cast<unsigned long long*>(smem + lay.meta_off);   // [W]
    uint32_t* const meta = reinterpret_cast<uint32_t*>(wsum + W);                 // [W][2] item starts, then a flag
    const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5;
    const int r8 = lane >> 2, c4 = lane & 3;               // operand row (or key column) and column group
    uint8_t* const mine = smem + lay.warp_off + warp * lay.warp_bytes;
    const uint32_t ring = smem_addr(mine), qmat = ring + lay.q_off, binit = ring + lay.init_off, bars = ring + lay.bar_off;

    if (lane < a.depth) mbar_init(bars + 8 * lane, 1);
    mbar_fence_init();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // ---- units per request, prefixed
    unsigned long long run = 0;
    bool bad_len = false, bad_page = false;
    for (int r0 = 0; r0 < a.n_req; r0 += 32 * W) {
        const int r = r0 + tid;
        unsigned long long n = 0;
        if (r < a.n_req) {
            const Request q = request_of<ROWS>(a, r, bad_len, bad_page);
            n = (unsigned long long)q.units * unsigned(q.tiles) * unsigned(a.n_kv);
        }
        unsigned long long s = n;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const unsigned long long up = __shfl_up_sync(kFull, s, d);
            if (lane >= d) s += up;
        }
        if (lane == 31) wsum[warp] = s;
        __syncthreads();
        unsigned long long before = run;
        for (int w = 0; w < W; ++w) {
            if (w < warp) before += wsum[w];
            run += wsum[w];
        }
        if (r < a.n_req) cum[r] = uint32_t(before + s - n);
        __syncthreads();
    }
    if (run >= 0x7FFFFFFFull) { bad_len = true; run = 0; }       // more units than the sequence can number
    if (tid == 0) cum[a.n_req] = uint32_t(run);
    if (tid < 2 * W) meta[tid] = kNoItem;
    if (blockIdx.x == 0 && bad_len) atomicOr(a.status, kStatusBadLength);
    if (blockIdx.x == 0 && bad_page) atomicOr(a.status, kStatusBadPage);
    __syncthreads();
    const uint32_t total = uint32_t(run);
    // At least one unit per warp: a smaller share would leave warps idle and more CTAs to join.
    const uint32_t share = max((total + gridDim.x - 1) / gridDim.x, uint32_t(W));
    const uint32_t c0 = min(share * blockIdx.x, total), c1 = min(c0 + share, total);
    if (c0 == c1) return;
    const uint32_t u0 = c0 + uint32_t((unsigned long long)(c1 - c0) * warp / W);
    const uint32_t u1 = c0 + uint32_t((unsigned long long)(c1 - c0) * (warp + 1) / W);

    // ---- page numbers, a batch (up to 16 units of one item) ahead of the copies
    uint32_t au = u0;                    // next unit to fetch page numbers for
    int ar = 0;
    int next_id = -1, next_rec = 0, next_head = 0, next_count = 0;
    uint64_t src = 0;                    // this lane's record of the current batch (0: none)
    uint32_t have = 0;
    int count = 0, at = 0;
    auto fetch = [&]() {
        next_count = 0;
        next_id = -1;
        if (au >= u1) return;
        ar = find_request(cum, ar, a.n_req, au);
        const Item it = item_at<ROWS>(a, cum, ar, au);
        next_count = min(min(16, it.rq.units - it.unit), int(u1 - au));
        next_head = it.head;
        next_rec = 2 * (it.rq.first_unit + it.unit) + lane;
        if (lane < 2 * next_count && (long long)next_rec * kRecordTokens < it.rq.seq) {
            next_id = a.table[(long long)ar * a.table_stride + next_rec / a.page_records];
            if (next_id < 0 || next_id >= a.n_pages) {
                atomicOr(a.status, kStatusBadPage);
                next_id = -1;
            }
        }
        au += next_count;
    };
    auto turn_batch = [&]() {
        src = 0;
        if (next_id >= 0)
            src = reinterpret_cast<uint64_t>(a.data) +
                  (((uint64_t)next_id * a.n_kv + next_head) * a.page_records + next_rec % a.page_records) * uint64_t(S::kRec);
        have = __ballot_sync(kFull, src != 0);
        count = next_count;
        at = 0;
        fetch();
    };
    // ---- the ring
    uint32_t issued = u0;
    int in_stage = 0, out_stage = 0;
    uint32_t out_phase = 0;
    bool dead = false;
    auto issue = [&]() {
        if (issued >= u1 || dead) return;
        if (at == count) turn_batch();
        const uint32_t bar = bars + 8 * in_stage;
        if (lane == 2 * at) {
            uint32_t bytes = __popc((have >> (2 * at)) & 3u) * S::kRec;
            if (issued == u0) bytes += a.test_extra_tx;
            mbar_arrive_expect_tx(bar, bytes);
        }
        __syncwarp();
        if ((lane >> 1) == at && src != 0) bulk_load(ring + in_stage * S::kStage + (lane & 1) * S::kRec, src, S::kRec, bar);
        ++at;
        ++issued;
        in_stage = in_stage + 1 == a.depth ? 0 : in_stage + 1;
    };
    if (u0 < u1) {
        fetch();
        for (int i = 0; i < a.depth; ++i) issue();
    }

    // ---- the warp's part, item by item
    uint32_t u = u0;
    int r = 0;
    while (u < u1) {
        r = find_request(cum, r, a.n_req, u);
        const Item it = item_at<ROWS>(a, cum, r, u);
        const int begin = it.rq.seq - it.rq.fresh;

        // Rows: what they see, their queries as matrix operands.
        Sight sight[PACKED ? 1 : 2];
        float factor[PACKED ? 1 : 2];
#pragma unroll
        for (int h = 0; h < (PACKED ? 1 : 2); ++h) {
            int j, head;
            row_of<ROWS>(a, it, r8 + 8 * h, j, head);
            sight[h].pos = begin + j;
            sight[h].begin = a.span_mask ? begin : 0x7FFFFFFF;
            sight[h].bits = a.span_mask && j >= 0 ? a.span_mask[it.rq.first_tok + j] : 0u;
            sight[h].low = a.window > 0 ? sight[h].pos - a.window : -1;
            if (j < 0) sight[h].pos = -1;
            float x[NG][8];
            const T* src_row = static_cast<const T*>(a.q) + (long long)(it.rq.first_tok + max(j, 0)) * a.q_stride +
                               (long long)head * D + 8 * c4;
            uint32_t top = 0;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                if (j >= 0) {
                    load8(src_row + 32 * g, x[g]);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[g][i] = 0.0f;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[g][i]) & 0x7FFFFFFFu);
            }
            top = max(top, __shfl_xor_sync(kFull, top, 1));
            top = max(top, __shfl_xor_sync(kFull, top, 2));
            // 2^s brings the row's largest magnitude to [2^14, 2^15) (s at most 126); a row with a
            // NaN or an infinity has NaN scores.
            const int e = int(top >> 23);
            const int sh = min(141 - e, 126);
            const float up = __uint_as_float(uint32_t(127 + sh) << 23), down = __uint_as_float(uint32_t(127 - sh) << 23);
            const bool finite = e < 255;
            factor[h] = finite ? a.scale_log2 * down : __uint_as_float(0x7FFFFFFFu);
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                uint32_t hi[4], lo[4];
                float sum_hi = 0.0f, sum_lo = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float p = finite ? x[g][i] * up : 0.0f, q = finite ? x[g][i + 4] * up : 0.0f;
                    split_pair(p, q, hi[i], lo[i]);
                    const float2 fh = __half22float2(bits_h2(hi[i])), fl = __half22float2(bits_h2(lo[i]));
                    sum_hi += fh.x + fh.y;
                    sum_lo += fl.x + fl.y;
                }
                if (TERMS == 1) sum_lo = 0.0f;
                if (!PACKED) sum_hi += sum_lo;
                sum_hi += __shfl_xor_sync(kFull, sum_hi, 1);
                sum_hi += __shfl_xor_sync(kFull, sum_hi, 2);
                if (PACKED) {
                    sum_lo += __shfl_xor_sync(kFull, sum_lo, 1);
                    sum_lo += __shfl_xor_sync(kFull, sum_lo, 2);
                }
                constexpr float kUlp = -8.0f / 1048576.0f;       // -8 codes of 2^-20
                float* const init = reinterpret_cast<float*>(mine + lay.init_off) + 16 * g;
                uint32_t* const m = reinterpret_cast<uint32_t*>(mine + lay.q_off);
                if (c4 == 0) {
                    init[r8 + 8 * h] = kUlp * sum_hi;
                    if (PACKED) init[r8 + 8] = kUlp * sum_lo;
                }
                // Operand words: (row, low columns), (row + 8, low), (row, high), (row + 8, high).
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                    uint32_t* const w = m + ((2 * g + ks) * 32 + lane) * 4;
                    w[h] = hi[2 * ks];
                    w[2 + h] = hi[2 * ks + 1];
                    if (PACKED) {
                        w[1] = lo[2 * ks];
                        w[3] = lo[2 * ks + 1];
                    } else if (TERMS == 2) {
                        uint32_t* const l = w + (D / 16) * 128;
                        l[h] = lo[2 * ks];
                        l[2 + h] = lo[2 * ks + 1];
                    }
                }
            }
        }
        __syncwarp();
        // Keys that every row sees lie in (full_low, full_high]; any row's in (any_low, any_high].
        int full_high = sight[0].pos, any_high = sight[0].pos;
        {
            const int i0 = it.tile * ROWS, i1 = min(i0 + ROWS, it.rq.fresh * a.group) - 1;
            full_high = begin + i0 / a.group;
            any_high = begin + i1 / a.group;
            if (a.span_mask) full_high = min(full_high, begin - 1);
        }
        const int full_low = a.window > 0 ? any_high - a.window : -1;
        const int any_low = a.window > 0 ? begin + it.tile * ROWS / a.group - a.window : -1;

        constexpr int H = PACKED ? 1 : 2;                  // rows of this lane
        f2_t o[4 * NG][H];                                 // columns 2 c4, 2 c4 + 1 of the output tiles
#pragma unroll
        for (int n = 0; n < 4 * NG; ++n)
#pragma unroll
            for (int h = 0; h < H; ++h) o[n][h] = 0ull;
        float ref[H], sum[H];
#pragma unroll
        for (int h = 0; h < H; ++h) { ref[h] = -INFINITY; sum[h] = 0.0f; }

        const uint32_t item_end = min(it.start + uint32_t(it.rq.units), u1);
        int key0 = (it.rq.first_unit + it.unit) * kUnit;
        for (; u < item_end; ++u, key0 += kUnit) {
            const uint32_t stage = ring + out_stage * S::kStage;
            if (dead) continue;
            dead = __any_sync(kFull, !mbar_wait(bars + 8 * out_stage, out_phase, a.wait_limit));
            if (dead) {
                // Gave up: no more copies; the ones in flight land (bounded again) before the
                // ring is reused or the CTA ends.  The rest of the part is passed over.
                if (lane == 0) atomicOr(a.status, kStatusWaitTimeout);
                for (uint32_t v = u; v < issued; ++v) {
                    mbar_wait(bars + 8 * out_stage, out_phase, a.drain_limit);
                    out_stage = out_stage + 1 == a.depth ? 0 : out_stage + 1;
                    if (out_stage == 0) out_phase ^= 1;
                }
                continue;
            }

            // ---- scores of 32 keys: four column tiles of 8
            uint32_t kw[4][NG], kd[4][NG];
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
                const uint32_t rec = stage + (nt >> 1) * S::kRec;
#pragma unroll
                for (int q = 0; q < NS; ++q) {
                    lds_words<GI>(rec + ((q * 16 + (nt & 1) * 8) * 4 + lane) * GI * 4, &kw[nt][q * GI]);
                    lds_words<GI>(rec + kv_k_scales(D) + (((nt & 1) * 4 + c4) * NG + q * GI) * 4, &kd[nt][q * GI]);
                }
            }
            f2_t s[4][H];
#pragma unroll
            for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                for (int h = 0; h < H; ++h) s[nt][h] = 0ull;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const uint4 qa = lds128(qmat + ((2 * g) * 32 + lane) * 16), qb = lds128(qmat + ((2 * g + 1) * 32 + lane) * 16);
                uint4 la, lb;
                if (!PACKED && TERMS == 2) {
                    la = lds128(qmat + ((D / 16 + 2 * g) * 32 + lane) * 16);
                    lb = lds128(qmat + ((D / 16 + 2 * g + 1) * 32 + lane) * 16);
                }
                const float i0 = __uint_as_float(lds32(binit + (16 * g + r8) * 4));
                const float i1 = __uint_as_float(lds32(binit + (16 * g + r8 + 8) * 4));
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) {
                    const uint32_t w = kw[nt][g], m = 0x00F000F0u;
                    const uint32_t b0 = (w << 4) & m, b1 = w & m, b2 = (w >> 4) & m, b3 = (w >> 8) & m;
                    float acc[4];
                    mma_f16(acc, qa, b0, b1, i0, i1);
                    mma_f16(acc, qb, b2, b3);
                    if (!PACKED && TERMS == 2) {
                        mma_f16(acc, la, b0, b1);
                        mma_f16(acc, lb, b2, b3);
                    }
                    const f2_t d = f2_of_h2(kd[nt][g]);
                    if (PACKED) {
                        s[nt][0] = f2_fma(f2_add(f2_of(acc[0], acc[1]), f2_of(acc[2], acc[3])), d, s[nt][0]);
                    } else {
                        s[nt][0] = f2_fma(f2_of(acc[0], acc[1]), d, s[nt][0]);
                        s[nt][H - 1] = f2_fma(f2_of(acc[2], acc[3]), d, s[nt][H - 1]);
                    }
                }
            }
            float p[4][H][2];
#pragma unroll
            for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const float2 t = f2_get(f2_mul(s[nt][h], f2_of(factor[h], factor[h])));
                    p[nt][h][0] = t.x;
                    p[nt][h][1] = t.y;
                }
            const bool masked = key0 + kUnit - 1 > full_high || key0 <= full_low;
            if (masked) {
#pragma unroll
                for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                    for (int h = 0; h < H; ++h)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            if (!sight[h].sees(key0 + 8 * nt + 2 * c4 + i)) p[nt][h][i] = -INFINITY;
            }

            // ---- running reference and sum
            bool grow = false;
            float top[H];
#pragma unroll
            for (int h = 0; h < H; ++h) {
                top[h] = fmaxf(p[0][h][0], p[0][h][1]);
#pragma unroll
                for (int nt = 1; nt < 4; ++nt) top[h] = fmaxf(top[h], fmaxf(p[nt][h][0], p[nt][h][1]));
                top[h] = fmaxf(top[h], __shfl_xor_sync(kFull, top[h], 1));
                top[h] = fmaxf(top[h], __shfl_xor_sync(kFull, top[h], 2));
                grow |= top[h] > ref[h] + kRefSlack;
            }
            float keep[H];                                  // what the outputs so far count for
#pragma unroll
            for (int h = 0; h < H; ++h) keep[h] = 1.0f;
            if (__any_sync(kFull, grow)) {
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const float to = fmaxf(ref[h], top[h]);
                    if (to != -INFINITY) keep[h] = exp2_fast(ref[h] - to);
                    ref[h] = to;
                    sum[h] *= keep[h];
                }
            }
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const float base = (ref[h] == -INFINITY ? 0.0f : ref[h]) - kProbShift;
                float add = 0.0f;
#pragma unroll
                for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        p[nt][h][i] = exp2_fast(p[nt][h][i] - base);
                        add += p[nt][h][i];
                    }
                sum[h] += add;
            }

            // ---- outputs: the unit's products go into accumulators of their own and are added to
            // the running outputs in fp32 (the tensor core truncates what it adds to: over a long
            // cache that bias would grow with the number of units)
            uint4 pa[2], pl[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (PACKED) {
                    split_pair(p[2 * k][0][0], p[2 * k][0][1], pa[k].x, pa[k].y);
                    split_pair(p[2 * k + 1][0][0], p[2 * k + 1][0][1], pa[k].z, pa[k].w);
                } else if (TERMS == 2) {
                    split_pair(p[2 * k][0][0], p[2 * k][0][1], pa[k].x, pl[k].x);
                    split_pair(p[2 * k][H - 1][0], p[2 * k][H - 1][1], pa[k].y, pl[k].y);
                    split_pair(p[2 * k + 1][0][0], p[2 * k + 1][0][1], pa[k].z, pl[k].z);
                    split_pair(p[2 * k + 1][H - 1][0], p[2 * k + 1][H - 1][1], pa[k].w, pl[k].w);
                } else {
                    pa[k].x = h2_bits(__floats2half2_rn(p[2 * k][0][0], p[2 * k][0][1]));
                    pa[k].y = h2_bits(__floats2half2_rn(p[2 * k][H - 1][0], p[2 * k][H - 1][1]));
                    pa[k].z = h2_bits(__floats2half2_rn(p[2 * k + 1][0][0], p[2 * k + 1][0][1]));
                    pa[k].w = h2_bits(__floats2half2_rn(p[2 * k + 1][H - 1][0], p[2 * k + 1][H - 1][1]));
                }
            }
#pragma unroll
            for (int q = 0; q < NS; ++q) {
                // Tokens 2 c4, 2 c4 + 1 of each half of each record.
                uint32_t w[4][GI], d[4][GI];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t rec = stage + (k >> 1) * S::kRec;
                    lds_words<GI>(rec + kv_v_codes(D) + ((q * 2 + (k & 1)) * 32 + lane) * GI * 4, w[k]);
                    lds_words<GI>(rec + kv_v_scales(D) + (((k & 1) * 4 + c4) * NG + q * GI) * 4, d[k]);
                }
                if (masked) {
                    // A scale that no row of the tile may see counts as zero, whatever is stored
                    // there; so does a NaN one, and the rows that see it turn NaN here.
                    bool odd = false;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int key = key0 + 8 * k + 2 * c4;
                        uint32_t m = 0;
                        if (key > any_low && key <= any_high) m |= 0xFFFFu;
                        if (key + 1 > any_low && key + 1 <= any_high) m |= 0xFFFF0000u;
#pragma unroll
                        for (int i = 0; i < GI; ++i) {
                            d[k][i] &= m;
                            odd |= (d[k][i] & 0x7C00u) == 0x7C00u || (d[k][i] & 0x7C000000u) == 0x7C000000u;
                        }
                    }
                    if (__any_sync(kFull, odd)) {
#pragma unroll
                        for (int i = 0; i < GI; ++i) {
                            bool spoil[H];
#pragma unroll
                            for (int h = 0; h < H; ++h) spoil[h] = false;
                            for (int t = 0; t < kUnit; ++t) {
                                const uint32_t x = lds16(stage + t / kRecordTokens * S::kRec + kv_v_scales(D) +
                                                         kv_scale(D, t % kRecordTokens, q * GI + i));
                                if ((x & 0x7C00u) != 0x7C00u) continue;
#pragma unroll
                                for (int h = 0; h < H; ++h) spoil[h] |= sight[h].sees(key0 + t);
                            }
#pragma unroll
                            for (int h = 0; h < H; ++h)
#pragma unroll
                                for (int n = 0; n < 4; ++n)
                                    if (spoil[h]) o[4 * (q * GI + i) + n][h] = f2_of(NAN, NAN);
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                if ((d[k][i] & 0x7C00u) == 0x7C00u) d[k][i] &= 0xFFFF0000u;
                                if ((d[k][i] & 0x7C000000u) == 0x7C000000u) d[k][i] &= 0xFFFFu;
                            }
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < GI; ++i) {
                    __half2 less[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) less[k] = __hmul2(bits_h2(d[k][i]), __float2half2_rn(-24.0f));
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        uint32_t v[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t x = w[k][i], t = n == 0 ? x << 6 : n == 1 ? x << 2 : n == 2 ? x >> 2 : x >> 6;
                            v[k] = h2_bits(__hfma2(bits_h2((t & 0x03C003C0u) | 0x4C004C00u), bits_h2(d[k][i]), less[k]));
                        }
                        float acc[4];
                        mma_f16(acc, pa[0], v[0], v[1], 0.0f, 0.0f);
                        mma_f16(acc, pa[1], v[2], v[3]);
                        if (!PACKED && TERMS == 2) {
                            mma_f16(acc, pl[0], v[0], v[1]);
                            mma_f16(acc, pl[1], v[2], v[3]);
                        }
                        f2_t(&to)[H] = o[4 * (q * GI + i) + n];
                        if (PACKED) {
                            to[0] = f2_fma(to[0], f2_of(keep[0], keep[0]), f2_add(f2_of(acc[0], acc[1]), f2_of(acc[2], acc[3])));
                        } else {
                            to[0] = f2_fma(to[0], f2_of(keep[0], keep[0]), f2_of(acc[0], acc[1]));
                            to[H - 1] = f2_fma(to[H - 1], f2_of(keep[H - 1], keep[H - 1]), f2_of(acc[2], acc[3]));
                        }
                    }
                }
            }
            __syncwarp();                                   // every lane has read the stage
            out_stage = out_stage + 1 == a.depth ? 0 : out_stage + 1;
            if (out_stage == 0) out_phase ^= 1;
            issue();
        }

        // ---- the item's end: written out, or left for the join
#pragma unroll
        for (int h = 0; h < H; ++h) {
            sum[h] += __shfl_xor_sync(kFull, sum[h], 1);
            sum[h] += __shfl_xor_sync(kFull, sum[h], 2);
        }
        const bool whole = it.start >= u0 && it.start + uint32_t(it.rq.units) <= u1;
        if (whole) {
#pragma unroll
            for (int h = 0; h < H; ++h) {
                int j, head;
                row_of<ROWS>(a, it, r8 + 8 * h, j, head);
                if (j < 0) continue;
                const float inv = sum[h] == 0.0f ? 0.0f : 1.0f / sum[h];
                const long long tok = it.rq.first_tok + j;
                T* const dst = static_cast<T*>(a.out) + tok * a.out_stride + (long long)head * D + 8 * c4;
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const float2 x0 = f2_get(o[4 * g][h]), x1 = f2_get(o[4 * g + 1][h]), x2 = f2_get(o[4 * g + 2][h]),
                                 x3 = f2_get(o[4 * g + 3][h]);
                    store4(dst + 32 * g, x0.x * inv, x1.x * inv, x2.x * inv, x3.x * inv);
                    store4(dst + 32 * g + 4, x0.y * inv, x1.y * inv, x2.y * inv, x3.y * inv);
                }
                if (a.lse && c4 == 0)
                    a.lse[tok * a.n_heads + head] = (ref[h] + log2f(sum[h]) - kProbShift) * 0.693147180559945309f;
            }
        } else {
            // The part's last item waits in the warp's ring (every copy into it has been consumed),
            // an earlier one, whose ring is still in use, in the workspace.
            const bool last = u == u1;
            float* const dst = last ? reinterpret_cast<float*>(mine)
                                    : a.partial + (2ll * gridDim.x + (long long)blockIdx.x * W + warp) * S::kPartial;
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const int row = r8 + 8 * h;
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const float2 x0 = f2_get(o[4 * g][h]), x1 = f2_get(o[4 * g + 1][h]), x2 = f2_get(o[4 * g + 2][h]),
                                 x3 = f2_get(o[4 * g + 3][h]);
                    store4(dst + row * D + 32 * g + 8 * c4, x0.x, x1.x, x2.x, x3.x);
                    store4(dst + row * D + 32 * g + 8 * c4 + 4, x0.y, x1.y, x2.y, x3.y);
                }
                if (c4 == 0) {
                    dst[ROWS * D + row] = ref[h];
                    dst[ROWS * D + ROWS + row] = sum[h];
                }
            }
            if (lane == 0) meta[2 * warp + (last ? 1 : 0)] = it.start;
        }
    }
    __syncthreads();

    // ---- join the warps' parts, in order; an item that other CTAs share leaves one partial
    auto part = [&](int i) -> const float* {
        return (i & 1) ? reinterpret_cast<const float*>(smem + lay.warp_off + (i >> 1) * lay.warp_bytes)
                       : a.partial + (2ll * gridDim.x + (long long)blockIdx.x * W + (i >> 1)) * S::kPartial;
    };
    auto put = [&](const Item& it, int row, int col, float4 v, float m, float l) {
        int j, head;
        row_of<ROWS>(a, it, row, j, head);
        if (j < 0) return;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const long long tok = it.rq.first_tok + j;
        store4(static_cast<T*>(a.out) + tok * a.out_stride + (long long)head * D + col, v.x * inv, v.y * inv, v.z * inv,
               v.w * inv);
        if (a.lse && col == 0) a.lse[tok * a.n_heads + head] = (m + log2f(l) - kProbShift) * 0.693147180559945309f;
    };
    uint32_t shared_item[2];
    int n_shared = 0;
    for (int i = 0; i < 2 * W;) {
        const uint32_t start = meta[i];
        if (start == kNoItem) { ++i; continue; }
        int end = i + 1, n = 1;
        while (end < 2 * W && (meta[end] == start || meta[end] == kNoItem)) n += meta[end++] == start;
        const Item it = item_at<ROWS>(a, cum, find_request(cum, 0, a.n_req, start), start);
        const bool all = start >= c0 && start + uint32_t(it.rq.units) <= c1;
        float* const dst = a.partial + (2ll * blockIdx.x + (start >= c0 ? 1 : 0)) * S::kPartial;
        for (int e = tid; e < ROWS * D / 4; e += 32 * W) {
            const int row = e / (D / 4), col = (e - row * (D / 4)) * 4;
            float m = -INFINITY;
            for (int k = i; k < end; ++k)
                if (meta[k] == start) m = fmaxf(m, part(k)[ROWS * D + row]);
            float l = 0.0f;
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int k = i; k < end; ++k) {
                if (meta[k] != start) continue;
                const float* const p = part(k);
                const float f = m == -INFINITY ? 1.0f : exp2_fast(p[ROWS * D + row] - m);
                const float4 x = *reinterpret_cast<const float4*>(p + row * D + col);
                l = fmaf(p[ROWS * D + ROWS + row], f, l);
                v.x = fmaf(x.x, f, v.x); v.y = fmaf(x.y, f, v.y); v.z = fmaf(x.z, f, v.z); v.w = fmaf(x.w, f, v.w);
            }
            if (all) {
                put(it, row, col, v, m, l);
            } else {
                *reinterpret_cast<float4*>(dst + row * D + col) = v;
                if (col == 0) { dst[ROWS * D + row] = m; dst[ROWS * D + ROWS + row] = l; }
            }
        }
        if (!all && n_shared < 2) shared_item[n_shared++] = start;
        i = end;
    }

    // ---- the last CTA of a shared item joins the CTAs' partials, in order
    int* const flag = reinterpret_cast<int*>(meta + 2 * W);
    for (int k = 0; k < n_shared; ++k) {
        const uint32_t start = shared_item[k];
        const Item it = item_at<ROWS>(a, cum, find_request(cum, 0, a.n_req, start), start);
        const uint32_t first = start / share, last = (start + uint32_t(it.rq.units) - 1) / share;
        const int n = int(last - first) + 1;
        __threadfence();
        __syncthreads();
        if (tid == 0) {
            const bool mine_last = atomicAdd(a.tickets + first, 1u) == uint32_t(n - 1);
            if (mine_last) a.tickets[first] = 0u;
            *flag = mine_last;
        }
        __syncthreads();
        if (!*flag) continue;
        __threadfence();
        auto cta_part = [&](int i) { return a.partial + (2ll * (first + i) + (i == 0 ? 1 : 0)) * S::kPartial; };
        // Weights of the partials, per row, where the rings were: [ROWS][n], then m[ROWS], l[ROWS].
        float* const wt = reinterpret_cast<float*>(smem + lay.warp_off);
        for (int row = warp; row < ROWS; row += W) {
            float m = -INFINITY;
            for (int i = lane; i < n; i += 32) m = fmaxf(m, __ldcg(cta_part(i) + ROWS * D + row));
#pragma unroll
            for (int d = 16; d > 0; d /= 2) m = fmaxf(m, __shfl_xor_sync(kFull, m, d));
            float l = 0.0f;
            for (int i = lane; i < n; i += 32) {
                const float f = m == -INFINITY ? 1.0f : exp2_fast(__ldcg(cta_part(i) + ROWS * D + row) - m);
                wt[row * n + i] = f;
                l = fmaf(__ldcg(cta_part(i) + ROWS * D + ROWS + row), f, l);
            }
#pragma unroll
            for (int d = 16; d > 0; d /= 2) l += __shfl_xor_sync(kFull, l, d);
            if (lane == 0) { wt[ROWS * n + row] = m; wt[ROWS * n + ROWS + row] = l; }
        }
        __syncthreads();
        for (int e = tid; e < ROWS * D / 4; e += 32 * W) {
            const int row = e / (D / 4), col = (e - row * (D / 4)) * 4;
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
            for (int i = 0; i < n; ++i) {
                const float f = wt[row * n + i];
                const float4 x = __ldcg(reinterpret_cast<const float4*>(cta_part(i) + row * D + col));
                v.x = fmaf(x.x, f, v.x); v.y = fmaf(x.y, f, v.y); v.z = fmaf(x.z, f, v.z); v.w = fmaf(x.w, f, v.w);
            }
            put(it, row, col, v, wt[ROWS * n + row], wt[ROWS * n + ROWS + row]);
        }
        __syncthreads();
    }
}

// What the host needs of an instantiation.
struct AttnKernel {
    const void* fn;
    int warps, partial;
    int (*smem)(int n_req, int depth);
};
template <typename T, int D, int ROWS, int TERMS> AttnKernel attn_kernel() {
    using S = AttnShape<D, ROWS, TERMS>;
    return {(const void*)&attention_kernel<T, D, ROWS, TERMS>, S::kWarps, S::kPartial,
            [](int n_req, int depth) { return attn_smem<D, ROWS, TERMS>(n_req, depth).total; }};
}

}  // namespace qg
