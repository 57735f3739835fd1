// Attention of new tokens over the paged 4-bit key/value cache (qg_attention): the kernel.
//
//     s_k = scale * q . key_k,   out = sum_k softmax(s)_k value_k,   lse = log sum_k exp(s_k)
//
// Work.  A row is one (new token, query head); the rows of a request that read the same
// key/value head are cut into tiles of ROWS, and an item is one (request, key/value head, row
// tile) with its visible keys in units of 32.  All items' units form one sequence, dealt in
// equal contiguous shares to the CTAs and, within a CTA, to its warps: a batch of any lengths
// loads every SM alike, and a single long request is split over all of them.  Each warp runs
// its part alone, with a running maximum and sum per row; parts of an item are joined in
// order, first the warps' within the CTA, then the CTAs' by the last of them to finish (a
// ticket; no CTA ever waits on another), so results do not change from run to run.
//
// Memory.  A unit's keys and values are two records of the cache, one bulk copy (two where
// they are not neighbours in a page) into the warp's own ring (mbarrier-counted, bounded
// waits), so the bytes in flight are set by shared memory and every byte is read from HBM
// once per row tile.  Page numbers are fetched a batch of 16 units ahead of their copies.
//
// Arithmetic.  The tensor cores' m16n8k16 (fp16 in, fp32 out) fits: a decode step has 1 to 32
// rows per key/value head, far below the 64 or 128 rows of a tcgen05 tile, and operands that
// come out of nibbles in registers would have to go back through shared or tensor memory for
// it.  Keys (then values, transposed) are the product's 16 rows, query rows its 8 columns.
// Every operand of the cache is exact:
//  * scores: a key's codes enter as they are, as fp16 subnormals (a shift and a mask per two
//    codes, no arithmetic); the sum starts at -8 * sum(q) of its block, and the block's scale
//    multiplies the fp32 result.  A query is scaled by a power of two to [2^14, 2^15) and split
//    into two fp16 terms (22 bits; one term is exact for bf16 queries).
//  * outputs: a value is (16 + code) * d - 24 * d in one fp16 FMA, exact because d has 8
//    significant bits (units with scales whose 24-fold fp16 does not hold take an addition and a
//    product instead); probabilities are two fp16 terms (one for bf16 outputs, below its
//    rounding), scaled by 2^7 relative to a reference that follows the running maximum within
//    2^8, so that outputs are rescaled rarely and a probability counts down to 2^-31 of the
//    row's largest.  Maxima, sums, outputs and joins are fp32.
//
// What bounds it (GB300, measured): per unit of a 128-wide head and 4 fp32 rows a warp issues
// about 670 instructions, 208 of them for the values' codes, 136 for the keys', 32 tensor
// products; on this tensor path a product (8 clocks per scheduler) does not overlap with fp32
// FMAs, which share its register ports.  The loop takes 0.80 ns per unit and GPU (4608 bytes:
// 5.8 TB/s; without its arithmetic 0.70 ns, 6.6 TB/s): memory and issue bound it together.  With
// 12 rows it takes about 990 instructions; neither memory, issue nor one pipe is full then, and three
// warps a scheduler do not cover the latencies that are left.
// Around the loop a call costs about 12 us (launch, lengths, first copies; the joins).
#pragma once

#include <type_traits>

#include <cuda_bf16.h>

#include "kv_layout.h"
#include "qgemv_kernels.cuh"

namespace qg {

constexpr int kUnit = 32;                 // keys per unit: two records
// An item's own cost (its queries, its outputs) in units, for the division of work: without it
// (0) a ragged batch of 64 took 133 us, with 2 it took 111; 3 to 9 measure alike.
constexpr int kItemCost = 4;
// The smallest share of a CTA, in units: 777 keys of 16 heads took 10.5 us with one unit per warp
// (16), 8.4 with 4, whose warps sit on the four schedulers; 2 measures as 4.
constexpr int kMinShare = 4;
constexpr int kMaxAttnReq = 1024;
constexpr int kAttnGrid = 160;             // most CTAs of a launch (one per SM; the workspace is sized by it)
static_assert(kAttnGrid * 4 <= QG_ATTENTION_ZERO_BYTES, "one ticket per CTA");
constexpr float kProbShift = 7.0f;        // probabilities are scaled by 2^7 ...
constexpr float kRefSlack = 8.0f;         // ... and the reference follows the maximum within 2^8: below 2^15
constexpr float kFarRef = 4096.0f;        // above it the exponent's argument is rounded like the reference (below)
constexpr float kNoRef = -3.0e38f;        // the reference before the first visible key: any score is above it
constexpr uint32_t kNoItem = 0xFFFFFFFFu;
constexpr uint32_t kMostPlaces = 0x7FFFFFFFu;    // a call's work, in places (units and kItemCost an item), stays below
constexpr int kMetaInts = 6;              // of an unfinished item: start, end, first token, new tokens, head, tile

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
    uint32_t group_inv, page_inv;    // floor(2^32 / x) (of 1: 2^32 - 1)
    float scale_log2;          // |scale| * log2(e) is scale_log2 * 2^scale_exp, scale_log2 in [0.5, 1]
    int scale_exp;             // (of a scale of 0: that of 1)
    float scale_sign;          // the scale's sign (0 for 0), which goes into the queries
    uint32_t wait_limit, drain_limit, test_extra_tx;
};

// How queries and probabilities enter the tensor core's fp16, in tiles of 8 columns:
//  kOne    one term a row, 8 rows to a tile (bf16 activations)
//  kSide   two terms side by side, 4 rows to a tile: for up to 4 rows half the products of kTwice
//          (and for 9 to 12 three quarters: 3 tiles against 2 of twice the products)
//  kTwice  two terms one after the other into one accumulator, 8 rows to a tile: as many products
//          per row in full tiles, without kSide's sums of neighbouring columns (8 rows of 32771
//          keys and 8 heads: 24.6 us against 25.5)
enum { kOne = 1, kSide = 2, kTwice = 3 };
template <int D, int TILES, int TERMS> struct AttnShape {
    static constexpr int kLaneRows = TERMS == kSide ? 1 : 2;         // rows a lane holds per tile
    static constexpr int kTileRows = 4 * kLaneRows;
    static constexpr int kMats = TERMS == kTwice ? 2 : 1;            // operand matrices
    static constexpr int kRows = TILES * kTileRows;
    // One tile leaves 128 registers a thread enough: 16 warps (262,100 keys of 8 heads: 64 us
    // against 68 with 12).  More tiles take 168 (12 warps; with 8 warps of 255, 12 rows of 32771
    // keys took 49 us against 44).  Heads of 256 have shared memory for 9 warps of one tile, but a
    // ninth gives one scheduler a warp more than the others, and all wait for that one: 12 requests
    // of up to 20000 keys took 42 us with 9 and 33 with 8 (bf16; fp32: 35 and 30).  Three tiles of
    // them leave room for 7.
    static constexpr int kWarps = D == 256 ? (kMats * TILES == 3 ? 7 : 8) : kMats * TILES == 1 ? 16 : 12;
    static constexpr int kCodeBits = TERMS == kOne ? 24 : 20;                    // a code of 1 stands for 2^-kCodeBits
    static constexpr float kCodeUnit = 1.0f / (1 << kCodeBits);
    static constexpr float kOddScale = TERMS == kOne ? 0.0625f : 1.0f;
    static constexpr int kRec = kv_record_bytes(D);
    static constexpr int kStage = 2 * kRec;
    static constexpr int kQBytes = kMats * TILES * kv_groups(D) * 512;    // queries in operand order
    static constexpr int kInitBytes = TILES * (kv_groups(D) + 1) * 32;    // -8 * sum(q) per block and column; factors
    static constexpr int kPartial = kRows * (D + 2);                 // floats: [rows][D], m[rows], l[rows]
};

// Shared memory: prefix of units per request, the warps' records of unfinished items, then
// per warp its barriers, queries and ring.
struct AttnSmem { int seq_off, new_off, meta_off, warp_off, bar_off, q_off, init_off, warp_bytes, total; };
template <int D, int TILES, int TERMS> __host__ __device__ inline AttnSmem attn_smem(int n_req, int depth) {
    using S = AttnShape<D, TILES, TERMS>;
    AttnSmem p;
    p.seq_off = (n_req + 1) * 4;                     // after the prefix: lengths, then first new tokens
    p.new_off = p.seq_off + n_req * 4;
    p.meta_off = p.new_off + (n_req + 1) * 4;
    p.warp_off = (p.meta_off + (S::kWarps + 2 * S::kWarps * kMetaInts + 2) * 4 + 127) / 128 * 128;
    p.q_off = depth * S::kStage;                     // a warp's ring comes first
    p.init_off = p.q_off + S::kQBytes;
    p.bar_off = p.init_off + S::kInitBytes;
    p.warp_bytes = (p.bar_off + depth * 8 + 127) / 128 * 128;
    p.total = p.warp_off + S::kWarps * p.warp_bytes;
    return p;
}

// ------------------------------------------------------------------------------ PTX helpers

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 :: "r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}
__device__ __forceinline__ void prefetch_l1(const void* p) { asm volatile("prefetch.global.L1 [%0];" :: "l"(p)); }
// d = a b + {c0, c1, c0, c1}: an accumulator of its own, so that a start value costs no moves.
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1, float c0, float c1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%10,%11};"
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
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
// The four pairs of codes of a key word (nibbles i and i + 4) as fp16 subnormals: code * 2^-20,
// or with COARSE code * 2^-24 and code * 2^-20 in turn (two shifts less; the queries of the odd
// pairs then carry 2^-4).  The tensor core aligns products by their exponent fields, so
// 2^-24 costs 6 bits of the sum (measured 9 ulps rms against 0.17): it serves bf16 only.
template <bool COARSE> __device__ __forceinline__ void key_codes(uint32_t w, uint32_t (&b)[4]) {
    const uint32_t m = 0x00F000F0u;
    if (COARSE) {
        const uint32_t v = w >> 8, l = 0x000F000Fu;
        b[0] = w & l;
        b[1] = w & m;
        b[2] = v & l;
        b[3] = v & m;
    } else {
        b[0] = (w << 4) & m;
        b[1] = w & m;
        b[2] = (w >> 4) & m;
        b[3] = (w >> 8) & m;
    }
}
// The four value pairs of a word (nibble n of two tokens) times the tokens' scales d: with the
// nibble in bits 6..9 under the exponent of 16, (16 + code) * d - 24 * d in one rounding, of
// an exact result.  The mask and the exponent come in registers, so that one three-input
// logic instruction places a pair.  24 * d is finite in fp16 for |d| <= 2720 (kFmaScale, blocks
// of magnitudes up to 21760); LARGE is for any scale: (16 + code) - 24, then times d, both exact.
constexpr uint32_t kFmaScale = 0x6950u;                  // 2720 in fp16
template <bool LARGE> __device__ __forceinline__ void value_pairs(uint32_t w, uint32_t d, uint32_t mask, uint32_t magic, uint32_t (&v)[4]) {
    const __half2 e = bits_h2(d), minus = __float2half2_rn(-24.0f), less = __hmul2(e, minus);
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        const uint32_t t = n == 0 ? w << 6 : n == 1 ? w << 2 : n == 2 ? w >> 2 : w >> 6;
        uint32_t x;
        asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(x) : "r"(t), "r"(mask), "r"(magic));
        v[n] = h2_bits(LARGE ? __hmul2(__hadd2(bits_h2(x), minus), e) : __hfma2(bits_h2(x), e, less));
    }
}
// A value the compiler does not see through.
__device__ __forceinline__ uint32_t opaque(uint32_t x) {
    uint32_t y;
    asm volatile("mov.b32 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// The transpose of an 8x8 matrix of fp16: lane 4 r + c holds row r, columns 2 c and 2 c + 1.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
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
__device__ __forceinline__ float2 lds_f2(uint32_t a) {
    float2 v;
    asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a));
    return v;
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

__device__ __forceinline__ void store2(float* p, float a, float b) { *reinterpret_cast<float2*>(p) = make_float2(a, b); }
__device__ __forceinline__ void store2(__nv_bfloat16* p, float a, float b) {
    *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(a, b);
}
// Takes a ticket: what the CTA wrote before (and a barrier ordered) is seen by whoever takes a
// later one, and what others wrote before theirs is seen here.
__device__ __forceinline__ uint32_t ticket_add(uint32_t* p) {
    uint32_t old;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(old) : "l"(p) : "memory");
    return old;
}

// A lane's V values of a row that another CTA wrote.
template <int V> __device__ __forceinline__ void load_row_l2(const float* p, int lane, float (&x)[V]) {
    if constexpr (V == 2) {
        const float2 y = __ldcg(reinterpret_cast<const float2*>(p + 2 * lane));
        x[0] = y.x; x[1] = y.y;
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 y = __ldcg(reinterpret_cast<const float4*>(p + 32 * i + 4 * lane));
            x[i] = y.x; x[i + 1] = y.y; x[i + 2] = y.z; x[i + 3] = y.w;
        }
    }
}

// ------------------------------------------------------------------------------ work

// i / d with inv = floor(2^32 / d): the high product is the quotient or one less.
__device__ __forceinline__ uint32_t divide(uint32_t i, uint32_t d, uint32_t inv) {
    const uint32_t q = __umulhi(i, inv);
    return q + (i - q * d >= d);
}

// A request's share of the work: its visible keys in units (from the first one a window
// leaves) and its row tiles.
struct Request {
    int seq, first_tok, fresh, first_unit, units, tiles;
};
template <int ROWS> __device__ __forceinline__ Request request_of(const AttnArgs& a, int seq, int first_tok, int end) {
    Request q;
    q.seq = seq;
    q.first_tok = first_tok;
    q.fresh = end - first_tok;
    q.first_unit = a.window > 0 ? max(0, seq - q.fresh + 1 - a.window) / kUnit : 0;
    q.units = max(1, int((unsigned(seq) + kUnit - 1) / kUnit) - q.first_unit);
    q.tiles = int((uint32_t(q.fresh) * uint32_t(a.group) + ROWS - 1) / ROWS);      // rows: below 2^32 (they are in memory)
    return q;
}

// The CTA's view of the batch: units prefixed over the requests, their lengths, their tokens.
struct Batch {
    const uint32_t* cum;
    const int *seq, *first;
    int n_req;
};

// An item, decoded from a place in the sequence: kItemCost places that stand for the item's own
// cost, so that CTAs with many short items get no more work than others, then its units.
struct Item {
    Request rq;
    int r, head, tile, unit;       // unit: within the item
    uint32_t start;                // the item's first unit in the sequence: its identity
    uint32_t end;
};
template <int ROWS> __device__ __forceinline__ Item item_at(const AttnArgs& a, const Batch& b, int r, uint32_t u) {
    int hi = b.n_req;              // the request whose units hold u, searched from r on (units only grow)
    while (hi - r > 1) {
        const int mid = (r + hi) >> 1;
        if (b.cum[mid] <= u) r = mid; else hi = mid;
    }
    Item it;
    it.r = r;
    it.rq = request_of<ROWS>(a, b.seq[r], b.first[r], b.first[r + 1]);
    const uint32_t length = uint32_t(it.rq.units + kItemCost), rem = u - b.cum[r], n = rem / length;
    it.head = it.rq.tiles == 1 ? int(n) : int(n / uint32_t(it.rq.tiles));
    it.tile = int(n - uint32_t(it.head) * uint32_t(it.rq.tiles));
    it.start = b.cum[r] + n * length + kItemCost;
    it.end = it.start + uint32_t(it.rq.units);
    it.unit = u > it.start ? int(u - it.start) : 0;
    return it;
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
    j = int(divide(uint32_t(i), uint32_t(a.group), a.group_inv));
    head = it.head * a.group + (i - j * a.group);
    if (j >= it.rq.fresh) j = -1;
}

// ------------------------------------------------------------------------------ kernel

template <typename T, int D, int TILES, int TERMS>
__global__ void __launch_bounds__(32 * AttnShape<D, TILES, TERMS>::kWarps, 1) attention_kernel(const AttnArgs a) {
    using S = AttnShape<D, TILES, TERMS>;
    constexpr int W = S::kWarps, NG = kv_groups(D), GI = kv_set(D), NS = NG / GI;
    constexpr int ROWS = S::kRows, H = S::kLaneRows;
    extern __shared__ __align__(128) uint8_t smem[];
    const AttnSmem lay = attn_smem<D, TILES, TERMS>(a.n_req, a.depth);
    uint32_t* const cum = reinterpret_cast<uint32_t*>(smem);
    int* const seqs = reinterpret_cast<int*>(smem + lay.seq_off);
    int* const firsts = reinterpret_cast<int*>(smem + lay.new_off);
    const Batch batch{cum, seqs, firsts, a.n_req};
    uint32_t* const wsum = reinterpret_cast<uint32_t*>(smem + lay.meta_off);      // [W]
    uint32_t* const meta = wsum + W;                                              // [W][2][kMetaInts], then two flags
    const int tid = int(threadIdx.x), lane = tid & 31;
    // A warp's place in the CTA's share: neighbours in the share sit on different schedulers, so
    // that a share of few units is spread over all four.
    const int warp = W % 4 == 0 ? (tid >> 5) % (W / 4) * 4 + (tid >> 5) / (W / 4) : tid >> 5;
    const int r8 = lane >> 2, c4 = lane & 3;               // operand row and column group
    uint8_t* const mine = smem + lay.warp_off + warp * lay.warp_bytes;
    const uint32_t ring = smem_addr(mine), qmat = ring + lay.q_off, binit = ring + lay.init_off, bars = ring + lay.bar_off;

    if (lane < a.depth) mbar_init(bars + 8 * lane, 1);
    mbar_fence_init();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // ---- units per request, prefixed
    uint32_t run = 0;
    bool bad_len = false, bad_page = false;
    // A request's units; its lengths go to shared memory for later decoding.
    auto units_of = [&](int r) -> uint32_t {
        const int seq = a.seq_len[r], first = a.cu_new[r], end = a.cu_new[r + 1];
        // (The new tokens are in the cache: with fewer tokens than those the positions would be negative.)
        const bool ok = first >= 0 && end >= first && seq >= end - first && end <= a.n_tok && !(a.span_mask && end - first > 32);
        // Records beyond the table's row cannot be found: such a request is left out whole.
        const bool fits = ((long long)seq + kRecordTokens - 1) / kRecordTokens <= a.table_stride * a.page_records;
        bad_len |= !ok;
        bad_page |= ok && !fits;
        seqs[r] = seq;
        firsts[r] = first;
        if (r == a.n_req - 1) firsts[r + 1] = end;
        if (!ok || !fits || end == first) return 0;
        const Request q = request_of<ROWS>(a, seq, first, end);
        const unsigned long long n = (unsigned long long)(q.units + kItemCost) * unsigned(q.tiles) * unsigned(a.n_kv);
        bad_len |= n >= kMostPlaces;
        return n < kMostPlaces ? uint32_t(n) : 0u;
    };
    // Sums of places stop at kMostPlaces, so a sequence that is too long shows in its total.
    auto add = [](uint32_t x, uint32_t y) { return min(x + y, kMostPlaces); };
    // Where it is: requests are taken in order, those that no longer fit are left out.
    auto take = [&](uint32_t& used, uint32_t n) -> uint32_t {
        const uint32_t at = used;
        if (n < kMostPlaces - used) used += n;
        else if (n > 0) bad_len = true;
        return at;
    };
    if (lane < 2) meta[(2 * warp + lane) * kMetaInts] = kNoItem;
    if (a.n_req <= 32) {
        // One warp's worth: every warp computes (and writes) the same values, none waits.
        const uint32_t n = lane < a.n_req ? units_of(lane) : 0u;
        run = n;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const uint32_t up = __shfl_up_sync(kFull, run, d);
            if (lane >= d) run = add(run, up);
        }
        uint32_t at = run - n;
        run = __shfl_sync(kFull, run, 31);
        if (run == kMostPlaces) {
            run = 0;
            for (int r = 0; r < a.n_req; ++r) {
                const uint32_t before = take(run, __shfl_sync(kFull, n, r));
                if (lane == r) at = before;
            }
        }
        if (lane < a.n_req) cum[lane] = at;
        if (lane == 0) cum[a.n_req] = run;
        __syncwarp();
    } else {
        for (int r0 = 0; r0 < a.n_req; r0 += 32 * W) {
            const int r = r0 + tid;
            const uint32_t n = r < a.n_req ? units_of(r) : 0u;
            uint32_t s = n;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const uint32_t up = __shfl_up_sync(kFull, s, d);
                if (lane >= d) s = add(s, up);
            }
            if (lane == 31) wsum[tid >> 5] = s;
            __syncthreads();
            uint32_t before = run;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const uint32_t x = wsum[w];
                if (w < (tid >> 5)) before = add(before, x);
                run = add(run, x);
            }
            if (r < a.n_req) cum[r] = add(before, s) - n;
            __syncthreads();
        }
        if (run == kMostPlaces) {                          // (the same for the whole CTA)
            for (int r = tid; r < a.n_req; r += 32 * W) cum[r] = units_of(r);
            __syncthreads();
            if (tid == 0) {
                run = 0;
                for (int r = 0; r < a.n_req; ++r) cum[r] = take(run, cum[r]);
                wsum[0] = run;
            }
            __syncthreads();
            run = wsum[0];
        }
        if (tid == 0) cum[a.n_req] = run;
        __syncthreads();
    }
    if (blockIdx.x == 0 && bad_len) atomicOr(a.status, kStatusBadLength);
    if (blockIdx.x == 0 && bad_page) atomicOr(a.status, kStatusBadPage);
    const uint32_t total = run;
    const uint32_t share = max((total + gridDim.x - 1) / gridDim.x, uint32_t(kMinShare));
    const uint32_t c0 = min(share * blockIdx.x, total), c1 = min(c0 + share, total);
    if (c0 == c1) return;
    const uint32_t u0 = c0 + uint32_t((unsigned long long)(c1 - c0) * warp / W);
    const uint32_t u1 = c0 + uint32_t((unsigned long long)(c1 - c0) * (warp + 1) / W);

    // ---- records, found a batch (up to 16 units of one item) ahead of their copies: lanes 2 i
    // and 2 i + 1 hold those of the batch's unit i.  A record past the request's last, or wholly
    // before its window (its page may be gone), is replaced by the unit's other one, a record of
    // a page that does not exist by the cache's first (and reported): every unit is two records,
    // and what a replacement brings is masked or not valid anyway.
    uint32_t au = u0, next_rec = 0, cur_rec = 0;
    int ar = 0, next_count = 0, count = 0, at = 0, next_page = 0;
    auto fetch_from = [&](const Item& it) {
        ar = it.r;
        if (it.start >= u1) return;
        next_count = min(min(16, it.rq.units - it.unit), int(u1 - max(au, it.start)));
        au = max(au, it.start) + next_count;
        const uint32_t base = 2 * uint32_t(it.rq.first_unit + it.unit);
        uint32_t rec = lane < 2 * next_count ? base + lane : base;
        if (rec * kRecordTokens >= unsigned(it.rq.seq)) rec &= ~1u;
        // (Records end at 2^31 at most: past int.)
        const int visible = a.window > 0 ? max(0, it.rq.seq - it.rq.fresh + 1 - a.window) : 0;
        if ((rec + 1) * kRecordTokens <= unsigned(visible)) rec |= 1u;
        const uint32_t page = divide(rec, uint32_t(a.page_records), a.page_inv);
        next_rec = uint32_t(it.head) * uint32_t(a.page_records) + (rec - page * uint32_t(a.page_records));
        next_page = it.rq.seq > 0 ? a.table[(long long)ar * a.table_stride + page] : 0;
        if (it.unit == 0) {                    // the item's queries, for when it begins
            for (int i = lane; i < ROWS * D * int(sizeof(T)) / 128; i += 32) {
                int j, head;
                row_of<ROWS>(a, it, i * 128 / (D * int(sizeof(T))), j, head);
                if (j >= 0)
                    prefetch_l1(static_cast<const T*>(a.q) + (long long)(it.rq.first_tok + j) * a.q_stride + (long long)head * D +
                                i * (128 / int(sizeof(T))) % D);
            }
        }
    };
    auto fetch = [&]() {
        next_count = 0;
        if (au < u1) fetch_from(item_at<ROWS>(a, batch, ar, au));
    };
    auto turn_batch = [&]() {
        if (next_page < 0 || next_page >= a.n_pages) {
            atomicOr(a.status, kStatusBadPage);
            next_page = 0;
        }
        cur_rec = uint32_t(next_page) * uint32_t(a.n_kv * a.page_records) + next_rec;
        count = next_count;
        at = 0;
        fetch();
    };
    // ---- the ring
    uint32_t issued = 0, consumed = 0;
    int in_stage = 0, out_stage = 0;
    uint32_t out_phase = 0;
    auto issue = [&](uint32_t extra_tx) {
        if (at == count) {
            if (next_count == 0) return;
            turn_batch();
        }
        const uint32_t rec0 = __shfl_sync(kFull, cur_rec, 2 * at), rec1 = __shfl_sync(kFull, cur_rec, 2 * at + 1);
        if (lane == 0) {
            const uint32_t bar = bars + 8 * in_stage, to = ring + in_stage * S::kStage;
            const uint8_t* const from = a.data + uint64_t(rec0) * S::kRec;
            mbar_arrive_expect_tx(bar, S::kStage + extra_tx);
            if (rec1 == rec0 + 1) {                        // neighbours in a page: one copy
                bulk_load(to, from, S::kStage, bar);
            } else {
                bulk_load(to, from, S::kRec, bar);
                bulk_load(to + S::kRec, a.data + uint64_t(rec1) * S::kRec, S::kRec, bar);
            }
        }
        ++at;
        ++issued;
        in_stage = in_stage + 1 == a.depth ? 0 : in_stage + 1;
    };

    // ---- the warp's part, item by item
    const uint32_t mask = opaque(0x03C003C0u), magic = opaque(0x4C004C00u);
    bool dead = false;
    uint32_t u = u0;
    int r = 0;
    while (u < u1) {
        const Item it = item_at<ROWS>(a, batch, r, u);
        if (u == u0) fetch_from(it);
        r = it.r;
        u = max(u, it.start);
        if (u >= u1) break;
        const int begin = it.rq.seq - it.rq.fresh;

        // Queries as operand columns: this lane's column is r8, a term of a row (or the row itself),
        // its values 8 c4 .. 8 c4 + 7 of every block.  The first item's are requested before the
        // ring's first copies, behind which they would wait.
        float x[TILES][NG][8];
#pragma unroll
        for (int t = 0; t < TILES; ++t) {
            int j, head;
            row_of<ROWS>(a, it, t * S::kTileRows + (TERMS == kSide ? r8 / 2 : r8), j, head);
            const T* src_row = static_cast<const T*>(a.q) + (long long)(it.rq.first_tok + max(j, 0)) * a.q_stride +
                               (long long)head * D + 8 * c4;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                if (j >= 0) {
                    load8(src_row + 32 * g, x[t][g]);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[t][g][i] = 0.0f;
                }
            }
        }
        // The first stage of every warp before the others: all warps start on the first bytes to
        // arrive, not on the last of a burst of whole rings.
        const bool starting = issued == 0;
        if (starting) issue(a.test_extra_tx);
#pragma unroll
        for (int t = 0; t < TILES; ++t) {
            float top = 0.0f;
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int i = 0; i < 8; ++i) top = max_nan(top, fabsf(x[t][g][i]));
            top = max_nan(top, __shfl_xor_sync(kFull, top, 1));
            top = max_nan(top, __shfl_xor_sync(kFull, top, 2));
            // 2^s brings the row's largest magnitude to [2^14, 2^15) (s at most 126); a row with a
            // NaN or an infinity has NaN scores.
            const int e = int((__float_as_uint(top) & 0x7FFFFFFFu) >> 23);
            const int sh = min(141 - e, 126);
            const float up = __uint_as_float(uint32_t(127 + sh) << 23) * a.scale_sign;
            const bool finite = e < 255;
            float* const init = reinterpret_cast<float*>(mine + lay.init_off) + t * (NG + 1) * 8;
            // The scores' factor in one step, so that no part of it leaves fp32's range; where the whole
            // does, it stays positive and finite: a masked -infinity stays one and a zero a zero.
            const float factor = fminf(fmaxf(ldexpf(a.scale_log2, a.scale_exp + S::kCodeBits - sh), 1.17549435e-38f), 3.40282347e38f);
            if (c4 == 0) init[NG * 8 + r8] = finite ? factor : __uint_as_float(0x7FFFFFFFu);
            // The first of two terms is cut off at 11 bits, the second is the rest (kSide: in the odd column).
            const float rest = TERMS == kSide && (r8 & 1) ? 1.0f : 0.0f;
            const uint32_t minus = TERMS == kSide && (r8 & 1) ? 0x80000000u : 0u;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                uint32_t v[S::kMats][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float w = (i & 1) ? up * S::kOddScale : up;
                    float p = finite ? x[t][g][i] * w : 0.0f, q = finite ? x[t][g][i + 4] * w : 0.0f;
                    if (TERMS != kOne) {
                        const float cp = __uint_as_float((__float_as_uint(p) & 0xFFFFE000u) ^ minus);
                        const float cq = __uint_as_float((__float_as_uint(q) & 0xFFFFE000u) ^ minus);
                        if (TERMS == kTwice) v[S::kMats - 1][i] = h2_bits(__floats2half2_rn(p - cp, q - cq));
                        p = TERMS == kSide ? fmaf(rest, p, cp) : cp;
                        q = TERMS == kSide ? fmaf(rest, q, cq) : cq;
                    }
                    v[0][i] = h2_bits(__floats2half2_rn(p, q));
                }
                // -8 * (sum of the column): a product with a matrix of -8 (-128 where the odd pairs
                // carry 2^-4), which also puts it where the scores' product wants it.
                const uint32_t eight = 0xC800C800u, odd8 = TERMS == kOne ? 0xD800D800u : eight;
                const uint4 a8 = make_uint4(eight, eight, odd8, odd8);
                float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int m = S::kMats - 1; m >= 0; --m) {
                    *reinterpret_cast<uint4*>(mine + lay.q_off + (((m * TILES + t) * NG + g) * 32 + lane) * 16) =
                        make_uint4(v[m][0], v[m][1], v[m][2], v[m][3]);
                    mma_f16(c, a8, v[m][0], v[m][1]);
                    mma_f16(c, a8, v[m][2], v[m][3]);
                }
                if (r8 == 0) *reinterpret_cast<float2*>(init + g * 8 + 2 * c4) = make_float2(c[0] * S::kCodeUnit, c[1] * S::kCodeUnit);
            }
        }
        __syncwarp();
        if (starting)
            for (int i = 1; i < a.depth; ++i) issue(0u);
        // Keys that every row sees lie in (full_low, full_high]; any row's in (any_low, any_high].
        const int i0 = it.tile * ROWS, i1 = min(i0 + ROWS, it.rq.fresh * a.group) - 1;
        const int low_pos = begin + int(divide(uint32_t(i0), uint32_t(a.group), a.group_inv));
        const int any_high = begin + int(divide(uint32_t(i1), uint32_t(a.group), a.group_inv));
        const int full_high = a.span_mask ? min(low_pos, begin - 1) : low_pos;
        const int full_low = a.window > 0 ? any_high - a.window : -1;
        const int any_low = a.window > 0 ? low_pos - a.window : -1;
        // What this lane's row h of tile t may see (in units that need it).
        auto sight = [&](int t, int h) {
            int j, head;
            row_of<ROWS>(a, it, t * S::kTileRows + H * c4 + h, j, head);
            Sight s;
            s.pos = j < 0 ? -1 : begin + j;
            s.low = a.window > 0 ? begin + j - a.window : -1;
            s.begin = a.span_mask ? begin : 0x7FFFFFFF;
            s.bits = a.span_mask && j >= 0 ? a.span_mask[it.rq.first_tok + j] : 0u;
            return s;
        };

        // Running outputs: of this lane's rows, value 4 r8 + n of block g.
        float o[TILES][4 * NG][H], ref[TILES][H], sum[TILES][H];
        bool far = false;                                  // some row's reference is above kFarRef (the warp's)
#pragma unroll
        for (int t = 0; t < TILES; ++t)
#pragma unroll
            for (int h = 0; h < H; ++h) {
#pragma unroll
                for (int n = 0; n < 4 * NG; ++n) o[t][n][h] = 0.0f;
                ref[t][h] = kNoRef;
                sum[t][h] = 0.0f;
            }

        const uint32_t item_end = min(it.end, u1);
        int key0 = (it.rq.first_unit + it.unit) * kUnit;
        for (; u < item_end; ++u, key0 = int(unsigned(key0) + kUnit)) {      // (past int after the last unit of 2^31 - 1 keys)
            const uint32_t stage = ring + out_stage * S::kStage;
            if (!__all_sync(kFull, mbar_try_wait(bars + 8 * out_stage, out_phase))) {
                if (!dead) dead = __any_sync(kFull, !mbar_wait(bars + 8 * out_stage, out_phase, a.wait_limit));
                if (dead) {
                    // Gave up: no more copies; the ones in flight land (bounded again) before the
                    // ring is reused or the CTA ends.  The rest of the part is passed over.
                    if (lane == 0) atomicOr(a.status, kStatusWaitTimeout);
                    for (; consumed < issued; ++consumed) {
                        mbar_wait(bars + 8 * out_stage, out_phase, a.drain_limit);
                        out_stage = out_stage + 1 == a.depth ? 0 : out_stage + 1;
                        if (out_stage == 0) out_phase ^= 1;
                    }
                    u = u1;
                    break;
                }
            }

            // ---- scores: keys are the product's rows (16 per record: r8 and r8 + 8), query columns
            // its columns
            float p[TILES][2][2][H];                       // [record][key r8, r8 + 8]
            uint32_t kw[2][2][NG];
            uint32_t kd[2][NG];                            // scales of keys r8 and r8 + 8
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t rec = stage + k * S::kRec;
#pragma unroll
                for (int q = 0; q < NS; ++q) {
                    uint32_t d0[GI], d1[GI];
                    lds_words<GI>(rec + ((q * 16) * 4 + lane) * GI * 4, &kw[k][0][q * GI]);
                    lds_words<GI>(rec + ((q * 16 + 8) * 4 + lane) * GI * 4, &kw[k][1][q * GI]);
                    lds_words<GI>(rec + kv_k_scales(D) + ((r8 >> 1) * NG + q * GI) * 4, d0);
                    lds_words<GI>(rec + kv_k_scales(D) + ((4 + (r8 >> 1)) * NG + q * GI) * 4, d1);
#pragma unroll
                    for (int i = 0; i < GI; ++i) kd[k][q * GI + i] = __byte_perm(d0[i], d1[i], (r8 & 1) ? 0x7632 : 0x5410);
                }
            }
            // Whether any value scale of the unit's 32 NG (a lane looks at NG / 2 pairs) is above kFmaScale:
            // its half of the sum reaches its top bit then.
            uint32_t above = 0;
#pragma unroll
            for (int i = 0; i < NG / 2; ++i) {
                const int at = 32 * i + lane;
                const uint32_t pair = lds32(stage + at / (8 * NG) * S::kRec + kv_v_scales(D) + at % (8 * NG) * 4);
                above |= (pair & 0x7FFF7FFFu) + (0x7FFFu - kFmaScale) * 0x10001u;
            }
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                uint4 qb[TILES], ql[TILES];
                float2 start[TILES];
#pragma unroll
                for (int t = 0; t < TILES; ++t) {
                    qb[t] = lds128(qmat + ((t * NG + g) * 32 + lane) * 16);
                    if (TERMS == kTwice) ql[t] = lds128(qmat + (((TILES + t) * NG + g) * 32 + lane) * 16);
                    start[t] = lds_f2(binit + ((t * (NG + 1) + g) * 8 + 2 * c4) * 4);
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    uint32_t x[4], y[4];
                    key_codes<TERMS == kOne>(kw[k][0][g], x);
                    key_codes<TERMS == kOne>(kw[k][1][g], y);
                    const uint4 a0 = make_uint4(x[0], y[0], x[1], y[1]), a1 = make_uint4(x[2], y[2], x[3], y[3]);
                    const float2 d = __half22float2(bits_h2(kd[k][g]));
#pragma unroll
                    for (int t = 0; t < TILES; ++t) {
                        float acc[4];
                        mma_f16(acc, a0, qb[t].x, qb[t].y, start[t].x, start[t].y);
                        mma_f16(acc, a1, qb[t].z, qb[t].w);
                        if (TERMS == kTwice) {
                            mma_f16(acc, a0, ql[t].x, ql[t].y);
                            mma_f16(acc, a1, ql[t].z, ql[t].w);
                        }
                        float(&to)[2][H] = p[t][k];
                        if (TERMS == kSide) {
                            const float v = acc[0] + acc[1], w = acc[2] + acc[3];
                            to[0][0] = g == 0 ? v * d.x : fmaf(v, d.x, to[0][0]);
                            to[1][0] = g == 0 ? w * d.y : fmaf(w, d.y, to[1][0]);
                        } else {
#pragma unroll
                            for (int h = 0; h < H; ++h) {
                                to[0][h] = g == 0 ? acc[h] * d.x : fmaf(acc[h], d.x, to[0][h]);
                                to[1][h] = g == 0 ? acc[2 + h] * d.y : fmaf(acc[2 + h], d.y, to[1][h]);
                            }
                        }
                    }
                }
            }
            const bool masked = key0 + kUnit - 1 > full_high || key0 <= full_low;
            uint32_t pb[S::kMats][TILES][2][2];            // probabilities as operand columns
            bool grow = false;
            float top[TILES][H], factor[TILES][H];
#pragma unroll
            for (int t = 0; t < TILES; ++t) {
                const float2 f = lds_f2(binit + ((t * (NG + 1) + NG) * 8 + 2 * c4) * 4);
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    factor[t][h] = h ? f.y : f.x;
                    if (masked) {
                        const Sight s = sight(t, h);
#pragma unroll
                        for (int k = 0; k < 2; ++k)
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                if (!s.sees(key0 + 16 * k + 8 * i + r8)) p[t][k][i][h] = -INFINITY;
                    }
                    float m = fmaxf(fmaxf(p[t][0][0][h], p[t][0][1][h]), fmaxf(p[t][1][0][h], p[t][1][1][h]));
                    m = fmaxf(m, __shfl_xor_sync(kFull, m, 4));
                    m = fmaxf(m, __shfl_xor_sync(kFull, m, 8));
                    m = fmaxf(m, __shfl_xor_sync(kFull, m, 16));
                    top[t][h] = __fmul_rn(m, factor[t][h]);
                    grow |= __fsub_rn(top[t][h], ref[t][h]) > kRefSlack;
                }
            }
            // ---- running reference and sum; what a unit seldom needs is behind one vote.  (Large values
            // and far scores cost the units that have neither 3%: 262,100 keys 65.3 -> 67.2 us, a large
            // batch 130 -> 134, a bf16 one 85.5 -> 88.3.  With a branch per block of values instead of a
            // second body for them, and far scores behind a vote of their own, it was 5%.)
            float base[TILES][H];
#pragma unroll
            for (int t = 0; t < TILES; ++t)
#pragma unroll
                for (int h = 0; h < H; ++h) base[t][h] = kProbShift - ref[t][h];
            bool large = false;
            if (__any_sync(kFull, grow || far || (above & 0x80008000u) != 0)) {
                large = __any_sync(kFull, (above & 0x80008000u) != 0);
                far = false;
#pragma unroll
                for (int t = 0; t < TILES; ++t)
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        const float to = fmaxf(ref[t][h], top[t][h]), keep = exp2_fast(ref[t][h] - to);
                        ref[t][h] = to;
                        base[t][h] = kProbShift - to;
                        far |= fabsf(to) > kFarRef && to != kNoRef;
                        sum[t][h] *= keep;
#pragma unroll
                        for (int n = 0; n < 4 * NG; ++n) o[t][n][h] *= keep;
                    }
                // A reference is a rounded product, the fused argument below an exact one: by half a last bit
                // of the reference apart (2^-12 at kFarRef, more than an exponent holds at 2^30).  Scores as
                // large as that are rounded as the reference was and subtracted from it, which is exact.
                far = __any_sync(kFull, far);
                if (far) {
#pragma unroll
                    for (int t = 0; t < TILES; ++t)
#pragma unroll
                        for (int h = 0; h < H; ++h) {
#pragma unroll
                            for (int k = 0; k < 2; ++k)
#pragma unroll
                                for (int i = 0; i < 2; ++i)
                                    p[t][k][i][h] = __fsub_rn(__fmul_rn(p[t][k][i][h], factor[t][h]), ref[t][h]);
                            factor[t][h] = 1.0f;
                            base[t][h] = kProbShift;
                        }
                }
            }
#pragma unroll
            for (int t = 0; t < TILES; ++t) {
#pragma unroll
                for (int h = 0; h < H; ++h) {
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int i = 0; i < 2; ++i) p[t][k][i][h] = exp2_fast(fmaf(p[t][k][i][h], factor[t][h], base[t][h]));
                    sum[t][h] += (p[t][0][0][h] + p[t][0][1][h]) + (p[t][1][0][h] + p[t][1][1][h]);
                }
                // A key's row of operand columns is the transpose of what the product takes.  The
                // first term is cut off at 11 bits (exact in fp16), the second is the rest rounded.
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float x = p[t][k][i][0], y = p[t][k][i][H - 1];
                        const float cx = __uint_as_float(__float_as_uint(x) & 0xFFFFE000u), cy = __uint_as_float(__float_as_uint(y) & 0xFFFFE000u);
                        pb[0][t][k][i] = transpose8(h2_bits(TERMS == kSide ? __floats2half2_rn(cx, x - cx)
                                                            : TERMS == kTwice ? __floats2half2_rn(cx, cy) : __floats2half2_rn(x, y)));
                        if (TERMS == kTwice) pb[S::kMats - 1][t][k][i] = transpose8(h2_bits(__floats2half2_rn(x - cx, y - cy)));
                    }
            }

            // ---- outputs, transposed: values are the product's rows.  The unit's products go into
            // accumulators of their own and are added to the running outputs in fp32 (the tensor
            // core truncates what it adds to: over a long cache that bias would grow with the
            // number of units).
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
#pragma unroll
                            for (int t = 0; t < TILES; ++t)
#pragma unroll
                                for (int h = 0; h < H; ++h) {
                                    const Sight s = sight(t, h);
                                    float spoil = 0.0f;
                                    for (int k = 0; k < kUnit; ++k) {
                                        const uint32_t x = lds16(stage + k / kRecordTokens * S::kRec + kv_v_scales(D) +
                                                                 kv_scale(D, k % kRecordTokens, q * GI + i));
                                        if ((x & 0x7C00u) == 0x7C00u && s.sees(key0 + k)) spoil = NAN;
                                    }
#pragma unroll
                                    for (int n = 0; n < 4; ++n) o[t][4 * (q * GI + i) + n][h] += spoil;
                                }
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                if ((d[k][i] & 0x7C00u) == 0x7C00u) d[k][i] &= 0xFFFF0000u;
                                if ((d[k][i] & 0x7C000000u) == 0x7C000000u) d[k][i] &= 0xFFFFu;
                            }
                        }
                    }
                }
                auto products = [&](auto any_scale) {
#pragma unroll
                    for (int i = 0; i < GI; ++i) {
                        uint32_t v[4][4];                      // [half][nibble]
#pragma unroll
                        for (int k = 0; k < 4; ++k) value_pairs<decltype(any_scale)::value>(w[k][i], d[k][i], mask, magic, v[k]);
#pragma unroll
                        for (int n = 0; n < 4; n += 2) {
                            const uint4 a0 = make_uint4(v[0][n], v[0][n + 1], v[1][n], v[1][n + 1]);
                            const uint4 a1 = make_uint4(v[2][n], v[2][n + 1], v[3][n], v[3][n + 1]);
#pragma unroll
                            for (int t = 0; t < TILES; ++t) {
                                float acc[4];
                                mma_f16(acc, a0, pb[0][t][0][0], pb[0][t][0][1], 0.0f, 0.0f);
                                mma_f16(acc, a1, pb[0][t][1][0], pb[0][t][1][1]);
                                if (TERMS == kTwice) {
                                    mma_f16(acc, a0, pb[S::kMats - 1][t][0][0], pb[S::kMats - 1][t][0][1]);
                                    mma_f16(acc, a1, pb[S::kMats - 1][t][1][0], pb[S::kMats - 1][t][1][1]);
                                }
                                float(&x)[H] = o[t][4 * (q * GI + i) + n];
                                float(&y)[H] = o[t][4 * (q * GI + i) + n + 1];
                                if (TERMS == kSide) {
                                    x[0] += acc[0] + acc[1];
                                    y[0] += acc[2] + acc[3];
                                } else {
#pragma unroll
                                    for (int h = 0; h < H; ++h) { x[h] += acc[h]; y[h] += acc[2 + h]; }
                                }
                            }
                        }
                    }
                };
                if (large) products(std::true_type{});
                else products(std::false_type{});
            }
            __syncwarp();                                   // every lane has read the stage
            ++consumed;
            out_stage = out_stage + 1 == a.depth ? 0 : out_stage + 1;
            if (out_stage == 0) out_phase ^= 1;
            issue(0u);
        }

        // ---- the item's end: written out, or left for the join
        const bool whole = it.start >= u0 && it.end <= u1;
        // The part's last item waits in the warp's ring (every copy into it has been consumed), an
        // earlier one, whose ring is still in use, in the workspace.
        const bool last = consumed == issued && at == count && next_count == 0;
        float* const keep_at = last ? reinterpret_cast<float*>(mine)
                                    : a.partial + (2ll * gridDim.x + (long long)blockIdx.x * W + warp) * S::kPartial;
#pragma unroll
        for (int t = 0; t < TILES; ++t)
#pragma unroll
            for (int h = 0; h < H; ++h) {
                float l = sum[t][h];
                l += __shfl_xor_sync(kFull, l, 4);
                l += __shfl_xor_sync(kFull, l, 8);
                l += __shfl_xor_sync(kFull, l, 16);
                const int row = t * S::kTileRows + H * c4 + h;
                if (!whole) {
#pragma unroll
                    for (int g = 0; g < NG; ++g)
                        store4(keep_at + row * D + 32 * g + 4 * r8, o[t][4 * g][h], o[t][4 * g + 1][h], o[t][4 * g + 2][h],
                               o[t][4 * g + 3][h]);
                    if (r8 == 0) {
                        keep_at[ROWS * D + row] = ref[t][h];
                        keep_at[ROWS * D + ROWS + row] = l;
                    }
                    continue;
                }
                int j, head;
                row_of<ROWS>(a, it, row, j, head);
                if (j < 0) continue;
                const long long tok = it.rq.first_tok + j;
                const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                T* const dst = static_cast<T*>(a.out) + tok * a.out_stride + (long long)head * D + 4 * r8;
#pragma unroll
                for (int g = 0; g < NG; ++g)
                    store4(dst + 32 * g, o[t][4 * g][h] * inv, o[t][4 * g + 1][h] * inv, o[t][4 * g + 2][h] * inv,
                           o[t][4 * g + 3][h] * inv);
                if (r8 == 0 && a.lse) a.lse[tok * a.n_heads + head] = (ref[t][h] + log2f(l) - kProbShift) * 0.693147180559945309f;
            }
        if (!whole && lane == 0) {
            uint32_t* const m = meta + (2 * warp + (last ? 1 : 0)) * kMetaInts;
            m[0] = it.start;
            m[1] = it.end;
            m[2] = uint32_t(it.rq.first_tok);
            m[3] = uint32_t(it.rq.fresh);
            m[4] = uint32_t(it.head);
            m[5] = uint32_t(it.tile);
        }
    }
    __syncthreads();

    // ---- join the warps' parts, in order.  Part i is warp i / 2's earlier (even) or last one; the
    // parts of one item are neighbours.  Every warp reads the list for itself and takes rows.
    constexpr int V = D / 32;                              // values of a row per lane
    auto load_row = [&](const float* p, float (&x)[V]) {
        if constexpr (V == 2) {
            const float2 y = *reinterpret_cast<const float2*>(p + 2 * lane);
            x[0] = y.x; x[1] = y.y;
        } else {
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                const float4 y = *reinterpret_cast<const float4*>(p + 32 * i + 4 * lane);
                x[i] = y.x; x[i + 1] = y.y; x[i + 2] = y.z; x[i + 3] = y.w;
            }
        }
    };
    auto store_row = [&](float* p, const float (&x)[V]) {
        if constexpr (V == 2) *reinterpret_cast<float2*>(p + 2 * lane) = make_float2(x[0], x[1]);
        else
#pragma unroll
            for (int i = 0; i < V; i += 4) store4(p + 32 * i + 4 * lane, x[i], x[i + 1], x[i + 2], x[i + 3]);
    };
    auto put_row = [&](const Item& it, int row, const float (&x)[V], float m, float l) {
        int j, head;
        row_of<ROWS>(a, it, row, j, head);
        if (j < 0) return;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const long long tok = it.rq.first_tok + j;
        T* const dst = static_cast<T*>(a.out) + tok * a.out_stride + (long long)head * D;
        if constexpr (V == 2) store2(dst + 2 * lane, x[0] * inv, x[1] * inv);
        else
#pragma unroll
            for (int i = 0; i < V; i += 4)
                store4(dst + 32 * i + 4 * lane, x[i] * inv, x[i + 1] * inv, x[i + 2] * inv, x[i + 3] * inv);
        if (a.lse && lane == 0) a.lse[tok * a.n_heads + head] = (m + log2f(l) - kProbShift) * 0.693147180559945309f;
    };
    auto unfinished = [&](int i) {
        const uint32_t* const m = meta + i * kMetaInts;
        Item it;
        it.start = m[0];
        it.end = m[1];
        it.rq.first_tok = int(m[2]);
        it.rq.fresh = int(m[3]);
        it.head = int(m[4]);
        it.tile = int(m[5]);
        return it;
    };
    float* const cta_parts = a.partial + 2ll * blockIdx.x * S::kPartial;
    const float* const early_parts = a.partial + (2ll * gridDim.x + (long long)blockIdx.x * W) * S::kPartial;
    static_assert(2 * W <= 32, "a lane per part");
    const uint32_t my_start = lane < 2 * W ? meta[lane * kMetaInts] : kNoItem;
    // This lane's part (odd lanes: in the ring of a warp, even ones: in the workspace).
    const float* const my_part = (lane & 1) ? reinterpret_cast<const float*>(smem + lay.warp_off + min(lane >> 1, W - 1) * lay.warp_bytes)
                                            : early_parts + (long long)min(lane >> 1, W - 1) * S::kPartial;
    uint32_t left = __ballot_sync(kFull, my_start != kNoItem);
    int shared_item[2] = {0, 0}, n_shared = 0;
    for (int turn = warp; left != 0; turn = (turn + W - ROWS % W) % W) {      // rows go round the warps, item after item
        const int first_part = __ffs(int(left)) - 1;
        const uint32_t parts = __ballot_sync(kFull, my_start == __shfl_sync(kFull, my_start, first_part));
        left &= ~parts;
        const Item it = unfinished(first_part);
        const bool all = it.start >= c0 && it.end <= c1, has = (parts >> lane) & 1u;
        if (!all) {                                        // at most two: the share's first item and its last
            if (n_shared == 0) shared_item[0] = first_part;
            else shared_item[1] = first_part;
            n_shared = n_shared == 0 ? 1 : 2;
        }
        for (int row = turn; row < ROWS; row += W) {
            const float mi = has ? my_part[ROWS * D + row] : kNoRef, li = has ? my_part[ROWS * D + ROWS + row] : 0.0f;
            float m = mi;
#pragma unroll
            for (int d = 16; d > 0; d /= 2) m = fmaxf(m, __shfl_xor_sync(kFull, m, d));
            const float f = exp2_fast(mi - m);
            float l = has ? li * f : 0.0f;
#pragma unroll
            for (int d = 16; d > 0; d /= 2) l += __shfl_xor_sync(kFull, l, d);
            float v[V] = {};
            for (uint32_t rest = parts; rest != 0;) {
                // Four parts' loads at a time; beyond the last, the first again, unused.
                float x[4][V], w[4];
                bool in[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int i = rest != 0 ? __ffs(int(rest)) - 1 : first_part;
                    w[k] = __shfl_sync(kFull, f, i);
                    in[k] = rest != 0;
                    rest &= rest - 1;
                    if (i & 1) load_row(reinterpret_cast<const float*>(smem + lay.warp_off + (i >> 1) * lay.warp_bytes) + row * D, x[k]);
                    else load_row(early_parts + (long long)(i >> 1) * S::kPartial + row * D, x[k]);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int i = 0; i < V; ++i) v[i] = in[k] ? fmaf(x[k][i], w[k], v[i]) : v[i];
            }
            if (all) {
                put_row(it, row, v, m, l);
            } else {
                float* const dst = cta_parts + (it.start >= c0 ? S::kPartial : 0);
                store_row(dst + row * D, v);
                if (lane == 0) { dst[ROWS * D + row] = m; dst[ROWS * D + ROWS + row] = l; }
            }
        }
    }

    // ---- the last CTA of a shared item joins the CTAs' partials, in order: a warp per row, or
    // several, which share the partials and add up what they have
    uint32_t* const flags = meta + 2 * W * kMetaInts;          // one per shared item
    constexpr int kSplit = W / ROWS > 1 ? W / ROWS : 1, kAhead = 8;
    if (n_shared == 0) return;
    __syncthreads();
    if (tid < n_shared) {
        const uint32_t* const m = meta + (tid == 0 ? shared_item[0] : shared_item[1]) * kMetaInts;
        const uint32_t first = m[0] / share, n = (m[1] - 1) / share - first + 1;
        const bool mine_last = ticket_add(a.tickets + first) == n - 1;
        if (mine_last) a.tickets[first] = 0u;
        flags[tid] = mine_last;
    }
    for (int k = 0; k < n_shared; ++k) {
        __syncthreads();
        if (flags[k] == 0) continue;
        const Item it = unfinished(k == 0 ? shared_item[0] : shared_item[1]);
        const uint32_t first = it.start / share;
        const int n = int((it.end - 1) / share - first) + 1;
        auto cta_part = [&](int i) { return a.partial + (2ll * (first + i) + (i == 0 ? 1 : 0)) * S::kPartial; };
        float* const sums = reinterpret_cast<float*>(smem + lay.warp_off);       // [kSplit][ROWS][D]: the rings are done with
        for (int job = warp; job < kSplit * ROWS; job += W) {
            const int row = job % ROWS, mod = job / ROWS;
            // The first partials' values are requested before their weights are known.
            float x[kAhead][V];
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (mod + i * kSplit < n) load_row_l2<V>(cta_part(mod + i * kSplit) + row * D, lane, x[i]);
            // Maximum and sum over the partials, a lane each (round after round where there are more).
            const bool in = lane < n;
            const float early_m = in ? __ldcg(cta_part(lane) + ROWS * D + row) : kNoRef;
            const float early_l = in ? __ldcg(cta_part(lane) + ROWS * D + ROWS + row) : 0.0f;
            float m = early_m;
            for (int i = lane + 32; i < n; i += 32) m = fmaxf(m, __ldcg(cta_part(i) + ROWS * D + row));
#pragma unroll
            for (int d = 16; d > 0; d /= 2) m = fmaxf(m, __shfl_xor_sync(kFull, m, d));
            const float early_w = exp2_fast(early_m - m);
            float l = early_l * early_w;
            for (int i = lane + 32; i < n; i += 32) {
                const float* const p = cta_part(i) + ROWS * D + row;
                l = fmaf(__ldcg(p + ROWS), exp2_fast(__ldcg(p) - m), l);
            }
#pragma unroll
            for (int d = 16; d > 0; d /= 2) l += __shfl_xor_sync(kFull, l, d);
            float v[V] = {};
            for (int i0 = mod; i0 < n; i0 += kAhead * kSplit) {
                if (i0 != mod) {
#pragma unroll
                    for (int i = 0; i < kAhead; ++i)
                        if (i0 + i * kSplit < n) load_row_l2<V>(cta_part(i0 + i * kSplit) + row * D, lane, x[i]);
                }
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    const int at = i0 + i * kSplit;
                    if (at >= n) break;
                    const float w = at < 32 ? __shfl_sync(kFull, early_w, at) : exp2_fast(__ldcg(cta_part(at) + ROWS * D + row) - m);
#pragma unroll
                    for (int q = 0; q < V; ++q) v[q] = fmaf(x[i][q], w, v[q]);
                }
            }
            if (kSplit > 1) {
                store_row(sums + (mod * ROWS + row) * D, v);
                if (mod == 0 && lane == 0) { sums[kSplit * ROWS * D + row] = m; sums[kSplit * ROWS * D + ROWS + row] = l; }
            } else {
                put_row(it, row, v, m, l);
            }
        }
        if (kSplit > 1) {
            __syncthreads();
            for (int row = warp; row < ROWS; row += W) {
                float v[V];
                load_row(sums + row * D, v);
#pragma unroll
                for (int i = 1; i < kSplit; ++i) {
                    float x[V];
                    load_row(sums + (i * ROWS + row) * D, x);
#pragma unroll
                    for (int q = 0; q < V; ++q) v[q] += x[q];
                }
                put_row(it, row, v, sums[kSplit * ROWS * D + row], sums[kSplit * ROWS * D + ROWS + row]);
            }
        }
    }
}

// What the host needs of an instantiation.
struct AttnKernel {
    const void* fn;
    int warps, partial;
    int (*smem)(int n_req, int depth);
};
template <typename T, int D, int TILES, int TERMS> AttnKernel attn_kernel() {
    using S = AttnShape<D, TILES, TERMS>;
    return {(const void*)&attention_kernel<T, D, TILES, TERMS>, S::kWarps, S::kPartial,
            [](int n_req, int depth) { return attn_smem<D, TILES, TERMS>(n_req, depth).total; }};
}

}  // namespace qg
