// The cache side of the attention sublayer: block tables and slots from request lengths
// (qg_cache_pages), norm and rotation of query and key heads (qg_qk_norm_rope), and the same
// with the quantizing store into the paged 4-bit cache (qg_cache_append).  Formulas, layouts
// and argument rules are in include/qgemv.h; the record layout in kv_layout.h.
#include <algorithm>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kv_layout.h"
#include "qgemv_host.h"

namespace qg {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kMostSets = 4;            // of a call without a store (with one: 2)
constexpr float kWhole = 12582912.0f;   // 1.5 * 2^23: adding it rounds a small number to a whole one
constexpr int kMaxPageReq = 16384;      // requests of one qg_cache_pages call (two prefix arrays in shared memory)
constexpr int kPageThreads = 512;       // most

__device__ __forceinline__ void grid_dependency() {
    // Let the next kernel start its prologue; this one's inputs may come from the previous.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ------------------------------------------------------------------------------ page tables

struct PageArgs {
    const int32_t* held;
    const int32_t* fresh;
    const int32_t* free_pages;
    const int32_t* free_begin;
    int32_t* free_end;
    int32_t* table;
    int32_t* seq_len;
    int32_t* cu_new;
    int64_t* slots;
    int32_t* positions;
    long long n_free, table_stride, n_tok;
    int n_req, page;
    bool in_place;            // free_end is free_begin: one cluster, which syncs before the write
    unsigned int* status;
};

// Prefix sums of new tokens and of new pages over the requests, kept in shared memory by
// every CTA for itself (n_req values from L2; no CTA waits on another), then one thread per
// new token: a binary search for its request, its page from the table (a page the request
// held) or from the free list, its slot and position; the first token of a page writes the
// table's entry.  Working per token rather than per request spreads one long prompt over the
// grid as evenly as many short ones.
// Bound by latency (GB300, measured): 48 requests with a token each 3.0 us, of which an empty
// launch is 2; 40 prompts of up to 16001 tokens 4.8 us, 0.76 TB/s of its 3.6 MB: one launch,
// the scan, a search in shared memory and two dependent loads.
__global__ void __launch_bounds__(kPageThreads) cache_pages_kernel(const PageArgs a) {
    extern __shared__ int32_t prefix[];                  // [n_req + 1] tokens, then [n_req] pages
    __shared__ long long warp_tok[kPageThreads / 32], warp_pg[kPageThreads / 32];
    int32_t* const cu = prefix;
    int32_t* const off = prefix + a.n_req + 1;
    const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5, threads = int(blockDim.x);
    grid_dependency();
    const long long begin = a.free_begin ? *a.free_begin : 0;
    bool bad = begin < 0;
    long long run_tok = 0, run_pg = 0;
    for (int r0 = 0; r0 < a.n_req; r0 += threads) {
        const int r = r0 + tid;
        long long tok = 0, pg = 0;
        if (r < a.n_req) {
            long long h = a.held[r], f = a.fresh[r];
            if (h < 0 || f < 0 || h + f > 0x7FFFFFFFll) { bad = true; h = f = 0; }
            tok = f;
            pg = (h + f + a.page - 1) / a.page - (h + a.page - 1) / a.page;
            if (blockIdx.x == 0) a.seq_len[r] = int32_t(h + f);
        }
        long long st = tok, sp = pg;                     // inclusive scans over the block
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const long long ut = __shfl_up_sync(kAll, st, d), up = __shfl_up_sync(kAll, sp, d);
            if (lane >= d) { st += ut; sp += up; }
        }
        if (lane == 31) { warp_tok[warp] = st; warp_pg[warp] = sp; }
        __syncthreads();
        long long bt = run_tok, bp = run_pg;
        for (int w = 0; w < threads / 32; ++w) {
            if (w < warp) { bt += warp_tok[w]; bp += warp_pg[w]; }
            run_tok += warp_tok[w];
            run_pg += warp_pg[w];
        }
        if (r < a.n_req) {
            // Clipped to the caller's n_tok (an excess is an error, reported below) and to 31 bits.
            cu[r] = int32_t(min(bt + st - tok, a.n_tok));
            off[r] = int32_t(min(bp + sp - pg, 0x7FFFFFFFll));
        }
        __syncthreads();
    }
    const long long total = min(run_tok, a.n_tok);
    if (tid == 0) cu[a.n_req] = int32_t(total);
    if (bad || run_tok > a.n_tok) atomicOr(a.status, kStatusBadLength);
    __syncthreads();
    for (long long t = (long long)blockIdx.x * threads + tid; t < a.n_tok; t += (long long)gridDim.x * threads) {
        long long slot = -1;
        int pos = -1;
        if (t < total) {
            int lo = 0, hi = a.n_req;                    // the last r with cu[r] <= t
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (cu[mid] <= t) lo = mid; else hi = mid;
            }
            const int held = a.held[lo];
            pos = held + int(t - cu[lo]);
            const int pg = pos / a.page, in = pos - pg * a.page, have = int((unsigned(held) + a.page - 1) / a.page);
            int32_t* const entry = a.table + (long long)lo * a.table_stride + pg;
            int page = -1;
            if (pg >= a.table_stride) {
                atomicOr(a.status, kStatusBadPage);
            } else if (pg < have) {
                page = *entry;
                if (page < 0) atomicOr(a.status, kStatusBadPage);
            } else {
                const long long i = begin + off[lo] + (pg - have);
                if (begin < 0 || i >= a.n_free) {
                    atomicOr(a.status, kStatusNoPages);
                } else {
                    page = a.free_pages[i];
                    if (page < 0) atomicOr(a.status, kStatusBadPage);
                }
                if (in == 0) *entry = page;
            }
            if (page >= 0) slot = (long long)page * a.page + in;
        }
        a.slots[t] = slot;
        a.positions[t] = pos;
    }
    if (a.in_place && gridDim.x > 1) {                   // every CTA has read free_begin
        asm volatile("barrier.cluster.arrive;" ::: "memory");
        asm volatile("barrier.cluster.wait;" ::: "memory");
    } else {
        __syncthreads();
    }
    if (blockIdx.x == 0) {
        for (int r = tid; r <= a.n_req; r += threads) a.cu_new[r] = cu[r];
        if (tid == 0 && a.free_end) *a.free_end = int32_t(min(max(begin, 0ll) + run_pg, a.n_free));
    }
}

// ------------------------------------------------------------------------- heads of a token

struct HeadArgs {
    const void *q, *k, *v;
    long long q_stride, k_stride, v_stride, q_out_stride, k_out_stride;      // elements
    const float *q_weight, *k_weight, *cos_sin;
    const int32_t* positions;
    const int64_t* slots;
    void *q_out, *k_out, *v_back;      // k_out: normed keys, or the cache's values when it is written
    uint8_t* data;                     // the cache, or null
    long long n_tok, n_pos, n_slots;
    int n_q, n_k, n_v, page, rot;
    float eps;
    unsigned flags;
    bool wide_rot, wide_weight;        // cos_sin, both weights: start on 16 bytes
    unsigned int* status;
};

template <typename T> struct Quad;                       // four elements of a lane
template <> struct Quad<float> { float4 v; };
template <> struct Quad<__nv_bfloat16> { uint2 v; };

__device__ __forceinline__ void widen(const Quad<float>& q, float (&x)[4]) { x[0] = q.v.x, x[1] = q.v.y, x[2] = q.v.z, x[3] = q.v.w; }
__device__ __forceinline__ void widen(const Quad<__nv_bfloat16>& q, float (&x)[4]) {
    x[0] = __uint_as_float(q.v.x << 16), x[1] = __uint_as_float(q.v.x & 0xFFFF0000u);
    x[2] = __uint_as_float(q.v.y << 16), x[3] = __uint_as_float(q.v.y & 0xFFFF0000u);
}
__device__ __forceinline__ void store(float* at, const float (&x)[4]) { *reinterpret_cast<float4*>(at) = make_float4(x[0], x[1], x[2], x[3]); }
__device__ __forceinline__ void store(__nv_bfloat16* at, const float (&x)[4]) {
    Quad<__nv_bfloat16> q;
    __nv_bfloat162* e = reinterpret_cast<__nv_bfloat162*>(&q);
    e[0] = __floats2bfloat162_rn(x[0], x[1]);            // nearest even
    e[1] = __floats2bfloat162_rn(x[2], x[3]);
    *reinterpret_cast<Quad<__nv_bfloat16>*>(at) = q;
}

// Sums of squares of the S rows of D values that each D / 8 neighbouring lanes hold, a lane the
// quads `sub` and D / 8 + `sub` of a row, as a tree of adjacent pairs: pairs and quads within
// the lane, then lanes 2i and 2i + 1, and so on, the row's two halves last.  The order is part
// of the operator's definition (the sum then does not depend on the kernel); the first steps
// halve the sums a lane still carries, so 2 S of them cost 2 S - 1 + log2(D / 8 / S) + 1 shuffles.
// A lane returns the sum of the row whose index its lane bits 1, 2 spell, high bit first (sum_lane).
template <int S> __host__ __device__ constexpr int sum_lane(int row) {       // a lane that holds row's sum
    int l = 0;
    for (int m = S / 2, d = 2; m >= 1; m /= 2, d *= 2) l += ((row / m) & 1) * d;
    return l;
}
template <int D, int S> __device__ __forceinline__ float square_sums(const float (&x)[S][2][4], int lane) {
    float s[2 * S];
#pragma unroll
    for (int j = 0; j < S; ++j)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const float* const v = x[j][q];
            s[q * S + j] = __fadd_rn(__fadd_rn(__fmul_rn(v[0], v[0]), __fmul_rn(v[1], v[1])),
                                     __fadd_rn(__fmul_rn(v[2], v[2]), __fmul_rn(v[3], v[3])));
        }
    int d = 1;
#pragma unroll
    for (int m = S; m >= 1; m /= 2, d *= 2) {
#pragma unroll
        for (int i = 0; i < m; ++i) {
            const bool up = (lane & d) != 0;
            const float send = up ? s[i] : s[i + m], mine = up ? s[i + m] : s[i];
            s[i] = __fadd_rn(mine, __shfl_xor_sync(kAll, send, d));
        }
    }
#pragma unroll
    for (; d < D / 8; d *= 2) s[0] = __fadd_rn(s[0], __shfl_xor_sync(kAll, s[0], d));
    return __fadd_rn(s[0], __shfl_xor_sync(kAll, s[0], 1));
}

// Levels (code - 8) and scale of the block this lane's four values belong to (8 neighbouring
// lanes hold a block).
__device__ __forceinline__ void quantize_block(const float (&x)[4], int lane, float (&level)[4], __half& scale) {
    float m = x[0];
    uint32_t top = __float_as_uint(x[0]) & 0x7FFFFFFFu;
#pragma unroll
    for (int i = 1; i < 4; ++i) {                        // the first of the largest (NaN above all)
        const uint32_t b = __float_as_uint(x[i]) & 0x7FFFFFFFu;
        if (b > top) { top = b; m = x[i]; }
    }
    uint32_t all = top;
#pragma unroll
    for (int d = 1; d < 8; d *= 2) all = max(all, __shfl_xor_sync(kAll, all, d));
    const uint32_t group = 0xFFu << (lane & 24);
    const uint32_t who = __ballot_sync(kAll, top == all) & group;
    m = __shfl_sync(kAll, m, __ffs(int(who)) - 1);
    const float d = __fmul_rn(m, -0.125f);
    const bool bad = !(all <= __float_as_uint(QG_CACHE_MAX)) || d == 0.0f;
    // x / d through the reciprocal where that cannot change the code (the quotient, within 2^-20
    // of the true one, is not that near to a half), by the division itself elsewhere.
    const float inv = d == 0.0f ? 0.0f : __frcp_rn(d);       // (a zero block, or a row that is not there, needs no division)
    float off = fabsf(inv) < 1e30f ? 0.0f : 1.0f;        // the quotients' largest distance from a whole number
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float t = __fmul_rn(x[i], inv);
        level[i] = __fsub_rn(__fadd_rn(t, kWhole), kWhole);      // the nearest whole number (|t| is at most 8)
        off = fmaxf(off, fabsf(__fsub_rn(t, level[i])));
    }
    if (!(off < 0.49999f) && !bad) {
#pragma unroll
        for (int i = 0; i < 4; ++i) level[i] = __fadd_rn(roundf(__fdiv_rn(x[i], d)), 0.0f);      // (no -0)
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) level[i] = bad ? 0.0f : fminf(level[i], 7.0f);
    scale = d == 0.0f ? __ushort_as_half(0u) : bad ? __ushort_as_half(0x7E00u) : __float2half_rn(float(__float2bfloat16_rn(d)));
}

// Four neighbouring floats, in one load where the array starts on 16 bytes.
__device__ __forceinline__ void read_quad(const float* p, bool wide, float (&x)[4]) {
    if (wide) {
        const float4 r = *reinterpret_cast<const float4*>(p);
        x[0] = r.x, x[1] = r.y, x[2] = r.z, x[3] = r.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = p[i];
    }
}

// One warp takes SETS * 256 / D consecutive heads of one kind (queries, keys or values) of a
// token: D / 8 lanes a row, a lane the row's quads `sub` and D / 8 + `sub`, so that a
// half-split rotation of the whole head pairs values of one lane, and a 32-value block of the
// cache lies in 8 neighbouring lanes.  All rows' loads are issued before the first is used, and
// the token's cosines and sines and the weights are read once for all of them.
//
// Bounds (GB300, measured): norm and rotation of 8191 tokens of 72 bf16 heads of 128 take 64 us,
// 4.7 TB/s (4 bytes an element and no more), 84 warp instructions a row at 2.7 a clock: memory
// latency and instruction issue together.  With quads of neighbouring lanes exchanged for the
// rotation and one row to a warp it was 115 instructions and 76 us; several tokens to a warp in a
// loop made it 59 and the store below 46 instead of 40.  4100 tokens of 32 + 8 + 8 fp32 heads
// with the store: 39 us, 5.3 TB/s; 4096 of 64 + 8 + 8 bf16 heads with it: 51 us, 3.4 TB/s.  A row
// stored takes about three times the instructions of one normed.  At 4 tokens: 2.1 and 3.1 us, a
// launch and two latencies.
template <int D, typename T, int SETS>
__global__ void __launch_bounds__(128, SETS > 1 ? 8 : 4) heads_kernel(const HeadArgs a) {
    constexpr int L = D / 8, PER = 32 / L, ROWS = PER * SETS;
    const int lane = int(threadIdx.x) & 31, sub = lane % L, row = lane / L;
    const int g_q = (a.n_q + ROWS - 1) / ROWS, g_k = (a.n_k + ROWS - 1) / ROWS, g_v = (a.n_v + ROWS - 1) / ROWS;
    const int per_tok = g_q + g_k + g_v;
    const uint32_t id = blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5);        // < 2^31 (host)
    grid_dependency();
    const uint32_t tok32 = id / uint32_t(per_tok);
    if (tok32 >= a.n_tok) return;
    const long long tok = tok32;
    const int group = int(id - tok32 * uint32_t(per_tok));
    const bool is_q = group < g_q, is_v = group >= g_q + g_k;
    const int h0 = (is_q ? group : is_v ? group - g_q - g_k : group - g_q) * ROWS;
    const int heads = (is_q ? a.n_q : is_v ? a.n_v : a.n_k) - h0;          // rows from here on
    const int ia = sub * 4, ib = D / 2 + ia;

    const T* const src = (is_q ? static_cast<const T*>(a.q) + tok * a.q_stride : is_v ? static_cast<const T*>(a.v) + tok * a.v_stride
                                                                               : static_cast<const T*>(a.k) + tok * a.k_stride) +
                         (long long)(h0 + row) * D + ia;
    Quad<T> raw[SETS][2] = {};
#pragma unroll
    for (int j = 0; j < SETS; ++j)
        if (j * PER + row < heads) {
            raw[j][0] = *reinterpret_cast<const Quad<T>*>(src + j * PER * D);
            raw[j][1] = *reinterpret_cast<const Quad<T>*>(src + j * PER * D + D / 2);
        }

    // The token's rotation: the cosines and sines a lane's values need.  Half-split over the whole
    // head: of its four pairs; over at most half of it: of its first quad, whose partner is the
    // first quad of another lane; interleaved: of the pairs in its two quads.
    const int half = a.rot / 2;
    const bool inter = (a.flags & QG_ROPE_INTERLEAVED) != 0, norm = !is_v && !(a.flags & QG_NORM_NONE);
    const bool turn = ia < a.rot, turn_b = ib < a.rot;
    float cs[4] = {}, sn[4] = {}, w[2][4];
    const float* angles = nullptr;
    bool dead = false;
    if (a.positions) {
        const int pos = a.positions[tok];
        dead = pos < 0 || (a.rot > 0 && pos >= a.n_pos);
        if (pos >= 0 && dead && lane == 0) atomicOr(a.status, kStatusBadLength);
        if (!dead && a.rot > 0 && !is_v) {
            angles = a.cos_sin + (long long)pos * a.rot;
            if (inter) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (turn) { cs[i] = angles[ia / 2 + i]; sn[i] = angles[half + ia / 2 + i]; }
                    if (turn_b) { cs[2 + i] = angles[ib / 2 + i]; sn[2 + i] = angles[half + ib / 2 + i]; }
                }
            } else if (turn) {
                const int at = ia < half ? ia : ia - half;
                read_quad(angles + at, a.wide_rot, cs);
                read_quad(angles + half + at, a.wide_rot, sn);
            }
        }
    }
    const float* const weight = is_q ? a.q_weight : a.k_weight;
    const bool weighted = norm && weight;
    if (weighted) {
        read_quad(weight + ia, a.wide_weight, w[0]);
        read_quad(weight + ib, a.wide_weight, w[1]);
        if (a.flags & QG_NORM_UNIT_OFFSET) {
#pragma unroll
            for (int i = 0; i < 4; ++i) { w[0][i] = __fadd_rn(w[0][i], 1.0f); w[1][i] = __fadd_rn(w[1][i], 1.0f); }
        }
    }

    float x[SETS][2][4];
#pragma unroll
    for (int j = 0; j < SETS; ++j) { widen(raw[j][0], x[j][0]); widen(raw[j][1], x[j][1]); }
    if (norm) {
        const float mean = __fmul_rn(square_sums<D, SETS>(x, lane), 1.0f / D);
        const float root = __frcp_rn(__fsqrt_rn(__fadd_rn(mean, a.eps)));
#pragma unroll
        for (int j = 0; j < SETS; ++j) {
            const float r = SETS == 1 ? root : __shfl_sync(kAll, root, (lane & ~(L - 1)) + sum_lane<SETS>(j));
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[j][q][i] = __fmul_rn(x[j][q][i], r);
        }
        if (weighted) {
#pragma unroll
            for (int j = 0; j < SETS; ++j)
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[j][q][i] = __fmul_rn(x[j][q][i], w[q][i]);
        }
    }
    if (angles) {                                        // (the same for the whole warp)
        if (inter) {
#pragma unroll
            for (int j = 0; j < SETS; ++j)
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    if (q ? turn_b : turn) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float u = x[j][q][2 * i], v = x[j][q][2 * i + 1], c = cs[2 * q + i], s = sn[2 * q + i];
                            x[j][q][2 * i] = __fsub_rn(__fmul_rn(u, c), __fmul_rn(v, s));
                            x[j][q][2 * i + 1] = __fadd_rn(__fmul_rn(v, c), __fmul_rn(u, s));
                        }
                    }
        } else if (a.rot == D) {
#pragma unroll
            for (int j = 0; j < SETS; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float u = x[j][0][i], v = x[j][1][i];
                    x[j][0][i] = __fsub_rn(__fmul_rn(u, cs[i]), __fmul_rn(v, sn[i]));
                    x[j][1][i] = __fadd_rn(__fmul_rn(v, cs[i]), __fmul_rn(u, sn[i]));
                }
        } else {
            // The partner of quad n of the rotated part is n +- half / 4; quads from L on are
            // second quads, which only a rotation of more than half the head reaches.
            const int hop = half / 4;
            const int pa = !turn ? sub : sub < hop ? sub + hop : sub - hop;
            const int pb = !turn_b ? L + sub : L + sub - hop;                    // (hop < L: a second quad is a high one)
            const int base = lane & ~(L - 1), from_a = base + pa % L, from_b = base + pb % L;
            float cb[4] = {}, sb[4] = {};
            if (turn_b) {
                read_quad(angles + ib - half, a.wide_rot, cb);
                read_quad(angles + ib, a.wide_rot, sb);
            }
#pragma unroll
            for (int j = 0; j < SETS; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {            // b' = b c + a s, a' = a c - b s
                    const float u = x[j][0][i], v = x[j][1][i];
                    float p = __shfl_sync(kAll, u, from_a);
                    if (a.rot > D / 2) {
                        const float p1 = __shfl_sync(kAll, v, from_a), r0 = __shfl_sync(kAll, u, from_b), r1 = __shfl_sync(kAll, v, from_b);
                        if (pa >= L) p = p1;
                        const float y = __fadd_rn(__fmul_rn(v, cb[i]), __fmul_rn(pb >= L ? r1 : r0, sb[i]));
                        if (turn_b) x[j][1][i] = y;
                    }
                    const float y = __fadd_rn(__fmul_rn(u, cs[i]), __fmul_rn(p, sub < hop ? -sn[i] : sn[i]));
                    if (turn) x[j][0][i] = y;
                }
        }
    }
    if (dead) {
#pragma unroll
        for (int j = 0; j < SETS; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[j][0][i] = x[j][1][i] = 0.0f;
    }
    if (SETS == kMostSets || is_q || !a.data) {
        T* const dst = (is_q ? static_cast<T*>(a.q_out) + tok * a.q_out_stride : static_cast<T*>(a.k_out) + tok * a.k_out_stride) +
                       (long long)(h0 + row) * D + ia;
#pragma unroll
        for (int j = 0; j < SETS; ++j)
            if (j * PER + row < heads) { store(dst + j * PER * D, x[j][0]); store(dst + j * PER * D + D / 2, x[j][1]); }
        return;
    }

    long long slot = a.slots[tok];
    if (slot >= a.n_slots || slot < -1) {
        if (lane == 0) atomicOr(a.status, kStatusBadPage);
        slot = -1;
    }
    const long long page = slot < 0 ? 0 : slot >> 31 ? slot / a.page : uint32_t(slot) / uint32_t(a.page);
    const int in = slot >= 0 ? int(slot - page * a.page) : 0, t = in % kRecordTokens;
    T* const back = static_cast<T*>(is_v ? a.v_back : a.k_out);
    // The lane's places in its first row's record, by quad; from set to set the record is PER heads on.
    const long long per_head = (long long)(a.page / kRecordTokens) * kv_record_bytes(D);
    uint8_t* rec = a.data + (page * a.n_k + h0 + row) * per_head + in / kRecordTokens * kv_record_bytes(D);
    int codes_at[2], scale_at[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int i0 = q ? ib : ia, g = i0 / 32, at = i0 % 32;
        codes_at[q] = is_v ? kv_v_codes(D) + kv_value_half(D, t, at / 4, g) : kv_key_word(D, t, at / 8, g) + at % 8 / 2;
        scale_at[q] = (is_v ? kv_v_scales(D) : kv_k_scales(D)) + kv_scale(D, t, g);
    }
#pragma unroll
    for (int j = 0; j < SETS; ++j, rec += PER * per_head) {
        if (j * PER >= heads) break;                     // (the same for the whole warp)
        const bool there = j * PER + row < heads;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            float level[4];
            __half scale;
            quantize_block(x[j][q], lane, level, scale);
            if (there && slot >= 0) {
                uint32_t c[4];                           // the codes are the last four bits
#pragma unroll
                for (int i = 0; i < 4; ++i) c[i] = __float_as_uint(__fadd_rn(level[i], kWhole + 8.0f)) & 15u;
                *reinterpret_cast<uint16_t*>(rec + codes_at[q]) = uint16_t(c[0] | c[1] << 4 | c[2] << 8 | c[3] << 12);
                if (sub % 8 == 0) *reinterpret_cast<__half*>(rec + scale_at[q]) = scale;
            }
            if (there && back) {
                const float d = __half2float(scale);
                float y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = __fmul_rn(level[i], d);
                store(back + (tok * a.n_k + h0 + j * PER + row) * D + (q ? ib : ia), y);
            }
        }
    }
}

template <int D, typename T> const void* heads_fn(int sets) {
    if constexpr (sizeof(T) == 2)
        if (sets == kMostSets) return (const void*)&heads_kernel<D, T, kMostSets>;
    return sets == 1 ? (const void*)&heads_kernel<D, T, 1> : (const void*)&heads_kernel<D, T, 2>;
}
template <typename T> const void* heads_fn(int D, int sets) {
    return D == 64 ? heads_fn<64, T>(sets) : D == 128 ? heads_fn<128, T>(sets) : heads_fn<256, T>(sets);
}

qg_status launch_heads(HeadArgs& a, qg_act act, int D, void* stream) {
    int dev = 0, sms = 0, optin = 0;
    qg_status st = device_info(&dev, &sms, &optin, &a.status);
    if (st != QG_OK) return st;
    a.wide_rot = aligned(a.cos_sin, 16);
    a.wide_weight = aligned(a.q_weight, 16) && aligned(a.k_weight, 16);
    const long long heads = a.n_q + a.n_k + a.n_v;
    if (heads == 0 || a.n_tok == 0) return QG_OK;
    // Warps of a token when a warp takes so many sets.
    auto warps_of = [&](int sets) {
        const long long rows = 256 / D * sets;
        return (a.n_q + rows - 1) / rows + (a.n_k + rows - 1) / rows + (a.n_v + rows - 1) / rows;
    };
    // More sets share a token's angles, weights and reductions, once there are enough warps without
    // it, and where a kind's last warp does not idle too much of it (at most half as many sets
    // again).  Norm and rotation of bf16 heads: with 1, 2 and 4 sets 64 + 8 heads of 128 take 4.9, 3.6
    // and 3.9 us for 256 tokens, 60, 44 and 33 for 4096; 8 + 4 heads of 64 take 6.1, 5.4 and 7.0 for
    // 4096.  fp32 and calls with a store have no registers for 4 (64 + 8 + 8 bf16 heads, 4096 tokens:
    // 73, 53 and 55), and a store hides its latency with 64 warps an SM (48 + 16 + 16 heads of 64, 256
    // tokens: 4.6 against 5.1 with two).
    const long long enough = (a.data ? 64ll : 32ll) * sms;
    const int most = act == QG_ACT_BF16 && !a.data ? kMostSets : 2;
    int sets = 1;
    while (sets < most && a.n_tok * warps_of(sets) > enough && 4 * sets * warps_of(2 * sets) <= 3 * warps_of(1)) sets *= 2;
    const void* fn = act == QG_ACT_F32 ? heads_fn<float>(D, sets) : heads_fn<__nv_bfloat16>(D, sets);
    const long long warps = a.n_tok * warps_of(sets);
    const int in_block = 4;
    const long long grid = (warps + in_block - 1) / in_block;
    if (warps > 0x7FFFFFFFll - 8) return QG_EUNSUPPORTED;
    void* params[] = {&a};
    return launch_early(fn, int(grid), 32 * in_block, 0, 1, params, stream);
}

constexpr unsigned kHeadFlags = QG_ROPE_INTERLEAVED | QG_NORM_UNIT_OFFSET | QG_NORM_NONE;

// Rows of `heads` heads of D values, `stride` elements apart: 16-byte aligned, not overlapping.
qg_status check_rows(const void* p, int64_t stride, int64_t heads, int D, qg_act act) {
    if (!p || stride < heads * D) return QG_EINVAL;
    const int64_t size = act == QG_ACT_F32 ? 4 : 2;
    return aligned(p, 16) && stride * size % 16 == 0 ? QG_OK : QG_EALIGN;
}

// Rows written over the rows they are made of need the same places: at another stride they would
// cover rows that other warps have yet to read.
bool in_place_ok(const void* in, int64_t in_stride, const void* out, int64_t out_stride, int64_t n_tok) {
    return in != out || in_stride == out_stride || n_tok <= 1;
}

qg_status check_heads(qg_act act, int64_t n_tok, int n_heads, int n_kv, int D, const float* qw, const float* kw,
                      float eps, unsigned flags, const float* cos_sin, int64_t n_pos, int rot,
                      const int32_t* positions) {
    if (act != QG_ACT_F32 && act != QG_ACT_BF16) return QG_EINVAL;
    if (n_tok < 0 || n_tok > (int64_t(1) << 31) - 1 || n_heads < 0 || n_heads > 65535 || n_kv < 0 || n_kv > 65535)
        return QG_EINVAL;
    if (!kv_dim_ok(D) || (flags & ~kHeadFlags) || !(eps >= 0.0f)) return QG_EINVAL;
    if (cos_sin ? (rot < 16 || rot > D || rot % 16 != 0 || n_pos < 1 || !positions) : rot != 0) return QG_EINVAL;
    return aligned(qw, 4) && aligned(kw, 4) && aligned(cos_sin, 4) && aligned(positions, 4) ? QG_OK : QG_EALIGN;
}

}  // namespace

static qg_status launch_with(bool early, const void* fn, int grid, int threads, size_t smem, int cluster, void** params, void* stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (early) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = unsigned(cluster);
        attr[n].val.clusterDim.y = 1;
        attr[n++].val.clusterDim.z = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = unsigned(n);
    if (cudaLaunchKernelExC(&cfg, fn, params) != cudaSuccess) { cudaGetLastError(); return QG_ECUDA; }
    return QG_OK;
}

qg_status launch_early(const void* fn, int grid, int threads, size_t smem, int cluster, void** params, void* stream) {
    return launch_with((launch_flags() & QG_LAUNCH_EARLY_START) != 0, fn, grid, threads, smem, cluster, params, stream);
}

qg_status launch_after(const void* fn, int grid, int threads, size_t smem, int cluster, bool early, void** params, void* stream) {
    return launch_with(early || (launch_flags() & QG_LAUNCH_EARLY_START) != 0, fn, grid, threads, smem, cluster, params, stream);
}

}  // namespace qg

using namespace qg;

extern "C" {

size_t qg_cache_bytes(int64_t n_pages, int page_tokens, int n_kv_heads, int head_dim) {
    const qg_cache c = {reinterpret_cast<void*>(16), n_pages, page_tokens, n_kv_heads, head_dim};
    if (kv_check(&c) != QG_OK) return 0;
    return size_t(n_pages) * size_t(n_kv_heads) * size_t(page_tokens / kRecordTokens) * size_t(kv_record_bytes(head_dim));
}

qg_status qg_cache_pages(const int32_t* held, const int32_t* fresh, int n_req, int page_tokens,
                         const int32_t* free_pages, int64_t n_free, const int32_t* free_begin, int32_t* free_end,
                         int32_t* table, int64_t table_stride, int32_t* seq_len, int32_t* cu_new, int64_t* slots,
                         int32_t* positions, int64_t n_tok, void* stream) {
    const int64_t most = (int64_t(1) << 31) - 1;
    if (n_req < 0 || page_tokens < 16 || page_tokens > 65536 || page_tokens % kRecordTokens != 0) return QG_EINVAL;
    if (n_free < 0 || n_free > most || table_stride < 0 || table_stride > most || n_tok < 0 || n_tok > most)
        return QG_EINVAL;
    if (!cu_new || (n_free > 0 && !free_pages) || (n_tok > 0 && (!slots || !positions))) return QG_EINVAL;
    if (n_req > 0 && (!held || !fresh || !table || !seq_len)) return QG_EINVAL;
    if (n_req > 0 && (seq_len == held || seq_len == fresh || cu_new == held || cu_new == fresh)) return QG_EINVAL;
    if (n_req > kMaxPageReq) return QG_EUNSUPPORTED;
    if (!aligned(held, 4) || !aligned(fresh, 4) || !aligned(free_pages, 4) || !aligned(free_begin, 4) ||
        !aligned(free_end, 4) || !aligned(table, 4) || !aligned(seq_len, 4) || !aligned(cu_new, 4) ||
        !aligned(slots, 8) || !aligned(positions, 4))
        return QG_EALIGN;
    int dev = 0, sms = 0, optin = 0;
    PageArgs a{};
    qg_status st = device_info(&dev, &sms, &optin, &a.status);
    if (st != QG_OK) return st;
    a.held = held;
    a.fresh = fresh;
    a.free_pages = free_pages;
    a.free_begin = free_begin;
    a.free_end = free_end;
    a.table = table;
    a.seq_len = seq_len;
    a.cu_new = cu_new;
    a.slots = slots;
    a.positions = positions;
    a.n_free = n_free;
    a.table_stride = table_stride;
    a.n_tok = n_tok;
    a.n_req = n_req;
    a.page = page_tokens;
    a.in_place = free_end && free_end == free_begin;
    const size_t smem = (2 * size_t(n_req) + 1) * sizeof(int32_t);
    const void* fn = (const void*)&cache_pages_kernel;
    // (The kernel's own shared memory counts towards the 48 KB that need no opt-in.)
    if (smem + kStaticSmemReserve > 48 * 1024 && blocks_per_sm(fn, dev, optin, kPageThreads, smem) < 1) return QG_EUNSUPPORTED;
    // CTAs of 256 threads, three to an SM, start and scan sooner than one of 512 (3.0 us against 3.5
    // at 48 tokens, 4.8 against 5.7 at 300,000).  Where 256 threads would scan in two rounds (300
    // requests: 4.3 us against 3.9), or a call in place, which has 8 CTAs, would take its tokens in
    // two (32,000: 12.8 us against 9.3), CTAs have 512.  A call in place has no more than its cluster's 8
    // CTAs: 3.5 us for 48 tokens, 8.1 to 9.6 for 32,000 and 70 for 292,000, where the whole grid with a
    // separate free_end takes 3.1, 2.8 and 5.1.
    const int threads = n_req > 256 || (a.in_place && n_tok > 8 * 256) ? kPageThreads : 256;
    int64_t grid = std::max<int64_t>(1, std::min<int64_t>((n_tok + threads - 1) / threads, threads == 256 ? 3 * sms : sms));
    // In place every CTA must have read free_begin before it is written: one cluster, which can wait for itself.
    const int cluster = a.in_place ? int(grid >= 8 ? 8 : grid) : 1;
    if (a.in_place) grid = cluster;
    void* params[] = {&a};
    return launch_early(fn, int(grid), threads, smem, cluster, params, stream);
}

qg_status qg_qk_norm_rope(qg_act act, const void* q, int64_t q_stride, const void* k, int64_t k_stride, int64_t n_tok,
                          int n_heads, int n_kv_heads, int head_dim, const float* q_weight, const float* k_weight,
                          float eps, unsigned int flags, const float* cos_sin, int64_t n_pos, int rot_dim,
                          const int32_t* positions, void* q_out, int64_t q_out_stride, void* k_out,
                          int64_t k_out_stride, void* stream) {
    qg_status st = check_heads(act, n_tok, n_heads, n_kv_heads, head_dim, q_weight, k_weight, eps, flags, cos_sin, n_pos,
                               rot_dim, positions);
    if (st != QG_OK) return st;
    if (n_tok > 0 && n_heads > 0) {
        if ((st = check_rows(q, q_stride, n_heads, head_dim, act)) != QG_OK) return st;
        if ((st = check_rows(q_out, q_out_stride, n_heads, head_dim, act)) != QG_OK) return st;
        if (!in_place_ok(q, q_stride, q_out, q_out_stride, n_tok)) return QG_EINVAL;
    }
    if (n_tok > 0 && n_kv_heads > 0) {
        if ((st = check_rows(k, k_stride, n_kv_heads, head_dim, act)) != QG_OK) return st;
        if ((st = check_rows(k_out, k_out_stride, n_kv_heads, head_dim, act)) != QG_OK) return st;
        if (!in_place_ok(k, k_stride, k_out, k_out_stride, n_tok)) return QG_EINVAL;
    }
    HeadArgs a{};
    a.q = q;
    a.k = k;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.cos_sin = cos_sin;
    a.positions = positions;
    a.q_out = q_out;
    a.k_out = k_out;
    a.q_out_stride = q_out_stride;
    a.k_out_stride = k_out_stride;
    a.n_tok = n_tok;
    a.n_pos = n_pos;
    a.n_q = n_heads;
    a.n_k = n_kv_heads;
    a.rot = rot_dim;
    a.eps = eps;
    a.flags = flags;
    return launch_heads(a, act, head_dim, stream);
}

qg_status qg_cache_append(const qg_cache* cache, qg_act act, const void* q, int64_t q_stride, const void* k,
                          int64_t k_stride, const void* v, int64_t v_stride, int64_t n_tok, int n_heads,
                          const float* q_weight, const float* k_weight, float eps, unsigned int flags,
                          const float* cos_sin, int64_t n_pos, int rot_dim, const int32_t* positions,
                          const int64_t* slots, void* q_out, int64_t q_out_stride, void* k_back, void* v_back,
                          void* stream) {
    qg_status st = kv_check(cache);
    if (st != QG_OK) return st;
    const int D = cache->head_dim, n_kv = cache->n_kv_heads;
    st = check_heads(act, n_tok, n_heads, n_kv, D, q_weight, k_weight, eps, flags, cos_sin, n_pos, rot_dim, positions);
    if (st != QG_OK) return st;
    if (n_tok > 0) {
        if (!slots) return QG_EINVAL;
        if (!aligned(slots, 8) || !aligned(k_back, 16) || !aligned(v_back, 16)) return QG_EALIGN;
        if (n_heads > 0) {
            if ((st = check_rows(q, q_stride, n_heads, D, act)) != QG_OK) return st;
            if ((st = check_rows(q_out, q_out_stride, n_heads, D, act)) != QG_OK) return st;
            if (!in_place_ok(q, q_stride, q_out, q_out_stride, n_tok)) return QG_EINVAL;
        }
        if ((st = check_rows(k, k_stride, n_kv, D, act)) != QG_OK) return st;
        if ((st = check_rows(v, v_stride, n_kv, D, act)) != QG_OK) return st;
        const int64_t row = int64_t(n_kv) * D;
        if (!in_place_ok(k, k_stride, k_back, row, n_tok) || !in_place_ok(v, v_stride, v_back, row, n_tok)) return QG_EINVAL;
    }
    HeadArgs a{};
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.cos_sin = cos_sin;
    a.positions = positions;
    a.slots = slots;
    a.q_out = q_out;
    a.q_out_stride = q_out_stride;
    a.k_out = k_back;
    a.v_back = v_back;
    a.data = static_cast<uint8_t*>(cache->data);
    a.n_tok = n_tok;
    a.n_pos = n_pos;
    a.n_slots = cache->n_pages * cache->page_tokens;
    a.n_q = n_heads;
    a.n_k = n_kv;
    a.n_v = n_kv;
    a.page = cache->page_tokens;
    a.rot = rot_dim;
    a.eps = eps;
    a.flags = flags;
    return launch_heads(a, act, D, stream);
}

}  // extern "C"
