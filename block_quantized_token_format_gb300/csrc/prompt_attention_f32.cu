// Causal attention of packed prompts, fp32: as the bf16 kernel, on two fp16 terms of every operand.
//
// stage_kernel writes, for every query, key and value of a head, its values times a power of two that
// takes their largest finite magnitude to [2^7, 2^15), as an fp16 value and another of what its
// rounding left: 22 bits of the largest and, of smaller ones, what is above 2^-32 of it.  The powers are a
// token's own: one for several tokens would take bits of a token for the size of another, which a row may
// not see.  Their exponents are multiples of 8, so that tokens of similar size have the same one: a tile in which all
// do, as the copying warp finds, has one factor for its scores and one for its part of the output.  In another
// tile the scores' columns and P's are multiplied by the powers, relative to the largest that the
// row sees, which gives the rows of both kinds the same bits.
// Three products of 16-bit terms (small ones first: the tensor cores truncate what they add) make S;
// P is 2^7 times the exponential, so that two terms of it reach 2^-31 of the row's largest; each
// tile's P V goes to fresh accumulators and is added in fp32 registers, in units of the largest power of values that the
// row has met, so that outputs next to the largest fp32 number do not pass it on the way.
//
// One CTA is 128 rows, two lanes a row (each half of a tile's keys and half of the output; one with heads
// of 256, whose operands leave no shared memory for the lanes' maxima); S and the tiles' P V have two buffers each, so that the next
// tile's S and this tile's P V run beside the softmax.  Heads of 256 take two CTAs, each 128 values of
// the output.
//
// Bound by the tensor cores, which work 68 % of the time on three products for each that counts as
// work, and by the softmax with its two terms in what is left: two prompts of up to 3500 tokens, 32
// heads of 128 on 8: 292 us with the staging (there four rows to a warp; one row to a warp took 12 us
// more); tokens of sizes from 1e-3 to 1, whose tiles are scaled by column, 331 us.  Heads of 64 209 us (283), 16
// heads of 256 on 4 525 us.  Two lanes a row instead of one: 377 to 306 us; four: 303 where two took 292, not kept.
// Powers of two in steps of 8: in single steps every tile was scaled by column, 340 us and heads of 64 283.
#include "prompt_attention.cuh"

namespace qg {
namespace {

constexpr int kStageThreads = 256;
constexpr float kSlack = 8.0f, kLift = 7.0f, kUnlift = 0.0078125f;     // log2: P is 2^7 times the exponential, at most 2^15
constexpr int kTileKeys = 64, kStageRows = 4;

template <int D> struct Shape {
    static constexpr int KT = kTileKeys, DV = D < 128 ? D : 128, HALVES = D / DV, STAGES = D == 256 ? 1 : 2;
    static constexpr int SIDES = D == 256 ? 1 : 2, WARPS = 4 * SIDES;        // lanes of a row, warps of the softmax
    static constexpr int SLOTS = STAGES + 1;             // tiles whose powers of two wait in shared memory
    static constexpr int CH = D / 64, CV = DV / 64;
    static constexpr int Q_TERM = CH * 128 * 128, K_TERM = CH * KT * 128, V_TERM = CV * KT * 128;
    static constexpr int SMEM = 1024 + 2 * Q_TERM + 2 * STAGES * (K_TERM + V_TERM);
    static constexpr uint32_t O_AT = 2 * KT, COLS = 2 * KT + 2 * DV <= 256 ? 256 : 512;
};

__device__ __forceinline__ bool finite_of(float x) { return (__float_as_uint(x) & 0x7F800000u) != 0x7F800000u; }
__device__ __forceinline__ uint32_t finite_bits(float x) { return finite_of(x) ? __float_as_uint(x) & 0x7FFFFFFFu : 0u; }
// The power of two, its exponent a multiple of 8, that takes a magnitude (its bits) to [2^7, 2^15), and its
// inverse; of zero the one of the smallest, which is nobody's largest.
__device__ __forceinline__ float lift_of(uint32_t top, float& inverse) {
    const int e = top ? min((14 - ilogbf(__uint_as_float(top))) & ~7, 120) : 120;
    inverse = __int_as_float((127 - e) << 23);
    return __int_as_float((e + 127) << 23);
}
// Four values: their terms.
__device__ __forceinline__ void terms4(float4 x, float lift, uint2& hi, uint2& lo) {
    float s[4] = {x.x * lift, x.y * lift, x.z * lift, x.w * lift};
    __half h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h[i] = __float2half_rn(s[i]);
        l[i] = finite_of(s[i]) ? __float2half_rn(s[i] - __half2float(h[i])) : __float2half_rn(0.0f);
    }
    hi = make_uint2(__half_as_ushort(h[0]) | uint32_t(__half_as_ushort(h[1])) << 16, __half_as_ushort(h[2]) | uint32_t(__half_as_ushort(h[3])) << 16);
    lo = make_uint2(__half_as_ushort(l[0]) | uint32_t(__half_as_ushort(l[1])) << 16, __half_as_ushort(l[2]) | uint32_t(__half_as_ushort(l[3])) << 16);
}

// One tensor's rows, [n_tok][heads][D].
struct StageRows {
    const float* x;
    long long stride;
    uint16_t* out;                               // [2 terms][n_tok][heads][D]
    float* scale;                                // [n_tok][heads]
    int heads;
};
struct StageArgs {
    StageRows q, k, v;
    const int32_t* cu_seq;
    int n_tok, n_seq;
    uint32_t q_blocks, kv_blocks;                // blocks of the queries, of the keys, of the values
};

// A warp four rows at a time.
template <int D> __global__ void __launch_bounds__(kStageThreads) stage_kernel(const __grid_constant__ StageArgs a) {
    tc::grid_launch_dependents();
    tc::grid_wait();
    const int tid = int(threadIdx.x), lane = tid & 31;
    uint32_t b = blockIdx.x;
    const bool queries = b < a.q_blocks;
    if (!queries) b -= a.q_blocks;
    const bool values = !queries && b >= a.kv_blocks;
    if (values) b -= a.kv_blocks;
    const StageRows& t = queries ? a.q : values ? a.v : a.k;
    const long long row0 = ((long long)b * (kStageThreads / 32) + (tid >> 5)) * kStageRows;
    const long long from = (long long)a.cu_seq[0] * t.heads, to = min((long long)a.cu_seq[a.n_seq], (long long)a.n_tok) * t.heads;
    constexpr int N = (D + 127) / 128;
    float4 x[kStageRows][N];
#pragma unroll
    for (int k = 0; k < kStageRows; ++k) {
        const long long row = row0 + k;
        const long long tok = row / t.heads;
        const float* const src = t.x + tok * t.stride + (row - tok * t.heads) * D;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at = (i * 32 + lane) * 4;
            x[k][i] = at < D && row >= from && row < to && row >= 0 ? *reinterpret_cast<const float4*>(src + at) : make_float4(0, 0, 0, 0);
        }
    }
#pragma unroll
    for (int k = 0; k < kStageRows; ++k) {
        const long long row = row0 + k;
        if (row < from || row >= to || row < 0) continue;
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < N; ++i)
            top = max(max(max(top, finite_bits(x[k][i].x)), finite_bits(x[k][i].y)), max(finite_bits(x[k][i].z), finite_bits(x[k][i].w)));
        top = __reduce_max_sync(tc::kFullMask, top);
        float inverse;
        const float lift = lift_of(top, inverse);
        bool fine = true;
#pragma unroll
        for (int i = 0; i < N; ++i) fine = fine && finite_of(x[k][i].x) && finite_of(x[k][i].y) && finite_of(x[k][i].z) && finite_of(x[k][i].w);
        // Two terms of a query or key that is not finite are no score: its power makes one that is NaN.
        if (!__all_sync(tc::kFullMask, fine) && !values) inverse = __int_as_float(0x7FC00000);
        if (lane == 0) t.scale[row] = inverse;
        uint16_t* const out = t.out + row * D;
        const size_t term = size_t(a.n_tok) * t.heads * D;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at = (i * 32 + lane) * 4;
            if (at >= D) break;
            uint2 hi, lo;
            terms4(x[k][i], lift, hi, lo);
            *reinterpret_cast<uint2*>(out + at) = hi;
            *reinterpret_cast<uint2*>(out + term + at) = lo;
        }
    }
}

// The inverse of a power of two from 2^-120 to 2^120 (of zero: 2^127).
__device__ __forceinline__ float inverse_of(float x) { return __int_as_float(0x7F000000 - __float_as_int(x)); }

// The largest of a tile's powers (in shared memory) from `lo` to `hi`; 0: none.
__device__ __forceinline__ float most_seen(uint32_t powers, int lo, int hi) {
    float most = 0.0f;
#pragma unroll 2
    for (int i = 0; i < kTileKeys; i += 4) {
        const float4 p = lds4(powers + i * 4);
        if (i >= lo && i <= hi) most = fmaxf(most, p.x);
        if (i + 1 >= lo && i + 1 <= hi) most = fmaxf(most, p.y);
        if (i + 2 >= lo && i + 2 <= hi) most = fmaxf(most, p.z);
        if (i + 3 >= lo && i + 3 <= hi) most = fmaxf(most, p.w);
    }
    return most;
}

template <int D> __global__ void __launch_bounds__(32 * (Shape<D>::WARPS + 2), 1) prompt_f32_kernel(const __grid_constant__ PromptArgs a) {
    using S = Shape<D>;
    constexpr int KT = S::KT, CH = S::CH, CV = S::CV, DV = S::DV, SIDES = S::SIDES, kSoftWarps = S::WARPS;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bar_mem[18 + S::SLOTS];
    __shared__ alignas(16) float scale_mem[S::SLOTS][2 * KT + 4];        // a tile's powers of keys and of values, their largest, whether they differ
    __shared__ uint32_t tmem_at, dead, odd;
    __shared__ float most_of[2][SIDES > 1 ? SIDES * 128 : 1], sum_of[SIDES > 1 ? SIDES * 128 : 1];      // the lanes' maxima, of even and odd tiles, and sums

    const int tid = int(threadIdx.x), warp = __shfl_sync(tc::kFullMask, tid >> 5, 0), lane = tid & 31;
    tc::grid_launch_dependents();
    tc::grid_wait();
    if (warp == 0) prompt_check(a, int(blockIdx.x));
    PromptItem it;
    const int parts = a.n_kv * S::HALVES, slots = int(gridDim.x) / parts, b = int(blockIdx.x) / parts;
    if (!prompt_piece(a.cu_seq, a.n_seq, a.n_tok, a.tokens, slots - 1 - b, it)) return;
    const int part = int(blockIdx.x) - b * parts, half = part % S::HALVES;
    it.head = part / S::HALVES;
    key_range<KT>(a, it, true);
    const int first = it.first, tiles = it.tiles;

    const uint32_t q_at = (smem_addr(smem_raw) + 1023u) & ~1023u, k_at = q_at + 2 * S::Q_TERM, v_at = k_at + 2 * S::STAGES * S::K_TERM;
    const uint32_t bars = smem_addr(bar_mem);
    const uint32_t q_full = bars, drained = bars + 8;
    auto k_full = [&](int s) { return bars + 16u + 8u * uint32_t(s); };
    auto k_empty = [&](int s) { return bars + 32u + 8u * uint32_t(s); };
    auto v_full = [&](int s) { return bars + 48u + 8u * uint32_t(s); };
    auto v_empty = [&](int s) { return bars + 64u + 8u * uint32_t(s); };
    auto s_full = [&](int s) { return bars + 80u + 8u * uint32_t(s); };
    auto p_full = [&](int s) { return bars + 96u + 8u * uint32_t(s); };
    auto o_full = [&](int s) { return bars + 112u + 8u * uint32_t(s); };
    auto o_empty = [&](int s) { return bars + 128u + 8u * uint32_t(s); };
    auto scales_full = [&](int s) { return bars + 144u + 8u * uint32_t(s); };
    const tc::Waits wait{&dead, a.status, a.wait_limit};

    if (tid == 0) {
        dead = odd = 0;
        mbar_init(q_full, 1);
        mbar_init(drained, 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(k_full(s), 1);
            mbar_init(k_empty(s), 1);
            mbar_init(v_full(s), 1);
            mbar_init(v_empty(s), 1);
            mbar_init(s_full(s), 1);
            mbar_init(p_full(s), kSoftWarps);
            mbar_init(o_full(s), 1);
            mbar_init(o_empty(s), kSoftWarps);
        }
        for (int s = 0; s < S::SLOTS; ++s) mbar_init(scales_full(s), 1);
        mbar_fence_init();
    }
    if (warp == kSoftWarps + 1) tc::tmem_alloc(smem_addr(&tmem_at), S::COLS);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = tmem_at;

    if (warp < kSoftWarps) {
        constexpr int K2 = KT / SIDES, D2 = DV / SIDES;
        const int rows = warp & 3, side = warp >> 2, row = rows * 32 + lane;
        const PromptRow r = prompt_row(a, it, row);
        const uint32_t mine = tmem + (uint32_t(rows) << 21);
        const int head = it.head * a.group + row % a.group;
        const long long token = it.seq0 + r.tok;
        const float c = r.there ? a.c * a.qscale[token * a.n_heads + head] : 0.0f;
        // The output is in units of the largest power of values so far: v_mine is the last tile's in these.
        float v_mine = 0.0f, v_unit = 0.0f;
        float top = -INFINITY, sum = 0.0f;               // the row's reference (log2 of an exponential), this lane's sum of P
        float o[D2];
#pragma unroll
        for (int i = 0; i < D2; ++i) o[i] = 0.0f;
        bool alive = true;
        // Adds the part of the output that tile j made, times its factor.
        auto gather = [&](int j) {
            const int ob = j & 1;
            if (!wait(o_full(ob), j >> 1 & 1)) return false;
            tc::fence_after();
#pragma unroll
            for (int i = 0; i < D2; i += 32) {
                uint32_t x[32];
                tc::tmem_load32(mine + S::O_AT + uint32_t(ob * DV + side * D2 + i), x);
                tc::tmem_load_wait32(x);
#pragma unroll
                for (int n = 0; n < 32; ++n) o[i + n] = fmaf(__uint_as_float(x[n]), v_mine, o[i + n]);
            }
            tc::fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(o_empty(ob));
            return true;
        };

        for (int j = 0; j < tiles; ++j) {
            const int k0 = first + j * KT, sb = j & 1;
            if (!wait(scales_full(j % S::SLOTS), j / S::SLOTS & 1)) { alive = false; break; }
            const float* const scales = scale_mem[j % S::SLOTS];
            const uint32_t powers = smem_addr(scales), k_pow = powers + uint32_t(side * K2 * 4), v_pow = k_pow + KT * 4;
            float k_this = scales[2 * KT], v_this = scales[2 * KT + 1], v_inverse = 1.0f;
            const bool edge = on_edge<KT>(a, it, k0), uneven = scales[2 * KT + 2] != 0.0f;
            if (!wait(s_full(sb), j >> 1 & 1)) { alive = false; break; }
            tc::fence_after();
            uint32_t x[K2];
            const uint32_t at = mine + uint32_t(sb * KT);
            tc::tmem_load(at + uint32_t(side * K2), x);
            const int hi = r.pos - k0 - side * K2, lo = r.low - k0 - side * K2;      // visible keys of this lane's
            if (uneven) {
                float k_inverse = 1.0f;
                if (edge) {                                  // the powers are as they are: relative to the largest that is seen
                    k_this = most_seen(powers, r.low - k0, r.pos - k0);
                    v_this = most_seen(powers + KT * 4, r.low - k0, r.pos - k0);
                    k_inverse = inverse_of(k_this);
                    v_inverse = inverse_of(v_this);
                }
#pragma unroll
                for (int i = 0; i < K2; i += 4) {
                    const float4 p = lds4(k_pow + i * 4);
                    x[i] = __float_as_uint(__uint_as_float(x[i]) * (p.x * k_inverse));
                    x[i + 1] = __float_as_uint(__uint_as_float(x[i + 1]) * (p.y * k_inverse));
                    x[i + 2] = __float_as_uint(__uint_as_float(x[i + 2]) * (p.z * k_inverse));
                    x[i + 3] = __float_as_uint(__uint_as_float(x[i + 3]) * (p.w * k_inverse));
                }
            }
            if (edge) {
#pragma unroll
                for (int i = 0; i < K2; ++i)
                    if (i > hi || i < lo) x[i] = 0xFF800000u;        // -infinity
            }
            float f = c * k_this;
            if (f < 1e-45f) f = 1e-45f;                          // (NaN stays; zero would make NaN of -infinity)
            float most = largest<K2>(x);
            if constexpr (SIDES > 1) {
                most_of[sb][side * 128 + row] = most;
                if (!meet<SIDES>(rows, dead)) { alive = false; break; }      // (all lanes have their S: P may lie over it now)
                most = largest_of<SIDES>(most_of[sb], row);
            }
            most *= f;
            const bool raise = most - top > kSlack || (top == -INFINITY && most > -INFINITY);
            float factor = 1.0f;
            if (raise) {
                factor = top == -INFINITY ? 0.0f : exp2_of(top - most);
                top = most;
                sum *= factor;
            }
            const bool grows = v_this > v_unit;
            if (grows) {
                factor *= v_unit * inverse_of(v_this);
                v_unit = v_this;
            }
            const unsigned long long f2 = pair_of(f), shift = pair_of(top == -INFINITY ? 0.0f : kLift - top);
            unsigned long long s2[2] = {};
            uint32_t lo16[K2 / 2];
            auto terms = [&](int i, float2 p) {
                const __half2 h = __floats2half2_rn(p.x, p.y);
                const float2 back = __half22float2(h);
                const __half2 l = __floats2half2_rn(p.x - back.x, p.y - back.y);
                x[i / 2] = *reinterpret_cast<const uint32_t*>(&h);
                lo16[i / 2] = *reinterpret_cast<const uint32_t*>(&l);
            };
            auto weights = [&](int i) {
                const float2 t = values_of(pair_fma(pair_of(x[i], x[i + 1]), f2, shift));
                const float2 p = make_float2(exp2_of(t.x), exp2_of(t.y));
                s2[i / 2 & 1] = pair_add(s2[i / 2 & 1], pair_of(__float_as_uint(p.x), __float_as_uint(p.y)));
                return p;
            };
            if (!uneven) {
#pragma unroll
                for (int i = 0; i < K2; i += 2) terms(i, weights(i));
            } else {
#pragma unroll
                for (int i = 0; i < K2; i += 4) {
                    const float4 w = lds4(v_pow + i * 4);
                    float2 p = weights(i), q = weights(i + 2);
                    // (A power of a token that the row does not see may be anything.)
                    p.x = p.x == 0.0f ? 0.0f : p.x * (w.x * v_inverse);
                    p.y = p.y == 0.0f ? 0.0f : p.y * (w.y * v_inverse);
                    q.x = q.x == 0.0f ? 0.0f : q.x * (w.z * v_inverse);
                    q.y = q.y == 0.0f ? 0.0f : q.y * (w.w * v_inverse);
                    terms(i, p);
                    terms(i + 2, q);
                }
            }
            const float2 s = values_of(pair_add(s2[0], s2[1]));
            sum += s.x + s.y;
            tc::tmem_store<K2 / 2>(at + uint32_t(side * (K2 / 2)), x);
            tc::tmem_store<K2 / 2>(at + KT / 2 + uint32_t(side * (K2 / 2)), lo16);
            if (edge) {                                  // values that are not finite
                if (!wait(v_full(j % S::STAGES), j / S::STAGES & 1)) { alive = false; break; }
                if (clear_not_finite<kFp16Exp, SIDES>(v_at + uint32_t(j % S::STAGES) * 2 * S::V_TERM, 2 * S::V_TERM, tid)) odd = 1;
                __syncwarp();
            }
            tc::tmem_store_wait();
            tc::fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full(sb));
            if (j > 0) {
                if (!gather(j - 1)) { alive = false; break; }
                if (__any_sync(tc::kFullMask, raise || grows)) {
#pragma unroll
                    for (int i = 0; i < D2; ++i) o[i] *= factor;
                }
            }
            v_mine = v_this * inverse_of(v_unit);
        }
        if constexpr (SIDES > 1) sum_of[side * 128 + row] = sum;
        if (alive && gather(tiles - 1) && (SIDES == 1 || meet<SIDES>(rows, dead))) {
            if constexpr (SIDES > 1) sum = sum_of_lanes<SIDES>(sum_of, row);
            const float inv = 1.0f / sum;
            const bool look = odd != 0;
            float* const to = static_cast<float*>(a.out) + token * a.out_stride + (long long)head * D + half * DV + side * D2;
            if (r.there) {
#pragma unroll
                for (int i = 0; i < D2; i += 32) {
                    float y[32];
#pragma unroll
                    for (int n = 0; n < 32; ++n) y[n] = o[i + n] * inv * v_unit;
                    if (look) add_not_finite<KT, float>(a, it, r, half * DV + side * D2 + i, D, y);      // visible values that were left out
#pragma unroll
                    for (int n = 0; n < 32; n += 4) *reinterpret_cast<float4*>(to + i + n) = make_float4(y[n], y[n + 1], y[n + 2], y[n + 3]);
                }
                if (a.lse && half == 0 && side == 0) a.lse[token * a.n_heads + head] = top * kLn2 + logf(sum * kUnlift);
            }
        }
        if (SIDES > 1 && dead) leave<SIDES>(rows);
    } else if (warp == kSoftWarps) {
        // --------------------------------------------------------------------- copies
        const int n_q = a.tokens * a.group * 128;        // bytes of a 64-wide piece
        if (tc::elect()) {
            mbar_arrive_expect_tx(q_full, uint32_t(2 * CH * n_q) + a.extra_tx);
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int n = 0; n < CH; ++n)
                    tc::load_3d(q_at + t * S::Q_TERM + n * 16384, &a.qmap, n * 64, it.head * a.group, t * a.n_tok + it.seq0 + it.t0, q_full);
        }
        __syncwarp();
        // The powers of two of a tile's keys and values, two of each to a lane: read ahead, and put into a
        // slot once the tile that had it has made its part of the output (which comes after v_empty).
        float k_pow[2], v_pow[2];
        auto fetch = [&](int t) {
            if (t >= tiles) return;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int tok = it.seq0 + first + t * KT + n * 32 + lane;
                const long long row = (long long)tok * a.n_kv + it.head;
                k_pow[n] = tok < a.n_tok ? a.kscale[row] : 1.0f;
                v_pow[n] = tok < a.n_tok ? a.vscale[row] : 1.0f;
            }
        };
        auto hand_out = [&](int t) {
            if (t >= tiles) return;
            float* const to = scale_mem[t % S::SLOTS];
            const uint32_t k_most = __reduce_max_sync(tc::kFullMask, max(__float_as_uint(k_pow[0]), __float_as_uint(k_pow[1])));
            const uint32_t v_most = __reduce_max_sync(tc::kFullMask, max(__float_as_uint(v_pow[0]), __float_as_uint(v_pow[1])));
            const bool even = k_most < 0x7F800000u &&            // (NaN is for the rows that see it)
                              __all_sync(tc::kFullMask, __float_as_uint(k_pow[0]) == k_most && __float_as_uint(k_pow[1]) == k_most &&
                                                            __float_as_uint(v_pow[0]) == v_most && __float_as_uint(v_pow[1]) == v_most);
            if (lane == 0) {
                to[2 * KT] = __uint_as_float(k_most);
                to[2 * KT + 1] = __uint_as_float(v_most);
                to[2 * KT + 2] = even ? 0.0f : 1.0f;
            }
            if (!even) {
                const bool edge = on_edge<KT>(a, it, first + t * KT);            // (there the rows see different ones)
                const float k_inverse = edge ? 1.0f : inverse_of(__uint_as_float(k_most)), v_inverse = edge ? 1.0f : inverse_of(__uint_as_float(v_most));
#pragma unroll
                for (int n = 0; n < 2; ++n) to[n * 32 + lane] = k_pow[n] * k_inverse, to[KT + n * 32 + lane] = v_pow[n] * v_inverse;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(scales_full(t % S::SLOTS));
        };
        fetch(0);
        int j = 0;
        for (; j < tiles; ++j) {
            const int s = j % S::STAGES;
            const uint32_t phase = (j / S::STAGES & 1) ^ 1;
            const int key = it.seq0 + first + j * KT;
            if (!wait(k_empty(s), phase)) break;
            if (tc::elect()) {
                mbar_arrive_expect_tx(k_full(s), 2 * S::K_TERM);
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int n = 0; n < CH; ++n)
                        tc::load_3d(k_at + (2 * s + t) * S::K_TERM + n * KT * 128, &a.kmap, n * 64, it.head, t * a.n_tok + key, k_full(s));
            }
            __syncwarp();
            if (!wait(v_empty(s), phase)) break;
            if (tc::elect()) {
                mbar_arrive_expect_tx(v_full(s), 2 * S::V_TERM);
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int n = 0; n < CV; ++n)
                        tc::load_3d(v_at + (2 * s + t) * S::V_TERM + n * KT * 128, &a.vmap, half * DV + n * 64, it.head, t * a.n_tok + key, v_full(s));
            }
            __syncwarp();
            if (j == 0) {
                hand_out(0);
                fetch(1);
            }
            hand_out(j + 1);
            fetch(j + 2);
        }
        if (dead) {                                      // copies still on their way end before the CTA does
            mbar_wait(q_full, 0, a.drain_limit);
            // (keys may have been requested for tile j where values were not)
            for (int t = j; t >= 0 && t > j - S::STAGES - 1; --t) {
                mbar_wait(k_full(t % S::STAGES), t / S::STAGES & 1, min(a.drain_limit, 65536u));
                mbar_wait(v_full(t % S::STAGES), t / S::STAGES & 1, min(a.drain_limit, 65536u));
            }
        }
    } else {
        // ------------------------------------------------------------------- products
        const uint32_t i_s = tc::instr(false, KT, false) | a.negate, i_o = tc::instr(false, DV, true);
        bool alive = wait(q_full, 0);
        auto scores = [&](int j) {
            const int s = j % S::STAGES, sb = j & 1;
            if (!wait(k_full(s), j / S::STAGES & 1)) return false;
            tc::fence_after();
            if (tc::elect()) {
                const uint64_t dq = tc::desc_k(q_at), dk = tc::desc_k(k_at + 2 * s * S::K_TERM);
                const uint32_t d = tmem + uint32_t(sb * KT);
                constexpr uint64_t ql = S::Q_TERM >> 4, kl = S::K_TERM >> 4;
#pragma unroll
                for (int n = 0; n < CH; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint64_t aq = dq + n * (16384 >> 4) + 2 * i, ak = dk + n * (KT * 128 >> 4) + 2 * i;
                        tc::mma(d, aq + ql, ak, i_s, n + i > 0);
                        tc::mma(d, aq, ak + kl, i_s, true);
                    }
#pragma unroll
                for (int n = 0; n < CH; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) tc::mma(d, dq + n * (16384 >> 4) + 2 * i, dk + n * (KT * 128 >> 4) + 2 * i, i_s, true);
                tc::commit(k_empty(s));
                tc::commit(s_full(sb));
            }
            __syncwarp();
            return true;
        };
        if (alive) alive = scores(0);
        for (int j = 0; j < tiles && alive; ++j) {
            const int s = j % S::STAGES, sb = j & 1;
            if (j + 1 < tiles) alive = scores(j + 1);
            if (!alive || !wait(v_full(s), j / S::STAGES & 1) || !wait(p_full(sb), j >> 1 & 1) || !wait(o_empty(sb), (j >> 1 & 1) ^ 1)) { alive = false; break; }
            tc::fence_after();
            if (tc::elect()) {
                const uint64_t dv = tc::desc_mn(v_at + 2 * s * S::V_TERM, KT * 128);
                const uint32_t p = tmem + uint32_t(sb * KT), d = tmem + S::O_AT + uint32_t(sb * DV);
                constexpr uint64_t vl = S::V_TERM >> 4;
#pragma unroll
                for (int i = 0; i < KT / 16; ++i) {
                    tc::mma_ts(d, p + KT / 2 + i * 8, dv + i * (2048 >> 4), i_o, i > 0);
                    tc::mma_ts(d, p + i * 8, dv + vl + i * (2048 >> 4), i_o, true);
                }
#pragma unroll
                for (int i = 0; i < KT / 16; ++i) tc::mma_ts(d, p + i * 8, dv + i * (2048 >> 4), i_o, true);
                tc::commit(v_empty(s));
                tc::commit(o_full(sb));
            }
            __syncwarp();
        }
        if (tc::elect()) tc::commit(drained);            // products under way end before the columns are given back
        __syncwarp();
        mbar_wait(drained, 0, a.drain_limit);
    }
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == kSoftWarps + 1) tc::tmem_free(tmem, S::COLS);
}

template <int D> PromptKernel kernel() {
    return {(const void*)&prompt_f32_kernel<D>, 32 * (Shape<D>::WARPS + 2), Shape<D>::SMEM, kTileKeys, Shape<D>::HALVES};
}

}  // namespace

PromptKernel prompt_f32(int D) { return D == 64 ? kernel<64>() : D == 128 ? kernel<128>() : kernel<256>(); }

qg_status prompt_stage(int D, const PromptStage& p, void* stream) {
    StageArgs a{};
    a.q = {p.q, p.q_stride, p.q_out, p.qscale, p.n_heads};
    a.k = {p.k, p.k_stride, p.k_out, p.kscale, p.n_kv};
    a.v = {p.v, p.v_stride, p.v_out, p.vscale, p.n_kv};
    a.cu_seq = p.cu_seq;
    a.n_tok = p.n_tok, a.n_seq = p.n_seq;
    const int64_t per = kStageThreads / 32 * kStageRows;
    const int64_t q_blocks = (int64_t(p.n_tok) * p.n_heads + per - 1) / per, kv_blocks = (int64_t(p.n_tok) * p.n_kv + per - 1) / per;
    if (q_blocks + 2 * kv_blocks > (int64_t(1) << 31) - 1) return QG_EUNSUPPORTED;
    a.q_blocks = uint32_t(q_blocks);
    a.kv_blocks = uint32_t(kv_blocks);
    void* params[] = {&a};
    const void* fn = D == 64 ? (const void*)&stage_kernel<64> : D == 128 ? (const void*)&stage_kernel<128> : (const void*)&stage_kernel<256>;
    return launch_early(fn, int(q_blocks + 2 * kv_blocks), kStageThreads, 0, 1, params, stream);
}

}  // namespace qg
