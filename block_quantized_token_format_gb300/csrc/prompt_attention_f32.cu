// Causal attention of packed prompts, fp32: as the bf16 kernel, on two fp16 terms of every operand.
//
// stage_kernel writes, for every query row and for every key tile (64 tokens of one prompt) of a head,
// the values times a power of two that takes the largest finite magnitude to [2^14, 2^15), as an fp16
// value and another of what its rounding left: 22 bits below the largest of the row or tile.  A
// score's factor is then one product per tile, and a tile's part of the output has one factor.
// Three products of 16-bit terms (small ones first: the tensor cores truncate what they add) make S;
// P is 2^7 times the exponential, so that two terms of it reach 2^-31 of the row's largest; each
// tile's P V goes to fresh accumulators and is added in fp32 registers.
//
// One CTA is 128 rows, two lanes a row (each half of a tile's keys and half of the output; one with heads
// of 256, whose operands leave no shared memory for the lanes' maxima); S and the tiles' P V have two buffers each, so that the next
// tile's S and this tile's P V run beside the softmax.  Heads of 256 take two CTAs, each 128 values of
// the output.
//
// Bound by the tensor cores, which work 68 % of the time on three products for each that counts as
// work, and by the softmax with its two terms in what is left: two prompts of up to 3500 tokens, 32
// heads of 128 on 8: 291 us with the staging (there four query rows to a warp; one row to a warp took 12 us
// more).  Two lanes a row instead of one: 377 to 306 us; four: 303 where two took 292, not kept.
#include "prompt_attention.cuh"

namespace qg {
namespace {

constexpr int kStageThreads = 256;
constexpr float kSlack = 8.0f, kLift = 7.0f;     // log2: P is 2^7 times the exponential, at most 2^15
constexpr int kTileKeys = 64, kStageRows = 4;

template <int D> struct Shape {
    static constexpr int KT = kTileKeys, DV = D < 128 ? D : 128, HALVES = D / DV, STAGES = D == 256 ? 1 : 2;
    static constexpr int SIDES = D == 256 ? 1 : 2, WARPS = 4 * SIDES;        // lanes of a row, warps of the softmax
    static constexpr int CH = D / 64, CV = DV / 64;
    static constexpr int Q_TERM = CH * 128 * 128, K_TERM = CH * KT * 128, V_TERM = CV * KT * 128;
    static constexpr int SMEM = 1024 + 2 * Q_TERM + 2 * STAGES * (K_TERM + V_TERM);
    static constexpr uint32_t O_AT = 2 * KT, COLS = 2 * KT + 2 * DV <= 256 ? 256 : 512;
};

__device__ __forceinline__ bool finite_of(float x) { return (__float_as_uint(x) & 0x7F800000u) != 0x7F800000u; }
__device__ __forceinline__ uint32_t finite_bits(float x) { return finite_of(x) ? __float_as_uint(x) & 0x7FFFFFFFu : 0u; }
// The power of two that takes a magnitude (its bits) to [2^14, 2^15), and its inverse.
__device__ __forceinline__ float lift_of(uint32_t top, float& inverse) {
    const int e = top ? min(14 - ilogbf(__uint_as_float(top)), 126) : 0;
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

struct StageArgs {
    const float *q, *k, *v;
    long long q_stride, k_stride, v_stride;
    const int32_t* cu_seq;
    uint16_t *q_out, *k_out, *v_out;             // [2 terms][n_tok][heads][D]
    float *qscale, *kscale, *vscale;             // [n_tok][heads]
    int n_tok, n_seq, n_heads, n_kv;
    uint32_t tile_blocks;                        // key tiles times heads, for keys and for values
};

template <int D> __global__ void __launch_bounds__(kStageThreads) stage_kernel(const StageArgs a) {
    tc::grid_launch_dependents();
    tc::grid_wait();
    const int tid = int(threadIdx.x), lane = tid & 31;
    if (blockIdx.x >= a.tile_blocks) {                   // queries, a warp four rows at a time
        const long long row0 = ((long long)(blockIdx.x - a.tile_blocks) * (kStageThreads / 32) + (tid >> 5)) * kStageRows;
        const long long from = (long long)a.cu_seq[0] * a.n_heads, to = min((long long)a.cu_seq[a.n_seq], (long long)a.n_tok) * a.n_heads;
        constexpr int N = (D + 127) / 128;
        float4 x[kStageRows][N];
#pragma unroll
        for (int k = 0; k < kStageRows; ++k) {
            const long long row = row0 + k;
            const long long tok = row / a.n_heads;
            const float* const src = a.q + tok * a.q_stride + (row - tok * a.n_heads) * D;
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
            if (lane == 0) a.qscale[row] = inverse;
            uint16_t* const out = a.q_out + row * D;
            const size_t term = size_t(a.n_tok) * a.n_heads * D;
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
        return;
    }
    __shared__ uint32_t most[kStageThreads / 32];
    uint32_t b = blockIdx.x;
    const bool values = b >= a.tile_blocks / 2;
    if (values) b -= a.tile_blocks / 2;
    const int slot = int(b / uint32_t(a.n_kv)), head = int(b - uint32_t(slot) * uint32_t(a.n_kv));
    PromptItem it;
    if (!prompt_piece(a.cu_seq, a.n_seq, a.n_tok, kTileKeys, slot, it)) return;
    const long long tok0 = it.seq0 + it.t0, stride = values ? a.v_stride : a.k_stride;
    const int rows = min(kTileKeys, it.len - it.t0);
    const float* const src = (values ? a.v : a.k) + tok0 * stride + (long long)head * D;
    constexpr int N = kTileKeys * D / 4 / kStageThreads, PER = D / 4;        // quads of a thread, of a row
    float4 x[N];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int n = i * kStageThreads + tid, row = n / PER;
        x[i] = row < rows ? *reinterpret_cast<const float4*>(src + row * stride + (n % PER) * 4) : make_float4(0, 0, 0, 0);
        top = max(max(max(top, finite_bits(x[i].x)), finite_bits(x[i].y)), max(finite_bits(x[i].z), finite_bits(x[i].w)));
    }
    top = __reduce_max_sync(tc::kFullMask, top);
    if (lane == 0) most[tid >> 5] = top;
    __syncthreads();
    for (int w = 0; w < kStageThreads / 32; ++w) top = max(top, most[w]);
    float inverse;
    const float lift = lift_of(top, inverse);
    if (tid == 0) (values ? a.vscale : a.kscale)[tok0 * a.n_kv + head] = inverse;
    uint16_t* const out = values ? a.v_out : a.k_out;
    const size_t term = size_t(a.n_tok) * a.n_kv * D;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int n = i * kStageThreads + tid, row = n / PER;
        if (row >= rows) break;
        uint2 hi, lo;
        terms4(x[i], lift, hi, lo);
        uint16_t* const to = out + ((tok0 + row) * a.n_kv + head) * D + (n % PER) * 4;
        *reinterpret_cast<uint2*>(to) = hi;
        *reinterpret_cast<uint2*>(to + term) = lo;
    }
}

template <int D> __global__ void __launch_bounds__(32 * (Shape<D>::WARPS + 2), 1) prompt_f32_kernel(const __grid_constant__ PromptArgs a) {
    using S = Shape<D>;
    constexpr int KT = S::KT, CH = S::CH, CV = S::CV, DV = S::DV, SIDES = S::SIDES, kSoftWarps = S::WARPS;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bar_mem[18];
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
        const float* const ks = a.kscale + (long long)(it.seq0 + first) * a.n_kv + it.head;
        const float* const vs = a.vscale + (long long)(it.seq0 + first) * a.n_kv + it.head;
        const long long hop = (long long)KT * a.n_kv;
        float k_next = ks[0], v_next = vs[0], v_mine = 0.0f;
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
            const float f = fmaxf(c * k_next, 1.17549435e-38f), v_this = v_next;
            if (j + 1 < tiles) {
                k_next = ks[(j + 1) * hop];
                v_next = vs[(j + 1) * hop];
            }
            if (!wait(s_full(sb), j >> 1 & 1)) { alive = false; break; }
            tc::fence_after();
            uint32_t x[K2];
            const uint32_t at = mine + uint32_t(sb * KT);
            tc::tmem_load(at + uint32_t(side * K2), x);
            const bool edge = on_edge<KT>(a, it, k0);
            if (edge) {
                const int hi = r.pos - k0 - side * K2, lo = r.low - k0 - side * K2;
#pragma unroll
                for (int i = 0; i < K2; ++i)
                    if (i > hi || i < lo) x[i] = 0xFF800000u;        // -infinity
            }
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
            const unsigned long long f2 = pair_of(f), shift = pair_of(top == -INFINITY ? 0.0f : kLift - top);
            unsigned long long s2[2] = {};
            uint32_t lo16[K2 / 2];
#pragma unroll
            for (int i = 0; i < K2; i += 2) {
                const float2 t = values_of(pair_fma(pair_of(x[i], x[i + 1]), f2, shift));
                const float p0 = exp2_of(t.x), p1 = exp2_of(t.y);
                s2[i / 2 & 1] = pair_add(s2[i / 2 & 1], pair_of(__float_as_uint(p0), __float_as_uint(p1)));
                const __half2 h = __floats2half2_rn(p0, p1);
                const float2 back = __half22float2(h);
                const __half2 l = __floats2half2_rn(p0 - back.x, p1 - back.y);
                x[i / 2] = *reinterpret_cast<const uint32_t*>(&h);
                lo16[i / 2] = *reinterpret_cast<const uint32_t*>(&l);
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
                if (__any_sync(tc::kFullMask, raise)) {
#pragma unroll
                    for (int i = 0; i < D2; ++i) o[i] *= factor;
                }
            }
            v_mine = v_this;
        }
        if constexpr (SIDES > 1) sum_of[side * 128 + row] = sum;
        if (alive && gather(tiles - 1) && (SIDES == 1 || meet<SIDES>(rows, dead))) {
            if constexpr (SIDES > 1) sum = sum_of_lanes<SIDES>(sum_of, row);
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            const bool look = odd != 0;
            float* const to = static_cast<float*>(a.out) + token * a.out_stride + (long long)head * D + half * DV + side * D2;
            if (r.there) {
#pragma unroll
                for (int i = 0; i < D2; i += 32) {
                    float y[32];
#pragma unroll
                    for (int n = 0; n < 32; ++n) y[n] = sum == 0.0f ? 0.0f : o[i + n] * inv;
                    if (look) add_not_finite<KT, float>(a, it, r, half * DV + side * D2 + i, D, y);      // visible values that were left out
#pragma unroll
                    for (int n = 0; n < 32; n += 4) *reinterpret_cast<float4*>(to + i + n) = make_float4(y[n], y[n + 1], y[n + 2], y[n + 3]);
                }
                if (a.lse && half == 0 && side == 0) a.lse[token * a.n_heads + head] = sum == 0.0f ? -INFINITY : (top - kLift) * kLn2 + logf(sum);
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
    a.q = p.q, a.k = p.k, a.v = p.v;
    a.q_stride = p.q_stride, a.k_stride = p.k_stride, a.v_stride = p.v_stride;
    a.cu_seq = p.cu_seq;
    a.q_out = p.q_out, a.k_out = p.k_out, a.v_out = p.v_out;
    a.qscale = p.qscale, a.kscale = p.kscale, a.vscale = p.vscale;
    a.n_tok = p.n_tok, a.n_seq = p.n_seq, a.n_heads = p.n_heads, a.n_kv = p.n_kv;
    const int64_t tiles = 2 * (int64_t(p.n_tok) / kTileKeys + p.n_seq) * p.n_kv;
    const int64_t per = kStageThreads / 32 * kStageRows, rows = (int64_t(p.n_tok) * p.n_heads + per - 1) / per;
    if (tiles + rows > (int64_t(1) << 31) - 1) return QG_EUNSUPPORTED;
    a.tile_blocks = uint32_t(tiles);
    void* params[] = {&a};
    const void* fn = D == 64 ? (const void*)&stage_kernel<64> : D == 128 ? (const void*)&stage_kernel<128> : (const void*)&stage_kernel<256>;
    return launch_early(fn, int(tiles + rows), kStageThreads, 0, 1, params, stream);
}

}  // namespace qg
