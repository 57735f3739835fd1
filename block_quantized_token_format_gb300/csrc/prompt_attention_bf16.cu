// Causal attention of packed prompts, bf16: S = Q K^T and O += P V on tcgen05, softmax by a thread
// a row.  Shapes and items in prompt_attention.cuh.
//
// One CTA is 128 rows.  Eight warps do the softmax, two lanes a row (each half of the tile's keys and
// half of the output); one warp copies keys and values, one issues
// the products.  S (fp32) and then P (bf16, over S) lie in tensor memory, P being the second
// product's operand there, and O is summed there.  A row's reference is raised, and O scaled,
// only where a tile's maximum is more than 2^8 above it: then rarely after the first tiles.  P is 2^-8 times the
// exponential, so that it stays below 1 and O below the sum of the values: they may be as large as that allows.
// CTAs stay and take one item after another, asking for the next that no CTA has begun: the next one's queries and first keys are copied, and its
// first S is made, while the last one's output is written.  Heads of 64 and 128 take 256 columns of
// tensor memory and at most 97 KB, so that two CTAs share an SM and the one's softmax runs beside the
// other's products; heads of 256 fill an SM with one CTA.  The next tile's S is issued before P is
// waited for.
//
// Bound by a tile's softmax, one dependent chain of tensor-memory load, maximum over two lanes,
// exponentials and store, which the two CTAs' tiles cover only in part, and by the scores' products,
// which read 6 KB of operands from shared memory in the 32 clocks that they would take: heads of
// 128 keep the tensor cores busy 71 % of the time and issue instructions in 52 % of the clocks, DRAM is
// at 8 %.  Back to back: 8191 tokens, 48 heads of 128 on 16: 614 us, 1340 TFLOP/s of
// visible keys' products; 60 packed prompts of up to 1500 tokens, 32 heads on 8: 299 us; 5 prompts of
// up to 5000, 24 heads of 256 on 4, window 1024: 193 us.  Steps (single calls): one lane a row to two and packed arithmetic 875 -> 707 us (8191 tokens); CTAs that
// stay 524 -> 425 (packed prompts); tiles of 64 keys, not 128, with two buffers of S 425 -> 352; items
// taken as CTAs come free, not in turn, 349 -> 287.  Four lanes a row with heads of 256: 203 -> 210, not kept.
//
// Numbers: products of bf16 values are exact, sums fp32; P is rounded to bf16 (2^-8 of each), its
// sum is not.  A tile on an edge (some row does not see some key) may hold values of keys that
// other rows, or none, see: one that is not finite would reach every row as 0 * inf.  Such tiles are looked
// through, those values made zeros for the product, and the rows that see them get them afterwards.
#include "prompt_attention.cuh"

namespace qg {
namespace {

constexpr int kItems = 4;          // that the copying warp may be ahead
constexpr float kSlack = 8.0f, kUnslack = 256.0f;     // log2: how far scores may pass the reference; P is 2^-8 times the exponential, at most 1

template <int D> struct Shape {
    static constexpr int KT = 64, STAGES = 2, SB = 2;
    static constexpr int SIDES = 2, WARPS = 4 * SIDES;    // lanes of a row, warps of the softmax
    static constexpr int THREADS = 32 * (WARPS + 2);
    static constexpr int CH = D / 64;                                // 64-wide pieces of a head
    static constexpr int Q_BYTES = CH * 128 * 128, T_BYTES = CH * KT * 128;      // (T: a key or value tile)
    static constexpr int SMEM = 1024 + Q_BYTES + 2 * STAGES * T_BYTES;
    static constexpr uint32_t O_AT = SB * KT, COLS = D == 256 ? 512 : 256;
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&p);
}

template <int D> __global__ void __launch_bounds__(Shape<D>::THREADS, D == 256 ? 1 : 2) prompt_bf16_kernel(const __grid_constant__ PromptArgs a) {
    using S = Shape<D>;
    constexpr int KT = S::KT, CH = S::CH, SIDES = S::SIDES, kSoftWarps = S::WARPS;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bar_mem[19 + 2 * kItems];
    __shared__ uint4 answer_mem;                         // the grid's next item
    __shared__ PromptItem item_mem[kItems];              // found by the copying warp, ahead of the others
    __shared__ uint32_t tmem_at, dead, odd;
    __shared__ float most_of[2][SIDES * 128], sum_of[SIDES * 128];       // the lanes' maxima, of even and odd tiles, and sums

    const int tid = int(threadIdx.x), warp = __shfl_sync(tc::kFullMask, tid >> 5, 0), lane = tid & 31;
    tc::grid_launch_dependents();
    tc::grid_wait();
    const int slots = a.n_tok / a.tokens + a.n_seq;      // (a CTA for each slot and key/value head)

    const uint32_t q_at = (smem_addr(smem_raw) + 1023u) & ~1023u, k_at = q_at + S::Q_BYTES, v_at = k_at + S::STAGES * S::T_BYTES;
    const uint32_t bars = smem_addr(bar_mem);
    const uint32_t q_full = bars, q_empty = bars + 8, o_full = bars + 16, o_empty = bars + 24, pv_done = bars + 32, drained = bars + 40;
    auto k_full = [&](int s) { return bars + 48u + 8u * uint32_t(s); };
    auto k_empty = [&](int s) { return bars + 64u + 8u * uint32_t(s); };
    auto v_full = [&](int s) { return bars + 80u + 8u * uint32_t(s); };
    auto v_empty = [&](int s) { return bars + 96u + 8u * uint32_t(s); };
    auto s_full = [&](int s) { return bars + 112u + 8u * uint32_t(s); };
    auto p_full = [&](int s) { return bars + 128u + 8u * uint32_t(s); };
    auto i_full = [&](int s) { return bars + 144u + 8u * uint32_t(s); };
    auto i_empty = [&](int s) { return bars + 144u + 8u * uint32_t(kItems + s); };
    const uint32_t answered = bars + 144u + 16u * uint32_t(kItems), answer = smem_addr(&answer_mem);
    const tc::Waits wait{&dead, a.status, a.wait_limit};

    if (tid == 0) {
        dead = odd = 0;
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        mbar_init(o_full, 1);
        mbar_init(o_empty, kSoftWarps);
        mbar_init(pv_done, 1);
        mbar_init(drained, 1);
        mbar_init(answered, 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(k_full(s), 1);
            mbar_init(k_empty(s), 1);
            mbar_init(v_full(s), 1);
            mbar_init(v_empty(s), 1);
            mbar_init(s_full(s), 1);
            mbar_init(p_full(s), kSoftWarps);
        }
        for (int s = 0; s < kItems; ++s) {
            mbar_init(i_full(s), 1);
            mbar_init(i_empty(s), kSoftWarps + 1);
        }
        mbar_fence_init();
    }
    if (warp == kSoftWarps + 1) tc::tmem_alloc(smem_addr(&tmem_at), S::COLS);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = tmem_at;
    // The CTA's n-th item, which the copying warp has found; false: there is none, or a wait gave up.
    auto next_item = [&](uint32_t n) { return wait(i_full(int(n % kItems)), n / kItems & 1) && item_mem[n % kItems].tiles > 0; };
    auto give_back = [&](uint32_t n) {
        __syncwarp();
        if (lane == 0) mbar_arrive(i_empty(int(n % kItems)));
    };

    if (warp < kSoftWarps) {
        constexpr int K2 = KT / SIDES, D2 = D / SIDES;
        const int rows = warp & 3, half = warp >> 2, row = rows * 32 + lane;
        const uint32_t mine = tmem + (uint32_t(rows) << 21), o_mine = mine + S::O_AT + uint32_t(half * D2);
        bool alive = true;
        uint32_t n = 0, g = 0;                           // items and key tiles so far
        while (alive && next_item(n)) {
            // What the loop over the tiles needs of the item: little, registers are what it lacks.
            int tiles, inside_lo, inside_hi, pos, low;   // tiles inside: every row sees every key; visible keys from the first tile on
            {
                const PromptItem it = item_mem[n % kItems];
                const PromptRow r = prompt_row(a, it, row);
                const int last = min(it.t0 + a.tokens, it.len) - 1;
                tiles = it.tiles;
                pos = r.pos - it.first - half * K2;
                low = r.low - it.first - half * K2;
                inside_lo = a.window > 0 ? (max(0, last - a.window + 1 - it.first) + KT - 1) / KT : 0;
                inside_hi = (it.t0 - it.first + 1) / KT;             // (exclusive)
            }
            float top = -INFINITY, sum = 0.0f;           // the row's reference (log2 of an exponential), this lane's sum of P
            for (int j = 0; j < tiles; ++j, ++g) {
                const int sb = int(g % S::SB);
                if (!wait(s_full(sb), g / S::SB & 1)) { alive = false; break; }
                tc::fence_after();
                uint32_t x[K2];
                const uint32_t at = mine + uint32_t(sb * KT);
                tc::tmem_load(at + uint32_t(half * K2), x);
                const bool edge = j < inside_lo || j >= inside_hi;
                if (edge) {
                    const int hi = pos - j * KT, lo = low - j * KT;
#pragma unroll
                    for (int i = 0; i < K2; ++i)
                        if (i > hi || i < lo) x[i] = 0xFF800000u;        // -infinity
                }
                float most = largest<K2>(x);
                float* const shared_most = most_of[g & 1];
                shared_most[half * 128 + row] = most;
                if (!meet<SIDES>(rows, dead)) { alive = false; break; }      // (all lanes have their S: P may lie over it now)
                most = largest_of<SIDES>(shared_most, row) * a.c;
                const bool raise = most - top > kSlack || (top == -INFINITY && most > -INFINITY);
                float factor = 1.0f;
                if (raise) {
                    factor = top == -INFINITY ? 0.0f : exp2_of(top - most);
                    top = most;
                    sum *= factor;
                }
                if (j > 0 && __any_sync(tc::kFullMask, raise)) {
                    if (!wait(pv_done, (g - 1) & 1)) { alive = false; break; }
                    tc::fence_after();
#pragma unroll
                    for (int i = 0; i < D2; i += 16) {
                        uint32_t o[16];
                        tc::tmem_load16(o_mine + i, o);
                        tc::tmem_load_wait16(o);
#pragma unroll
                        for (int n = 0; n < 16; ++n) o[n] = __float_as_uint(__uint_as_float(o[n]) * factor);
                        tc::tmem_store16(o_mine + i, o);
                    }
                }
                const unsigned long long c2 = pair_of(a.c), shift = pair_of(top == -INFINITY ? 0.0f : -top - kSlack);
                unsigned long long s2[2] = {};
#pragma unroll
                for (int i = 0; i < K2; i += 2) {
                    const float2 t = values_of(pair_fma(pair_of(x[i], x[i + 1]), c2, shift));
                    const float p0 = exp2_of(t.x), p1 = exp2_of(t.y);
                    s2[i / 2 & 1] = pair_add(s2[i / 2 & 1], pair_of(__float_as_uint(p0), __float_as_uint(p1)));
                    x[i / 2] = pack_bf16(p0, p1);
                }
                const float2 s = values_of(pair_add(s2[0], s2[1]));
                sum += s.x + s.y;
                tc::tmem_store<K2 / 2>(at + uint32_t(half * (K2 / 2)), x);
                if (edge) {                                  // values that are not finite
                    if (!wait(v_full(int(g % S::STAGES)), g / S::STAGES & 1)) { alive = false; break; }
                    if (clear_not_finite<kBf16Exp, SIDES>(v_at + (g % S::STAGES) * S::T_BYTES, S::T_BYTES, tid)) odd = 1;
                    __syncwarp();
                }
                tc::tmem_store_wait();
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full(sb));
            }
            sum_of[half * 128 + row] = sum;
            alive = alive && wait(o_full, n & 1) && meet<SIDES>(rows, dead);
            if (alive) {
                tc::fence_after();
                sum = sum_of_lanes<SIDES>(sum_of, row);
                const float inv = 1.0f / sum;                // (all scores -infinity: the sum is 0, the average NaN)
                const PromptItem it = item_mem[n % kItems];
                const PromptRow r = prompt_row(a, it, row);
                const long long token = it.seq0 + r.tok;
                const int head = it.head * a.group + row % a.group;
                const bool look = odd != 0;
                uint16_t* const to = static_cast<uint16_t*>(a.out) + token * a.out_stride + (long long)head * D + half * D2;
#pragma unroll 1
                for (int d = 0; d < D2; d += 32) {
                    uint32_t o[32];
                    tc::tmem_load32(o_mine + d, o);
                    tc::tmem_load_wait32(o);
                    if (d + 32 >= D2) {                      // the next item's output may come
                        tc::fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(o_empty);
                    }
                    float y[32];
#pragma unroll
                    for (int n = 0; n < 32; ++n) y[n] = __uint_as_float(o[n]) * inv;
                    if (look && r.there) add_not_finite<KT, __nv_bfloat16>(a, it, r, half * D2 + d, D, y);      // visible values that were left out
                    uint32_t w[16];
#pragma unroll
                    for (int n = 0; n < 16; ++n) w[n] = pack_bf16(y[2 * n], y[2 * n + 1]);
                    store_rows(to + d, r.there, w, lane);
                }
                if (r.there && a.lse && half == 0) a.lse[token * a.n_heads + head] = top * kLn2 + logf(sum * kUnslack);
            }
            give_back(n);
            ++n;
        }
        if (dead) leave<SIDES>(rows);
    } else if (warp == kSoftWarps) {
        // --------------------------------------------------------------------- copies
        const int n_q = a.tokens * a.group * 128;        // bytes of a 64-wide piece
        uint32_t n = 0, gk = 0, gv = 0;                  // items, key and value tiles requested
        uint32_t extra = a.extra_tx;
        PromptItem it;
        auto hand_out = [&](uint32_t n) {                // the n-th item to the other warps
            const int s = int(n % kItems);
            if (!wait(i_empty(s), (n / kItems & 1) ^ 1)) return false;
            if (lane == 0) {
                item_mem[s] = it;
                mbar_arrive(i_full(s));
            }
            __syncwarp();
            return true;
        };
        // After its own item those of CTAs that have not begun, one asked for ahead: items differ in their
        // tiles by far (in equal turns the most loaded CTA of 60 packed prompts had 1.32 times the mean).
        uint32_t asked = 0, heard = 0;
        auto ask = [&]() {
            tc::fence_async();                           // the last answer has been read
            if (tc::elect()) {
                mbar_arrive_expect_tx(answered, 16);
                tc::ask_block(answer, answered);
            }
            __syncwarp();
            ++asked;
        };
        auto next_block = [&]() {
            if (dead || !wait(answered, heard & 1)) return -1;
            ++heard;
            const int block = tc::block_of(answer);
            __syncwarp();
            return block;
        };
        for (int at = int(blockIdx.x); at >= 0; at = a.asks ? next_block() : -1) {
            if (a.asks) ask();
            const int b = at / a.n_kv;
            it.head = at - b * a.n_kv;
            prompt_check(a, at);
            if (!prompt_piece(a.cu_seq, a.n_seq, a.n_tok, a.tokens, slots - 1 - b, it)) continue;
            key_range<KT>(a, it, false);
            if (!hand_out(n)) break;
            if (!wait(q_empty, (n & 1) ^ 1)) break;
            if (tc::elect()) {
                mbar_arrive_expect_tx(q_full, uint32_t(CH * n_q) + extra);
#pragma unroll
                for (int c = 0; c < CH; ++c) tc::load_3d(q_at + c * 16384, &a.qmap, c * 64, it.head * a.group, it.seq0 + it.t0, q_full);
            }
            __syncwarp();
            extra = 0;
            ++n;
            for (int j = 0; j < it.tiles; ++j) {
                const int s = int(gk % S::STAGES), key = it.seq0 + it.first + j * KT;
                const uint32_t phase = (gk / S::STAGES & 1) ^ 1;
                if (!wait(k_empty(s), phase)) break;
                if (tc::elect()) {
                    mbar_arrive_expect_tx(k_full(s), S::T_BYTES);
#pragma unroll
                    for (int c = 0; c < CH; ++c) tc::load_3d(k_at + s * S::T_BYTES + c * KT * 128, &a.kmap, c * 64, it.head, key, k_full(s));
                }
                __syncwarp();
                ++gk;
                if (!wait(v_empty(s), phase)) break;
                if (tc::elect()) {
                    mbar_arrive_expect_tx(v_full(s), S::T_BYTES);
#pragma unroll
                    for (int c = 0; c < CH; ++c) tc::load_3d(v_at + s * S::T_BYTES + c * KT * 128, &a.vmap, c * 64, it.head, key, v_full(s));
                }
                __syncwarp();
                ++gv;
            }
        }
        it.tiles = 0;                                    // no more items
        hand_out(n);
        if (dead) {                                      // copies still on their way end before the CTA does
            if (heard < asked) mbar_wait(answered, heard & 1, a.drain_limit);
            if (n > 0) mbar_wait(q_full, (n - 1) & 1, a.drain_limit);
            for (uint32_t i = 1; i <= S::STAGES; ++i) {
                if (gk >= i) mbar_wait(k_full(int((gk - i) % S::STAGES)), (gk - i) / S::STAGES & 1, a.drain_limit);
                if (gv >= i) mbar_wait(v_full(int((gv - i) % S::STAGES)), (gv - i) / S::STAGES & 1, a.drain_limit);
            }
        }
    } else {
        // ------------------------------------------------------------------- products
        const uint32_t i_s = tc::instr(true, KT, false) | a.negate, i_o = tc::instr(true, D, true);
        bool alive = true;
        uint32_t n = 0, g = 0;                           // items and key tiles so far
        // S of the CTA's g-th tile.
        auto scores = [&](uint32_t g, bool last) {
            const int s = int(g % S::STAGES), sb = int(g % S::SB);
            if (!wait(k_full(s), g / S::STAGES & 1)) return false;
            tc::fence_after();
            if (tc::elect()) {
                const uint64_t dq = tc::desc_k(q_at), dk = tc::desc_k(k_at + s * S::T_BYTES);
#pragma unroll
                for (int c = 0; c < CH; ++c)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        tc::mma(tmem + uint32_t(sb * KT), dq + c * (16384 >> 4) + 2 * i, dk + c * (KT * 128 >> 4) + 2 * i, i_s, c + i > 0);
                tc::commit(k_empty(s));
                tc::commit(s_full(sb));
                if (last) tc::commit(q_empty);
            }
            __syncwarp();
            return true;
        };
        while (alive && next_item(n)) {
            const int tiles = item_mem[n % kItems].tiles;
            give_back(n);
            alive = wait(q_full, n & 1);
            if (alive) alive = scores(g, tiles == 1);
            for (int j = 0; j < tiles && alive; ++j, ++g) {
                const int s = int(g % S::STAGES), sb = int(g % S::SB);
                if (j + 1 < tiles) alive = scores(g + 1, j + 2 == tiles);
                if (!alive || (j == 0 && !wait(o_empty, (n & 1) ^ 1)) || !wait(v_full(s), g / S::STAGES & 1) || !wait(p_full(sb), g / S::SB & 1)) {
                    alive = false;
                    break;
                }
                tc::fence_after();
                if (tc::elect()) {
                    const uint64_t dv = tc::desc_mn(v_at + s * S::T_BYTES, KT * 128);
#pragma unroll
                    for (int i = 0; i < KT / 16; ++i)
                        tc::mma_ts(tmem + S::O_AT, tmem + uint32_t(sb * KT + i * 8), dv + i * (2048 >> 4), i_o, j > 0 || i > 0);
                    tc::commit(v_empty(s));
                    tc::commit(pv_done);
                    if (j + 1 == tiles) tc::commit(o_full);
                }
                __syncwarp();
            }
            ++n;
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

template <int D> PromptKernel kernel() { return {(const void*)&prompt_bf16_kernel<D>, Shape<D>::THREADS, Shape<D>::SMEM, Shape<D>::KT, 1}; }

}  // namespace

PromptKernel prompt_bf16(int D) { return D == 64 ? kernel<64>() : D == 128 ? kernel<128>() : kernel<256>(); }

}  // namespace qg
