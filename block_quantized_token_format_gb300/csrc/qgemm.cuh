// The product of block-quantized weights with many tokens' activations (qgemm) and the same
// grouped by expert (qgemm_experts): y = f(W x + bias) + residual.  Argument rules and formulas
// are in include/qgemv.h.
//
// A tile is 128 rows of W times `bn` tokens; the products run on tcgen05 with W's rows as M (the
// accumulators' lanes) and tokens as N, in steps of 64 along K:
//   * one thread copies, with tensor copies, W's raw codes (each step) and scales (every fourth)
//     into one ring and the tokens' operand (staged by stage_kernel, qgemm.cu) into another;
//   * groups of four warps turn the codes into 16-bit floats, a lane a row, a group a step, and put
//     them into tensor memory, from where the products take them: through shared memory, which
//     bounded the kernel, it was 32 of a step's 58 KB there (Q8_0, 32 tokens: 270 ns a step, now 209);
//   * one thread issues the products;
//   * eight warps empty the accumulators, of which there are two sets, so that a tile's epilogue
//     runs beside the next one's products.
// A CTA takes tiles in turn; consecutive tiles share their tokens (which then come from L2).
// Where tiles are few, a cluster of up to eight CTAs shares each tile's K; they join their sums through
// one another's shared memory, in the order of K (2560 x 6144, 17 tokens fp32: 61 -> 17 us).
//
// What bounds it.  Quantized weights with many tokens: the decoding (Q8_0: 209 to 213 ns a step up to 96
// tokens; instructions are issued in 69 % of the clocks, the tensor cores work in 60 %), which every tile
// of tokens does anew, and for tiles of 128 tokens and more the way of the operands into the SM, about 60 bytes
// a clock: Q8_0, bf16, 10240 x 2560, 8191 tokens 340 us, 1260 TFLOP/s (318 us, 1350 TFLOP/s where the same
// buffers come again); bf16 weights, which need no decoding, 262 us, 1640 TFLOP/s, 2560 x 6144 158 us (the same buffers
// again).  fp32: its three products and the sums' moves to registers, 2047 tokens of
// 2560 x 12288 with swiglu 327 us.  Experts: their weights' way from memory (61 tokens of ten experts out of 512,
// 1.22 GB: 221 us, 5.5 TB/s; 2048 tokens, 1.82 GB: 378 us, 4.8 TB/s), with 40 rows each and more beside the
// decoding.  A few tokens: two launches, the first copies and the join.
//
// Tried and not kept: five decoding groups (10240 x 2560, 8191 tokens 320 -> 333 us); raw codes in rows of 128
// bytes, two or four steps to a copy (320 -> 332, 2048 tokens' experts 404 -> 434).
//
// Numbers.  Quantized formats enter as fp16: a code times its fp16 scale has at most 19 bits.
// bf16 activations, which a row's power of two moves into fp16's range exactly (but for values
// 2^-29 and more below the row's largest), meet weights rounded to 11 bits: 2^-11 of a weight at most,
// an eighth of what rounding the output to bf16 costs.  fp32 activations are two fp16 terms (22
// bits), weights two (exact; affine 22 bits), in three products; the two small ones have accumulators of their
// own, and every 256 values of K the sums move to fp32 registers: the tensor cores truncate what
// they add, and a long chain of additions would lose what the terms keep.
// bf16 weights meet bf16 activations as they are, fp32 ones as three bf16 terms (all 24 bits).
#pragma once

#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "qg_layout.h"
#include "umma.cuh"

namespace qg {

constexpr int kGemmRows = 128, kGemmK = 64;
// Decoding warps: groups of four, each group a step of its own in turn.  A step's way through a group
// (its codes' arrival, the arithmetic, the stage's release, the stores) takes 1500 clocks, its
// products 512 or less, so bf16 has four groups; fp32, with three times the products and registers for
// the sums, two.
constexpr int kDrainWarps = 8;
__host__ __device__ constexpr int decode_groups(int fmt, bool f32) { return fmt == QG_BF16 ? 0 : f32 ? 2 : 4; }
__host__ __device__ constexpr int gemm_threads(int fmt, bool f32) { return 32 * (kDrainWarps + 4 * decode_groups(fmt, f32) + 3); }
constexpr int kChunkSteps = 4;               // fp32: steps of K between moves to registers
// bf16: rows of W of more than kChainValues are summed in chains of kChainSteps steps of K (512 additions on the
// tensor cores, which cut off a bit: 2^-14 of the sum), whose sums are added in fp32 in a third set of columns.
// One chain for 4 million products of one sign lost more than the output's rounding.
constexpr int kChainValues = 16384, kChainSteps = 128;
constexpr int kMostRaws = 16;

constexpr int kOperandA = kGemmRows * kGemmK * 2;

// Raw codes of a step (64 weights of 128 rows) and raw scales of four steps, as their copies' boxes
// bring them: bytes of a row.
constexpr int kScaleSteps = 4, kScaleSlots = 4;
__host__ __device__ constexpr int raw_codes(int fmt) { return fmt == QG_Q8_0 ? 64 : fmt == QG_BF16 ? 0 : 32; }
__host__ __device__ constexpr int raw_scales(int fmt) { return fmt == QG_BF16 ? 0 : fmt == QG_Q5_0 ? 48 : 16; }
__host__ __device__ constexpr int terms_x(int fmt, bool f32) { return !f32 ? 1 : fmt == QG_BF16 ? 3 : 2; }
// Tokens of the largest tile: two sets of sums (three with chains) and the stages of W's operand share
// tensor memory's 512 columns.
__host__ __device__ constexpr int gemm_sets(bool f32, int n_in) { return !f32 && n_in > kChainValues ? 3 : 2; }
__host__ __device__ constexpr int gemm_most_tokens(int fmt, bool f32, int sets = 2) {
    return fmt == QG_BF16 ? (f32 ? 128 : sets == 3 ? 160 : 256) : f32 ? 96 : sets == 3 ? 128 : 192;
}
__host__ __device__ constexpr int w_columns(int fmt, bool f32) { return fmt == QG_BF16 ? 0 : f32 ? 64 : 32; }      // of a step

struct GemmArgs {
    CUtensorMap xmap, wmap, smap;  // staged tokens [terms][n_slots][n_in]; rows of W: codes (or bf16), scales
    int n_out, n_in, n_slots, n_experts;      // n_experts 0: one matrix
    const int32_t* offsets;                   // experts: the caller's, and the tiles before each expert
    const int32_t* tile_start;
    const float* xscale;                      // a power of two per slot, or null
    const float* bias;
    const void* residual;
    void* y;
    long long residual_stride, y_stride;
    int f, bn, box, subs, stages, raws, m_tiles, n_tiles;      // box: tokens of a copy; subs: steps of K in a stage
    int parts;                                            // CTAs of a cluster that share a tile's K
    unsigned int* status;
    uint32_t wait_limit, drain_limit, extra_tx;
};

enum { kFNone = 0, kFSilu = 1, kFGelu = 2, kFGeluTanh = 3, kFSwiglu = 4 };

// (bf16 outputs: the fast exponential and division, 2^-20 of the value for |v| below 16.)
template <bool F32> __device__ __forceinline__ float silu_of(float v) {
    return F32 ? v / (1.0f + expf(-v)) : __fdividef(v, 1.0f + __expf(-v));
}

// row0: in the expert's matrix; w_row0: in the stack.  n: tokens that are copied and multiplied (experts: no more
// than the tile has, in sixteens, so that a tile for an expert's most rows costs no more where it has few).
struct GemmTile { int row0, w_row0, slot0, cols, n; };

__device__ __forceinline__ int gemm_tiles(const GemmArgs& a) {
    return (a.n_experts ? a.tile_start[a.n_experts] : a.n_tiles) * a.m_tiles;
}
// (Whole warps.)
__device__ __forceinline__ GemmTile gemm_tile(const GemmArgs& a, int t) {
    GemmTile g;
    const int nt = t / a.m_tiles;
    g.row0 = (t - nt * a.m_tiles) * kGemmRows;
    if (!a.n_experts) {
        g.w_row0 = g.row0;
        g.slot0 = nt * a.bn;
        g.cols = min(a.bn, a.n_slots - g.slot0);
        g.n = a.bn;
        return g;
    }
    int lo = 0, hi = a.n_experts;                        // the last expert with tile_start <= nt, 32 probes at a time
    const int lane = int(threadIdx.x) & 31;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, probe = lo + (lane + 1) * step;
        const bool before = probe < hi && a.tile_start[probe] <= nt;
        lo += __popc(__ballot_sync(tc::kFullMask, before)) * step;
        hi = min(hi, lo + step);
    }
    g.slot0 = a.offsets[lo] + (nt - a.tile_start[lo]) * a.bn;
    g.cols = min(a.bn, a.offsets[lo + 1] - g.slot0);
    g.n = (g.cols + 15) / 16 * 16;
    g.w_row0 = lo * a.n_out + g.row0;
    return g;
}

// ------------------------------------------------------------------------- codes to fp16

// The order of a step's values along K: eight nibbles of a word come as the pairs (0,4), (1,5),
// (2,6), (3,7), which one mask each takes out of the word; the tokens are staged in that order.
__host__ __device__ constexpr bool pairs_by_four(int fmt) { return fmt == QG_Q4_0 || fmt == QG_AFFINE4_G64 || fmt == QG_Q5_0; }

__device__ __forceinline__ __half2 as_h2(uint32_t b) { return *reinterpret_cast<__half2*>(&b); }
__device__ __forceinline__ uint32_t as_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }

// 32 weights of one row: codes (Q8_0: 8 words, else 4), fifth bits, scale (and bias) -> 16 pairs,
// and with F32 the 16 pairs of what their rounding left.
template <int FMT, bool F32>
__device__ __forceinline__ void decode32(const uint32_t* code, uint32_t fifth, __half2 d, __half2 b, uint32_t (&hi)[16], uint32_t (&lo)[16]) {
    constexpr uint32_t kThousand = 0x64006400u;          // 1024 in both halves: its last bits are a whole number
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        uint32_t u;
        float off;
        if constexpr (FMT == QG_Q8_0) {
            u = __byte_perm(code[i / 2], 0x64646464u, i % 2 ? 0x4342 : 0x4140);
            off = 1024.0f + 128.0f;
        } else {
            const int m = i % 4, j = i / 4;
            u = ((code[j] >> (4 * m)) & 0x000F000Fu) | kThousand;
            off = FMT == QG_Q4_0 ? 1024.0f + 8.0f : 1024.0f;
            if constexpr (FMT == QG_Q5_0) {
                const int s = 8 * (m / 2) + 2 * j + m % 2;           // element 8 j + m; m + 4 is 16 bits up
                u |= (s >= 4 ? fifth >> (s - 4 < 0 ? 0 : s - 4) : fifth << (4 - s < 0 ? 0 : 4 - s)) & 0x00100010u;
                off = 1024.0f + 16.0f;
            }
        }
        const __half2 q = __hsub2(as_h2(u), __float2half2_rn(off));
        if constexpr (FMT == QG_AFFINE4_G64) {
            if constexpr (F32) {
                const float2 w = make_float2(fmaf(__low2float(q), __low2float(d), __low2float(b)),
                                             fmaf(__high2float(q), __low2float(d), __low2float(b)));
                const __half2 h = __floats2half2_rn(w.x, w.y);
                hi[i] = as_bits(h);
                lo[i] = as_bits(__floats2half2_rn(w.x - __low2float(h), w.y - __high2float(h)));
            } else {
                hi[i] = as_bits(__hfma2(q, d, b));
            }
        } else {
            const __half2 h = __hmul2_rn(q, d);
            hi[i] = as_bits(h);
            if constexpr (F32) lo[i] = as_bits(__hfma2(q, d, __hneg2(h)));       // exact
        }
    }
}

// ------------------------------------------------------------------------------ the kernel

template <int FMT, bool F32, bool CHAINS> __global__ void __launch_bounds__(gemm_threads(FMT, F32), 1) qgemm_kernel(const __grid_constant__ GemmArgs a) {
    constexpr bool kQuant = FMT != QG_BF16;
    constexpr int kGroups = decode_groups(FMT, F32), kDecodeWarps = 4 * kGroups;
    constexpr int TX = terms_x(FMT, F32);
    constexpr int kStepWeights = FMT == QG_Q8_0 ? 512 : 1024;        // of a layout step
    using Out = typename std::conditional<F32, float, __nv_bfloat16>::type;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bar_mem[3 * 8 + 5 + 2 * kMostRaws + 2 * kScaleSlots];
    __shared__ uint32_t tmem_at, dead;

    const int tid = int(threadIdx.x), warp = __shfl_sync(tc::kFullMask, tid >> 5, 0), lane = tid & 31;
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    constexpr uint32_t a_bytes = kQuant ? 0 : kOperandA;             // (quantized weights' operand is in tensor memory)
    const uint32_t b_bytes = uint32_t(a.bn) * kGemmK * 2, sub_bytes = a_bytes + TX * b_bytes, stage_bytes = uint32_t(a.subs) * sub_bytes;
    const uint32_t raw0 = base + uint32_t(a.stages) * stage_bytes;
    const uint32_t bars = smem_addr(bar_mem);
    auto full = [&](int s) { return bars + 8u * uint32_t(s); };
    auto empty = [&](int s) { return bars + 8u * uint32_t(16 + s); };
    auto acc_full = [&](int b) { return bars + 8u * uint32_t(24 + b); };
    auto acc_empty = [&](int b) { return bars + 8u * uint32_t(26 + b); };
    const uint32_t drained = bars + 8u * 28u;
    auto raw_full = [&](int r) { return bars + 8u * uint32_t(29 + r); };
    auto raw_empty = [&](int r) { return bars + 8u * uint32_t(29 + kMostRaws + r); };
    auto sc_full = [&](int r) { return bars + 8u * uint32_t(29 + 2 * kMostRaws + r); };
    auto sc_empty = [&](int r) { return bars + 8u * uint32_t(29 + 2 * kMostRaws + kScaleSlots + r); };
    const uint32_t acc_cols = uint32_t(a.bn) * (F32 ? 2 : 1);                    // of one set
    const uint32_t sums_cols = (CHAINS ? 3 : 2) * acc_cols;                      // of all sets; behind them W's operand
    const uint32_t tmem_cols = kQuant ? 512 : sums_cols <= 64 ? 64 : sums_cols <= 128 ? 128 : sums_cols <= 256 ? 256 : 512;
    const tc::Waits wait{&dead, a.status, a.wait_limit};
    // (A last stage that K does not fill gets zeros.)
    const int ksteps = ((a.n_in + kGemmK - 1) / kGemmK + a.subs - 1) / a.subs * a.subs;
    // Its steps of K: all, or this CTA's part of a cluster's (in units of the scales' four).
    const int units = (ksteps + kScaleSteps - 1) / kScaleSteps, rank = a.parts > 1 ? int(blockIdx.x) % a.parts : 0;
    const int kb = units * rank / a.parts * kScaleSteps, ke = min(ksteps, units * (rank + 1) / a.parts * kScaleSteps);
    const int tile0 = int(blockIdx.x) / a.parts, tile_step = int(gridDim.x) / a.parts;

    if (tid == 0) {
        dead = 0;
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(full(s), kQuant ? 1 + 4 * a.subs : 1);
            mbar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(acc_full(b), 1);
            mbar_init(acc_empty(b), kDrainWarps);
        }
        for (int r = 0; r < a.raws; ++r) {
            mbar_init(raw_full(r), 1);
            mbar_init(raw_empty(r), 4);
        }
        for (int r = 0; r < kScaleSlots; ++r) {
            mbar_init(sc_full(r), 1);
            mbar_init(sc_empty(r), kQuant ? kDecodeWarps : 1);
        }
        mbar_init(drained, 1);
        mbar_fence_init();
    }
    if (warp == kDrainWarps + kDecodeWarps + 1) tc::tmem_alloc(smem_addr(&tmem_at), tmem_cols);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = tmem_at;
    tc::grid_launch_dependents();

    if (warp < kDrainWarps) {
        // ---------------------------------------------------------------- accumulators to y
        tc::grid_wait();
        const int half = warp >> 2;
        const uint32_t lanes = uint32_t(warp & 3) << 21;             // 32 (warp % 4) in the address's high half
        const int chunks = F32 ? (ke - kb + kChunkSteps - 1) / kChunkSteps : CHAINS ? (ke - kb + kChainSteps - 1) / kChainSteps : 1;
        const int tiles = gemm_tiles(a);
        uint32_t it = 0;
        bool alive = true;
        for (int t = tile0; t < tiles && alive; t += tile_step) {
            const GemmTile g = gemm_tile(a, t);
            const int split = (g.n / 2 + 15) / 16 * 16, from = half * split, hc = half ? g.n - split : split;      // its part of the columns
            const int row = g.row0 + (warp & 3) * 32 + lane;
            const bool there = row < a.n_out;
            const float bias = a.bias && there ? a.bias[row] : 0.0f;
            const int col = a.f == kFSwiglu ? row >> 1 : row;
            const bool writes = there && (a.f != kFSwiglu || (lane & 1) == 0);
            constexpr int kSums = !F32 ? 1 : (gemm_most_tokens(FMT, true) / 2 + 15) / 16;   // fp32: sets of 16 sums of a lane
            float sum[F32 ? 16 * kSums : 1];
            uint32_t v[16];
            // 16 columns of this lane's row: one pass per part of the epilogue that the call has, so that
            // none of them asks again for every column.
            auto put = [&](int c0, float* x) {
                const int n = min(16, g.cols - c0);
                if (n <= 0) return;
                if (a.xscale) {
                    const float mine = (lane & 15) < n ? a.xscale[g.slot0 + c0 + (lane & 15)] : 1.0f;
#pragma unroll
                    for (int c = 0; c < 16; ++c) x[c] *= __shfl_sync(tc::kFullMask, mine, c);
                }
                if (a.bias) {
#pragma unroll
                    for (int c = 0; c < 16; ++c) x[c] += bias;
                }
                if (a.f == kFSwiglu) {
#pragma unroll
                    for (int c = 0; c < 16; ++c) x[c] = silu_of<F32>(x[c]) * __shfl_xor_sync(tc::kFullMask, x[c], 1);
                } else if (a.f == kFSilu) {
#pragma unroll
                    for (int c = 0; c < 16; ++c) x[c] = silu_of<F32>(x[c]);
                } else if (a.f == kFGelu) {
#pragma unroll
                    for (int c = 0; c < 16; ++c) x[c] = 0.5f * x[c] * (1.0f + erff(x[c] * 0.70710678f));
                } else if (a.f == kFGeluTanh) {
#pragma unroll
                    for (int c = 0; c < 16; ++c) x[c] = 0.5f * x[c] * (1.0f + tanhf(0.79788456f * (x[c] + 0.044715f * x[c] * x[c] * x[c])));
                }
                if (!writes) return;
                if (a.residual) {
                    const Out* r = static_cast<const Out*>(a.residual) + (g.slot0 + c0) * a.residual_stride + col;
#pragma unroll
                    for (int c = 0; c < 16; ++c, r += a.residual_stride)
                        if (c < n) x[c] += float(*r);
                }
                Out* to = static_cast<Out*>(a.y) + (g.slot0 + c0) * a.y_stride + col;
                if (n == 16) {
#pragma unroll
                    for (int c = 0; c < 16; ++c, to += a.y_stride) *to = Out(x[c]);
                } else {
#pragma unroll
                    for (int c = 0; c < 16; ++c, to += a.y_stride)
                        if (c < n) *to = Out(x[c]);
                }
            };
            // The CTA's part of the sums, in the operands' memory (all products are done): [column][row].
            auto stash = [&](int c0, const float* x) {
#pragma unroll
                for (int c = 0; c < 16; ++c)
                    asm volatile("st.shared.f32 [%0], %1;" :: "r"(base + uint32_t(((c0 + c) * kGemmRows + (warp & 3) * 32 + lane) * 4)), "f"(x[c]) : "memory");
            };
            for (int ch = 0; ch < chunks; ++ch, ++it) {
                const int b = int(it & 1);
                if (!wait(acc_full(b), (it >> 1) & 1)) { alive = false; break; }
                tc::fence_after();
                const uint32_t acc = tmem + lanes + uint32_t(b) * acc_cols + uint32_t(from);
                if constexpr (F32) {
#pragma unroll
                    for (int u = 0; u < kSums; ++u)
                        if (u * 16 < hc) {
                            tc::tmem_load16(acc + uint32_t(g.n) + u * 16, v);
                            tc::tmem_load_wait16(v);
#pragma unroll
                            for (int c = 0; c < 16; ++c) sum[u * 16 + c] = ch == 0 ? __uint_as_float(v[c]) : sum[u * 16 + c] + __uint_as_float(v[c]);
                            tc::tmem_load16(acc + u * 16, v);
                            tc::tmem_load_wait16(v);
#pragma unroll
                            for (int c = 0; c < 16; ++c) sum[u * 16 + c] += __uint_as_float(v[c]);
                        }
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(acc_empty(b));
                } else {
                    if constexpr (CHAINS) {              // the sum so far, in the third set; of the last chain, in its own
                        for (int u = 0; u * 16 < hc; ++u) {
                            const uint32_t so_far = tmem + lanes + 2 * acc_cols + uint32_t(from + u * 16);
                            float x[16];
                            tc::tmem_load16(acc + u * 16, v);
                            tc::tmem_load_wait16(v);
                            if (ch > 0) {
#pragma unroll
                                for (int c = 0; c < 16; ++c) x[c] = __uint_as_float(v[c]);
                                tc::tmem_load16(so_far, v);
                                tc::tmem_load_wait16(v);
#pragma unroll
                                for (int c = 0; c < 16; ++c) v[c] = __float_as_uint(x[c] + __uint_as_float(v[c]));
                            }
                            tc::tmem_store16(ch + 1 < chunks ? so_far : acc + u * 16, v);
                        }
                        tc::tmem_store_wait();
                        if (ch + 1 < chunks) {
                            tc::fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(acc_empty(b));
                            continue;
                        }
                    }
                    if (hc == 0 && lane == 0) mbar_arrive(acc_empty(b));     // (16 tokens: all in the first half)
                    for (int u = 0; u * 16 < hc; ++u) {
                        tc::tmem_load16(acc + u * 16, v);
                        tc::tmem_load_wait16(v);
                        float x[16];
#pragma unroll
                        for (int c = 0; c < 16; ++c) x[c] = __uint_as_float(v[c]);
                        if ((u + 1) * 16 >= hc) {                    // the set is free before it is written out
                            tc::fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(acc_empty(b));
                        }
                        if (a.parts == 1) put(from + u * 16, x); else stash(from + u * 16, x);
                    }
                }
            }
            if constexpr (F32) {
                if (alive) {
#pragma unroll
                    for (int u = 0; u < kSums; ++u)
                        if (u * 16 < hc) {
                            if (a.parts == 1) put(from + u * 16, sum + u * 16); else stash(from + u * 16, sum + u * 16);
                        }
                }
            }
            if (a.parts > 1) {                           // (one tile)
                tc::cluster_sync();
                // Every CTA of the cluster joins and writes some of the tile's columns; the parts are
                // added in the order of K.
                if (alive)
                    for (int c0 = (rank + (warp >> 2) * a.parts) * 16; c0 < g.n; c0 += 2 * a.parts * 16) {
                        float x[16];
#pragma unroll
                        for (int c = 0; c < 16; ++c) x[c] = 0.0f;
                        for (int p = 0; p < a.parts; ++p) {
                            const uint32_t at = tc::of_cluster(base + uint32_t((c0 * kGemmRows + (warp & 3) * 32 + lane) * 4), p);
#pragma unroll
                            for (int c = 0; c < 16; ++c) x[c] += tc::load_cluster(at + uint32_t(c * kGemmRows * 4));
                        }
                        put(c0, x);
                    }
            }
        }
    } else if (warp < kDrainWarps + kDecodeWarps) {
        // --------------------------------------------------------------- codes to operand A
        if constexpr (kQuant) {
            constexpr int CB = raw_codes(FMT), SB = raw_scales(FMT);
            if (a.n_experts) tc::grid_wait();
            const int w = warp - kDrainWarps, row = (w & 3) * 32 + lane, which = w >> 2;
            const uint32_t scales0 = raw0 + uint32_t(a.raws) * (kGemmRows * CB);
            const int tiles = gemm_tiles(a);
            int s = 0, sub = 0, r = 0, sr = 0;
            uint32_t phase = 0, raw_phase = 0, n = 0, groups = 0;
            bool alive = true;
            for (int t = tile0; t < tiles && alive; t += tile_step) {
                for (int k = kb; k < ke; ++k, ++n) {
                    if (k % kScaleSteps == 0) {          // the next four steps' scales
                        if (groups && lane == 0) mbar_arrive(sc_empty(sr));
                        sr = int(groups % kScaleSlots);
                        if (!wait(sc_full(sr), groups / kScaleSlots & 1)) { alive = false; break; }
                        ++groups;
                    }
                    if (n % uint32_t(kGroups > 0 ? kGroups : 1) == uint32_t(which)) {
                        if (!wait(raw_full(r), raw_phase)) { alive = false; break; }
                        uint32_t code[2][CB / 8];
                        const uint32_t at = raw0 + uint32_t(r) * (kGemmRows * CB) + uint32_t(row) * CB + uint32_t(CB == 64 ? (row >> 1) & 3 : (row >> 2) & 1) * 16;
#pragma unroll
                        for (int c = 0; c < CB / 16; ++c) {          // the copy's swizzle: no two lanes of a phase in a bank
                            const uint4 q = tc::lds128(at ^ uint32_t(c * 16));
                            uint32_t* const to = &code[c * 16 / (CB / 2)][c * 4 % (CB / 8)];
                            to[0] = q.x, to[1] = q.y, to[2] = q.z, to[3] = q.w;
                        }
                        const uint32_t sc = scales0 + uint32_t(sr) * (kGemmRows * SB) + uint32_t(row) * SB + uint32_t(k % kScaleSteps) * (SB / 4);
                        uint32_t fifth[2] = {0, 0}, half[2];
                        if constexpr (FMT == QG_Q5_0) {
                            const uint32_t w0 = tc::lds32(sc), w1 = tc::lds32(sc + 4), w2 = tc::lds32(sc + 8);
                            fifth[0] = w0, half[0] = w1 & 0xFFFFu;
                            fifth[1] = (w1 >> 16) | (w2 << 16), half[1] = w2 >> 16;
                        } else {
                            const uint32_t w0 = tc::lds32(sc);
                            half[0] = w0 & 0xFFFFu, half[1] = w0 >> 16;
                        }
                        const int left = a.n_in - k * kGemmK;                    // weights from here to the row's end
                        const uint32_t to = tmem + (uint32_t(w & 3) << 21) + sums_cols + uint32_t((s * a.subs + sub) * w_columns(FMT, F32));
                        bool ready = false;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t hi[16], lo[16];
                            __half2 d, b;
                            if constexpr (FMT == QG_AFFINE4_G64) {
                                d = __half2half2(__ushort_as_half(static_cast<unsigned short>(half[0])));
                                b = __half2half2(__ushort_as_half(static_cast<unsigned short>(half[1])));
                            } else {
                                d = b = __half2half2(__ushort_as_half(static_cast<unsigned short>(half[h])));
                            }
                            decode32<FMT, F32>(code[h], fifth[h], d, b, hi, lo);
                            if (32 * h >= left) {                                // codes there are other bytes of the row
#pragma unroll
                                for (int i = 0; i < 16; ++i) hi[i] = lo[i] = 0;
                            }
                            // (Two phases ahead a wait would pass too soon.  The group's last step was in a stage
                            // filled since this one's last but one filling: there are at least as many stages
                            // as groups, or half as many of two steps.)
                            if (h == 0) {
                                if (!wait(empty(s), phase ^ 1)) { alive = false; break; }
                                tc::fence_after();
                            }
                            ready = true;
                            tc::tmem_store16(to + uint32_t(16 * h), hi);
                            if constexpr (F32) tc::tmem_store16(to + uint32_t(32 + 16 * h), lo);
                        }
                        if (!ready) break;
                        tc::tmem_store_wait();
                        tc::fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(full(s));
                            mbar_arrive(raw_empty(r));           // (what was read has been used: no load is still under way)
                        }
                    }
                    if (++sub == a.subs) {
                        sub = 0;
                        if (++s == a.stages) { s = 0; phase ^= 1; }
                    }
                    if (++r == a.raws) { r = 0; raw_phase ^= 1; }
                }
            }
        }
    } else if (warp == kDrainWarps + kDecodeWarps) {
        // ------------------------------------------------------------- tokens (and bf16 W)
        {
            tc::grid_wait();
            const int tiles = gemm_tiles(a);
            uint32_t extra = a.extra_tx;
            int s = 0;
            uint32_t phase = 0, filled = 0;
            bool alive = true;
            for (int t = tile0; t < tiles && alive; t += tile_step) {
                const GemmTile g = gemm_tile(a, t);
                const uint32_t term = uint32_t(g.n) * kGemmK * 2, bytes = TX * term + a_bytes;
                for (int k = kb; k < ke; k += a.subs) {
                    if (!wait(empty(s), phase ^ 1)) { alive = false; break; }
                    uint32_t at = base + uint32_t(s) * stage_bytes;
                    if (tc::elect()) {
                        mbar_arrive_expect_tx(full(s), uint32_t(a.subs) * bytes + extra);
                        for (int u = 0; u < a.subs; ++u, at += sub_bytes) {
                            if constexpr (!kQuant) tc::load_2d(at, &a.wmap, (k + u) * kGemmK, g.w_row0, full(s));
#pragma unroll
                            for (int x = 0; x < TX; ++x)
                                for (int c = 0; c < g.n; c += a.box)
                                    tc::load_3d(at + a_bytes + x * term + uint32_t(c) * kGemmK * 2, &a.xmap, (k + u) * kGemmK, g.slot0 + c, x, full(s));
                        }
                    }
                    __syncwarp();
                    extra = 0;
                    ++filled;
                    if (++s == a.stages) { s = 0; phase ^= 1; }
                }
            }
            // Copies still on their way end before the CTA does: those of the last stages.
            if (dead) {
                for (uint32_t i = 0; i < uint32_t(a.stages) && i < filled; ++i) {
                    const uint32_t n = filled - 1 - i;
                    mbar_wait(full(int(n % a.stages)), (n / a.stages) & 1, a.drain_limit);
                }
            }
        }
    } else if (warp == kDrainWarps + kDecodeWarps + 2) {
        // ------------------------------------------------------------- raw codes and scales
        if constexpr (kQuant) {
            {
                constexpr int CB = raw_codes(FMT), SB = raw_scales(FMT), kSteps = kStepWeights / kGemmK;
                if (a.n_experts) tc::grid_wait();
                const int tiles = gemm_tiles(a);
                const uint32_t scales0 = raw0 + uint32_t(a.raws) * (kGemmRows * CB);
                constexpr int kStepBytes = 512 + kSteps / kScaleSteps * SB;
                const int last = (a.n_in - 1) / kStepWeights, last_codes = (a.n_in - last * kStepWeights) * CB / kGemmK;
                int r = 0;
                uint32_t phase = 0, filled = 0, groups = 0;
                bool alive = true;
                for (int t = tile0; t < tiles && alive; t += tile_step) {
                    const GemmTile g = gemm_tile(a, t);
                    for (int k = kb; k < ke; ++k) {
                        if (!wait(raw_empty(r), phase ^ 1)) { alive = false; break; }
                        const int step = k / kSteps, in = k % kSteps;
                        if (k % kScaleSteps == 0) {
                            const int sr = int(groups % kScaleSlots);
                            if (!wait(sc_empty(sr), (groups / kScaleSlots & 1) ^ 1)) { alive = false; break; }
                            ++groups;
                            if (tc::elect()) {
                                mbar_arrive_expect_tx(sc_full(sr), kGemmRows * SB);
                                tc::load_2d(scales0 + uint32_t(sr) * (kGemmRows * SB), &a.smap,
                                            step * kStepBytes + (step == last ? last_codes : 512) + in / kScaleSteps * SB, g.w_row0, sc_full(sr));
                            }
                            __syncwarp();
                        }
                        if (tc::elect()) {
                            mbar_arrive_expect_tx(raw_full(r), kGemmRows * CB);
                            tc::load_2d(raw0 + uint32_t(r) * (kGemmRows * CB), &a.wmap, step * kStepBytes + in * CB, g.w_row0, raw_full(r));
                        }
                        __syncwarp();
                        ++filled;
                        if (++r == a.raws) { r = 0; phase ^= 1; }
                    }
                }
                if (dead) {
                    for (uint32_t i = 0; i < uint32_t(a.raws) && i < filled; ++i) {
                        const uint32_t n = filled - 1 - i;
                        mbar_wait(raw_full(int(n % a.raws)), (n / a.raws) & 1, a.drain_limit);
                    }
                    for (uint32_t i = 0; i < uint32_t(kScaleSlots) && i < groups; ++i) {
                        const uint32_t n = groups - 1 - i;
                        mbar_wait(sc_full(int(n % kScaleSlots)), (n / kScaleSlots) & 1, a.drain_limit);
                    }
                }
            }
        }
    } else if (warp == kDrainWarps + kDecodeWarps + 1) {
        // ---------------------------------------------------------------------- products
        {
            if (a.n_experts) tc::grid_wait();
            const int tiles = gemm_tiles(a);
            // fp32: the tokens' first two terms are neighbours, and so are the sums of the large products
            // and of the small ones.
            int s = 0;
            uint32_t phase = 0, it = 0;
            bool alive = true;
            for (int t = tile0; t < tiles && alive; t += tile_step) {
                const int n = a.n_experts ? gemm_tile(a, t).n : a.bn;
                const uint32_t idesc = tc::instr(!kQuant, F32 ? 2 * n : n, false), ione = tc::instr(!kQuant, n, false);
                for (int k = kb; k < ke; k += a.subs) {
                    const bool first = F32 ? k % kChunkSteps == 0 : k == kb || (CHAINS && (k - kb) % kChainSteps == 0);
                    const bool lastk = k + a.subs == ke || (F32 && (k + a.subs) % kChunkSteps == 0) || (CHAINS && (k + a.subs - kb) % kChainSteps == 0);
                    const int b = int(it & 1);
                    if (first && !wait(acc_empty(b), ((it >> 1) & 1) ^ 1)) { alive = false; break; }
                    if (!wait(full(s), phase)) { alive = false; break; }
                    tc::fence_after();
                    const uint32_t acc = tmem + uint32_t(b) * acc_cols;
                    uint32_t at = base + uint32_t(s) * stage_bytes;
                    if (tc::elect()) {
                        uint32_t wt = tmem + sums_cols + uint32_t(s * a.subs * w_columns(FMT, F32));
                        for (int u = 0; u < a.subs; ++u, at += sub_bytes, wt += w_columns(FMT, F32)) {
                            const uint64_t da = tc::desc_k(at), db = tc::desc_k(at + a_bytes);
#pragma unroll
                            for (int j = 0; j < kGemmK / 16; ++j) {
                                const bool add = j > 0 || u > 0 || !first;
                                const uint64_t bj = db + 2 * j;                      // 32 bytes along K
                                const uint32_t cross = acc + uint32_t(n);
                                if constexpr (kQuant) {                              // (fp32: the tokens' two terms at once)
                                    tc::mma_ts(acc, wt + 8 * j, bj, idesc, add);
                                    if constexpr (F32) tc::mma_ts(cross, wt + 32 + 8 * j, bj, ione, true);
                                } else {
                                    tc::mma(acc, da + 2 * j, bj, idesc, add);
                                    if constexpr (F32) tc::mma(cross, da + 2 * j, bj + 2 * (uint32_t(n) * kGemmK * 2 >> 4), ione, true);
                                }
                            }
                        }
                        tc::commit(empty(s));
                        if (lastk) tc::commit(acc_full(b));
                    }
                    __syncwarp();
                    if (lastk) ++it;
                    if (++s == a.stages) { s = 0; phase ^= 1; }
                }
            }
            // Products still under way end before the accumulators are given back.
            if (tc::elect()) tc::commit(drained);
            __syncwarp();
            mbar_wait(drained, 0, a.drain_limit);
        }
    }
    if (a.parts > 1) {
        if (warp >= kDrainWarps) tc::cluster_sync();         // the drain warps' first (each of them has had its tile)
        tc::cluster_sync();                                  // no CTA ends while another reads its sums
    }
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == kDrainWarps + kDecodeWarps + 1) tc::tmem_free(tmem, tmem_cols);
}

const void* qgemm_lookup(int fmt, bool f32, bool chains);

}  // namespace qg
