// qgemm and qgemm_experts: argument checks, the kernel that stages the tokens, the choice of the
// tile's tokens, the launch.  Formulas and argument rules are in include/qgemv.h; the product's
// kernel in qgemm.cuh.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdio>

#include "qgemm.cuh"
#include "qgemv_host.h"

namespace qg {

const void* qgemm_lookup_fmt0(bool, bool);
const void* qgemm_lookup_fmt1(bool, bool);
const void* qgemm_lookup_fmt2(bool, bool);
const void* qgemm_lookup_fmt3(bool, bool);
const void* qgemm_lookup_fmt4(bool, bool);
const void* qgemm_lookup(int fmt, bool f32, bool chains) {
    switch (fmt) {
        case 0: return qgemm_lookup_fmt0(f32, chains);
        case 1: return qgemm_lookup_fmt1(f32, chains);
        case 2: return qgemm_lookup_fmt2(f32, chains);
        case 3: return qgemm_lookup_fmt3(f32, chains);
        default: return qgemm_lookup_fmt4(f32, chains);
    }
}

namespace {

constexpr int kStageThreads = 256;
constexpr int kMostExperts = 65536;

struct StageArgs {
    const void* x;
    void* staged;                  // [terms][n_slots][n_in]; null: nothing to stage
    float* xscale;
    const int32_t* rows;           // experts: the token of each slot, or null
    const int32_t* offsets;
    int32_t* tile_start;
    long long x_stride, n_x;
    int n_slots, n_in, n_experts, bn;
    unsigned int* status;
};

// Tiles of `bn` slots before each expert; offsets that do not grow from 0 on or pass n_slots leave
// no tile at all.  One CTA.
__device__ void plan_tiles(const StageArgs& a) {
    __shared__ long long warp_sum[kStageThreads / 32];
    __shared__ int bad;
    const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5;
    if (tid == 0) bad = 0;
    __syncthreads();
    long long run = 0;
    for (int e0 = 0; e0 < a.n_experts; e0 += kStageThreads) {
        const int e = e0 + tid;
        long long tiles = 0;
        if (e < a.n_experts) {
            const int lo = a.offsets[e], hi = a.offsets[e + 1];
            if (lo < 0 || hi < lo || hi > a.n_slots) bad = 1;
            else tiles = (hi - lo + a.bn - 1) / a.bn;
        }
        long long sum = tiles;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const long long up = __shfl_up_sync(tc::kFullMask, sum, d);
            if (lane >= d) sum += up;
        }
        if (lane == 31) warp_sum[warp] = sum;
        __syncthreads();
        long long before = run;
        for (int w = 0; w < kStageThreads / 32; ++w) {
            if (w < warp) before += warp_sum[w];
            run += warp_sum[w];
        }
        if (e < a.n_experts) a.tile_start[e] = int32_t(min(before + sum - tiles, 0x7FFFFFFFll));
        __syncthreads();
    }
    // (Tiles are numbered with 31 bits: the host has checked n_slots and n_experts for that.)
    if (bad)
        for (int e = tid; e <= a.n_experts; e += kStageThreads) a.tile_start[e] = 0;
    else if (tid == 0)
        a.tile_start[a.n_experts] = int32_t(run);
    if (bad && tid == 0) atomicOr(a.status, 4u);         // QG_DEVICE_BAD_PLAN
}

// Eight neighbouring values of a row.
__device__ __forceinline__ void read8(const float* p, float (&x)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void read8(const __nv_bfloat16* p, float (&x)[8]) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
}
__device__ __forceinline__ bool finite_of(float x) { return (__float_as_uint(x) & 0x7F800000u) != 0x7F800000u; }

// The tokens' operand, one row per slot.  With quantized weights: fp16 terms of the row times the
// power of two that takes its largest magnitude to [2^14, 2^15) (a second term holds what the
// first one's rounding left: 22 bits together); with bf16 weights: the bf16 values, or three
// bf16 terms of fp32 ones, each the next 8 bits (cut off, so that they add up exactly).  A value
// that is not finite is its own first term.  `PER` threads take a row: a warp, or a CTA where rows are
// too few to fill the GPU with warps (17 tokens of 6144: the row's latency, not its bytes).  Bound by
// the launch for few rows, else by memory (a bf16 row is read twice, out of L2 the second time).
template <typename T, int FMT, int PER> __global__ void __launch_bounds__(kStageThreads) stage_kernel(const StageArgs a) {
    constexpr bool kQuant = FMT != QG_BF16, kF32 = sizeof(T) == 4;
    __shared__ uint32_t most[kStageThreads / 32];
    // What ran before is done, W's writer among it, when the product's kernel begins to copy W.
    tc::grid_wait();
    tc::grid_launch_dependents();
    if (a.n_experts && blockIdx.x == gridDim.x - 1) {
        plan_tiles(a);
        return;
    }
    const int tid = int(threadIdx.x), sub = tid % PER;
    const long long slot = (long long)blockIdx.x * (kStageThreads / PER) + tid / PER;
    const int unused = a.n_experts ? a.offsets[0] : 0, used = a.n_experts ? min(a.offsets[a.n_experts], a.n_slots) : a.n_slots;
    if (slot < unused || slot >= used) return;           // of no expert (PER = 256: the whole block)
    long long at = a.rows ? (long long)a.rows[slot] : slot;
    const bool bad = at < 0 || at >= a.n_x;
    if (bad) {
        if (sub == 0) atomicOr(a.status, 4u);            // QG_DEVICE_BAD_PLAN; the row counts as zeros
        at = 0;
    }
    const T* const src = static_cast<const T*>(a.x) + at * a.x_stride;
    float scale = 1.0f;
    if constexpr (kQuant) {
        uint32_t top = 0;                                // the largest finite magnitude's bits
        for (int i = sub * 8; i < a.n_in; i += PER * 8) {
            float x[8];
            read8(src + i, x);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (finite_of(x[j])) top = max(top, __float_as_uint(x[j]) & 0x7FFFFFFFu);
        }
#pragma unroll
        for (int d = 16; d >= 1; d /= 2) top = max(top, __shfl_xor_sync(tc::kFullMask, top, d));
        if constexpr (PER > 32) {
            if ((tid & 31) == 0) most[tid >> 5] = top;
            __syncthreads();
            for (int w = 0; w < kStageThreads / 32; ++w) top = max(top, most[w]);
        }
        if (bad) top = 0;
        int e = 0;
        if (top) e = min(14 - ilogbf(__uint_as_float(top)), 126);        // at least -113
        scale = __int_as_float((e + 127) << 23);
        if (sub == 0) a.xscale[slot] = __int_as_float((127 - e) << 23);
    }
    const size_t term = size_t(a.n_slots) * size_t(a.n_in);
    uint16_t* const out = static_cast<uint16_t*>(a.staged) + size_t(slot) * size_t(a.n_in);
    for (int i = sub * 8; i < a.n_in; i += PER * 8) {
        float x[8];
        read8(src + i, x);
        uint16_t t0[8], t1[8], t2[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float v = bad ? 0.0f : x[pairs_by_four(FMT) ? j / 2 + j % 2 * 4 : j];
            if constexpr (kQuant) {
                const float s = v * scale;
                const __half h = __float2half_rn(s);
                t0[j] = __half_as_ushort(h);
                t1[j] = finite_of(s) ? __half_as_ushort(__float2half_rn(s - __half2float(h))) : uint16_t(0);
            } else {
                const bool fine = finite_of(v);
                const uint32_t b0 = __float_as_uint(v) & 0xFFFF0000u;
                const float r1 = fine ? v - __uint_as_float(b0) : 0.0f;
                const uint32_t b1 = __float_as_uint(r1) & 0xFFFF0000u;
                const float r2 = r1 - __uint_as_float(b1);
                // (A NaN whose bits would all be cut off stays one.)
                t0[j] = fine || (b0 & 0x007F0000u) || !(__float_as_uint(v) & 0x007FFFFFu) ? uint16_t(b0 >> 16) : uint16_t(0x7FC0);
                t1[j] = uint16_t(b1 >> 16);
                t2[j] = uint16_t(__float_as_uint(r2) >> 16);
            }
        }
        auto put = [&](uint16_t* to, const uint16_t (&t)[8]) {
            *reinterpret_cast<uint4*>(to) = make_uint4(t[0] | uint32_t(t[1]) << 16, t[2] | uint32_t(t[3]) << 16, t[4] | uint32_t(t[5]) << 16,
                                                       t[6] | uint32_t(t[7]) << 16);
        };
        put(out + i, t0);
        if constexpr (kF32) put(out + term + i, t1);
        if constexpr (kF32 && !kQuant) put(out + 2 * term + i, t2);
    }
}

template <typename T, int PER> const void* stage_fn(int fmt) {
    return fmt == QG_BF16 ? (const void*)&stage_kernel<T, QG_BF16, PER>
           : fmt == QG_Q8_0 ? (const void*)&stage_kernel<T, QG_Q8_0, PER> : (const void*)&stage_kernel<T, QG_Q4_0, PER>;
}
const void* stage_fn(int fmt, bool f32, bool wide) {
    return f32 ? (wide ? stage_fn<float, 256>(fmt) : stage_fn<float, 32>(fmt))
               : (wide ? stage_fn<__nv_bfloat16, 256>(fmt) : stage_fn<__nv_bfloat16, 32>(fmt));
}

// What a call needs of its workspace: tiles per expert, powers of two, staged tokens.
struct GemmSpace { size_t tile_start, xscale, staged, total; };
GemmSpace gemm_space(int fmt, bool f32, bool gathers, int64_t n_in, int64_t n_slots, int64_t n_experts) {
    GemmSpace s{};
    auto take = [&](size_t bytes) { const size_t at = s.total; s.total = (at + bytes + 255) / 256 * 256; return at; };
    const bool quant = fmt != QG_BF16;
    s.tile_start = take(n_experts ? size_t(n_experts + 1) * 4 : 0);
    s.xscale = take(quant ? size_t(n_slots) * 4 : 0);
    s.staged = take(quant || f32 || gathers ? size_t(terms_x(fmt, f32)) * size_t(n_slots) * size_t(n_in) * 2 : 0);
    return s;
}

struct GemmCall {
    int fmt;
    const void* W;
    int64_t n_out, n_in, n_experts;
    qg_act act;
    const void* x;
    int64_t x_stride, n_x, n_slots;
    const int32_t *offsets, *rows;
    const float* bias;
    const void* residual;
    int64_t residual_stride;
    qg_activation f;
    void* y;
    int64_t y_stride;
    void* workspace;
    size_t workspace_bytes;
    void* stream;
};

qg_status check(const GemmCall& c) {
    const int64_t most = (int64_t(1) << 31) - 1;
    if (!shape_valid(c.fmt, c.n_out, c.n_in) || (c.act != QG_ACT_F32 && c.act != QG_ACT_BF16)) return QG_EINVAL;
    if (c.n_slots < 0 || c.n_slots > most - 1024 || c.n_x < 0 || c.n_x > most) return QG_EINVAL;
    if (c.f < QG_F_NONE || c.f > QG_F_SWIGLU || (c.f == QG_F_SWIGLU && c.n_out % 2 != 0)) return QG_EINVAL;
    const int64_t width = c.f == QG_F_SWIGLU ? c.n_out / 2 : c.n_out;
    if (c.x_stride < c.n_in || c.y_stride < width || (c.residual && c.residual_stride < width)) return QG_EINVAL;
    if (c.x_stride > most || c.y_stride > most || c.residual_stride > most) return QG_EINVAL;
    if (c.n_slots == 0) return QG_OK;
    if (!c.W || !c.x || !c.y || c.x == c.y) return QG_EINVAL;
    const int64_t size = c.act == QG_ACT_F32 ? 4 : 2;
    if (!aligned(c.W, 16) || !aligned(c.x, 16) || c.x_stride * size % 16 != 0 || !aligned(c.y, uintptr_t(size)) ||
        !aligned(c.residual, uintptr_t(size)) || !aligned(c.bias, 4) || !aligned(c.offsets, 4) || !aligned(c.rows, 4))
        return QG_EALIGN;
    // Rows written over residual rows need the same places.
    if (c.residual == c.y && c.residual_stride != c.y_stride && c.n_slots > 1) return QG_EINVAL;
    return QG_OK;
}

// Clusters of `parts` CTAs, an SM each, that run at once (cached: every geometry of these kernels
// fills an SM).
int clusters_at_once(const void* fn, int dev, int threads, size_t smem, int parts) {
    static std::atomic<int> cache[64][9];                // one more than the number; 0: not known yet
    if (dev < 0 || dev >= 64) return 0;
    const int known = cache[dev][parts].load(std::memory_order_relaxed);
    if (known) return known - 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(parts));
    cfg.blockDim = dim3(unsigned(threads));
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(parts);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess) { cudaGetLastError(); n = 0; }
    cache[dev][parts].store(n + 1, std::memory_order_relaxed);
    return n;
}

// A kernel's shared memory for tiles of bn tokens.
struct Geometry { int subs, stages, raws; size_t smem; };
Geometry geometry(int fmt, bool f32, int bn, int sets, int optin) {
    // Stages of one step of K, or of two where they are small (a stage's waits and bookkeeping take
    // about 200 clocks of the warp that issues the products): four or three of them; the rest of
    // shared memory holds raw codes on their way, which is what few tokens to a tile need.  Their slots
    // are a multiple of the decoding groups: a slot then always belongs to the same group, which waits
    // for its fills one by one.
    const bool quant = fmt != QG_BF16;
    const int groups = decode_groups(fmt, f32);
    const size_t raw = size_t(kGemmRows) * size_t(raw_codes(fmt)), scales = size_t(kGemmRows) * kScaleSlots * size_t(raw_scales(fmt));
    const size_t room = size_t(optin) - kStaticSmemReserve - 1024 - scales;
    Geometry g{};
    g.subs = bn <= (quant ? (f32 ? 64 : sets == 3 ? 96 : 160) : f32 ? 0 : 128) ? 2 : 1;
    const size_t stage = size_t(g.subs) * ((quant ? 0 : size_t(kOperandA)) + size_t(terms_x(fmt, f32)) * size_t(bn) * kGemmK * 2);
    auto slots = [&](int stages) { return int(std::min<size_t>(kMostRaws, (room - size_t(stages) * stage) / std::max<size_t>(raw, 1))) / std::max(groups, 1) * groups; };
    g.stages = int(std::min<size_t>(quant ? (g.subs == 2 ? 3 : 4) : 8, (room - size_t(groups) * raw) / stage));
    if (quant) g.stages = std::min(g.stages, (512 - sets * bn * (f32 ? 2 : 1)) / (g.subs * w_columns(fmt, f32)));
    g.raws = quant ? slots(g.stages) : 0;
    g.smem = 1024 + scales + size_t(g.raws) * raw + size_t(g.stages) * stage;
    return g;
}

// Nanoseconds of a step of K (64) of a tile of bn tokens, all SMs at work: the decoding of the codes, or from
// some size on the tokens' way from L2 and the products.  Fitted to measurements on GB300, in calls short enough that
// the clocks stay up; calls of 150 steps to a tile measured, in ns, at 32 / 96 / 192 tokens (bf16) and 32 / 64 / 96
// (fp32): Q8_0 209 / 213 / 472 and 350 / 364 / 548, Q4_0 246 / 253 / 451 and 372 / 393 / 534, affine 252 / 255 / 452 and
// 531 / 555 / 566, Q5_0 298 / 311 / 489 and 454 / 473 / 581, bf16 166 / 188 / 301 and 388 / 455 / 525.
double step_ns(int fmt, bool f32, int bn) {
    if (fmt == QG_BF16) return f32 ? 300.0 + 2.75 * bn : std::max(160.0, 1.55 * bn);
    if (!f32) return std::max(fmt == QG_Q8_0 ? 215.0 : fmt == QG_Q5_0 ? 300.0 : 255.0, 1.8 * bn);
    return std::max(fmt == QG_Q8_0 ? 0.0 : fmt == QG_Q4_0 ? 375.0 : fmt == QG_Q5_0 ? 450.0 : 535.0, 290.0 + 1.8 * bn + (bn > 80 ? 70.0 : 0.0));      // (two stages)
}

// The tile's tokens, and the CTAs that share its K.  Tiles run on all SMs in rounds, each with about
// 1.5 us of its own (fp32 2.5); a cluster's join takes 2.5 us.
struct Shape { int bn, parts; };
template <typename Clusters>
Shape tile_shape(int fmt, bool f32, int64_t n_in, int64_t m_tiles, int64_t n_slots, int64_t n_experts, int sms, Clusters clusters) {
    Shape best{32, 1};
    double least = 0;
    const double ksteps = double((n_in + kGemmK - 1) / kGemmK);
    // Experts' rows: spread like independent choices, and by half their mean for the experts' popularity, which the
    // host does not know.  A larger tile costs little more where an expert has few rows, so the guess matters little:
    // with popularities exp(sigma N(0, 1)), sigma 0 / 0.5 / 1 / 1.5, 512 experts of Q8_0 1280 x 2560 took, in us (in
    // parentheses the best of all widths), 20,480 rows 372 / 372 / 388 / 392 (372 / 370 / 388 / 392), 5120 rows
    // 319 / 318 / 310 / 285 (319 / 318 / 306 / 279), 60,000 rows 582 / 639 / 658 / 663 (535 / 617 / 634 / 663); of
    // 2560 x 640 in fp32 7000 rows 269 / 269 / 270 / 262 (268 / 268 / 266 / 253).
    const double mean = n_experts ? double(n_slots) / double(n_experts) : 0.0, spread = std::sqrt(mean + 0.25 * mean * mean);
    for (int bn = 32; bn <= gemm_most_tokens(fmt, f32, gemm_sets(f32, int(n_in))); bn += 16) {
        // (An expert's tile has no more tokens than the expert.)
        const double step = step_ns(fmt, f32, n_experts && mean + spread < bn ? std::min(bn, int(mean + spread) / 16 * 16 + 16) : bn);
        for (int parts = 1; parts <= 8; ++parts) {
            double rounds;
            if (n_experts == 0) {
                const int64_t tiles = m_tiles * ((n_slots + bn - 1) / bn);
                if (parts > 1 && (tiles * parts > sms || ksteps < 8 * parts)) break;
                if (parts > 1 && clusters(parts) < tiles) continue;
                rounds = double((tiles + sms - 1) / sms);
            } else {
                if (parts > 1) break;
                double per_expert = 1.0 - std::exp(-mean);               // the mean of a count's tiles
                if (mean > 16.0 * bn)
                    per_expert = mean / bn + 0.5;                        // (the sum below comes to that)
                else
                    for (int j = 1; j * bn < mean + 4.0 * spread; ++j)
                        per_expert += 0.5 * std::erfc((j * bn - mean) / (spread * 1.41421356));
                rounds = std::max(1.0, double(m_tiles) * double(n_experts) * per_expert / sms);
            }
            const double steps = parts > 1 ? kScaleSteps * std::ceil(std::ceil(ksteps / kScaleSteps) / parts) : ksteps;      // of a CTA
            const double cost = rounds * (steps * step + (f32 ? 2500.0 : 1500.0)) + (parts > 1 ? 2500.0 : 0.0);
            if (least == 0 || cost < least) {
                best = {bn, parts};
                least = cost;
            }
        }
    }
    return best;
}

qg_status encode_tokens(CUtensorMap* map, const void* p, int64_t inner, int64_t rows, int64_t terms, int64_t pitch, int box_rows) {
    const EncodeTiledFn enc = encode_tiled();
    if (!enc) return QG_ECUDA;
    const cuuint64_t dims[3] = {cuuint64_t(inner), cuuint64_t(rows), cuuint64_t(terms)};
    const cuuint64_t strides[2] = {cuuint64_t(pitch), terms > 1 ? cuuint64_t(pitch) * cuuint64_t(rows) : cuuint64_t(pitch)};
    const cuuint32_t box[3] = {kGemmK, cuuint32_t(box_rows), 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(p), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? QG_OK : QG_ECUDA;
}
// Boxes of 128 rows of W, `width` elements wide.
qg_status encode_2d(CUtensorMap* map, CUtensorMapDataType type, const void* W, int64_t inner, int64_t rows, int64_t pitch, int width,
                    CUtensorMapSwizzle swizzle) {
    const EncodeTiledFn enc = encode_tiled();
    if (!enc) return QG_ECUDA;
    const cuuint64_t dims[2] = {cuuint64_t(inner), cuuint64_t(rows)};
    const cuuint64_t strides[1] = {cuuint64_t(pitch)};
    const cuuint32_t box[2] = {cuuint32_t(width), kGemmRows};
    const cuuint32_t estr[2] = {1, 1};
    return enc(map, type, 2, const_cast<void*>(W), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? QG_OK : QG_ECUDA;
}

// A call's kernel, tile and shared memory on the current device.
struct Choice {
    int dev, sms, optin;
    unsigned int* status;
    const void* fn;
    int threads;
    int64_t m_tiles, n_tiles;
    Shape shape;
    Geometry geo;
};
qg_status choose(int fmt, bool f32, int64_t n_out, int64_t n_in, int64_t n_slots, int64_t n_experts, Choice* ch) {
    qg_status st = device_info(&ch->dev, &ch->sms, &ch->optin, &ch->status);
    if (st != QG_OK) return st;
    const int sets = gemm_sets(f32, int(n_in)), groups = decode_groups(fmt, f32);
    ch->fn = qgemm_lookup(fmt, f32, sets == 3);
    ch->threads = gemm_threads(fmt, f32);
    ch->m_tiles = (n_out + kGemmRows - 1) / kGemmRows;
    ch->shape = tile_shape(fmt, f32, n_in, ch->m_tiles, n_slots, n_experts, ch->sms, [&](int parts) {
        const size_t smem = geometry(fmt, f32, 32, sets, ch->optin).smem;
        return blocks_per_sm(ch->fn, ch->dev, ch->optin, ch->threads, smem) < 1 ? 0 : clusters_at_once(ch->fn, ch->dev, ch->threads, smem, parts);
    });
    ch->n_tiles = (n_slots + ch->shape.bn - 1) / ch->shape.bn;
    if ((ch->n_tiles + n_experts) * ch->m_tiles > (int64_t(1) << 31) - 4096) return QG_EUNSUPPORTED;
    const Geometry& g = ch->geo = geometry(fmt, f32, ch->shape.bn, sets, ch->optin);
    if (g.stages < 2 || g.stages * g.subs < groups || g.raws < groups) return QG_EUNSUPPORTED;
    return blocks_per_sm(ch->fn, ch->dev, ch->optin, ch->threads, g.smem) < 1 ? QG_EUNSUPPORTED : QG_OK;
}

qg_status launch_gemm(const GemmCall& c) {
    const bool f32 = c.act == QG_ACT_F32, quant = c.fmt != QG_BF16;
    const GemmSpace sp = gemm_space(c.fmt, f32, c.rows != nullptr, c.n_in, c.n_slots, c.n_experts);
    if (sp.total > 0 && (!c.workspace || c.workspace_bytes < sp.total)) return QG_EWORKSPACE;
    if (!aligned(c.workspace, 16)) return QG_EALIGN;
    Choice ch{};
    qg_status st = choose(c.fmt, f32, c.n_out, c.n_in, c.n_slots, c.n_experts, &ch);
    if (st != QG_OK) return st;
    const int bn = ch.shape.bn, parts = ch.shape.parts;
    uint8_t* const ws = static_cast<uint8_t*>(c.workspace);
    const bool stages_x = quant || f32 || c.rows;

    GemmArgs a{};
    a.n_out = int(c.n_out);
    a.n_in = int(c.n_in);
    a.n_slots = int(c.n_slots);
    a.n_experts = int(c.n_experts);
    a.offsets = c.offsets;
    a.tile_start = reinterpret_cast<const int32_t*>(ws + sp.tile_start);
    a.xscale = quant ? reinterpret_cast<const float*>(ws + sp.xscale) : nullptr;
    a.bias = c.bias;
    a.residual = c.residual;
    a.y = c.y;
    a.residual_stride = c.residual_stride;
    a.y_stride = c.y_stride;
    a.f = int(c.f);
    a.bn = bn;
    a.box = c.n_experts ? 16 : bn;
    a.m_tiles = int(ch.m_tiles);
    a.n_tiles = int(ch.n_tiles);
    a.status = ch.status;
    a.wait_limit = wait_limit();
    a.drain_limit = std::max<uint32_t>(a.wait_limit, 1u << 16);
    a.extra_tx = test_extra_tx();
    a.subs = ch.geo.subs;
    a.stages = ch.geo.stages;
    a.raws = ch.geo.raws;
    a.parts = parts;
    const int64_t rows = std::max<int64_t>(1, c.n_experts) * c.n_out, pitch = row_stride(c.fmt, c.n_in);
    st = stages_x ? encode_tokens(&a.xmap, ws + sp.staged, c.n_in, c.n_slots, terms_x(c.fmt, f32), c.n_in * 2, a.box)
                  : encode_tokens(&a.xmap, c.x, c.n_in, c.n_x, 1, c.x_stride * 2, a.box);
    if (st == QG_OK && !quant)
        st = encode_2d(&a.wmap, CU_TENSOR_MAP_DATA_TYPE_UINT16, c.W, c.n_in, rows, pitch, kGemmK, CU_TENSOR_MAP_SWIZZLE_128B);
    if (st == QG_OK && quant)
        st = encode_2d(&a.wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, c.W, pitch, rows, pitch, raw_codes(c.fmt),
                       c.fmt == QG_Q8_0 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B);
    if (st == QG_OK && quant)
        st = encode_2d(&a.smap, CU_TENSOR_MAP_DATA_TYPE_UINT8, c.W, pitch, rows, pitch, raw_scales(c.fmt), CU_TENSOR_MAP_SWIZZLE_NONE);
    if (st != QG_OK) return st;

    const bool before = stages_x || c.n_experts > 0;
    if (before) {
        StageArgs s{};
        s.x = c.x;
        s.staged = ws + sp.staged;
        s.xscale = reinterpret_cast<float*>(ws + sp.xscale);
        s.rows = c.rows;
        s.offsets = c.offsets;
        s.tile_start = reinterpret_cast<int32_t*>(ws + sp.tile_start);
        s.x_stride = c.x_stride;
        s.n_x = c.n_x;
        s.n_slots = int(c.n_slots);
        s.n_in = int(c.n_in);
        s.n_experts = int(c.n_experts);
        s.bn = bn;
        s.status = ch.status;
        // A row takes a CTA where there are too few rows to fill the GPU with a warp each.
        const bool wide = c.n_slots < 8 * ch.sms;
        const int64_t per = wide ? 1 : kStageThreads / 32;
        const int64_t grid = (stages_x ? (c.n_slots + per - 1) / per : 0) + (c.n_experts > 0 ? 1 : 0);
        void* params[] = {&s};
        st = launch_early(stage_fn(c.fmt, f32, wide), int(grid), kStageThreads, 0, 1, params, c.stream);
        if (st != QG_OK) return st;
    }
    const int64_t tiles = c.n_experts ? ch.sms : ch.n_tiles * ch.m_tiles;
    void* params[] = {&a};
    return launch_after(ch.fn, parts > 1 ? int(tiles) * parts : int(std::min<int64_t>(ch.sms, tiles)), ch.threads, ch.geo.smem, parts, before, params,
                        c.stream);
}

}  // namespace
}  // namespace qg

using namespace qg;

extern "C" {

size_t qgemm_workspace_bytes(qg_fmt fmt, qg_act act, int64_t n_out, int64_t n_in, int64_t n_slots, int64_t n_experts) {
    if (!shape_valid(fmt, n_out, n_in) || (act != QG_ACT_F32 && act != QG_ACT_BF16) || n_slots < 0 ||
        n_slots > (int64_t(1) << 31) - 1025 || n_experts < 0 || n_experts > kMostExperts)
        return 0;
    return std::max<size_t>(256, gemm_space(fmt, act == QG_ACT_F32, true, n_in, n_slots, n_experts).total);
}

qg_status qgemm(qg_fmt fmt, const void* W, int64_t n_out, int64_t n_in, qg_act act, const void* x, int64_t x_stride, int64_t ntok,
                const float* bias, qg_activation f, const void* residual, int64_t residual_stride, void* y, int64_t y_stride,
                void* workspace, size_t workspace_bytes, void* stream) {
    GemmCall c{fmt, W, n_out, n_in, 0, act, x, x_stride, ntok, ntok, nullptr, nullptr, bias, residual, residual ? residual_stride : 0,
               f, y, y_stride, workspace, workspace_bytes, stream};
    const qg_status st = check(c);
    if (st != QG_OK || ntok == 0) return st;
    return launch_gemm(c);
}

qg_status qgemm_experts(qg_fmt fmt, const void* W, int64_t n_experts, int64_t n_out, int64_t n_in, qg_act act, const void* x,
                        int64_t x_stride, int64_t n_x, const int32_t* offsets, const int32_t* rows, int64_t n_slots, qg_activation f,
                        void* y, int64_t y_stride, void* workspace, size_t workspace_bytes, void* stream) {
    GemmCall c{fmt, W, n_out, n_in, n_experts, act, x, x_stride, n_x, n_slots, offsets, rows, nullptr, nullptr, 0,
               f, y, y_stride, workspace, workspace_bytes, stream};
    if (n_experts < 1 || n_experts > kMostExperts || n_experts * n_out > (int64_t(1) << 31) - 1024) return QG_EINVAL;
    if (n_slots > 0 && (!offsets || n_x < 1 || (!rows && n_x < n_slots))) return QG_EINVAL;
    const qg_status st = check(c);
    if (st != QG_OK || n_slots == 0) return st;
    return launch_gemm(c);
}

qg_status qg_describe_gemm_tile(qg_fmt fmt, qg_act act, int64_t n_out, int64_t n_in, int64_t n_slots, int64_t n_experts, char* buf, size_t len) {
    if (!buf || len == 0 || !shape_valid(fmt, n_out, n_in) || (act != QG_ACT_F32 && act != QG_ACT_BF16)) return QG_EINVAL;
    if (n_slots < 1 || n_slots > (int64_t(1) << 31) - 1025 || n_experts < 0 || n_experts > kMostExperts) return QG_EINVAL;
    Choice ch{};
    const qg_status st = choose(fmt, act == QG_ACT_F32, n_out, n_in, n_slots, n_experts, &ch);
    if (st != QG_OK) return st;
    std::snprintf(buf, len, "tokens=%d,parts=%d,steps=%d,stages=%d,raws=%d", ch.shape.bn, ch.shape.parts, ch.geo.subs, ch.geo.stages, ch.geo.raws);
    return QG_OK;
}

}  // extern "C"
