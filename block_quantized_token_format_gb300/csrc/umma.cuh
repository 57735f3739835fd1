// Helpers of the kernels whose products run on the fifth-generation tensor cores (tcgen05):
// shared-memory matrix descriptors, instruction descriptors, tensor-memory loads and stores,
// tensor copies, and waits that end.
//
// Operands lie in shared memory in the 128-byte swizzle: rows of 64 16-bit values (128 bytes),
// eight rows an atom of 1024 bytes, the 16-byte chunk c of row r at chunk c ^ (r % 8).  That is
// what a tensor copy with CU_TENSOR_MAP_SWIZZLE_128B and a box 64 values wide writes.
#pragma once

#include "qgemv_kernels.cuh"

namespace qg {
namespace tc {

constexpr uint32_t kFullMask = 0xFFFFFFFFu;

// ---------------------------------------------------------------------------- descriptors

// A matrix whose rows (of M or N) lie along the swizzled rows' order, K along a row: 64 values
// of K to an atom row; a step of 16 along K is 32 bytes further.
// `stride`: bytes from one group of eight rows to the next.
__device__ __forceinline__ uint64_t desc_k(uint32_t addr, uint32_t stride = 1024) {
    return uint64_t((addr & 0x3FFFF) >> 4) | uint64_t(1) << 16 | uint64_t(stride >> 4) << 32 | uint64_t(1) << 46 | uint64_t(2) << 61;
}
// A matrix with N along a row (64 values to an atom row) and K from row to row: eight rows of K
// are an atom, `k_stride` bytes from one to the next; the next 64 values of N are `n_stride`
// bytes further.  A step of 16 along K is 2 * k_stride bytes further.
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr, uint32_t n_stride, uint32_t k_stride = 1024) {
    return uint64_t((addr & 0x3FFFF) >> 4) | uint64_t(n_stride >> 4) << 16 | uint64_t(k_stride >> 4) << 32 | uint64_t(1) << 46 |
           uint64_t(2) << 61;
}
// 16-bit operands, fp32 accumulators, M = 128 rows.
__device__ __forceinline__ constexpr uint32_t instr(bool bf16, int n, bool b_along_n) {
    return 1u << 4 | (bf16 ? 1u << 7 | 1u << 10 : 0u) | (b_along_n ? 1u << 16 : 0u) | uint32_t(n >> 3) << 17 | uint32_t(128 >> 4) << 24;
}

// D[128][n] += A[128][16] B[n][16]^T (or =, without `add`), one thread of the CTA issues.
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
                 " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}"
                 :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(add)) : "memory");
}
// The same with A in tensor memory: lane = row, a 32-bit column two neighbouring values of K.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
                 " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}"
                 :: "r"(d), "r"(a), "l"(b), "r"(idesc), "r"(uint32_t(add)) : "memory");
}
// Arrives on `bar` when all products this thread has issued are done.
__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" :: "r"(bar) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// Plain shared-memory writes before this are seen by the tensor cores and the copy engine after it.
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// ---------------------------------------------------------------------------- tensor memory

// Whole warp; columns a power of two from 32 on; the address is written to shared memory.
__device__ __forceinline__ void tmem_alloc(uint32_t dst, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(dst), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(addr), "r"(cols) : "memory");
}

// Lane l of the warp gets `n` columns of row 32 (warp % 4) + l; the address carries the row in its high half.
#define QG_R4(v, i) "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3])
#define QG_R16(v, i) QG_R4(v, i), QG_R4(v, i + 4), QG_R4(v, i + 8), QG_R4(v, i + 12)
__device__ __forceinline__ void tmem_load16(uint32_t addr, uint32_t* v) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : QG_R16(v, 0) : "r"(addr) : "memory");
}
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t* v) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : QG_R16(v, 0), QG_R16(v, 16) : "r"(addr) : "memory");
}
#undef QG_R16
#undef QG_R4
#define QG_R4(v, i) "r"(v[i]), "r"(v[i + 1]), "r"(v[i + 2]), "r"(v[i + 3])
#define QG_R16(v, i) QG_R4(v, i), QG_R4(v, i + 4), QG_R4(v, i + 8), QG_R4(v, i + 12)
__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};"
                 :: QG_R16(v, 0), "r"(addr) : "memory");
}
#undef QG_R16
#undef QG_R4
// Waits for the warp's loads; their values pass through, so that no use of them comes before.
#define QG_R4(v, i) "+r"(v[i]), "+r"(v[i + 1]), "+r"(v[i + 2]), "+r"(v[i + 3])
#define QG_R16(v, i) QG_R4(v, i), QG_R4(v, i + 4), QG_R4(v, i + 8), QG_R4(v, i + 12)
__device__ __forceinline__ void tmem_load_wait16(uint32_t* v) { asm volatile("tcgen05.wait::ld.sync.aligned;" : QG_R16(v, 0) :: "memory"); }
__device__ __forceinline__ void tmem_load_wait32(uint32_t* v) {
    // (30 operands are the most that one statement takes both ways: a wait that is over costs nothing.)
    tmem_load_wait16(v);
    tmem_load_wait16(v + 16);
}
#undef QG_R16
#undef QG_R4
template <int N> __device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&v)[N]) {
    static_assert(N % 32 == 0, "columns");
#pragma unroll
    for (int i = 0; i < N; i += 32) tmem_load32(addr + uint32_t(i), v + i);
#pragma unroll
    for (int i = 0; i < N; i += 32) tmem_load_wait32(v + i);
}
// (of a larger array's first N)
template <int N> __device__ __forceinline__ void tmem_store(uint32_t addr, const uint32_t* v) {
    static_assert(N % 16 == 0, "columns");
#pragma unroll
    for (int i = 0; i < N; i += 16) tmem_store16(addr + uint32_t(i), v + i);
}
__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// True in one lane of a whole warp.  The loops that issue products and copies run in the whole warp
// and only their instructions in this lane: what they take is then known to be the same in all
// lanes, and stays in the registers that they read it from.
__device__ __forceinline__ bool elect() {
    uint32_t one;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(one));
    return one != 0;
}

// ---------------------------------------------------------------------------- copies

__device__ __forceinline__ void load_3d(uint32_t dst, const void* map, int x, int y, int z, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
                 :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}
__device__ __forceinline__ void load_2d(uint32_t dst, const void* map, int x, int y, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
                 :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar) : "memory");
}

// Shared-memory loads that stay between the barrier operations around them.
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a) : "memory");
    return r;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t r;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(a) : "memory");
    return r;
}

__device__ __forceinline__ void grid_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ---------------------------------------------------------------------------- the grid's next block

// Asks for a CTA of the grid that has not begun, to do its work instead of it: the answer's 16 bytes
// arrive on `bar`.  Not asked again after an answer that there is none.
__device__ __forceinline__ void ask_block(uint32_t answer, uint32_t bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];"
                 :: "r"(answer), "r"(bar) : "memory");
}
// The block's x, or -1.
__device__ __forceinline__ int block_of(uint32_t answer) {
    uint32_t x, got;
    asm volatile("{\n .reg .pred p;\n .reg .b128 h;\n .reg .b64 lo, hi;\n"
                 " ld.shared.v2.b64 {lo, hi}, [%2];\n mov.b128 h, {lo, hi};\n"
                 " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n"
                 " selp.u32 %1, 1, 0, p;\n mov.u32 %0, 0;\n"
                 " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, h;\n}"
                 : "=r"(x), "=r"(got) : "r"(answer) : "memory");
    return got ? int(x) : -1;
}

// ---------------------------------------------------------------------------- clusters

// Whole warps; every thread of the cluster's CTAs comes here.
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.aligned;\n barrier.cluster.wait.aligned;" ::: "memory");
}
// The same shared-memory address in CTA `rank` of the cluster, and a load from there.
__device__ __forceinline__ uint32_t of_cluster(uint32_t addr, int rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float load_cluster(uint32_t addr) {
    float x;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(addr) : "memory");
    return x;
}

// ---------------------------------------------------------------------------- waits that end

// A wait on a barrier's phase that gives up after `limit` polls, or once another thread of the
// CTA has given up; the CTA's roles then leave their loops.
struct Waits {
    volatile uint32_t* dead;       // shared memory
    unsigned int* status;
    uint32_t limit;
    // The whole warp, with one result.
    __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const {
        if (__all_sync(kFullMask, mbar_try_wait(bar, parity))) return true;
        for (uint32_t i = 0; i < limit; ++i) {
            if (__all_sync(kFullMask, mbar_try_wait(bar, parity))) return true;
            if ((i & 31) == 31 && __any_sync(kFullMask, *dead != 0)) return false;
        }
        *dead = 1;
        atomicOr(status, 1u);      // QG_DEVICE_WAIT_TIMEOUT
        return false;
    }
};

}  // namespace tc
}  // namespace qg
