// gq_tc.cuh -- tensor cores, tensor memory and tensor maps as the products use them (gq_wgrad.cu,
// gq_fp8_linear.cu): thin names for the instructions, and what a pair of blocks says to each other.
// CG: blocks that work on a tile, one or a pair.
#pragma once
#include "gq_kernels.cuh"

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace gqa {

#define GQA_CG(CG, one, two, ...)                     \
    do {                                              \
        if constexpr ((CG) == 1) asm volatile(one __VA_ARGS__); \
        else asm volatile(two __VA_ARGS__);           \
    } while (0)
template <int CG> __device__ __forceinline__ void tmem_alloc(uint32_t smem, uint32_t cols) {
    GQA_CG(CG, "tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;",
           "tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;",
           ::"r"(smem), "r"(cols) : "memory");
    GQA_CG(CG, "tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;",
           "tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;", ::);
}
template <int CG> __device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
    GQA_CG(CG, "tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;",
           "tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;", ::"r"(addr), "r"(cols));
}
// Arrives on this barrier of every block of the tile when the MMAs issued so far are done.
template <int CG> __device__ __forceinline__ void mma_commit(uint32_t bar) {
    if constexpr (CG == 1)
        asm volatile(
            "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
            : "memory");
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
            "[%0], %1;" ::"r"(bar), "h"(static_cast<uint16_t>(3))
            : "memory");
}
// The pair: this block's rank, an arrival on the same barrier in the first block, and a barrier of both
// blocks.  What an arrival announces are operands in shared memory, made visible to the tensor cores
// by a proxy fence or written by the TMA, and registers read from TMEM, ordered by a tcgen05 fence; no
// thread of the other block reads them with ordinary loads, so the arrival is not a release at cluster
// scope (which waits for every store of the thread: 1,600 cycles, most of a step).  The PTX memory model
// promises the order of ordinary accesses between two blocks for the cluster's scope alone; what is relied
// on here instead is that a proxy fence makes the stores before it visible to the async proxy, through which
// the tensor cores read the shared memory of both blocks, before the arrival behind it is counted.
template <int CG> __device__ __forceinline__ uint32_t pair_rank() {
    uint32_t r = 0;
    if constexpr (CG == 2) asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
template <int CG> __device__ __forceinline__ void arrive_first(uint32_t bar) {
    if constexpr (CG == 1) {
        gq::mbar_arrive(bar);
    } else {
        uint32_t there;
        asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(there) : "r"(bar));
        asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(there) : "memory");
    }
}
template <int CG> __device__ __forceinline__ void pair_sync() {
    if constexpr (CG == 2) {
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    } else {
        __syncthreads();
    }
}
// One thread of a warp that is here as a whole.  Instructions of the tensor cores that it issues take their
// operands from registers of the warp; behind a branch on the lane's number each one waited for its operands to
// be moved there (4 tcgen05.mma and a commit 406 cycles, longer than their products take).
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xFFFFFFFF;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ void fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// 32 columns of this warp's 32 lanes.  One statement, so that nothing that uses the registers moves between
// the load and the wait for it.
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr)
        : "memory");
}
// The same for 16 columns.
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(addr)
        : "memory");
}

// The same for 64 columns.
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&r)[64]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
        "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
        "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
        "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63"
        "}, [%64];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
          "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
          "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
          "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]),
          "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]),
          "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]),
          "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]),
          "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(addr)
        : "memory");
}

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int y,
                                         uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// The same for a pair of blocks, counted on a barrier of either one (its address in the cluster).
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
// The address in the cluster of a place in another block's shared memory.
__device__ __forceinline__ uint32_t place_in(uint32_t smem, uint32_t rank) {
    uint32_t there;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(smem), "r"(rank));
    return there;
}

// gq::mbar_wait for a thread that others' shared memory traffic depends on: it asks to be put to sleep until the
// phase ends instead of asking again (whose loads take their turn with operands and copies: a product of
// 16,384 x 4,096 x 4,096 in 8 bits 200 us, so 180).
__device__ __forceinline__ bool mbar_rest(uint32_t bar, uint32_t parity) {
    uint64_t t0 = 0;
    for (;;) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(bar), "r"(parity), "r"(1000000u)  // ns, at most
            : "memory");
        if (done) return true;
        const uint64_t now = gq::global_ns();
        if (t0 == 0) t0 = now;
        else if (now - t0 > gq::kWaitLimitNs) return false;
    }
}

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                             const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                             CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                             CUtensorMapFloatOOBfill);
inline EncodeFn encode_fn() {
    static EncodeFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeFn>(p);
    }();
    return fn;
}

}  // namespace gqa
