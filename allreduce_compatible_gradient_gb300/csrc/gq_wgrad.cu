// gq_wgrad.cu -- weight and bias gradient of a linear layer whose input was kept as an 8-bit
// checkpoint (C ABI in include/gq.h).
//
//   dW[o, i] = sum_t dy[t, o] X[t, i],   X = V  or  V scale + shift (a layer norm's affine part)
//            = scale[i] (dy^T V)[o, i] + shift[i] db[o],   db[o] = sum_t dy[t, o]
//
// with V the values of the checkpoint.  They are exact in bf16, so the tensor cores see the
// checkpoint itself: dy^T V is a product of bf16 matrices with fp32 accumulation, and the affine
// part is applied to the finished sums.  fp32 gradients are cut into three bf16 parts (8 + 8 + 8
// bits, exact), laid one after another along t.
//
// Persistent blocks compute tiles of outs x columns; a large tile (512 x 256) belongs to a pair of
// blocks, each with 256 of its outs (two accumulators of 128 x 256, all of TMEM) and 128 of its columns
// as operands, on which one tcgen05.mma of both tensor cores works.  In each block:
//   warp 0      TMA loads of dy (64 tokens x 64 outs per box, 128-byte swizzle, outs contiguous)
//   warp 1      one thread (of the pair's first block) issues tcgen05.mma, accumulators in TMEM
//   the others  read codes and exponents from global memory into registers one turn ahead, widen
//               them to bf16 in shared memory in the layout of the other operand, and store
//               finished tiles from TMEM; two teams take turns at the steps, so that the latency
//               of a load or of a barrier is that of two steps' time
// Both operands are contiguous along their outer dimension ("MN-major"), so neither is transposed.
// Why pairs: shared memory moves 128 bytes per cycle, and one block with a 256 x 256 tile asks for 160
// (operands 96, dy's arrival 32, the widened codes 32).  A pair shares the widened codes, and asks for 112.
//
// Each block or pair first works on whole tiles of its own, beside the others' in the matrix (so that they
// read the same rows of dy and the same codes at the same time: 0.76 GB from memory at 4,096 x 4,096 x
// 16,384 tokens, 1.03 where each began elsewhere); the steps (64 tokens) of the tiles that are left are
// one list, cut into equal contiguous pieces.  A tile that two or more blocks work on leaves fp32 partial
// tiles in the workspace, which join_kernel adds in a fixed order.
//
// The tensor cores' fp32 accumulation rounds each sum of 16 products towards zero or nearly so, an error
// that grows with the length of the chain (5.8e-6 of the result's norm over 16,384 tokens in one): a chain
// ends after kChain steps, and the rest is added to it in fp32 outside.  Errors against 64 bits, normal
// numbers: 1.7e-6 at 6,144 and at 16,384 tokens (the library's product of the same bf16 matrices 2.0e-6 and
// 7.5e-6, its product of fp32 ones 0.3e-6 and 0.5e-6), 4.8e-7 at 2,048 (4.8e-7, 1.3e-7), 7.8e-8 at 384
// (7.8e-8, 4.9e-8).
//
// What bounds it: the tensor cores, and the ends of the chains, when 256 KB of sums per block leave or
// cross the L2.  4,096 x 4,096 x 16,384 tokens, bf16: 335 us without db (the library's product of two
// bf16 matrices 285; chains of 256 steps would take 310), 383 with it, inputs changing.  Tiles side by side, a chain's
// steps widened ahead, its accumulators finished one after the other, and first chains of different
// lengths took it there from 352 and 379.
#include "gq_act.cuh"

#include <cuda.h>

using namespace gqa;

namespace {

constexpr int kTok = 64;              // tokens per step
constexpr int kChain = 96;            // steps of one accumulation (error and time above)
constexpr int kEarly = 2;             // steps widened for the next chain before one's sums are stored
constexpr int kTeams = 2;             // teams of widening warps that take turns at the steps
constexpr int kChunk = kTok * 128;    // bytes of 64 outs (or columns) x 64 tokens in bf16

// CG blocks work on a tile, each on MH x 128 of its outs; BN columns, BN / CG widened by each block.
// WARPS widening warps: 8 keep up with both (16 leave 96 registers each, and gained nothing: 600 cycles
// of a small tile's step are its operands' way through shared memory).
template <int CG_, int MH_, int BN_, int WARPS> struct Tile {
    static constexpr int CG = CG_, MH = MH_, BN = BN_;
    static constexpr int kConv = WARPS;               // warps 2 .. WARPS + 1
    static constexpr int kTeam = 32 * WARPS / kTeams; // threads of a team
    static constexpr int kThreads = 64 + 32 * WARPS;
    static constexpr int kOuts = 128 * MH;            // of a block
    static constexpr int kRows = kOuts * CG;          // of the tile
    static constexpr int kOwn = BN / CG;              // columns widened by a block
    static constexpr int kABytes = kOuts * kTok * 2;
    static constexpr int kBBytes = kOwn * kTok * 2;
    static constexpr int kStages = 192 * 1024 / (kABytes + kBBytes);
    static_assert(kEarly <= kStages, "a chain's ends are in shared memory at once");
    static constexpr int kCols = MH * BN;             // TMEM columns: a power of two >= 32
    static constexpr int kSmem = kStages * (kABytes + kBBytes) + 1024;
};
using Large = Tile<2, 2, 256, 8>;
using Small = Tile<1, 1, 128, 8>;

struct WArgs {
    int64_t rows, outs, cols, pitch, epitch, ldw;
    const int8_t* codes;
    const uint8_t* exps;
    const float* scale;   // nullable, with shift
    const float* shift;
    const float* db;
    void* dw;
    int out_f32;
    float* partial;
    int64_t ktok;         // tokens of one part, rounded up to whole steps, in steps
    int ksteps;           // steps of a tile: parts * ktok
    int tiles_m, tiles_n;
    int shares, own;      // blocks or pairs at work; whole tiles that each has to itself
    int64_t units;        // steps of the remaining tiles, in
    int64_t base;         // pieces of base steps, one more in the first `rest` shares
    int rest;
    int packed;           // dy is what pack_kernel wrote
    int fast;             // whole 32-byte pieces of dw, and of scale and shift, are aligned
};

// ---- tcgen05 -------------------------------------------------------------------------------
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
template <int CG>
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         bool add) {
    GQA_CG(CG,
           "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
           "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}",
           "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
           "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}",
           ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(add ? 1u : 0u) : "memory");
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
__device__ __forceinline__ void fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// Shared-memory descriptor of an operand that is contiguous along its outer dimension, 128-byte
// swizzle: rows of 64 elements (one token each, 128 bytes), 8 tokens every 1,024 bytes (stride
// offset), the next 64 outer elements kChunk bytes on (leading offset).
__device__ __forceinline__ uint64_t operand(uint32_t smem) {
    return static_cast<uint64_t>((smem & 0x3FFFFu) >> 4) |
           (static_cast<uint64_t>(kChunk >> 4) << 16) | (static_cast<uint64_t>(1024 >> 4) << 32) |
           (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
// fp32 accumulator, bf16 operands, both contiguous along their outer dimension, M = 128 per block.
template <int CG, int BN> struct Instruction {
    static constexpr uint32_t value = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (1u << 16) |
                                      (static_cast<uint32_t>(BN >> 3) << 17) | ((128u * CG) >> 4 << 24);
};

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int y,
                                         uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// Two codes (the low bytes of the halves of p, 0x43 above them) times a power of two.  0x43cc is
// 128 + (c & 127) if c's sign bit is taken out, and 0x4300 or 0x4380, 128 or 256, from the sign
// bit alone: their difference is the code, and the product is exact.
__device__ __forceinline__ uint32_t widen2(uint32_t p, __nv_bfloat162 s) {
    uint32_t a = p & 0xFF7FFF7Fu, b = p & 0xFF80FF80u;
    const __nv_bfloat162 d = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&a),
                                     *reinterpret_cast<__nv_bfloat162*>(&b));
    const __nv_bfloat162 r = __hmul2(d, s);
    return *reinterpret_cast<const uint32_t*>(&r);
}

// A place in a share's steps: a tile, and a step of that tile.  First come `own` whole tiles (share,
// share + shares, ...), then a contiguous piece of the remaining tiles' steps (of the first `rest`
// shares one step longer).  The place moves on by counting; a 64-bit division per step and thread had
// cost a third of the issue slots, and even one per thread is felt by a call of a few steps.
__device__ __forceinline__ int64_t share_begin(const WArgs& a, int share) {
    return a.base * share + min(share, a.rest);
}
struct At {
    int left;  // steps of the share from here on
    int tile, k;
    int own;   // whole tiles from this one on
    __device__ __forceinline__ At(const WArgs& a, int share)
        : left(a.own * a.ksteps + static_cast<int>(a.base) + (share < a.rest ? 1 : 0)), own(a.own) {
        tile = share;
        k = 0;
        if (own == 0) split(a, share);
    }
    // to the piece of the tiles that several shares work on
    __device__ __forceinline__ void split(const WArgs& a, int share) {
        const int64_t u = share_begin(a, share);
        if (a.units <= INT32_MAX) {
            const uint32_t v = static_cast<uint32_t>(u);
            tile = static_cast<int>(v / static_cast<uint32_t>(a.ksteps));
            k = static_cast<int>(v % static_cast<uint32_t>(a.ksteps));
        } else {
            tile = static_cast<int>(u / a.ksteps);
            k = static_cast<int>(u % a.ksteps);
        }
        tile += a.own * a.shares;
    }
    // `steps` more, which stay in the tile or end it
    __device__ __forceinline__ void skip(const WArgs& a, int steps) {
        left -= steps;
        k += steps;
        if (k < a.ksteps) return;
        k = 0;
        if (own == 0) ++tile;
        else if (--own > 0) tile += a.shares;
        else split(a, tile - (a.own - 1) * a.shares);
    }
    __device__ __forceinline__ void next(const WArgs& a) { skip(a, 1); }
    // steps of the tile at hand that are in the share
    __device__ __forceinline__ int segment(const WArgs& a) const { return min(left, a.ksteps - k); }
};

// Steps of the next chain of a segment with `left` steps.  The first chains of neighbouring shares are of
// different lengths, where the number of chains leaves the room, so that not all of them store their
// sums at the same time.
__device__ __forceinline__ int chain_steps(int left, bool first, int share) {
    if (left <= kChain) return left;
    if (!first) return kChain;
    const int room = (left + kChain - 1) / kChain * kChain - left;
    return kChain - room * (share & 7) / 8;
}

// 8 columns of a row of dw from fp32 sums, element by element: the last columns, and rows that are
// not aligned.  Kept out of the kernels' straight path, whose instructions a short call fetches cold.
__device__ __noinline__ void finish_slow(const WArgs& a, int64_t o, int64_t i, const float (&v)[8]) {
    for (int k = 0; k < 8 && i + k < a.cols; ++k) {
        float x = v[k];
        if (a.scale) x = x * a.scale[i + k];
        if (a.shift) x = fmaf(a.db[o], a.shift[i + k], x);
        if (a.out_f32) static_cast<float*>(a.dw)[o * a.ldw + i + k] = x;
        else static_cast<bf16*>(a.dw)[o * a.ldw + i + k] = __float2bfloat16_rn(x);
    }
}
// N columns (a multiple of 8) of row o from column i on: the sums times scale, plus db shift, rounded.
template <int N>
__device__ __forceinline__ void finish(const WArgs& a, int64_t o, int64_t i, float (&v)[N]) {
    if (o >= a.outs || i >= a.cols) return;
    if (a.fast && i + N <= a.cols) {
        if (a.scale) {
#pragma unroll
            for (int k = 0; k < N; k += 4) {
                const float4 f = __ldg(reinterpret_cast<const float4*>(a.scale + i + k));
                v[k] *= f.x; v[k + 1] *= f.y; v[k + 2] *= f.z; v[k + 3] *= f.w;
            }
        }
        if (a.shift) {
            const float d = a.db[o];  // not __ldg: written while the main kernel already runs
#pragma unroll
            for (int k = 0; k < N; k += 4) {
                const float4 f = __ldg(reinterpret_cast<const float4*>(a.shift + i + k));
                v[k] = fmaf(d, f.x, v[k]); v[k + 1] = fmaf(d, f.y, v[k + 1]);
                v[k + 2] = fmaf(d, f.z, v[k + 2]); v[k + 3] = fmaf(d, f.w, v[k + 3]);
            }
        }
        if (a.out_f32) {
            float* p = static_cast<float*>(a.dw) + o * a.ldw + i;
#pragma unroll
            for (int k = 0; k < N; k += 8) {
                uint32_t u[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) u[j] = __float_as_uint(v[k + j]);
                st32<32>(p + k, u);
            }
        } else {
            bf16* p = static_cast<bf16*>(a.dw) + o * a.ldw + i;
#pragma unroll
            for (int k = 0; k < N; k += 8)
                *reinterpret_cast<uint4*>(p + k) =
                    make_uint4(pack2(v[k], v[k + 1], bf16()), pack2(v[k + 2], v[k + 3], bf16()),
                               pack2(v[k + 4], v[k + 5], bf16()), pack2(v[k + 6], v[k + 7], bf16()));
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < N; k += 8) {
        float w[8] = {v[k], v[k + 1], v[k + 2], v[k + 3], v[k + 4], v[k + 5], v[k + 6], v[k + 7]};
        if constexpr (N > 8) {
            if (i + k < a.cols) finish(a, o, i + k, w);
        } else {
            finish_slow(a, o, i + k, w);
        }
    }
}

// Where a partial tile keeps 8 columns of a row: blocks of 32 rows x 32 columns, in which the 32 rows'
// 32 bytes of the same 8 columns lie side by side, so that a warp with a row per lane writes and reads
// 1,024 bytes in a row.
template <int BN> __device__ __forceinline__ int64_t partial_at(int row, int col) {
    return static_cast<int64_t>((row >> 5) * (BN / 32) + (col >> 5)) * 1024 + (col >> 3 & 3) * 256 +
           (row & 31) * 8;
}

template <typename C>
__global__ void __launch_bounds__(C::kThreads, 1)
    wgrad_kernel(const __grid_constant__ CUtensorMap dy_map, const WArgs a) {
    constexpr int CG = C::CG, MH = C::MH, BN = C::BN, S = C::kStages;
    extern __shared__ uint8_t raw[];
    // full: everything of a step is there (in the pair's first block); full_a: the second block's dy
    __shared__ alignas(8) uint64_t full[S], full_a[S], empty[S], acc_full[MH], acc_empty[MH], drain;
    __shared__ uint32_t tmem_slot;
    const uint32_t base = (gq::smem_u32(raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = pair_rank<CG>();
    auto a_stage = [&](int s) { return base + s * C::kABytes; };
    auto b_stage = [&](int s) { return base + S * C::kABytes + s * C::kBBytes; };

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            // the widening warps of a team in each block, and each block's dy
            gq::mbar_init(gq::smem_u32(&full[s]), CG * (C::kConv / kTeams + 1));
            gq::mbar_init(gq::smem_u32(&full_a[s]), 1u);
            gq::mbar_init(gq::smem_u32(&empty[s]), 1u);
        }
        for (int h = 0; h < MH; ++h) {
            gq::mbar_init(gq::smem_u32(&acc_full[h]), 1u);
            gq::mbar_init(gq::smem_u32(&acc_empty[h]), CG * C::kConv);
        }
        gq::mbar_init(gq::smem_u32(&drain), 1u);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc<CG>(gq::smem_u32(&tmem_slot), C::kCols);
    fence_before();
    __syncthreads();
    pair_sync<CG>();
    fence_after();
    const uint32_t tmem = tmem_slot;
    const int share = blockIdx.x / CG;

    if (warp == 0) {
        if (lane == 0) {
            uint32_t n = 0;
            bool ok = true;
            if (a.packed) gq::pdl_wait();  // dy is the launch before's work
            for (At at(a, share); at.left > 0 && ok; at.next(a), ++n) {
                const int s = n % S;
                if (n >= S) ok = gq::mbar_wait(gq::smem_u32(&empty[s]), ((n / S) - 1) & 1);
                if (!ok) break;
                const uint32_t bar = gq::smem_u32(rank == 0 ? &full[s] : &full_a[s]);
                gq::mbar_arrive_expect_tx(bar, C::kABytes);
                const int o0 = (at.tile / a.tiles_n) * C::kRows + static_cast<int>(rank) * C::kOuts;
#pragma unroll
                for (int c = 0; c < 2 * MH; ++c)
                    tma_load(a_stage(s) + c * kChunk, &dy_map, o0 + 64 * c, at.k * kTok, bar);
            }
            // nothing of this block's is in flight when it ends, whatever the others did
            for (uint32_t j = n > S ? n - S : 0; j < n; ++j)
                gq::mbar_wait(gq::smem_u32(rank == 0 ? &full[j % S] : &full_a[j % S]), (j / S) & 1);
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            uint32_t n = 0, seg = 0;
            bool ok = true, first = true;
            auto wait_full = [&](uint32_t m) {
                if (ok) ok = gq::mbar_wait(gq::smem_u32(&full[m % S]), (m / S) & 1);
                fence_after();
            };
            auto issue = [&](uint32_t m, int h, bool add) {  // step m on accumulator h
                const int s = m % S;
#pragma unroll
                for (int kk = 0; kk < kTok / 16; ++kk)
                    mma_bf16<CG>(tmem + h * BN, operand(a_stage(s) + h * 2 * kChunk + kk * 2048),
                                 operand(b_stage(s) + kk * 2048), Instruction<CG, BN>::value,
                                 add || kk > 0);
            };
            auto wait_empty = [&](int h) {
                if (seg > 0 && ok) ok = gq::mbar_wait(gq::smem_u32(&acc_empty[h]), (seg - 1) & 1);
                fence_after();
            };
            for (At at(a, share); at.left > 0 && ok; ++seg) {
                const int left = at.segment(a), steps = chain_steps(left, first, share);
                at.skip(a, steps);
                first = steps == left;
                // With two accumulators a chain's first and last kEarly steps run on the first one, then
                // on the second: each works on while the other's sums are stored.
                const int head = MH > 1 ? min(steps, kEarly) : 0, tail = MH > 1 ? min(steps - head, kEarly) : 0;
                const uint32_t from = n, back = n + steps - tail, end = n + steps;
                wait_empty(0);
                for (; n < from + head && ok; ++n) {
                    wait_full(n);
                    if (ok) issue(n, 0, n > from);
                }
                if constexpr (MH > 1) {
                    if (tail == 0 && ok) mma_commit<CG>(gq::smem_u32(&acc_full[0]));
                    wait_empty(1);
                    if (ok) {
                        for (n = from; n < from + head; ++n) {
                            issue(n, 1, n > from);
                            mma_commit<CG>(gq::smem_u32(&empty[n % S]));
                        }
                    }
                }
                for (; n < back && ok; ++n) {
                    wait_full(n);
                    if (!ok) break;
#pragma unroll
                    for (int h = 0; h < MH; ++h) issue(n, h, n > from);
                    mma_commit<CG>(gq::smem_u32(&empty[n % S]));
                }
                for (; n < end && ok; ++n) {
                    wait_full(n);
                    if (ok) issue(n, 0, true);
                }
                if (ok && (MH == 1 || tail > 0)) mma_commit<CG>(gq::smem_u32(&acc_full[0]));
                if constexpr (MH > 1) {
                    if (ok) {
                        for (uint32_t m = back; m < end; ++m) {
                            issue(m, 1, true);
                            mma_commit<CG>(gq::smem_u32(&empty[m % S]));
                        }
                        mma_commit<CG>(gq::smem_u32(&acc_full[1]));
                    }
                }
            }
            if (!ok) {  // let what was issued finish before TMEM is given back
                mma_commit<CG>(gq::smem_u32(&drain));
                gq::mbar_wait(gq::smem_u32(&drain), 0);
            }
        } else if (lane == 0) {  // the second block: tells the first that its dy has arrived
            uint32_t n = 0;
            bool ok = true;
            for (At at(a, share); at.left > 0 && ok; at.next(a), ++n) {
                ok = gq::mbar_wait(gq::smem_u32(&full_a[n % S]), (n / S) & 1);
                if (ok) arrive_first<CG>(gq::smem_u32(&full[n % S]));
            }
        }
    } else {
        const int team = (threadIdx.x - 64) / C::kTeam, ct = (threadIdx.x - 64) % C::kTeam;
        constexpr int kPer = C::kOwn * kTok / 16 / C::kTeam;  // 16-code pieces per thread and step
        constexpr int kRowPieces = C::kOwn / 16;
        // this thread's pieces of a step: every kTokStep-th token, the same 16 columns.  Eight lanes
        // that store together hold 64 columns of two tokens, whose swizzles differ in the last bit: 8
        // different bank groups (128 columns of one token would be 4 groups twice).
        static_assert(kRowPieces == 8, "the bits of ct below");
        const int col = ((ct & 3) | (ct >> 1 & 4)) * 16, tok = (ct >> 2 & 1) | (ct >> 4 << 1);
        constexpr int kTokStep = C::kTeam / kRowPieces;
        uint4 w[kPer];
        uint32_t e[kPer];
        At ahead(a, share);
        int part = ahead.k % static_cast<int>(a.ktok);  // step within the part of dy
        const int8_t* pc = nullptr;   // codes and exponents of the thread's first piece of the
        const uint8_t* pe = nullptr;  // step `ahead`
        bool in_cols = false;
        const int rows_left = static_cast<int>(min(a.rows - tok, int64_t(1) << 30));
        auto place = [&]() {
            const int64_t i = static_cast<int64_t>(ahead.tile % a.tiles_n) * BN + rank * C::kOwn + col;
            const int64_t t = static_cast<int64_t>(part) * kTok + tok;
            in_cols = i < a.pitch;
            pc = a.codes + t * a.pitch + i;
            pe = a.exps + t * a.epitch + (i >> 5);
        };
        // on by `steps` (at most kTeams)
        auto advance = [&](int steps) {
            if (ahead.k + steps < a.ksteps && part + steps < a.ktok) {
                ahead.left -= steps;
                ahead.k += steps;
                part += steps;
                pc += steps * (kTok * a.pitch);
                pe += steps * (kTok * a.epitch);
            } else {  // a part of dy, or a tile, begins
                for (int j = 0; j < steps; ++j) ahead.next(a);
                part = ahead.k % static_cast<int>(a.ktok);
                place();
            }
        };
        auto fetch = [&]() {  // the step `ahead`, and on to the team's next
            const int left = rows_left - part * kTok;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const bool in = in_cols && j * kTokStep < left;
                w[j] = in ? __ldg(reinterpret_cast<const uint4*>(pc + j * kTokStep * a.pitch))
                          : make_uint4(0, 0, 0, 0);
                e[j] = in ? __ldg(pe + j * kTokStep * a.epitch) : 0u;
            }
            advance(kTeams);
        };
        place();
        if (team > 0) advance(team);
        if (ahead.left > 0) fetch();
        uint32_t n = team, end = 0, seg = 0;
        bool ok = true;
        At at(a, share);
        const uint32_t total = at.left;
        auto widen = [&](uint32_t to) {  // the team's steps below `to`
            for (; n < to; n += kTeams) {
                const int s = n % S;
                uint4 cw[kPer];
                uint32_t ce[kPer];
#pragma unroll
                for (int j = 0; j < kPer; ++j) { cw[j] = w[j]; ce[j] = e[j]; }
                if (ahead.left > 0) fetch();
                if (n >= S && ok) ok = gq::mbar_wait(gq::smem_u32(&empty[s]), ((n / S) - 1) & 1);
                ok = __all_sync(kFull, ok);
                if (!ok) continue;
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
                    const int t = tok + j * kTokStep, c = col / 16;  // token, 16-column piece
                    const uint32_t sc = ce[j] << 7 | ce[j] << 23;
                    const __nv_bfloat162 sv = *reinterpret_cast<const __nv_bfloat162*>(&sc);
                    const uint32_t in[4] = {cw[j].x, cw[j].y, cw[j].z, cw[j].w};
                    uint32_t o[8];
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        o[2 * m] = widen2(__byte_perm(in[m], 0x43434343u, 0x4140), sv);
                        o[2 * m + 1] = widen2(__byte_perm(in[m], 0x43434343u, 0x4342), sv);
                    }
                    // 16-byte unit v of row t of a 64-column chunk sits at unit v ^ (t mod 8)
                    const uint32_t row = b_stage(s) + (c >> 2) * kChunk + t * 128;
                    const uint32_t v0 = (2 * (c & 3)) ^ (t & 7);
                    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(row + v0 * 16),
                                 "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3])
                                 : "memory");
                    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(row + (v0 ^ 1) * 16),
                                 "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
                                 : "memory");
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) arrive_first<CG>(gq::smem_u32(&full[s]));
            }
        };
        while (at.left > 0) {
            const int tile = at.tile;
            int left = at.segment(a);
            const bool whole = at.k == 0 && left == a.ksteps, from_first = at.k == 0;
            for (bool first = true; left > 0; first = false, ++seg) {  // the chains of the segment
                const int steps = chain_steps(left, first, share);
                left -= steps;
                at.skip(a, steps);
                end += steps;
                widen(end);
                // the chain's sums: 4 warps take the 128 lanes of TMEM, the groups of 4 share the
                // columns
                const int quad = warp & 3, group = (warp - 2) >> 2;
                constexpr int kShare = BN / (C::kConv / 4);
                const int c0 = group * kShare;
                const int64_t i0 = static_cast<int64_t>(tile % a.tiles_n) * BN;
                float* part_tile = a.partial + (static_cast<int64_t>(blockIdx.x / CG) * 2 +
                                                (from_first ? 1 : 0)) * (C::kRows * BN);
                const bool last = whole && left == 0;
                if (last && a.shift) gq::pdl_wait();  // db, if the sums of dy still run
#pragma unroll 1
                for (int h = 0; h < MH; ++h) {
                    const int r = static_cast<int>(rank) * C::kOuts + h * 128 + quad * 32 + lane;
                    const int64_t o = static_cast<int64_t>(tile / a.tiles_n) * C::kRows + r;
                    float4 x[8];  // what the chains before left of the next 32 columns, on its way
                    auto before = [&](int c) {
                        const float* p = part_tile + partial_at<BN>(r, c);
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            x[k] = reinterpret_cast<const float4*>(p + 256 * (k >> 1))[k & 1];
                    };
                    if (!first) before(c0);
                    if (h == MH - 1) widen(min(end + kEarly, total));
                    if (ok) ok = gq::mbar_wait(gq::smem_u32(&acc_full[h]), seg & 1);
                    ok = __all_sync(kFull, ok);
                    fence_after();
#pragma unroll 1
                    for (int c = c0; c < c0 + kShare; c += 32) {
                        uint32_t acc[32];
                        if (ok) {
                            tmem_load(tmem + (static_cast<uint32_t>(quad * 32) << 16) + h * BN + c, acc);
                        } else {  // a wait gave up: the tile is marked, not left as it was
#pragma unroll
                            for (int k = 0; k < 32; ++k) acc[k] = 0x7FFFFFFFu;
                        }
                        float v[32];
#pragma unroll
                        for (int k = 0; k < 32; ++k) v[k] = __uint_as_float(acc[k]);
                        if (!first) {
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                v[4 * k] += x[k].x; v[4 * k + 1] += x[k].y;
                                v[4 * k + 2] += x[k].z; v[4 * k + 3] += x[k].w;
                            }
                            if (c + 32 < c0 + kShare) before(c + 32);
                        }
                        if (last) {
                            finish(a, o, i0 + c, v);
                        } else {
                            float* p = part_tile + partial_at<BN>(r, c);
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                uint32_t u[8];
#pragma unroll
                                for (int j = 0; j < 8; ++j) u[j] = __float_as_uint(v[8 * k + j]);
                                st32<32>(p + 256 * k, u);
                            }
                        }
                    }
                    fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_first<CG>(gq::smem_u32(&acc_empty[h]));
                }
            }
        }
    }
    gq::pdl_wait();
    __syncwarp();
    fence_before();
    __syncthreads();
    pair_sync<CG>();  // neither block's memory is in use any more
    if (warp == 1) tmem_free<CG>(tmem, C::kCols);
    pair_sync<CG>();
}

// Adds the partial tiles of every tile that more than one share has a part of, in the shares' order.
// blockIdx.x = tile after the shares' own; thread = 8 columns of a row, 32 rows of the same columns per warp.
template <typename C> __global__ void __launch_bounds__(256) join_kernel(const WArgs a) {
    constexpr int BN = C::BN;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * a.ksteps, last = first + a.ksteps - 1;
    const int tile = a.own * a.shares + static_cast<int>(blockIdx.x);
    __shared__ int owners[2];
    if (threadIdx.x < 2) {  // the share that holds the tile's first step, and its last
        const int64_t u = threadIdx.x ? last : first;
        const int64_t longer = (a.base + 1) * a.rest;  // steps of the shares that have one more
        const int64_t b = u < longer ? u / (a.base + 1) : a.rest + (u - longer) / a.base;
        // a share that begins at the tile's first step keeps it in slot 1, any other in slot 0
        owners[threadIdx.x] = static_cast<int>(2 * b + (share_begin(a, static_cast<int>(b)) <= first ? 1 : 0));
    }
    __syncthreads();
    const int b0 = owners[0], b1 = owners[1];
    if (b0 / 2 == b1 / 2) return;  // stored by its one share
    // q counts rows of 32, then the four 8-column pieces of a 32-column block, then blocks
    const int q = blockIdx.y * 256 + threadIdx.x;
    const int r = (q >> 7) / (BN / 32) * 32 + (q & 31);
    const int c = (q >> 7) % (BN / 32) * 32 + (q >> 5 & 3) * 8;
    float v[8] = {};
    const float* p = a.partial + partial_at<BN>(r, c);
    for (int b = b0; b <= b1;) {  // slot b0, then slot 0 of the shares after it; four in flight
        uint32_t w[4][8];
        int n = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (b <= b1) {
                ld32<32>(p + static_cast<int64_t>(b) * (C::kRows * BN), w[j]);
                b = (b | 1) + 1;
                n = j + 1;
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j < n) {
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] += __uint_as_float(w[j][k]);
            }
        }
    }
    finish(a, static_cast<int64_t>(tile / a.tiles_n) * C::kRows + r,
           static_cast<int64_t>(tile % a.tiles_n) * BN + c, v);
}

// dy as the TMA needs it, in one pass that also takes its column sums (partial not null, as below): rows
// of `pitch` bf16 (a multiple of 8), `tokens` per part (whole steps), zeros behind the last row and
// column.  fp32 is cut into three parts of 8 bits each by truncation, whose sum is the number itself; an
// infinity or a NaN stays in the first.  Thread = 8 columns, read by the 16-byte granules that hold them
// (10,744 x 1,854 bf16 element by element: 33 us); two rows' loads are on their way at a time.
template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(512, 2)
    pack_kernel(const T* __restrict__ dy, int64_t ld, int64_t rows, int64_t outs,
                float* __restrict__ partial, bf16* __restrict__ out, int64_t pitch, int64_t tokens) {
    __shared__ float tile[16][257];
    gq::pdl_launch_dependents();  // what follows waits before it reads
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int64_t c = (static_cast<int64_t>(blockIdx.x) * 32 + x) * 8;
    const int left = c < outs ? static_cast<int>(min(outs - c, int64_t(8))) : 0;
    float s[8] = {};
    const int64_t stride = static_cast<int64_t>(gridDim.y) * 16;
    constexpr int P = sizeof(T) / 2 + (ALIGNED ? 0 : 1), B = 2;
    for (int64_t t = static_cast<int64_t>(blockIdx.y) * 16 + y; t < tokens; t += B * stride) {
        uint32_t r[B][4 * P], m[B];
#pragma unroll
        for (int k = 0; k < B; ++k) {
            const uint8_t* q = reinterpret_cast<const uint8_t*>(dy + (t + k * stride) * ld + c);
            m[k] = ALIGNED ? 0u : static_cast<uint32_t>(reinterpret_cast<uintptr_t>(q)) & 15u;
            const int bytes =
                t + k * stride < rows && left > 0 ? static_cast<int>(m[k]) + left * static_cast<int>(sizeof(T)) : 0;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const uint4 g = 16 * i < bytes ? __ldg(reinterpret_cast<const uint4*>(q - m[k]) + i)
                                               : make_uint4(0u, 0u, 0u, 0u);
                r[k][4 * i] = g.x; r[k][4 * i + 1] = g.y; r[k][4 * i + 2] = g.z; r[k][4 * i + 3] = g.w;
            }
        }
#pragma unroll
        for (int k = 0; k < B; ++k) {
            if (t + k * stride >= tokens) break;
            const Raw8<T> w = shifted<T, ALIGNED>(r[k], m[k], left);
            F2 h[4];
            pairs(w, h);
            float v[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) split(h[i], v[2 * i], v[2 * i + 1]);
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i] += v[i];
            if (c >= pitch) continue;
            bf16* to = out + (t + k * stride) * pitch + c;
            if constexpr (sizeof(T) == 2) {
                *reinterpret_cast<uint4*>(to) = make_uint4(w.w[0], w.w[1], w.w[2], w.w[3]);
            } else {
#pragma unroll
                for (int p = 0; p < 3; ++p) {
                    uint32_t top[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t bits = __float_as_uint(v[i]);
                        top[i] = (bits & 0x7FFFFFFFu) > 0x7F800000u ? 0x7FFF0000u : bits & 0xFFFF0000u;
                        const bool special = (bits & 0x7F800000u) == 0x7F800000u;
                        v[i] = special ? 0.0f : v[i] - __uint_as_float(top[i]);
                    }
                    *reinterpret_cast<uint4*>(to + p * tokens * pitch) =
                        make_uint4(top[0] >> 16 | top[1], top[2] >> 16 | top[3],
                                   top[4] >> 16 | top[5], top[6] >> 16 | top[7]);
                }
            }
        }
    }
    if (!partial) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) tile[y][x * 8 + i] = s[i];
    __syncthreads();
    const int64_t to = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (threadIdx.x < 256 && to < outs) {
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < 16; ++k) v += tile[k][threadIdx.x];
        partial[blockIdx.y * outs + to] = v;
    }
}

// Column sums of a bf16 dy with aligned rows, 32 rows at a time per block, thread = 8 columns:
// partial[blockIdx.y][outs], or db itself where one block row does.  Eight rows' loads are on their way
// at a time (16,384 x 4,096: 32 us with four, 27 with eight, of which the memory needs 20).
__global__ void __launch_bounds__(1024)
    bias_kernel(const bf16* __restrict__ dy, int64_t ld, int64_t rows, int64_t outs,
                float* __restrict__ partial) {
    __shared__ float tile[32][257];
    gq::pdl_launch_dependents();  // what follows waits where it reads the sums
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int64_t c = (static_cast<int64_t>(blockIdx.x) * 32 + x) * 8;
    float s[8] = {};
    const int64_t stride = static_cast<int64_t>(gridDim.y) * 32;
    const int64_t t0 = static_cast<int64_t>(blockIdx.y) * 32 + y;
    const bf16* p = dy + t0 * ld + c;
    int64_t left = rows - t0;
    // (the test for the last columns is outside, and rows that are not there are read as the first and
    // left out, so that the loads are issued together)
    if (c + 8 <= outs) {
        constexpr int B = 8;
        for (; left > 0; left -= B * stride, p += B * stride * ld) {
            uint4 r[B];
#pragma unroll
            for (int k = 0; k < B; ++k)
                r[k] = __ldg(reinterpret_cast<const uint4*>(p + (left > k * stride ? k * stride * ld : 0)));
#pragma unroll
            for (int k = 0; k < B; ++k) {
                F2 v[4];
                pairs(Raw8<bf16>{{r[k].x, r[k].y, r[k].z, r[k].w}}, v);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float lo, hi;
                    split(v[i], lo, hi);
                    s[2 * i] += left > k * stride ? lo : 0.0f;
                    s[2 * i + 1] += left > k * stride ? hi : 0.0f;
                }
            }
        }
    } else if (c < outs) {
        for (; left > 0; left -= stride, p += stride * ld) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c + i < outs) s[i] += up(p[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) tile[y][x * 8 + i] = s[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // a warp adds up a column
        const int col = y * 8 + i;
        float v = tile[x][col];
#pragma unroll
        for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
        const int64_t to = static_cast<int64_t>(blockIdx.x) * 256 + col;
        if (x == 0 && to < outs) partial[blockIdx.y * outs + to] = v;
    }
}
// (partial is not __restrict__: the launch before may still write it when this one starts, so its loads
// must be ordinary ones, which stay behind the wait)
__global__ void __launch_bounds__(256)
    bias_sum_kernel(const float* partial, int parts, int64_t outs, float* db) {
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + (threadIdx.x & 31);
    __shared__ float tile[8][32];
    gq::pdl_launch_dependents();
    gq::pdl_wait();
    float s = 0.0f;
    if (c < outs) {
#pragma unroll 4
        for (int p = threadIdx.x >> 5; p < parts; p += 8) s += partial[p * outs + c];
    }
    tile[threadIdx.x >> 5][threadIdx.x & 31] = s;
    __syncthreads();
    if (threadIdx.x < 32 && c < outs) {
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) v += tile[k][threadIdx.x];
        db[c] = v;
    }
}

// dw from finished fp32 sums in rows of `ld`: for a dw whose rows are not aligned, which the main kernel
// could only store element by element.
__global__ void __launch_bounds__(256)
    finish_kernel(const WArgs a, const float* __restrict__ sums, int64_t ld) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= a.cols) return;
    const float f = a.scale ? a.scale[i] : 1.0f, g = a.shift ? a.shift[i] : 0.0f;
#pragma unroll 4
    for (int64_t o = blockIdx.y; o < a.outs; o += gridDim.y) {
        float x = sums[o * ld + i];
        if (a.scale) x = x * f;
        if (a.shift) x = fmaf(a.db[o], g, x);
        if (a.out_f32) static_cast<float*>(a.dw)[o * a.ldw + i] = x;
        else static_cast<bf16*>(a.dw)[o * a.ldw + i] = __float2bfloat16_rn(x);
    }
}

// ---- host ----------------------------------------------------------------------------------

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                             const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                             CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                             CUtensorMapFloatOOBfill);
EncodeFn encode_fn() {
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

struct WPlan {
    bool big;            // pairs of blocks on 512 x 256 tiles, else 128 x 128
    bool pack;
    int parts;           // bf16 parts of dy
    int64_t ktok, ksteps, tiles_m, tiles_n, pitch;
    int shares, bias_shares;  // of the steps; of the rows in the bias sums
    size_t pack_off, bias_off, db_off, sums_off, bytes;
    int64_t sums_ld;     // of the fp32 sums for a dw with unaligned rows (0: none)
};

WPlan wgrad_plan(const void* dy, int dtype, int64_t rows, int64_t outs, int64_t ld, int64_t cols) {
    WPlan p;
    const int sms = gqh::sm_count();
    p.parts = dtype == GQ_F32 ? 3 : 1;
    p.pack = dtype == GQ_F32 || row_align(dy, dtype, rows, ld) == 0;
    p.ktok = (rows + kTok - 1) / kTok;
    p.ksteps = p.ktok * p.parts;
    // Small or large tiles, and how many shares: the smallest of the times that the steps, a launch's
    // ends and the partial tiles take, in microseconds as measured (a step of a 512 x 256 tile 0.55, of
    // a 128 x 128 tile 0.36; splitting tiles costs 12 or 6 more).  Both sides, in graphs, outs x columns x
    // tokens: 2,048 x 2,048 x 8,192 66 us in large tiles and 114 in small ones, 4,096 x 1,024 x 512 23.0 and
    // 25.5, 768 x 768 x 384 21 and 12, 3,840 x 41 x 15,872 66 and 53; 768 x 768 x 384 in 54 shares of the
    // small tiles instead of 36 whole ones 14.5 and 10.4.
    double best = 0.0;
    for (int large = 0; large < 2; ++large) {
        const int rows_of = large ? Large::kRows : Small::kRows, cols_of = large ? Large::BN : Small::BN;
        const int64_t tiles = ((outs + rows_of - 1) / rows_of) * ((cols + cols_of - 1) / cols_of);
        const int64_t most = large ? sms / 2 : sms;
        const double step = large ? 0.55 : 0.36, ends = large ? 4.0 : 3.0, split = large ? 12.0 : 6.0;
        auto consider = [&](int64_t shares, double steps, bool whole) {
            const double t = ends + steps * step + (whole ? 0.0 : split);
            if (best == 0.0 || t < best) {
                best = t;
                p.big = large != 0;
                p.shares = static_cast<int>(shares);
            }
        };
        if (tiles <= most) {
            consider(tiles, static_cast<double>(p.ksteps), true);
            // k shares for each tile; where k does not divide the steps some lie across two tiles and leave
            // two partial tiles, which is not counted (adding them takes about 0.15 us for each of a tile's)
            const int64_t q = most / tiles;
            for (int64_t k = 2; k <= q && p.ksteps >= 2 * k; k = k < 8 ? k + 1 : k * 5 / 4)
                consider(tiles * k, static_cast<double>((p.ksteps + k - 1) / k) + 0.15 * k / step, false);
        }
        const double even = static_cast<double>(tiles) * p.ksteps / most;
        if (tiles > most || even >= 4.0) consider(most, even + 2.0, tiles % most == 0);
    }
    const int rows_of = p.big ? Large::kRows : Small::kRows, cols_of = p.big ? Large::BN : Small::BN;
    p.tiles_m = (outs + rows_of - 1) / rows_of;
    p.tiles_n = (cols + cols_of - 1) / cols_of;
    p.pitch = (outs + 7) / 8 * 8;
    // the pass over dy: up to 512 rows in one go if there are only sums to take, else one wave of blocks
    // (one per SM, two where dy is packed)
    const int64_t groups = (outs + 255) / 256;
    const int64_t wave = p.pack ? 2 * sms : sms;
    int64_t sh = rows <= 512 && !p.pack ? 1 : groups < wave ? wave / groups : 1;
    const int64_t rows_each = p.pack ? 32 : 128;
    if (sh > (rows + rows_each - 1) / rows_each) sh = (rows + rows_each - 1) / rows_each;
    p.bias_shares = static_cast<int>(sh);
    auto up256 = [](size_t v) { return (v + 255) / 256 * 256; };
    p.pack_off = up256(static_cast<size_t>(p.shares) * 2 * rows_of * cols_of * sizeof(float));
    p.bias_off = p.pack_off +
                 (p.pack ? up256(static_cast<size_t>(p.ksteps) * kTok * p.pitch * 2) : 0);
    p.db_off = p.bias_off + up256(static_cast<size_t>(p.bias_shares) * outs * sizeof(float));
    p.sums_off = p.db_off + up256(static_cast<size_t>(outs) * sizeof(float));
    p.sums_ld = cols % 8 ? (cols + 7) / 8 * 8 : 0;
    p.bytes = p.sums_off + up256(static_cast<size_t>(outs) * p.sums_ld * sizeof(float)) + 256;  // to align
                                                                                               // the start
    return p;
}

bool wgrad_sizes(int64_t rows, int64_t outs, int64_t cols) {
    // 32-bit TMA coordinates: tokens of three parts, and outs
    return size_ok(rows, cols) && rows < (int64_t(1) << 29) && outs >= 1 &&
           outs < (int64_t(1) << 30) && cols < (int64_t(1) << 30) &&
           ((outs + 127) / 128) * ((cols + 127) / 128) < (int64_t(1) << 31) &&
           // steps of a share, in 32 bits
           static_cast<double>(rows) * outs * cols < 1e17;
}

// early: the launch before this one on the stream is of the sums of dy or of its packed form, which the
// kernel waits for only where it reads them; what came before those is done when it starts.
template <typename C>
gq_status launch_wgrad(const CUtensorMap& map, const WArgs& a, bool early, cudaStream_t st) {
    auto k = wgrad_kernel<C>;
    gqh::blocks_per_sm(k, C::kSmem, C::kThreads);  // raises the shared-memory limit once
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.shares * C::CG));
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = early ? 1 : 0;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C::CG;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = C::CG > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, k, map, a) != cudaSuccess) return GQ_ERR_CUDA;
    if (a.units > 0) {  // tiles that several shares work on
        const dim3 grid(static_cast<unsigned>(a.units / a.ksteps), C::kRows * C::BN / 8 / 256);
        join_kernel<C><<<grid, 256, 0, st>>>(a);
    }
    return gqh::launch_status();
}

}  // namespace

extern "C" {

size_t gq_linear_wgrad_workspace_bytes(const void *dy, int dtype, int64_t rows, int64_t outs,
                                       int64_t lddy, int64_t cols) {
    if (!in_type(dtype) || !wgrad_sizes(rows, outs, cols)) return 0;
    if (rows == 0) return 16;
    return wgrad_plan(dy, dtype, rows, outs, lddy, cols).bytes;
}

gq_status gq_linear_wgrad_plan(const void *dy, int dtype, int64_t rows, int64_t outs, int64_t lddy,
                               int64_t cols, int64_t *plan) {
    if (!in_type(dtype) || !wgrad_sizes(rows, outs, cols) || !plan) return GQ_ERR_INVALID;
    for (int i = 0; i < 8; ++i) plan[i] = 0;
    if (rows == 0) return GQ_OK;
    const WPlan p = wgrad_plan(dy, dtype, rows, outs, lddy, cols);
    const int64_t tiles = p.tiles_m * p.tiles_n, own = tiles / p.shares, left = tiles % p.shares;
    int64_t longest = own ? p.ksteps : 0, u = 0;
    for (int64_t b = 0; b < p.shares; ++b) {
        const int64_t end = u + left * p.ksteps / p.shares + (b < left * p.ksteps % p.shares ? 1 : 0);
        while (u < end) {  // as far as the tile goes
            const int64_t stop = (u / p.ksteps + 1) * p.ksteps, n = (stop < end ? stop : end) - u;
            if (n > longest) longest = n;
            u += n;
        }
    }
    const int64_t out[8] = {p.big ? Large::kRows : Small::kRows, p.big ? Large::BN : Small::BN,
                            p.ksteps, p.shares, own, left, longest, kChain};
    for (int i = 0; i < 8; ++i) plan[i] = out[i];
    return GQ_OK;
}

gq_status gq_linear_wgrad(const void *dy, int dtype, int64_t rows, int64_t outs, int64_t lddy,
                          const int8_t *codes, const uint8_t *exps, int64_t cols,
                          const float *scale, const float *shift, void *dw, int out_dtype,
                          int64_t lddw, float *dbias, void *ws, size_t ws_bytes, void *stream) {
    if (!in_type(dtype) || !in_type(out_dtype) || !wgrad_sizes(rows, outs, cols))
        return GQ_ERR_INVALID;
    if (!matrix_ok(dw, out_dtype, outs, cols, lddw) || !matrix_ok(dy, dtype, rows, outs, lddy))
        return GQ_ERR_INVALID;
    if (!mult(scale, 4) || !mult(shift, 4) || !mult(dbias, 4)) return GQ_ERR_INVALID;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (rows == 0) {  // sums over no tokens
        const size_t elt = elt_bytes(out_dtype);
        if (cudaMemset2DAsync(dw, lddw * elt, 0, cols * elt, outs, st) != cudaSuccess)
            return GQ_ERR_CUDA;
        if (dbias && cudaMemsetAsync(dbias, 0, outs * sizeof(float), st) != cudaSuccess)
            return GQ_ERR_CUDA;
        return GQ_OK;
    }
    if (!saved_ok(codes, exps)) return GQ_ERR_INVALID;
    const WPlan p = wgrad_plan(dy, dtype, rows, outs, lddy, cols);
    if (!ws || !mult(ws, 16) || ws_bytes < p.bytes) return GQ_ERR_WORKSPACE;
    EncodeFn encode = encode_fn();
    if (!encode) return GQ_ERR_CUDA;
    uint8_t* w = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(ws) + 255) / 256 * 256);
    float* db = dbias ? dbias : reinterpret_cast<float*>(w + p.db_off);

    const void* src = dy;
    int64_t src_ld = lddy, src_rows = rows, src_outs = outs;
    const bool sums = dbias || shift;
    if (p.pack || sums) {
        float* part = !sums ? nullptr : p.bias_shares > 1 ? reinterpret_cast<float*>(w + p.bias_off) : db;
        const int64_t tokens = p.ktok * kTok;
        bf16* out = p.pack ? reinterpret_cast<bf16*>(w + p.pack_off) : nullptr;
        const bool vec = row_align(dy, dtype, rows, lddy) != 0;
        const dim3 grid(static_cast<unsigned>((outs + 255) / 256), p.bias_shares);
#define GQA_PACK(T, ALIGNED)                                                                             \
    pack_kernel<T, ALIGNED><<<grid, 512, 0, st>>>(static_cast<const T*>(dy), lddy, rows, outs, part, out, \
                                                  p.pitch, tokens)
        if (dtype == GQ_F32) {
            if (vec) GQA_PACK(float, true); else GQA_PACK(float, false);
        } else if (p.pack) {
            GQA_PACK(bf16, false);
        } else {
            bias_kernel<<<grid, 1024, 0, st>>>(static_cast<const bf16*>(dy), lddy, rows, outs, part);
        }
#undef GQA_PACK
        if (sums && p.bias_shares > 1) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(static_cast<unsigned>((outs + 31) / 32));
            cfg.blockDim = dim3(256);
            cfg.stream = st;
            cudaLaunchAttribute attr;
            attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
            attr.val.programmaticStreamSerializationAllowed = 1;
            cfg.attrs = &attr;
            cfg.numAttrs = 1;
            if (cudaLaunchKernelEx(&cfg, bias_sum_kernel, static_cast<const float*>(part), p.bias_shares,
                                   outs, db) != cudaSuccess)
                return GQ_ERR_CUDA;
        }
        if (p.pack) {
            src = out;
            src_ld = p.pitch;
            src_rows = tokens * p.parts;
            src_outs = p.pitch;
        }
    }
    CUtensorMap map;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(src_outs), static_cast<cuuint64_t>(src_rows)};
    // one row's stride is not used, but has to be a multiple of 16 bytes like any other
    const cuuint64_t strides[1] = {src_rows > 1 ? static_cast<cuuint64_t>(src_ld) * 2
                                                : (static_cast<cuuint64_t>(src_outs) * 2 + 15) / 16 * 16};
    const cuuint32_t box[2] = {64, kTok}, one[2] = {1, 1};
    if (encode(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(src), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return GQ_ERR_CUDA;

    WArgs a;
    a.rows = rows; a.outs = outs; a.cols = cols;
    a.pitch = code_pitch(cols); a.epitch = exp_pitch(cols); a.ldw = lddw;
    a.codes = codes; a.exps = exps;
    a.scale = scale; a.shift = shift; a.db = db;
    a.dw = dw; a.out_f32 = out_dtype == GQ_F32;
    a.fast = row_align(dw, out_dtype, outs, lddw) >= (a.out_f32 ? 32 : 16) && mult(scale, 16) && mult(shift, 16);
    a.partial = reinterpret_cast<float*>(w);
    a.ktok = p.ktok; a.ksteps = static_cast<int>(p.ksteps);
    a.tiles_m = static_cast<int>(p.tiles_m); a.tiles_n = static_cast<int>(p.tiles_n);
    const int64_t tiles = p.tiles_m * p.tiles_n;
    a.shares = p.shares;
    a.own = static_cast<int>(tiles / p.shares);
    a.units = tiles % p.shares * p.ksteps;
    a.base = a.units / p.shares; a.rest = static_cast<int>(a.units % p.shares);
    const WArgs wanted = a;
    float* raw = p.sums_ld && !a.fast ? reinterpret_cast<float*>(w + p.sums_off) : nullptr;
    if (raw) {  // aligned fp32 sums first, padding columns among them (their codes are 0)
        a.scale = a.shift = nullptr;
        a.dw = raw;
        a.ldw = a.cols = p.sums_ld;
        a.out_f32 = a.fast = 1;
    }
    a.packed = p.pack;
    const bool early = sums || p.pack;
    const gq_status r = p.big ? launch_wgrad<Large>(map, a, early, st)
                              : launch_wgrad<Small>(map, a, early, st);
    if (r != GQ_OK || !raw) return r;
    const dim3 grid(static_cast<unsigned>((cols + 255) / 256),
                    static_cast<unsigned>(outs < 16384 ? (outs + 3) / 4 : 4096));
    finish_kernel<<<grid, 256, 0, st>>>(wanted, raw, p.sums_ld);
    return gqh::launch_status();
}

}  // extern "C"
