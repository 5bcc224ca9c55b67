// gq_fp8_linear.cu -- products of a linear layer on operands in 8-bit floating point (C ABI in
// include/gq.h; the format is described in gq_fp8.cuh).
//
//   forward   y[t, o]  = sum_i X[t, i] W[o, i] + bias[o]
//   gradient  dx[t, i] = sum_o DY[t, o] W[o, i]
//
// Both are D[m, t] = sum_k A[m, k] B[t, k] with A = W or its transposed matrix and B the tokens' operand.
// The outputs are the tensor cores' rows (128 of them) and the tokens their columns (16 to 128), so that a
// few tokens leave no tensor core idle rows to work on, and a warp with a lane per output stores 32
// neighbouring ones.  W is stored once: the gradient's product reads the same bytes with the outer dimension
// contiguous.  Scales are block scales of tcgen05.mma: the four instructions of a step of 128 take the
// same byte of each operand's exponents.
//
// Small form: a block per tile, and where there are few tiles a cluster of up to 8 blocks per tile, each with
// a part of the sum; the parts are added through distributed shared memory in the blocks' order.
//   warp 0   TMA loads of both operands (128 of k per step) and bulk copies of exponents (512 of k each)
//   warp 1   one thread copies exponents to TMEM and issues tcgen05.mma, accumulators in TMEM
//   2 on     (4 or 8) the sums from TMEM to memory; in calls of few steps a block, and of up to 16 tokens, they also put x
//            into 8 bits on its way to shared memory, so that the call is one launch
// What bounds it: latency.  With bf16 tokens, in a graph, the weights in the L2: one token through 4,096 x 4,096
// weights 6.6 to 8.0 us (their 16.8 MB would take 2.5 from memory), 384 tokens through 768 x 768 7.8 to 9.2; of
// tokens in 8 bits already 7.5 and 6.3 to 7.4.  A launch's ends, an operand's way, a chain of four steps or so, a join.
//
// The sums of the tensor cores: 32 products are added at a time, and the sum is cut each time, so the error of a chain
// grows with its length.  Of normal numbers, in one chain: 5.9e-8 of the result's norm at a depth of 1,024 (a
// product of the same values in fp32 4.1e-8), 2.2e-7 at 4,096 (8.4e-8) and 5.0e-7 at 8,192 (1.3e-7); where a
// cluster shares a sum (100 tokens, 1,280 outputs) 3.5e-8, 6.2e-8 and 8.1e-8.  Beside operands of 4 bits chains of the
// large form are not shortened for it: a second accumulator does not fit.
#include "gq_fp8.cuh"
#include "gq_tc.cuh"

#include <type_traits>

using namespace gqa;

namespace {

constexpr int kStep = 128;             // of k per step: bytes of a row of an operand's tile
constexpr int kTile = 128 * kStep;     // bytes of a tile of W

struct LArgs {
    int rows, m;                 // tokens, outputs
    int steps;                   // of k
    int tiles_m;
    const uint8_t* a_exps;       // of W (or its transposed matrix), of the tokens' operand
    const uint8_t* b_exps;
    const float* bias;           // nullable
    void* y;
    int64_t ldy;
    int out_f32, wide;           // wide: four neighbouring outputs of a row can be stored at once
    const void* x;               // of a fused call
    int64_t ldx;
};

template <int CG>
__device__ __forceinline__ void mma_fp8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa,
                                        uint32_t sb, bool add) {
    GQA_CG(CG,
           "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
           "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}",
           "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
           "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}",
           ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(add ? 1u : 0u) : "memory");
}
// 32 rows of 16 bytes to 4 columns of TMEM, in each of its four quarters (of both blocks of a pair, from the
// same place in each one's shared memory).
template <int CG> __device__ __forceinline__ void copy_exps(uint32_t tmem, uint64_t smem) {
    GQA_CG(CG, "tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;", "tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;",
           ::"r"(tmem), "l"(smem) : "memory");
}
// Rows of 128 bytes, 128-byte swizzle, 8 rows every 1,024 bytes: along k (128 of k of a row of the matrix)
// and along the outer dimension (128 outer elements of a k) alike.
__device__ __forceinline__ uint64_t operand(uint32_t smem) {
    return static_cast<uint64_t>((smem & 0x3FFFFu) >> 4) | (uint64_t(1) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
// Exponents: rows of 16 bytes one after the other, 8 of them every 128 bytes, no swizzle.
__device__ __forceinline__ uint64_t exp_operand(uint32_t smem) {
    return static_cast<uint64_t>((smem & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(128 >> 4) << 32) |
           (uint64_t(1) << 46);
}
// e4m3 operands, exponent bytes as scales, N columns, M = 128 per block; A_OUTER: A is contiguous along its
// outer dimension.  The scales' byte of a word is added per step.
template <int CG, int N, bool A_OUTER> struct Instruction {
    static constexpr uint32_t value = (A_OUTER ? 1u << 15 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
                                      (1u << 23) | (128u * CG >> 4 << 24);
    static __device__ __forceinline__ uint32_t of(uint32_t byte) { return value | byte << 4 | byte << 29; }
};
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float4 peer_load(uint32_t smem, uint32_t rank) {
    uint32_t there;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(smem), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(there)
                 : "memory");
    return v;
}
__device__ __forceinline__ void put(const LArgs& a, int64_t token, int out, float v) {
    if (a.out_f32) static_cast<float*>(a.y)[token * a.ldy + out] = v;
    else static_cast<bf16*>(a.y)[token * a.ldy + out] = __float2bfloat16_rn(v);
}

// Four neighbouring outputs of a token.
__device__ __forceinline__ void put4(const LArgs& a, int64_t token, int out, float4 v) {
    if (a.wide && out + 4 <= a.m) {
        if (a.out_f32)
            *reinterpret_cast<float4*>(static_cast<float*>(a.y) + token * a.ldy + out) = v;
        else
            *reinterpret_cast<uint2*>(static_cast<bf16*>(a.y) + token * a.ldy + out) =
                make_uint2(pack2(v.x, v.y, bf16()), pack2(v.z, v.w, bf16()));
        return;
    }
    const float w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (out + i < a.m) put(a, token, out + i, w[i]);
}

// BN tokens per tile: fewer than 128 only where one tile holds all of them.  A tile's exponents then begin with
// its first row, at an address in TMEM that is a multiple of 4 columns, as the scales of an instruction have to.
template <int BN_> struct Small {
    static constexpr int BN = BN_;
    static constexpr int kBytes = kTile + BN * kStep;      // of a step's operands
    static constexpr int kStages = BN <= 16 ? 8 : 6;
    static constexpr int kCols = BN <= 16 ? 32 : BN <= 64 ? 128 : 256;  // of TMEM
    // columns behind the accumulator: two sets of 4 for W's exponents, two of 4 for the tokens'
    static constexpr int kExps = BN;
    static_assert(kExps + 16 <= kCols, "exponents fit behind the accumulator");
    static constexpr int kSmem = kStages * (kBytes + 2 * kExpTile) + 1024;
    static_assert(128 * BN * 4 <= kStages * kBytes, "a block's sums fit in its operands' place");
};

// Warps that take the sums, and x in a fused call (8 where a step has much of it: 384 x 768 x 768 in two steps a
// block 9.2 us with four).
template <int BN, typename T> constexpr int kWarpsOf = !std::is_void<T>::value && BN > 16 ? 8 : 4;

// The tokens' side of a step, 128 columns of BN tokens from token t0 on, from x: 16 lanes hold a row's block, 2 W
// rows at a time by W warps.  Behind the last row and column stand zeros.
template <typename T, int BN, int W> struct Squeeze {
    static constexpr int S = 2 * W, R = BN / S;
    Raw8<T> w[R];
    __device__ __forceinline__ void fetch(const LArgs& a, int t0, int k, int depth, int thread, bool wide) {
        const int c = k * kStep + (thread & 15) * 8;
        const int left = depth - c, rows = a.rows - t0;
        const T* p = static_cast<const T*>(a.x) + (t0 + (thread >> 4)) * a.ldx + c;
#pragma unroll
        for (int i = 0; i < R; ++i, p += S * a.ldx) {
#pragma unroll
            for (int j = 0; j < static_cast<int>(sizeof(T)) * 2; ++j) w[i].w[j] = 0u;
            if ((thread >> 4) + S * i >= rows || left <= 0) continue;
            if (wide && left >= 8) {
#pragma unroll
                for (int j = 0; j < static_cast<int>(sizeof(T)) / 2; ++j) {
                    const uint4 g = reinterpret_cast<const uint4*>(p)[j];
                    w[i].w[4 * j] = g.x; w[i].w[4 * j + 1] = g.y; w[i].w[4 * j + 2] = g.z; w[i].w[4 * j + 3] = g.w;
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j < left) {
                        if constexpr (sizeof(T) == 4) w[i].w[j] = __float_as_uint(p[j]);
                        else w[i].w[j >> 1] |= static_cast<uint32_t>(__bfloat16_as_ushort(p[j])) << (16 * (j & 1));
                    }
            }
        }
    }
    // codes in the layout of a swizzled box, exponents at the step's byte of each row's word
    __device__ __forceinline__ void store(uint32_t codes, uint32_t exps, int k, int thread) {
        uint32_t top[R];
        tops<R>(w, top);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int row = (thread >> 4) + S * i, unit = (thread & 15) >> 1;
            const uint32_t e = fp8_exp_byte(top[i]);
            F2 v[4];
            pairs(w[i], v);
            uint2 q = fp8_codes8(v, inv_step(e));
            if (e == 255u) q = make_uint2(0u, 0u);
            asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(codes + row * 128 + ((unit ^ (row & 7)) << 4) +
                                                                  (thread & 1) * 8),
                         "r"(q.x), "r"(q.y)
                         : "memory");
            if ((thread & 15) == 0)
                asm volatile("st.shared.b8 [%0], %1;" ::"r"(exps + (row & 31) * 16 + (row >> 5) * 4 + (k & 3)), "r"(e)
                             : "memory");
        }
    }
};

// Adds the parts of tokens c, c + W PARTS, ... below `end` (W warps, each block a PARTS-th) and stores them;
// eight loads are on their way at a time (one by one, 128 tokens took 4 us).
template <int PARTS, int W>
__device__ __forceinline__ void join(const LArgs& a, uint32_t from, int c, int end, int t0, int out, float4 b) {
    constexpr int B = 8 / PARTS;
    for (; c < end; c += B * W * PARTS) {
        float4 p[B][PARTS];
#pragma unroll
        for (int j = 0; j < B; ++j)
#pragma unroll
            for (int r = 0; r < PARTS; ++r) {
                // (tokens behind the last are read as the last, and left out)
                const uint32_t at = from + min(c + j * W * PARTS, end - 1) * 512;
                if constexpr (PARTS == 1)
                    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                                 : "=f"(p[j][r].x), "=f"(p[j][r].y), "=f"(p[j][r].z), "=f"(p[j][r].w)
                                 : "r"(at)
                                 : "memory");
                else
                    p[j][r] = peer_load(at, r);
            }
#pragma unroll
        for (int j = 0; j < B; ++j) {
            float4 v = p[j][0];
#pragma unroll
            for (int r = 1; r < PARTS; ++r) {
                v.x += p[j][r].x; v.y += p[j][r].y; v.z += p[j][r].z; v.w += p[j][r].w;
            }
            v.x += b.x; v.y += b.y; v.z += b.z; v.w += b.w;
            if (c + j * W * PARTS < end) put4(a, t0 + c + j * W * PARTS, out, v);
        }
    }
}

// T: the type of x in a fused call, else void.
template <typename C, bool A_OUTER, typename T>
__global__ void __launch_bounds__(64 + 32 * kWarpsOf<C::BN, T>, 1)
    small_kernel(const __grid_constant__ CUtensorMap a_map, const __grid_constant__ CUtensorMap b_map,
                 const LArgs a, const int depth) {
    constexpr bool FUSED = !std::is_void<T>::value;
    constexpr int BN = C::BN, S = C::kStages, W = kWarpsOf<BN, T>;
    extern __shared__ uint8_t raw[];
    __shared__ alignas(8) uint64_t full[S], empty[S], acc_full, drain;
    __shared__ uint32_t tmem_slot;
    const uint32_t base = (gq::smem_u32(raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank(), parts = cluster_size();
    auto a_stage = [&](int s) { return base + s * C::kBytes; };
    auto b_stage = [&](int s) { return base + s * C::kBytes + kTile; };
    auto e_stage = [&](int s) { return base + S * C::kBytes + s * 2 * kExpTile; };

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            gq::mbar_init(gq::smem_u32(&full[s]), FUSED ? 1u + W : 1u);
            gq::mbar_init(gq::smem_u32(&empty[s]), 1u);
        }
        gq::mbar_init(gq::smem_u32(&acc_full), 1u);
        gq::mbar_init(gq::smem_u32(&drain), 1u);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc<1>(gq::smem_u32(&tmem_slot), C::kCols);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_slot;
    const int tile = blockIdx.x / parts;
    const int m0 = tile % a.tiles_m * 128, t0 = tile / a.tiles_m * BN;
    const int words = (a.steps + 3) / 4;
    const int k0 = static_cast<int>(static_cast<int64_t>(a.steps) * rank / parts);
    const int k1 = static_cast<int>(static_cast<int64_t>(a.steps) * (rank + 1) / parts);
    // exponents come with the first step of the block's, and with each that begins 512 of k
    auto with_exps = [&](int k) { return k == k0 || (k & 3) == 0; };

    if (warp == 0) {
        if (lane == 0) {
            bool ok = true;
            // W's side of a step, then the tokens': the launch before may still write those
            auto load_a = [&](int k, int s) {
                const uint32_t bar = gq::smem_u32(&full[s]);
                gq::mbar_arrive_expect_tx(bar, (FUSED ? kTile : C::kBytes) +
                                                   (with_exps(k) ? (FUSED ? 1 : 2) * kExpTile : 0));
                tma_load(a_stage(s), &a_map, A_OUTER ? m0 : k * kStep, A_OUTER ? k * kStep : m0, bar);
                if (with_exps(k))
                    bulk_load(e_stage(s), a.a_exps + (static_cast<int64_t>(m0 / 128) * words + k / 4) * kExpTile,
                              kExpTile, bar);
            };
            auto load_b = [&](int k, int s) {
                if constexpr (!FUSED) {
                    const uint32_t bar = gq::smem_u32(&full[s]);
                    tma_load(b_stage(s), &b_map, k * kStep, t0, bar);
                    if (with_exps(k))
                        bulk_load(e_stage(s) + kExpTile,
                                  a.b_exps + (static_cast<int64_t>(t0 / 128) * words + k / 4) * kExpTile, kExpTile, bar);
                }
            };
            const int first = min(k1 - k0, S);
            // W may be the work of the launch before too, but not where that one puts x into 8 bits: it let this
            // one begin when all before it had ended
            if constexpr (FUSED) gq::pdl_wait();
            for (int n = 0; n < first; ++n) load_a(k0 + n, n);
            if constexpr (!FUSED) gq::pdl_wait();
            for (int n = 0; n < first; ++n) load_b(k0 + n, n);
            int n = first;
            for (; n < k1 - k0; ++n) {
                ok = mbar_rest(gq::smem_u32(&empty[n % S]), ((n / S) - 1) & 1);
                if (!ok) break;
                load_a(k0 + n, n % S);
                load_b(k0 + n, n % S);
            }
            // nothing of this block's is in flight when it ends, whatever the others did
            for (int j = n > S ? n - S : 0; j < n; ++j) mbar_rest(gq::smem_u32(&full[j % S]), (j / S) & 1);
        }
    } else if (warp == 1) {
        bool ok = true;
        uint32_t set = 1, set_b = 1;  // of exponents' columns
        for (int n = 0; n < k1 - k0; ++n) {
            const int k = k0 + n, s = n % S;
            ok = __all_sync(kFull, mbar_rest(gq::smem_u32(&full[s]), (n / S) & 1));
            if (!ok) break;
            fence_after();
            const bool exps = with_exps(k), exps_b = FUSED || exps;  // (a fused call has a step's bytes with the step)
            if (exps) set ^= 1u;
            if (exps_b) set_b ^= 1u;
            const uint32_t sa = tmem + C::kExps + 4 * set, sb = tmem + C::kExps + 8 + 4 * set_b;
            const uint64_t da = operand(a_stage(s)), db = operand(b_stage(s));
            const uint32_t idesc = Instruction<1, BN, A_OUTER>::of(k & 3);
            if (elect_one()) {
                if (exps) copy_exps<1>(sa, exp_operand(e_stage(s)));
                if (exps_b) copy_exps<1>(sb, exp_operand(e_stage(s) + kExpTile));
#pragma unroll
                for (int kk = 0; kk < kStep / 32; ++kk)
                    mma_fp8<1>(tmem, da + kk * ((A_OUTER ? 32 * 128 : 32) >> 4), db + kk * (32 >> 4), idesc, sa, sb,
                               n > 0 || kk > 0);
                mma_commit<1>(gq::smem_u32(&empty[s]));
                if (n + 1 == k1 - k0) mma_commit<1>(gq::smem_u32(&acc_full));
            }
            __syncwarp();
        }
        if (!ok) {  // what was issued finishes before TMEM is freed
            if (elect_one()) mma_commit<1>(gq::smem_u32(&drain));
            __syncwarp();
            mbar_rest(gq::smem_u32(&drain), 0);
        }
    } else {
        const int q = warp & 3, m = q * 32 + lane;
        bool ok = true;
        if constexpr (FUSED) {
            const int thread = threadIdx.x - 64;
            const bool wide = ((reinterpret_cast<uintptr_t>(a.x) | static_cast<uintptr_t>(a.ldx * sizeof(T))) & 15u) == 0;
            // steps' loads on their way while as many are put into 8 bits
            constexpr int B = BN == 16 ? 8 / static_cast<int>(sizeof(T)) : 1;
            Squeeze<T, BN, W> now[B], next[B];
            auto fetch = [&](int n) {
#pragma unroll
                for (int j = 0; j < B; ++j)
                    if (n + j < k1 - k0) next[j].fetch(a, t0, k0 + n + j, depth, thread, wide);
            };
            gq::pdl_wait();
            fetch(0);
            for (int n0 = 0; n0 < k1 - k0 && ok; n0 += B) {
#pragma unroll
                for (int j = 0; j < B; ++j) now[j] = next[j];
                fetch(n0 + B);
#pragma unroll
                for (int j = 0; j < B; ++j) {
                    const int n = n0 + j, s = n % S;
                    if (n >= k1 - k0 || !ok) break;
                    if (n >= S) ok = mbar_rest(gq::smem_u32(&empty[s]), ((n / S) - 1) & 1);
                    ok = __all_sync(kFull, ok);
                    if (!ok) break;
                    now[j].store(b_stage(s), e_stage(s) + kExpTile, k0 + n, thread);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) gq::mbar_arrive(gq::smem_u32(&full[s]));
                }
            }
        }
        if (ok) ok = mbar_rest(gq::smem_u32(&acc_full), 0);
        ok = __all_sync(kFull, ok);
        fence_after();
        float* sums = reinterpret_cast<float*>(raw + (base - gq::smem_u32(raw)));
        if constexpr (!FUSED) gq::pdl_wait();  // y may be what the launch before still reads
#pragma unroll 1
        for (int c = (warp - 2) / 4 * 16; c < BN; c += W * 4) {
            if (t0 + c >= a.rows) break;
            uint32_t v[16];
            tmem_load(tmem + (static_cast<uint32_t>(q * 32) << 16) + c, v);
            if (!ok) {  // a wait gave up: the tile is marked
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = 0x7FFFFFFFu;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) sums[(c + i) * 128 + m] = __uint_as_float(v[i]);
        }
    }
    fence_before();
    __syncwarp();
    if (parts > 1) cluster_sync();
    else __syncthreads();
    if (warp >= 2) {  // every parts-th token, four outputs a lane, and of those every fourth a warp
        const int m = lane * 4;
        float4 b = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (a.bias) {
            float* w = reinterpret_cast<float*>(&b);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (m0 + m + i < a.m) w[i] = a.bias[m0 + m + i];
        }
        const uint32_t from = base + m * 4;
        const int c = static_cast<int>(rank) + (warp - 2) * static_cast<int>(parts), end = min(BN, a.rows - t0);
        switch (parts) {
            case 1: join<1, W>(a, from, c, end, t0, m0 + m, b); break;
            case 2: join<2, W>(a, from, c, end, t0, m0 + m, b); break;
            case 4: join<4, W>(a, from, c, end, t0, m0 + m, b); break;
            default: join<8, W>(a, from, c, end, t0, m0 + m, b); break;
        }
    }
    __syncwarp();
    if (parts > 1) cluster_sync();  // no block's sums are read any more
    if (warp == 1) tmem_free<1>(tmem, C::kCols);
}

// ---- the large form ------------------------------------------------------------------------
//
// A pair of blocks works on 256 outputs x 256 tokens: each block loads 128 of the outputs and 128 of the
// tokens, and one tcgen05.mma of both tensor cores reads both blocks' shared memory (a step of 128 x 256 in
// one block would ask for 48 KB of operands in the time of 32).  Pairs stay and take tile after tile; the
// sums leave TMEM for registers at once, so that the next tile's products go on while they are stored.
// What bounds it: the tensor cores, 86 % busy; a step takes 537 cycles of the 512 that its products need (copies of
// both blocks count on the first one's barrier, and waiting threads sleep), the change of tiles 1,400, and the
// last wave is not full.  16,384 tokens x 4,096 x 4,096: 141 us at 2,070 MHz (3.9 PFLOP/s; the library's product
// of matrices with one scale 124), 173 to 183 as the power cap lets random numbers run (146 to 167).
struct Large {
    static constexpr int BN = 256, kStages = 6, kWarps = 8;         // warps that take the sums
    static constexpr int kThreads = 64 + 32 * kWarps;
    static constexpr int kBytes = 2 * kTile;                        // of a step's operands, per block
    static constexpr int kExps = BN;                                // columns of exponents: two sets, in turn,
    static constexpr int kSet = 12;                                 // of 4 for the outputs and 8 for the tokens
    static constexpr int kCols = 512;
    // rows of y on their way out: two groups of warps, three buffers of 16 tokens each
    static constexpr int kOut = 16, kRing = 3, kOutBytes = kOut * 256;
    static constexpr int kOperands = kStages * (kBytes + 3 * kExpTile);
    static constexpr int kSmem = kOperands + 2 * kRing * kOutBytes + 1024;
};

// 64 tokens' sums of this lane's output, from token t on, element by element: fp32, and rows of y that the TMA
// cannot write.
__device__ __forceinline__ void put_column(const LArgs& a, int t, int m, float b, const uint32_t (&v)[64]) {
    if (m >= a.m) return;
    if (a.out_f32) {
        float* p = static_cast<float*>(a.y) + static_cast<int64_t>(t) * a.ldy + m;
#pragma unroll
        for (int j = 0; j < 64; ++j, p += a.ldy)
            if (t + j < a.rows) *p = __uint_as_float(v[j]) + b;
    } else {
        bf16* p = static_cast<bf16*>(a.y) + static_cast<int64_t>(t) * a.ldy + m;
#pragma unroll
        for (int j = 0; j < 64; ++j, p += a.ldy)
            if (t + j < a.rows) *p = __float2bfloat16_rn(__uint_as_float(v[j]) + b);
    }
}
__device__ __forceinline__ void group_sync(int group) { asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory"); }

// The same through shared memory, in bf16: four warps fill 16 tokens' rows of 128 outputs, which the TMA takes
// to y while they fill the next (two stores of 64 bytes in every instruction, straight from registers, took
// 4 us a tile).  next: the ring's place, the same for the group.
__device__ __forceinline__ void put_rows(const CUtensorMap* y_map, uint32_t ring, int group, int warp, int lane, int t,
                                         int m0, int rows, float b, const uint32_t (&v)[64],
                                         int& next) {
    using C = Large;
    const bool leads = warp == 0 && lane == 0;
#pragma unroll
    for (int c = 0; c < 64; c += C::kOut) {
        const uint32_t at = ring + next * C::kOutBytes;
        if (leads) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(C::kRing - 1) : "memory");
        group_sync(group);
#pragma unroll
        for (int j = 0; j < C::kOut; j += 2) {
            const uint32_t w = pack2(__uint_as_float(v[c + j]) + b, __uint_as_float(v[c + j + 1]) + b, bf16());
            const uint32_t to = at + j * 256 + (warp * 32 + lane) * 2;
            asm volatile("st.shared.b16 [%0], %1;" ::"r"(to), "h"(static_cast<uint16_t>(w)) : "memory");
            asm volatile("st.shared.b16 [%0], %1;" ::"r"(to + 256), "h"(static_cast<uint16_t>(w >> 16)) : "memory");
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        group_sync(group);
        if (leads && t + c < rows) {
            asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(y_map),
                         "r"(m0), "r"(t + c), "r"(at)
                         : "memory");
        }
        if (leads) asm volatile("cp.async.bulk.commit_group;" ::: "memory");  // (the ring counts empty ones too)
        next = next + 1 == C::kRing ? 0 : next + 1;
    }
}

template <bool A_OUTER>
__global__ void __launch_bounds__(Large::kThreads, 1)
    large_kernel(const __grid_constant__ CUtensorMap a_map, const __grid_constant__ CUtensorMap b_map,
                 const __grid_constant__ CUtensorMap a_exps, const __grid_constant__ CUtensorMap b_exps,
                 const __grid_constant__ CUtensorMap y_map, const LArgs a) {
    using C = Large;
    constexpr int S = C::kStages;
    extern __shared__ uint8_t raw[];
    __shared__ alignas(8) uint64_t full[S], empty[S], acc_full, acc_empty, drain;  // full: in the first block
    __shared__ uint32_t tmem_slot;
    const uint32_t base = (gq::smem_u32(raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = pair_rank<2>();
    auto a_stage = [&](int s) { return base + s * C::kBytes; };
    auto b_stage = [&](int s) { return base + s * C::kBytes + kTile; };
    auto e_stage = [&](int s) { return base + S * C::kBytes + s * 3 * kExpTile; };

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            gq::mbar_init(gq::smem_u32(&full[s]), 1u);
            gq::mbar_init(gq::smem_u32(&empty[s]), 1u);
        }
        gq::mbar_init(gq::smem_u32(&acc_full), 1u);
        gq::mbar_init(gq::smem_u32(&acc_empty), 2 * C::kWarps);
        gq::mbar_init(gq::smem_u32(&drain), 1u);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc<2>(gq::smem_u32(&tmem_slot), C::kCols);
    fence_before();
    __syncthreads();
    pair_sync<2>();
    fence_after();
    const uint32_t tmem = tmem_slot;
    const int pairs = gridDim.x / 2, first = blockIdx.x / 2;
    const int across = (a.m + 255) / 256, tiles = across * ((a.rows + C::BN - 1) / C::BN);
    const int words = (a.steps + 3) / 4;
    const int last_a = (a.m - 1) / 128, last_b = (a.rows - 1) / 128;  // 128 rows of exponents that exist

    if (warp == 0) {
        if (lane == 0) {
            int n = 0;
            bool ok = true;
            gq::pdl_wait();  // the tokens' operand may be the launch before's work
            for (int tile = first; tile < tiles && ok; tile += pairs) {
                const int am = tile % across * 2 + static_cast<int>(rank);  // in 128 rows
                const int bt = tile / across * 2;
                const int ea = min(am, last_a) * words, eb0 = bt * words, eb1 = min(bt + 1, last_b) * words;
                for (int k = 0; k < a.steps; ++k, ++n) {
                    const int s = n % S;
                    if (n >= S) ok = mbar_rest(gq::smem_u32(&empty[s]), ((n / S) - 1) & 1);
                    if (!ok) break;
                    const uint32_t bar = place_in(gq::smem_u32(&full[s]), 0);
                    const bool exps = (k & 3) == 0;
                    if (rank == 0)  // what both blocks will load
                        gq::mbar_arrive_expect_tx(gq::smem_u32(&full[s]), 2 * (C::kBytes + (exps ? 3 * kExpTile : 0)));
                    tma_load_pair(a_stage(s), &a_map, A_OUTER ? am * 128 : k * kStep, A_OUTER ? k * kStep : am * 128,
                                  bar);
                    tma_load_pair(b_stage(s), &b_map, k * kStep, (bt + static_cast<int>(rank)) * 128, bar);
                    if (exps) {
                        tma_load_pair(e_stage(s), &a_exps, 0, ea + k / 4, bar);
                        tma_load_pair(e_stage(s) + kExpTile, &b_exps, 0, eb0 + k / 4, bar);
                        tma_load_pair(e_stage(s) + 2 * kExpTile, &b_exps, 0, eb1 + k / 4, bar);
                    }
                }
            }
            // nothing that comes to this block is in flight when it ends: what was loaded has been read, and
            // the word of that has come
            for (int j = n > S ? n - S : 0; j < n; ++j) mbar_rest(gq::smem_u32(&empty[j % S]), (j / S) & 1);
        }
    } else if (warp == 1) {
        if (rank == 0) {
            int n = 0, done = 0;
            bool ok = true;
            uint32_t set = 1;  // of exponents' columns
            auto wait = [&](uint64_t* bar, int phase) {
                ok = __all_sync(kFull, mbar_rest(gq::smem_u32(bar), phase & 1));
                fence_after();
            };
            for (int tile = first; tile < tiles && ok; tile += pairs, ++done) {
                if (done > 0) wait(&acc_empty, done - 1);
                for (int k = 0; k < a.steps && ok; ++k, ++n) {
                    const int s = n % S;
                    wait(&full[s], n / S);
                    if (!ok) break;
                    const bool exps = (k & 3) == 0;
                    if (exps) set ^= 1u;
                    const uint32_t sa = tmem + C::kExps + C::kSet * set;
                    const uint64_t da = operand(a_stage(s)), db = operand(b_stage(s));
                    const uint32_t idesc = Instruction<2, C::BN, A_OUTER>::of(k & 3);
                    if (elect_one()) {
                        if (exps) {
#pragma unroll
                            for (int j = 0; j < 3; ++j)
                                copy_exps<2>(sa + 4 * j, exp_operand(e_stage(s) + j * kExpTile));
                        }
#pragma unroll
                        for (int kk = 0; kk < kStep / 32; ++kk)
                            mma_fp8<2>(tmem, da + kk * ((A_OUTER ? 32 * 128 : 32) >> 4), db + kk * (32 >> 4), idesc, sa,
                                       sa + 4, k > 0 || kk > 0);
                        mma_commit<2>(gq::smem_u32(&empty[s]));
                        if (k + 1 == a.steps) mma_commit<2>(gq::smem_u32(&acc_full));
                    }
                    __syncwarp();
                }
            }
            if (!ok) {  // let what was issued finish before TMEM is given back
                if (elect_one()) mma_commit<2>(gq::smem_u32(&drain));
                __syncwarp();
                mbar_rest(gq::smem_u32(&drain), 0);
            }
        }
    } else {
        const int quad = warp & 3, group = (warp - 2) >> 2;
        const uint32_t ring = base + C::kOperands + group * (C::kRing * C::kOutBytes);
        int done = 0, next = 0;
        bool ok = true;
        gq::pdl_wait();  // y may be what the launch before still reads
        for (int tile = first; tile < tiles; tile += pairs, ++done) {
            const int m0 = (tile % across * 2 + static_cast<int>(rank)) * 128, m = m0 + quad * 32 + lane;
            const int t0 = tile / across * C::BN + group * 128;
            const float b = a.bias && m < a.m ? a.bias[m] : 0.0f;
            if (ok) ok = mbar_rest(gq::smem_u32(&acc_full), done & 1);
            ok = __all_sync(kFull, ok);
            fence_after();
            uint32_t v[2][64];
            if (ok) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    tmem_load(tmem + (static_cast<uint32_t>(quad * 32) << 16) + group * 128 + j * 64, v[j]);
            } else {  // a wait gave up: the tile is marked
#pragma unroll
                for (int j = 0; j < 128; ++j) v[j >> 6][j & 63] = 0x7FFFFFFFu;
            }
            fence_before();
            __syncwarp();
            if (lane == 0) arrive_first<2>(gq::smem_u32(&acc_empty));
            if (a.wide) {
                if (m0 >= a.m) continue;  // (the whole group)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    if (t0 + 64 * j < a.rows)
                        put_rows(&y_map, ring, group, quad, lane, t0 + 64 * j, m0, a.rows, b, v[j],
                                 next);
            } else {
                put_column(a, t0, m, b, v[0]);
                put_column(a, t0 + 64, m, b, v[1]);
            }
        }
        // nothing leaves shared memory any more when the block ends
        if (quad == 0 && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    pair_sync<2>();  // neither block's memory is in use any more
    if (warp == 1) tmem_free<2>(tmem, C::kCols);
    pair_sync<2>();
}

// ---- host ----------------------------------------------------------------------------------

// A matrix of bytes, `rows` of them `pitch` apart with `width` elements each, in boxes of 128 x `box`.
bool byte_map(CUtensorMap* map, const uint8_t* p, int64_t width, int64_t rows, int64_t pitch, int box) {
    EncodeFn encode = encode_fn();
    if (!encode) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch)};
    const cuuint32_t sizes[2] = {kStep, static_cast<cuuint32_t>(box)}, one[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(p), dims, strides, sizes, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Exponents of a matrix of `rows` rows as rows of 512 bytes, one of them per box.
bool exp_map(CUtensorMap* map, const uint8_t* p, int64_t rows, int64_t steps) {
    EncodeFn encode = encode_fn();
    if (!encode) return false;
    const cuuint64_t dims[2] = {kExpTile / 4, static_cast<cuuint64_t>((rows + 127) / 128 * ((steps + 3) / 4))};
    const cuuint64_t strides[1] = {kExpTile};
    const cuuint32_t sizes[2] = {kExpTile / 4, 1}, one[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<uint8_t*>(p), dims, strides, sizes, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// y in bf16, in boxes of 128 outputs x 16 tokens; false where its rows do not suit the TMA, which writes whole
// 16-byte pieces also where a row ends inside one.
bool out_map(CUtensorMap* map, const LArgs& a) {
    EncodeFn encode = encode_fn();
    if (!encode) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(a.m), static_cast<cuuint64_t>(a.rows)};
    const cuuint64_t strides[1] = {a.rows > 1 ? static_cast<cuuint64_t>(a.ldy) * 2
                                              : (static_cast<cuuint64_t>(a.m) * 2 + 15) / 16 * 16};
    const cuuint32_t sizes[2] = {128, Large::kOut}, one[2] = {1, 1};
    return strides[0] < (cuuint64_t(1) << 40) &&
           encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.y, dims, strides, sizes, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// early: this launch may begin while the one before it on the stream ends (and waits for that before it reads
// what may be its work).
template <typename C, bool A_OUTER, typename T>
gq_status launch_small(const CUtensorMap& a_map, const CUtensorMap& b_map, const LArgs& a, int64_t depth, int parts,
                       bool early, cudaStream_t st) {
    auto k = small_kernel<C, A_OUTER, T>;
    constexpr int kThreadsS = 64 + 32 * kWarpsOf<C::BN, T>;
    gqh::blocks_per_sm(k, C::kSmem, kThreadsS);  // raises the shared-memory limit once
    const int64_t tiles = static_cast<int64_t>(a.tiles_m) * ((a.rows + C::BN - 1) / C::BN);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * parts));
    cfg.blockDim = dim3(kThreadsS);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (parts > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = static_cast<unsigned>(parts);
        attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (early) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return gqh::status_of(cudaLaunchKernelEx(&cfg, k, a_map, b_map, a, static_cast<int>(depth)));
}

template <bool A_OUTER>
gq_status launch_large(const CUtensorMap& a_map, const CUtensorMap& b_map, LArgs a, bool early, cudaStream_t st) {
    auto k = large_kernel<A_OUTER>;
    gqh::blocks_per_sm(k, Large::kSmem, Large::kThreads);  // raises the shared-memory limit once
    const int64_t tiles = (static_cast<int64_t>(a.m) + 255) / 256 * ((static_cast<int64_t>(a.rows) + Large::BN - 1) / Large::BN);
    const int64_t pairs = gqh::sm_count() / 2;
    CUtensorMap a_exps, b_exps;
    if (!exp_map(&a_exps, a.a_exps, a.m, a.steps) || !exp_map(&b_exps, a.b_exps, a.rows, a.steps)) return GQ_ERR_CUDA;
    CUtensorMap y_map = a_map;  // not used where it cannot be made
    a.wide = !a.out_f32 && mult(a.y, 16) && a.m % 8 == 0 && (a.ldy % 8 == 0 || a.rows == 1) && out_map(&y_map, a);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * (tiles < pairs ? tiles : pairs)));
    cfg.blockDim = dim3(Large::kThreads);
    cfg.dynamicSmemBytes = Large::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = early ? 2 : 1;
    return gqh::status_of(cudaLaunchKernelEx(&cfg, k, a_map, b_map, a_exps, b_exps, y_map, a));
}

// The form that a call takes: bn tokens per tile and parts of the sums, Large::BN for the large form; fused: one
// launch, which puts x into 8 bits itself.  The smallest of the times that the waves of blocks take, in
// microseconds as measured in graphs: 5 for a launch's ends, and for each wave 2 and 0.28 a step (0.7 more for a
// join); 6 and 1 in the large form, whose pairs stay.  Both sides, depth x outputs for so many tokens: 768 x
// 768 for 384 in four parts 6.3 and in one 7.1, 4,096 x 4,096 for 256 in two parts 11.9, in one 15.6, large
// 15.6; for 1,024 tokens of 1,024 x 4,096 large 8.9 and small 15.4, 256 x 256 for 4,096 large 6.9 and small
// 5.7.  Fused or not, 4,096 x 4,096: 1 token 6.6 and 7.8, 16 tokens 7.8 and 8.4, 32 tokens 8.9 and 8.1; a step of
// 64 or 128 tokens takes the warps 0.3 or 0.6 us more, and what is saved is a launch: 64 tokens x 1,024 x 1,024 5.3 for
// 5.8 in one step a block, 384 x 768 x 768 7.8 for 7.4 in two, 200 x 2,048 x 1,024 9.9 for 7.9 in four, and 2.7 us
// of the host in each.  So up to 1.5 us of the GPU are given for the host's 2.7: a call is faster, its replay in a graph
// up to 0.5 us slower (384 x 768 x 768; 128 x 1,024 x 4,096 8.1 for 7.6; 512 x 1,024 x 1,024 8.1 for 7.8).
struct Choice {
    int bn, parts;
    bool fused;
};
Choice choose(int64_t rows, int64_t outs, int64_t steps, int64_t sms, bool from_x) {
    const int bn = rows <= 16 ? 16 : rows <= 64 ? 64 : 128;
    const int64_t tiles = (outs + 127) / 128 * ((rows + bn - 1) / bn);
    const int64_t large = (outs + 255) / 256 * ((rows + Large::BN - 1) / Large::BN), pairs = sms / 2;
    double best = 6.0 + static_cast<double>((large + pairs - 1) / pairs) * (1.0 + 0.28 * steps);
    Choice c{Large::BN, 1, false};
    for (int parts = 1; parts <= 8 && parts <= steps; parts *= 2) {
        const double waves = static_cast<double>((tiles * parts + sms - 1) / sms);
        const double t = 5.0 + waves * (2.0 + 0.28 * ((steps + parts - 1) / parts)) + (parts > 1 ? 0.7 : 0.0);
        if (t <= best) {
            best = t;
            const double squeeze = (bn == 16 ? 0.0 : 0.6 * bn / 128.0) * ((steps + parts - 1) / parts) * waves;
            c = {bn, parts, from_x && squeeze <= 1.5};
        }
    }
    return c;
}

// D = A B^T as above: `outs` rows of A, sums over `depth`.
template <bool A_OUTER>
gq_status product(const void* x, int dtype, int64_t ldx, uint8_t* xcodes, uint8_t* xexps, int64_t rows,
                  int64_t depth, const uint8_t* wcodes, const uint8_t* wexps, int64_t outs, const float* bias,
                  void* y, int out_dtype, int64_t ldy, cudaStream_t st) {
    const int64_t most = int64_t(1) << 30;
    if (!in_type(out_dtype) || !size_ok(rows, depth) || outs < 1 || rows >= most || depth >= most || outs >= most)
        return GQ_ERR_INVALID;
    if (!matrix_ok(y, out_dtype, rows, outs, ldy) || !mult(bias, 4)) return GQ_ERR_INVALID;
    if (x && (!in_type(dtype) || !matrix_ok(x, dtype, rows, depth, ldx))) return GQ_ERR_INVALID;
    if (rows == 0) return GQ_OK;
    if (!saved_ok(wcodes, wexps)) return GQ_ERR_INVALID;
    const int64_t sms = gqh::sm_count(), tiles_m = (outs + 127) / 128, steps = (depth + kStep - 1) / kStep;
    if (tiles_m * ((rows + 15) / 16) * 8 >= int64_t(1) << 31) return GQ_ERR_INVALID;
    LArgs a;
    a.rows = static_cast<int>(rows); a.m = static_cast<int>(outs);
    a.steps = static_cast<int>(steps); a.tiles_m = static_cast<int>(tiles_m);
    a.a_exps = wexps; a.b_exps = xexps; a.bias = bias;
    a.y = y; a.ldy = ldy; a.out_f32 = out_dtype == GQ_F32;
    a.wide = mult(y, a.out_f32 ? 16 : 8) && (ldy % 4 == 0 || rows == 1);
    a.x = x; a.ldx = ldx;
    const Choice c = choose(rows, outs, steps, sms, x != nullptr);
    if (c.bn < 128 && rows > c.bn) return GQ_ERR_INVALID;  // see Small
    if (!c.fused && !saved_ok(xcodes, xexps)) return GQ_ERR_INVALID;
    CUtensorMap a_map, b_map;
    if (!byte_map(&a_map, wcodes, A_OUTER ? outs : depth, A_OUTER ? depth : outs,
                  fp8_pitch(A_OUTER ? outs : depth), 128))
        return GQ_ERR_CUDA;
    if (c.fused) {
        b_map = a_map;  // not used
    } else {
        if (!byte_map(&b_map, xcodes, depth, rows, fp8_pitch(depth), c.bn < 128 ? c.bn : 128)) return GQ_ERR_CUDA;
        if (x) {
            const gq_status r = gq_fp8_quantize(x, dtype, rows, depth, ldx, 1, xcodes, xexps, nullptr, st);
            if (r != GQ_OK) return r;
        }
    }
    if (c.bn == Large::BN) return launch_large<A_OUTER>(a_map, b_map, a, x != nullptr, st);
#define GQA_SMALL(BN, T) launch_small<Small<BN>, A_OUTER, T>(a_map, b_map, a, depth, c.parts, x != nullptr, st)
#define GQA_TOKENS(T) \
    (c.bn == 16 ? GQA_SMALL(16, T) : c.bn == 64 ? GQA_SMALL(64, T) : GQA_SMALL(128, T))
    if (!c.fused) return GQA_TOKENS(void);
    return dtype == GQ_F32 ? GQA_TOKENS(float) : GQA_TOKENS(bf16);
#undef GQA_TOKENS
#undef GQA_SMALL
}

}  // namespace

extern "C" {

size_t gq_fp8_linear_workspace_bytes(int64_t rows, int64_t depth, int64_t outs) {
    if (!size_ok(rows, depth) || rows < 1 || outs < 1) return 0;
    if (choose(rows, outs, (depth + kStep - 1) / kStep, gqh::sm_count(), true).fused) return 0;
    return static_cast<size_t>(rows * fp8_pitch(depth) + exp_bytes(rows, depth));
}

gq_status gq_fp8_linear(const void *x, int dtype, int64_t ldx, uint8_t *xcodes, uint8_t *xexps, int64_t rows,
                        int64_t cols, const uint8_t *wcodes, const uint8_t *wexps, int64_t outs,
                        const float *bias, void *y, int out_dtype, int64_t ldy, void *stream) {
    return product<false>(x, dtype, ldx, xcodes, xexps, rows, cols, wcodes, wexps, outs, bias, y, out_dtype, ldy,
                          static_cast<cudaStream_t>(stream));
}

gq_status gq_fp8_linear_dgrad(const void *dy, int dtype, int64_t lddy, uint8_t *dycodes, uint8_t *dyexps,
                              int64_t rows, int64_t outs, const uint8_t *wcodes, const uint8_t *wexps_t,
                              int64_t cols, void *dx, int out_dtype, int64_t lddx, void *stream) {
    return product<true>(dy, dtype, lddy, dycodes, dyexps, rows, outs, wcodes, wexps_t, cols, nullptr, dx,
                         out_dtype, lddx, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
