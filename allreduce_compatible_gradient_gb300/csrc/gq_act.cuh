// gq_act.cuh -- device and host pieces shared by the activation kernels (gq_act.cu, gq_layernorm_fwd.cu,
// gq_layernorm_bwd.cu, gq_wgrad.cu): element access, the 8-bit block format and its two roundings.
//
// Format: a row of `cols` elements is cut into blocks of 32 columns.  A block with largest
// magnitude a has the exponent byte E = min{ E >= 1 : a <= 127 * 2^(E - 127) }, 255 if it holds
// a NaN, an infinity or a magnitude above 127 * 2^121 (its codes are then 0 and it reads back as
// NaN: 0 * 2^128); an element stands for code * 2^(E - 127).  A power-of-two step costs at most one
// bit against a free step (the code of the block's largest element lies in 64..127) and makes every
// value, 7 bits times a power of two, exact in bf16: what reads a checkpoint rounds nothing.
#pragma once
#include "gq.h"
#include "gq_host.cuh"
#include "gq_kernels.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

namespace gqa {

constexpr int kBlk = 32;         // columns of one exponent
constexpr uint32_t kFull = 0xFFFFFFFFu;

// Random words of a launch: the Philox round keys of the seed, and the step.
struct Rng {
    uint32_t rk[20];
    uint32_t step_lo, step_hi;
};

inline Rng make_rng(uint64_t seed, uint64_t step) {
    Rng r;
    const uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
    for (int i = 0; i < 10; ++i) {
        r.rk[2 * i] = k0 + static_cast<uint32_t>(i) * 0x9E3779B9u;
        r.rk[2 * i + 1] = k1 + static_cast<uint32_t>(i) * 0xBB67AE85u;
    }
    r.step_lo = static_cast<uint32_t>(step);
    r.step_hi = static_cast<uint32_t>(step >> 32);
    return r;
}

inline int64_t code_pitch(int64_t cols) { return (cols + 31) / 32 * 32; }
inline int64_t exp_pitch(int64_t cols) { return ((cols + 31) / 32 + 15) / 16 * 16; }

// n / d for n < 2^31 by a multiplication: m = ceil(2^(31 + l) / d), l = ceil(log2 d) >= 1; the
// excess m d - 2^(31 + l) is below 2^l, so its contribution n * excess stays below 2^(31 + l).
struct Div {
    uint32_t d, m, s;
};
inline Div make_div(uint32_t d) {  // d >= 2
    uint32_t l = 1;
    while ((uint64_t(1) << l) < d) ++l;
    return Div{d, static_cast<uint32_t>(((uint64_t(1) << (31 + l)) + d - 1) / d), l - 1};
}
__device__ __forceinline__ uint32_t quot(uint32_t n, const Div& v) { return __umulhi(n, v.m) >> v.s; }

// ---- elements ------------------------------------------------------------------------------
using bf16 = __nv_bfloat16;

__device__ __forceinline__ float up(float v) { return v; }
__device__ __forceinline__ float up(bf16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void down(float v, float& o) { o = v; }
__device__ __forceinline__ void down(float v, bf16& o) { o = __float2bfloat16_rn(v); }
__device__ __forceinline__ void down(float v, __half& o) { o = __float2half_rn(v); }

__device__ __forceinline__ uint32_t pack2(float a, float b, bf16) {
    __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&t);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
    __half2 t = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&t);
}

// 32 bytes in one access (sm_100 and later), or two 16-byte ones where rows are only 16-byte
// aligned.
template <int ALIGN>
__device__ __forceinline__ void ld32(const void* p, uint32_t (&w)[8]) {
    if constexpr (ALIGN == 32) {
        asm volatile("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                       "=r"(w[6]), "=r"(w[7])
                     : "l"(p));
    } else {
        const uint4 a = __ldg(static_cast<const uint4*>(p));
        const uint4 b = __ldg(static_cast<const uint4*>(p) + 1);
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    }
}
template <int ALIGN>
__device__ __forceinline__ void st32(void* p, const uint32_t (&w)[8]) {
    if constexpr (ALIGN == 32) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]),
                     "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        static_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        static_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// V consecutive elements starting at column c of the row at p, widened to fp32; columns at and
// past `cols` read as 0.  V = 1: one element.  V = 8: p + c is 16-byte aligned.
template <typename T, int V>
__device__ __forceinline__ void load(const T* p, int64_t c, int64_t cols, float (&v)[V]) {
    if constexpr (V > 1) {
        if (c + V <= cols) {
            if constexpr (sizeof(T) == 4) {
                uint32_t w[8];
                ld32<16>(p + c, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
            } else {
                const uint4 a = __ldg(reinterpret_cast<const uint4*>(p + c));
                const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[2 * i] = __uint_as_float(w[i] << 16);
                    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
                }
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = c + i < cols ? up(p[c + i]) : 0.0f;
}

// The same for storing; V = 8 or 16: p + c is ALIGN-byte aligned.
template <typename T, int V, int ALIGN>
__device__ __forceinline__ void store(T* p, int64_t c, int64_t cols, const float (&v)[V]) {
    if constexpr (V > 1) {
        if (c + V <= cols) {
            if constexpr (sizeof(T) == 4) {
#pragma unroll
                for (int k = 0; k < V / 8; ++k) {
                    uint32_t w[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[8 * k + i]);
                    st32<ALIGN>(p + c + 8 * k, w);
                }
            } else if constexpr (V == 16) {
                uint32_t w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = pack2(v[2 * i], v[2 * i + 1], T());
                st32<ALIGN>(p + c, w);
            } else {
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = pack2(v[2 * i], v[2 * i + 1], T());
                *reinterpret_cast<uint4*>(p + c) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (c + i < cols) down(v[i], p[c + i]);
}

// ---- copies in flight ----------------------------------------------------------------------
// Every thread brings what it will read itself to its own places in shared memory, kDepth - 1 rows
// ahead, so that no thread waits for another's copy: about 70 KB in flight per SM where latency
// times bandwidth asks for 36, without a register for it.
constexpr int kDepth = 4;
// Through L1: a thread's 32 bytes are two copies, and past L1 (cp.async.cg) each would fetch the
// 32-byte sector that they share (32,768 x 4,096 bf16 to codes: 95 us so, 64 us through L1).
template <int BYTES> __device__ __forceinline__ void copy_async(uint32_t to, const void* from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(from), "n"(BYTES)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the last D - 1 groups have landed.
template <int D = kDepth> __device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(D - 1) : "memory");
}
__device__ __forceinline__ void copy_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// `bytes` of 16 (0..16), the rest zeros.
__device__ __forceinline__ void copy_part(uint32_t to, const void* from, uint32_t bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes)
                 : "memory");
}

// ---- pairs of fp32 -------------------------------------------------------------------------
// One instruction on two fp32 numbers (sm_100 and later), each rounded as its scalar form: what
// bounds these kernels beside memory is the number of instructions issued.
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ F2 f2(float a) { return f2(a, a); }
__device__ __forceinline__ void split(F2 a, float& x, float& y) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(a.v));
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ float sum2(F2 a) {
    float x, y;
    split(a, x, y);
    return x + y;
}

// ---- the 8-bit block format ----------------------------------------------------------------

// The exponent byte: with a = 1.f * 2^k, a <= 127 * 2^(k - 6) iff 1.f <= 127 / 64, that is iff
// the fraction field is at most 0x7E0000; adding 0x1FFFF carries into the exponent otherwise.
__device__ __forceinline__ uint32_t exp_byte(uint32_t top) {
    const int e = static_cast<int>((top + 0x1FFFFu) >> 23) - 6;
    return top > 0x7F7E0000u ? 255u : static_cast<uint32_t>(max(e, 1));
}
// 2^(127 - E): exact, normal for 1 <= E <= 248 (the largest that a block not marked has).
__device__ __forceinline__ float inv_step(uint32_t e) { return __uint_as_float((254u - e) << 23); }
// 2^(E - 127); infinity for E = 255.
__device__ __forceinline__ float step_of(uint32_t e) { return __uint_as_float(e << 23); }

// Bytes B of a, b, c, d as one word.
template <int B>
__device__ __forceinline__ uint32_t gather_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    constexpr uint32_t sel = B | ((4 + B) << 4);
    return __byte_perm(__byte_perm(a, b, sel), __byte_perm(c, d, sel), 0x5410);
}

// Largest magnitude of the 32-column block that 4 neighbouring lanes hold, 8 columns each as pairs, as fp32
// bits (which order like the magnitudes, with NaN above infinity).  Every lane of the warp calls it.
// Maxima of floating-point numbers pass over a NaN, so `plain` says that there is none (and no
// infinity); otherwise the bits are compared.
__device__ __forceinline__ uint32_t block_top8(const F2 (&h)[4], bool plain) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) split(h[i], v[2 * i], v[2 * i + 1]);
    uint32_t m;
    if (plain) {
        float a = fmaxf(fabsf(v[0]), fabsf(v[1]));
#pragma unroll
        for (int i = 2; i < 8; ++i) a = fmaxf(a, fabsf(v[i]));
        m = __float_as_uint(a);
    } else {
        m = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    }
    m = max(m, __shfl_xor_sync(kFull, m, 1));
    return max(m, __shfl_xor_sync(kFull, m, 2));
}

// Codes of 8 columns; r: their Philox call (not read when rounding to nearest).  Nearest: x / step + 1.5 *
// 2^23 leaves the integer nearest to x / step, ties to even, in the low byte (one rounding, the product
// is exact).  Random: x / step * 2^16 + 1.5 * 2^24 keeps 128 + x / step in units of 2^-15 in the
// fraction; doubled and increased by the 16-bit random number, bits 16..23 hold floor(128 + x / step + u).
template <bool RANDOM>
__device__ __forceinline__ uint2 codes8(const F2 (&h)[4], uint32_t e, const uint4& r) {
    const F2 inv = f2(inv_step(e));
    uint32_t t[8];
    const uint32_t word[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a, b;
        if constexpr (RANDOM) {
            split(fma2(mul2(h[i], inv), f2(65536.0f), f2(25165824.0f)), a, b);
            t[2 * i] = (__float_as_uint(a) << 1) + (word[i] & 0xFFFFu);
            t[2 * i + 1] = (__float_as_uint(b) << 1) + (word[i] >> 16);
        } else {
            split(fma2(h[i], inv, f2(12582912.0f)), a, b);
            t[2 * i] = __float_as_uint(a);
            t[2 * i + 1] = __float_as_uint(b);
        }
    }
    constexpr int B = RANDOM ? 2 : 0;
    constexpr uint32_t flip = RANDOM ? 0x80808080u : 0u;
    uint2 w = make_uint2(gather_bytes<B>(t[0], t[1], t[2], t[3]) ^ flip,
                         gather_bytes<B>(t[4], t[5], t[6], t[7]) ^ flip);
    if (e == 255u) w = make_uint2(0u, 0u);
    return w;
}

// Codes and exponent of 8 columns of a row from column c on; `live`: they are to be stored.
template <bool RANDOM>
__device__ __forceinline__ void save8(const F2 (&h)[4], bool live, uint32_t row, uint32_t c, int64_t pitch,
                                      int64_t epitch, const Rng& rng, int8_t* codes, uint8_t* exps) {
    const uint32_t e = exp_byte(block_top8(h, false));
    uint4 r = make_uint4(0u, 0u, 0u, 0u);
    if constexpr (RANDOM)
        r = gq::philox_row(gq::philox_group(c >> 3, rng.step_lo, rng.step_hi, rng.rk), row, rng.step_lo, rng.rk);
    const uint2 q = codes8<RANDOM>(h, e, r);
    if (!live) return;
    *reinterpret_cast<uint2*>(codes + static_cast<int64_t>(row) * pitch + c) = q;
    if ((c & (kBlk - 1)) == 0)
        exps[static_cast<int64_t>(row) * epitch + (c >> 5)] = static_cast<uint8_t>(e);
}

// The values of 8 codes as pairs.  A code byte plus 128 in the low byte of the fp32 number 2^23 gives
// 2^23 + 128 + code without a conversion instruction.
__device__ __forceinline__ void values8(uint2 w, uint32_t e, F2 (&v)[4]) {
    const F2 s = f2(step_of(e)), off = f2(-8388736.0f);
    const uint32_t u[2] = {w.x ^ 0x80808080u, w.y ^ 0x80808080u};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t q = u[i >> 1];
        const int k = 2 * (i & 1);
        v[i] = mul2(add2(f2(__uint_as_float(__byte_perm(q, 0x4B000000u, 0x7650 + k)),
                            __uint_as_float(__byte_perm(q, 0x4B000000u, 0x7651 + k))), off), s);
    }
}

// 8 elements as loaded (bf16: 4 words, fp32: 8), and as pairs of fp32.
template <typename T> struct Raw8 {
    uint32_t w[sizeof(T) * 2];
};
// 8 elements out of the words of the 16-byte granules that hold them: the first is m bytes behind the
// first granule's start (0 where ALIGNED); `left` of them are wanted, the others read as 0.
template <typename T, bool ALIGNED, int N>
__device__ __forceinline__ Raw8<T> shifted(uint32_t (&r)[N], uint32_t m, int left) {
    constexpr int W = 2 * sizeof(T);
    if constexpr (!ALIGNED) {
#pragma unroll
        for (int i = 0; i < W + 2; ++i) r[i] = (m & 8u) ? r[i + 2] : r[i];
#pragma unroll
        for (int i = 0; i < W + 1; ++i) r[i] = (m & 4u) ? r[i + 1] : r[i];
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < W; ++i) r[i] = __funnelshift_r(r[i], r[i + 1], (m & 2u) * 8u);
        }
    }
    if (left < 8) {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            if constexpr (sizeof(T) == 4) {
                if (i >= left) r[i] = 0u;
            } else {
                if (2 * i >= left) r[i] = 0u;
                else if (2 * i + 1 >= left) r[i] &= 0xFFFFu;
            }
        }
    }
    Raw8<T> w;
#pragma unroll
    for (int i = 0; i < W; ++i) w.w[i] = r[i];
    return w;
}
template <typename T>
__device__ __forceinline__ void pairs(const Raw8<T>& r, F2 (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4)
            v[i] = f2(__uint_as_float(r.w[2 * i]), __uint_as_float(r.w[2 * i + 1]));
        else
            v[i] = f2(__uint_as_float(r.w[i] << 16), __uint_as_float(r.w[i] & 0xFFFF0000u));
    }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const F2 (&v)[4]) {
    float o[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) split(v[i], o[2 * i], o[2 * i + 1]);
    store<T, 8, 16>(p, 0, 8, o);
}

// p + row * ld elements, in one multiplication: rows and their distance in bytes fit 32 bits each.
template <typename P>
__device__ __forceinline__ P* row_of(P* p, uint32_t row, uint32_t ld_bytes) {
    return reinterpret_cast<P*>(reinterpret_cast<uintptr_t>(p) + static_cast<uint64_t>(row) * ld_bytes);
}

// ---- host checks ---------------------------------------------------------------------------

inline bool mult(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline int elt_bytes(int dtype) { return dtype == GQ_F32 ? 4 : 2; }
inline bool in_type(int dtype) { return dtype == GQ_F32 || dtype == GQ_BF16; }

// A rows x cols matrix whose rows are ld elements apart, of an element type already checked.
inline bool matrix_ok(const void* p, int dtype, int64_t rows, int64_t cols, int64_t ld) {
    if (rows == 0) return true;
    return p && mult(p, elt_bytes(dtype)) && ld >= cols;
}
inline bool size_ok(int64_t rows, int64_t cols) {
    return rows >= 0 && rows < (int64_t(1) << 31) && cols >= 1 && cols < (int64_t(1) << 31) - 32;
}
// Codes and exponent bytes: 16-byte aligned (their row pitches are multiples of 16 bytes).
inline bool saved_ok(const void* codes, const void* exps) {
    return codes && exps && mult(codes, 16) && mult(exps, 16);
}
// Widest alignment (32, 16 or 0 bytes) that every row start of the matrix has.
inline int row_align(const void* p, int dtype, int64_t rows, int64_t ld) {
    const int64_t step = rows > 1 ? ld * elt_bytes(dtype) : 0;
    if (mult(p, 32) && step % 32 == 0) return 32;
    return mult(p, 16) && step % 16 == 0 ? 16 : 0;
}

// Blocks of a kernel that are resident on the whole GPU.  The query is remembered; the kernel's limit
// on shared memory is raised first where it asks for much.
template <typename K> int64_t resident_blocks(K kernel, int threads, size_t smem) {
    struct Entry {
        const void* fn;
        int dev, threads, blocks;
        size_t smem;
    };
    static std::mutex mu;
    static Entry table[512];
    static int used = 0;
    const void* fn = reinterpret_cast<const void*>(kernel);
    int dev = 0, nb = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) dev = 0;
    {
        std::lock_guard<std::mutex> lock(mu);
        for (int i = 0; i < used && nb == 0; ++i)
            if (table[i].fn == fn && table[i].dev == dev && table[i].threads == threads &&
                table[i].smem == smem)
                nb = table[i].blocks;
        if (nb == 0) {
            if (smem > 32 * 1024)
                cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     227 * 1024 - 4096);
            if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&nb, kernel, threads, smem) != cudaSuccess ||
                nb < 1)
                nb = 1;
            if (used < 512) table[used++] = Entry{fn, dev, threads, nb, smem};
        }
    }
    return static_cast<int64_t>(nb) * gqh::sm_count();
}

}  // namespace gqa
