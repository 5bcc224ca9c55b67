// gq_fp8.cuh -- matrices in 8-bit floating point: e4m3 codes with a power-of-two scale for each block of 128
// columns of a row, or of 128 x 128 elements.  Shared by gq_fp8.cu and gq_fp8_linear.cu.
//
// A block with largest magnitude a has the exponent byte E = min{ E >= 1 : a <= 448 * 2^(E - 127) }, 255
// if it holds a NaN or an infinity (its codes are then 0); an element stands for code * 2^(E - 127).  That is
// the form in which the tensor cores take scales, so a product needs no instruction for them, and a byte of
// 255 makes the sums that it takes part in NaN.  A power-of-two step costs at most one bit of the range that
// e4m3 has below its largest number, and no precision above that: codes are floating-point numbers.
//
// Exponents lie as tensor memory holds them: 512 bytes for 128 rows and 4 blocks (512 columns), the byte of
// row 32 j + r and block b at 16 r + 4 j + b, so that one bulk copy and one tcgen05.cp bring them there.
#pragma once
#include "gq_act.cuh"

namespace gqa {

constexpr int kScaled = 128;   // columns (and rows, of a tile) of one exponent
constexpr int kExpTile = 512;  // bytes of the exponents of 128 rows and 4 blocks

inline int64_t up_to(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
inline int64_t fp8_pitch(int64_t cols) { return up_to(cols, 16); }
__host__ __device__ inline int64_t exp_words(int64_t cols) { return (cols + 4 * kScaled - 1) / (4 * kScaled); }
inline int64_t exp_bytes(int64_t rows, int64_t cols) {
    return (rows + 127) / 128 * exp_words(cols) * kExpTile;
}

// With a = 1.f * 2^k, a <= 448 * 2^(k - 8) iff 1.f <= 1.75, that is iff the fraction field is at most 0x600000.
__device__ __forceinline__ uint32_t fp8_exp_byte(uint32_t top) {
    const int e = static_cast<int>((top + 0x1FFFFFu) >> 23) - 8;
    return top >= 0x7F800000u ? 255u : static_cast<uint32_t>(max(e, 1));
}
// Largest magnitude of 8 elements as fp32 bits, above infinity's where one is a NaN.
__device__ __forceinline__ uint32_t top8(const Raw8<float>& r) {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i += 2)
        asm("max.NaN.abs.f32 %0, %1, %2, %3;"
            : "=f"(a)
            : "f"(a), "f"(__uint_as_float(r.w[i])), "f"(__uint_as_float(r.w[i + 1])));
    return __float_as_uint(a);
}
// (bf16 magnitudes order like their bits)
__device__ __forceinline__ uint32_t max16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t top8(const Raw8<bf16>& r) {
    uint32_t m = r.w[0] & 0x7FFF7FFFu;
#pragma unroll
    for (int i = 1; i < 4; ++i) m = max16x2(m, r.w[i] & 0x7FFF7FFFu);
    return max(m & 0xFFFF0000u, m << 16);
}
// The same over the 16 lanes of a block, for R rows.
template <int R> __device__ __forceinline__ void tops(const Raw8<float> (&r)[R], uint32_t (&top)[R]) {
#pragma unroll
    for (int j = 0; j < R; ++j) {
        top[j] = top8(r[j]);
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) top[j] = max(top[j], __shfl_xor_sync(kFull, top[j], o));
    }
}
template <int R> __device__ __forceinline__ void tops(const Raw8<bf16> (&r)[R], uint32_t (&top)[R]) {
#pragma unroll
    for (int j = 0; j < R; j += 2) {  // two rows in a register
        uint32_t m = top8(r[j]) >> 16 | top8(r[j + 1]);
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) m = max16x2(m, __shfl_xor_sync(kFull, m, o));
        top[j] = m << 16;
        top[j + 1] = m & 0xFFFF0000u;
    }
}
// Codes of 8 elements times inv, the reciprocal of their block's step (products of at most 448, so nothing
// saturates): rounded to nearest even.
__device__ __forceinline__ uint2 fp8_codes8(const F2 (&h)[4], float inv) {
    uint32_t p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a, b;
        split(mul2(h[i], f2(inv)), a, b);
        uint16_t c;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(b), "f"(a));
        p[i] = c;
    }
    return make_uint2(p[0] | p[1] << 16, p[2] | p[3] << 16);
}
// Two codes (the low 16 bits of w) as fp32.
__device__ __forceinline__ F2 fp8_values2(uint32_t w) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(w)));
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
    return f2(v.x, v.y);
}

// A launch that may begin while the one before it on the stream ends.  Its kernel waits for that one
// (gq::pdl_wait) before it reads or writes memory, and lets a launch behind it begin only after.
template <typename... Params, typename... Args>
void launch_early(void (*k)(Params...), int64_t blocks, int threads, cudaStream_t st, const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, k, args...);
}

}  // namespace gqa
