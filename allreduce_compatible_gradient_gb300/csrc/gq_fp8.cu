// gq_fp8.cu -- a matrix into 8-bit floating point with a scale for each block of 128, and back (C ABI in
// include/gq.h; the format is described in gq_fp8.cuh).
//
// Both directions are one pass over the data, bound by memory: bytes in flight and few instructions.  32,768 x
// 4,096 bf16: 67 us there and 60 back, 6.0 and 6.6 TB/s; a 4,096 x 4,096 fp32 weight 15 and 9 us.
#include "gq_fp8.cuh"

using namespace gqa;

namespace {

// The granules that hold 8 elements at p: nothing is read where left <= 0, and no granule behind the last one
// with an element that is wanted.
template <typename T, bool ALIGNED> struct Granules {
    static constexpr int P = sizeof(T) / 2 + (ALIGNED ? 0 : 1);
    uint32_t w[4 * P];
    uint32_t m;
    __device__ __forceinline__ void fetch(const T* p, int left) {
        const uint8_t* q = reinterpret_cast<const uint8_t*>(p);
        m = ALIGNED ? 0u : static_cast<uint32_t>(reinterpret_cast<uintptr_t>(q)) & 15u;
        const int bytes = left > 0 ? static_cast<int>(m) + min(left, 8) * static_cast<int>(sizeof(T)) : 0;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            // an ordinary load: a read-only one may pass the wait for the launch before, whose work x may be
            const uint4 g = 16 * i < bytes ? reinterpret_cast<const uint4*>(q - m)[i] : make_uint4(0u, 0u, 0u, 0u);
            w[4 * i] = g.x; w[4 * i + 1] = g.y; w[4 * i + 2] = g.z; w[4 * i + 3] = g.w;
        }
    }
    __device__ __forceinline__ Raw8<T> wanted(int left) {
        return shifted<T, ALIGNED>(w, m, min(max(left, 0), 8));
    }
};

// One exponent per row and 128 columns.  A warp's task is rows r, r + 32, r + 64, r + 96 of 128 and 256 columns:
// 16 lanes hold a block, and the 8 exponents lie in 16 bytes.  The next task's loads are on their way while
// one is computed.
template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(256)
    rows_kernel(const T* x, int64_t ld, int64_t rows, int64_t cols, int64_t pitch, uint32_t across,
                Div by, uint32_t tasks, uint8_t* codes, uint8_t* exps) {
    gq::pdl_wait();
    gq::pdl_launch_dependents();  // a product that follows waits before it reads the codes; all before has ended
    const int lane = threadIdx.x & 31;
    const uint32_t stride = gridDim.x * 8;
    Granules<T, ALIGNED> g[4];
    // neighbouring warps take neighbouring columns of the same rows
    auto fetch = [&](uint32_t t) {
        const uint32_t q = across > 1 ? quot(t, by) : t;
        const int64_t r = static_cast<int64_t>(q >> 5) * 128 + (q & 31);
        const int64_t c = static_cast<int64_t>(t - q * across) * 256 + lane * 8;
        const int left = static_cast<int>(min(cols - c, int64_t(8)));
#pragma unroll
        for (int j = 0; j < 4; ++j) g[j].fetch(x + (r + 32 * j) * ld + c, r + 32 * j < rows ? left : 0);
    };
    uint32_t t = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (t < tasks) fetch(t);
    for (; t < tasks; t += stride) {
        const uint32_t q = across > 1 ? quot(t, by) : t;
        const int64_t r = static_cast<int64_t>(q >> 5) * 128 + (q & 31);
        const uint32_t piece = t - q * across;
        const int64_t c = static_cast<int64_t>(piece) * 256 + lane * 8;
        const int left = static_cast<int>(min(cols - c, int64_t(8)));
        Raw8<T> now[4];
        uint32_t top[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) now[j] = g[j].wanted(r + 32 * j < rows ? left : 0);
        if (t < tasks - min(stride, tasks)) fetch(t + stride);
        tops<4>(now, top);
        uint32_t e4 = 0u;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t e = fp8_exp_byte(top[j]);
            F2 v[4];
            pairs(now[j], v);
            uint2 w = fp8_codes8(v, inv_step(e));
            if (e == 255u) w = make_uint2(0u, 0u);
            if (r + 32 * j < rows && c < pitch) *reinterpret_cast<uint2*>(codes + (r + 32 * j) * pitch + c) = w;
            e4 |= e << (8 * j);
        }
        // lane j < 4: row j's two blocks
        const uint32_t other = __shfl_xor_sync(kFull, e4, 16);
        if (lane < 4)
            *reinterpret_cast<uint16_t*>(exps + (static_cast<int64_t>(q >> 5) * ((across + 1) / 2) + piece / 2) * kExpTile +
                                         (q & 31) * 16 + lane * 4 + (piece & 1) * 2) =
                static_cast<uint16_t>(__byte_perm(e4, other, lane | (4 + lane) << 4));
    }
}

// One exponent per 128 x 128 elements, written for every row (exps) and every column (exps_t, nullable).
// Block = one tile, 32 elements per thread.
template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(512)
    tiles_kernel(const T* x, int64_t ld, int64_t rows, int64_t cols, int64_t pitch, uint32_t across,
                 uint8_t* codes, uint8_t* exps, uint8_t* exps_t) {
    gq::pdl_wait();
    gq::pdl_launch_dependents();
    __shared__ uint32_t most[16];
    const int64_t tr = blockIdx.x / across, tc = blockIdx.x % across;
    const int64_t r0 = tr * 128 + (threadIdx.x >> 4), c = tc * 128 + (threadIdx.x & 15) * 8;
    const int left = static_cast<int>(min(cols - c, int64_t(8)));
    Granules<T, ALIGNED> g[4];
    Raw8<T> now[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) g[i].fetch(x + (r0 + 32 * i) * ld + c, r0 + 32 * i < rows ? left : 0);
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        now[i] = g[i].wanted(r0 + 32 * i < rows ? left : 0);
        m = max(m, top8(now[i]));
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) m = max(m, __shfl_xor_sync(kFull, m, o));
    if ((threadIdx.x & 31) == 0) most[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, most[i]);
    const uint32_t e = fp8_exp_byte(m);
    const float inv = inv_step(e);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        F2 v[4];
        pairs(now[i], v);
        uint2 q = fp8_codes8(v, inv);
        if (e == 255u) q = make_uint2(0u, 0u);
        if (r0 + 32 * i < rows && c < pitch)
            *reinterpret_cast<uint2*>(codes + (r0 + 32 * i) * pitch + c) = q;
    }
    const int k = threadIdx.x & 127;  // 4-byte places of 128 rows, each for 4 blocks
    if (threadIdx.x < 128)
        exps[(tr * exp_words(cols) + (tc >> 2)) * kExpTile + k * 4 + (tc & 3)] = static_cast<uint8_t>(e);
    else if (threadIdx.x < 256 && exps_t)
        exps_t[(tc * exp_words(rows) + (tr >> 2)) * kExpTile + k * 4 + (tr & 3)] = static_cast<uint8_t>(e);
}

// 16 columns of a row per thread, which are in one block.
template <typename O, int ALIGN>
__global__ void __launch_bounds__(256)
    values_kernel(const uint8_t* codes, const uint8_t* exps, int64_t cols, int64_t pitch, int64_t words,
                  int64_t pieces, uint32_t across, Div by, O* out, int64_t ld) {
    constexpr int B = 2;
    gq::pdl_wait();
    const int64_t stride = static_cast<int64_t>(gridDim.x) * 256;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; t < pieces; t += B * stride) {
        uint4 q[B];
        uint32_t e[B];
        int64_t row[B], c[B];
#pragma unroll
        for (int k = 0; k < B; ++k) {
            const int64_t at = t + k * stride;
            if (at >= pieces) break;
            if (pieces <= INT32_MAX) {
                const uint32_t n = across > 1 ? quot(static_cast<uint32_t>(at), by) : static_cast<uint32_t>(at);
                row[k] = n;
                c[k] = static_cast<int64_t>(static_cast<uint32_t>(at) - n * across) * 16;
            } else {
                row[k] = at / across;
                c[k] = at % across * 16;
            }
            q[k] = *reinterpret_cast<const uint4*>(codes + row[k] * pitch + c[k]);
            e[k] = exps[((row[k] >> 7) * words + (c[k] >> 9)) * kExpTile + (row[k] & 31) * 16 + (row[k] >> 5 & 3) * 4 +
                        (c[k] >> 7 & 3)];
        }
#pragma unroll
        for (int k = 0; k < B; ++k) {
            if (t + k * stride >= pieces) break;
            const uint32_t w[4] = {q[k].x, q[k].y, q[k].z, q[k].w};
            const F2 s = f2(step_of(e[k]));
            float v[16];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const F2 p = mul2(fp8_values2(w[i >> 1] >> (16 * (i & 1))), s);
                split(p, v[2 * i], v[2 * i + 1]);
            }
            O* to = out + row[k] * ld;
            if constexpr (ALIGN > 0) {
                store<O, 16, ALIGN>(to, c[k], cols, v);
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (c[k] + i < cols) down(v[i], to[c[k] + i]);
            }
        }
    }
}

Div div_by(int64_t d) { return d > 1 ? make_div(static_cast<uint32_t>(d)) : Div{1, 0, 0}; }

template <typename T>
gq_status quantize(const T* x, int64_t rows, int64_t cols, int64_t ld, bool tiles, uint8_t* codes,
                   uint8_t* exps, uint8_t* exps_t, cudaStream_t st) {
    const int64_t pitch = fp8_pitch(cols);
    const bool aligned = row_align(x, sizeof(T) == 4 ? GQ_F32 : GQ_BF16, rows, ld) != 0;
    if (tiles) {
        const int64_t across = (cols + 127) / 128, n = (rows + 127) / 128 * across;
        auto k = aligned ? tiles_kernel<T, true> : tiles_kernel<T, false>;
        launch_early(k, n, 512, st, x, ld, rows, cols, pitch, static_cast<uint32_t>(across), codes, exps, exps_t);
        return gqh::launch_status();
    }
    const int64_t across = (cols + 255) / 256, tasks = (rows + 127) / 128 * 32 * across;
    if (tasks >= int64_t(1) << 31) return GQ_ERR_INVALID;
    auto k = aligned ? rows_kernel<T, true> : rows_kernel<T, false>;
    const int64_t most = resident_blocks(k, 256, 0), need = (tasks + 7) / 8;
    launch_early(k, need < most ? need : most, 256, st, x, ld, rows, cols, pitch, static_cast<uint32_t>(across),
                 div_by(across), static_cast<uint32_t>(tasks), codes, exps);
    return gqh::launch_status();
}

template <typename O>
gq_status dequantize(const uint8_t* codes, const uint8_t* exps, int64_t rows, int64_t cols, O* out, int dtype,
                     int64_t ld, cudaStream_t st) {
    const int64_t across = (cols + 15) / 16, pieces = rows * across;
    const int a = row_align(out, dtype, rows, ld);
    auto k = a == 32 ? values_kernel<O, 32> : a == 16 ? values_kernel<O, 16> : values_kernel<O, 0>;
    const int64_t most = resident_blocks(k, 256, 0), need = (pieces + 255) / 256;
    launch_early(k, need < most ? need : most, 256, st, codes, exps, cols, fp8_pitch(cols), exp_words(cols), pieces,
                 static_cast<uint32_t>(across), div_by(across), out, ld);
    return gqh::launch_status();
}

}  // namespace

extern "C" {

int64_t gq_fp8_code_pitch(int64_t cols) { return cols < 1 ? 0 : fp8_pitch(cols); }

size_t gq_fp8_exp_bytes(int64_t rows, int64_t cols) {
    return !size_ok(rows, cols) ? 0 : static_cast<size_t>(exp_bytes(rows, cols));
}

gq_status gq_fp8_quantize(const void *x, int dtype, int64_t rows, int64_t cols, int64_t ldx, int block_rows,
                          uint8_t *codes, uint8_t *exps, uint8_t *exps_t, void *stream) {
    if (!in_type(dtype) || !size_ok(rows, cols) || !matrix_ok(x, dtype, rows, cols, ldx)) return GQ_ERR_INVALID;
    if ((block_rows != 1 && block_rows != 128) || (block_rows == 1 && exps_t)) return GQ_ERR_INVALID;
    if ((rows + 127) / 128 * ((cols + 127) / 128) >= (int64_t(1) << 31)) return GQ_ERR_INVALID;
    if (rows == 0) return GQ_OK;
    if (!saved_ok(codes, exps) || !mult(exps_t, 16)) return GQ_ERR_INVALID;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return dtype == GQ_F32 ? quantize(static_cast<const float*>(x), rows, cols, ldx, block_rows > 1, codes, exps,
                                      exps_t, st)
                           : quantize(static_cast<const bf16*>(x), rows, cols, ldx, block_rows > 1, codes, exps,
                                      exps_t, st);
}

gq_status gq_fp8_dequantize(const uint8_t *codes, const uint8_t *exps, int64_t rows, int64_t cols, void *out,
                            int out_dtype, int64_t ldout, void *stream) {
    if ((!in_type(out_dtype) && out_dtype != GQ_F16) || !size_ok(rows, cols) ||
        !matrix_ok(out, out_dtype, rows, cols, ldout))
        return GQ_ERR_INVALID;
    if (rows == 0) return GQ_OK;
    if (!saved_ok(codes, exps)) return GQ_ERR_INVALID;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (out_dtype == GQ_F32)
        return dequantize(codes, exps, rows, cols, static_cast<float*>(out), out_dtype, ldout, st);
    if (out_dtype == GQ_BF16)
        return dequantize(codes, exps, rows, cols, static_cast<bf16*>(out), out_dtype, ldout, st);
    return dequantize(codes, exps, rows, cols, static_cast<__half*>(out), out_dtype, ldout, st);
}

}  // extern "C"
