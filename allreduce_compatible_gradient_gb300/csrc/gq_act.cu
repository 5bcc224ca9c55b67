// gq_act.cu -- 8-bit activation checkpoints and GELU over them (C ABI in include/gq.h).
//
// Every kernel here reads each input once and writes each output once: it is bound by memory.
// A thread takes 16 columns at a time (one 32-byte load of bf16, one 16-byte store of codes), two
// lanes share a block's exponent (one shuffle), and two such pieces are in flight per thread.
// Matrices whose rows are not 16-byte aligned take the V = 1 form: a warp holds one block, lane =
// column, so that its accesses stay contiguous whatever the alignment.
#include "gq_act.cuh"

#include <type_traits>

using namespace gqa;

namespace {

constexpr int kT = 256;  // threads per block
constexpr int kU = 2;    // pieces of V columns per thread

// ---- GELU ----------------------------------------------------------------------------------
// Normal distribution function at -|u|: q(|u|) = t P(t) exp(-u^2 / 2), t = 1 / (1 + p |u|).  The
// polynomials are least-maximum fits of erfc(z) exp(z^2) / 2 over 0 <= u <= 14 (computed for this
// file by iteratively reweighted least squares on Chebyshev nodes); relative error below 1.5e-7
// (8 coefficients, fp32 outputs) or 5e-6 (6 coefficients, bf16 outputs, whose own rounding is
// 2e-3).  One exponential serves the distribution and the density.
template <bool WIDE> struct Tail;
template <> struct Tail<true> {
    static constexpr float p = 0.30f;
    __device__ __forceinline__ static float poly(float t) {
        float a = 0.03567477688193321f;
        a = fmaf(a, t, -0.15720310807228088f);
        a = fmaf(a, t, 0.20635353028774261f);
        a = fmaf(a, t, -0.05368367210030556f);
        a = fmaf(a, t, 0.12856164574623108f);
        a = fmaf(a, t, 0.09991348534822464f);
        a = fmaf(a, t, 0.12075395882129669f);
        a = fmaf(a, t, 0.11962930113077164f);
        return a * t;
    }
};
template <> struct Tail<false> {
    static constexpr float p = 0.31f;
    __device__ __forceinline__ static float poly(float t) {
        float a = -0.07392916828393936f;
        a = fmaf(a, t, 0.1804504245519638f);
        a = fmaf(a, t, 0.01574462652206421f);
        a = fmaf(a, t, 0.13342982530593872f);
        a = fmaf(a, t, 0.1204412654042244f);
        a = fmaf(a, t, 0.1238607019186019f);
        return a * t;
    }
};

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Phi(u), and with DENSITY u phi(u) too.
template <bool WIDE, bool DENSITY>
__device__ __forceinline__ float normal_cdf(float u, float* u_phi) {
    const float t = rcp_fast(fmaf(fabsf(u), Tail<WIDE>::p, 1.0f));
    const float g = exp2_fast(u * u * -0.72134752044448170f);  // exp(-u^2 / 2)
    const float q = Tail<WIDE>::poly(t) * g;
    if constexpr (DENSITY) *u_phi = u * (g * 0.39894228040143268f);
    return u < 0.0f ? q : 1.0f - q;
}

// 1 / (1 + exp(-2 z)) with z = sqrt(2/pi) (u + 0.044715 u^3), which is (1 + tanh z) / 2; u is
// held to +-16, where it is 0 or 1 already and u^3 cannot overflow.
template <bool DENSITY>
__device__ __forceinline__ float tanh_cdf(float u, float* u_phi) {
    const float k = 0.79788456080286536f, b = 0.044715f;
    const float c = fminf(fmaxf(u, -16.0f), 16.0f);
    const float c2 = c * c;
    const float z = c * fmaf(c2, k * b, k);
    const float p = rcp_fast(1.0f + exp2_fast(z * -2.8853900817779268f));
    if constexpr (DENSITY) *u_phi = u * (2.0f * p * (1.0f - p)) * fmaf(c2, 3.0f * k * b, k);
    return p;
}

enum Op { kSave = 0, kGeluErf = GQ_GELU_ERF + 1, kGeluTanh = GQ_GELU_TANH + 1 };

template <int OP, bool WIDE>
__device__ __forceinline__ float gelu(float u) {
    return u * (OP == kGeluErf ? normal_cdf<WIDE, false>(u, nullptr) : tanh_cdf<false>(u, nullptr));
}

struct Flat {  // pieces of V columns of a row range, numbered row by row
    uint32_t pieces;
    Div per_row;
    int64_t cols, pitch, epitch;
};

// x -> codes and exponents (OP = kSave), or h = gelu(x) with or without them.
template <typename T, int V, int ALIGN, int OP, int RND>
__global__ void __launch_bounds__(kT) save_kernel(const T* __restrict__ x, int64_t ldx,
                                                  T* __restrict__ h, int64_t ldh, Flat f,
                                                  uint32_t row0, Rng rng,
                                                  int8_t* __restrict__ codes,
                                                  uint8_t* __restrict__ exps) {
    float v[kU][V];
    uint32_t row[kU], col[kU];
    bool live[kU];
#pragma unroll
    for (int k = 0; k < kU; ++k) {
        const uint32_t i = (blockIdx.x * kU + k) * kT + threadIdx.x;
        live[k] = i < f.pieces;
        const uint32_t r = quot(live[k] ? i : 0u, f.per_row);
        row[k] = row0 + r;
        col[k] = ((live[k] ? i : 0u) - r * f.per_row.d) * V;
        if (live[k]) {
            load<T, V, ALIGN>(x + static_cast<int64_t>(row[k]) * ldx, col[k], f.cols, v[k]);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) v[k][j] = 0.0f;
        }
    }
#pragma unroll
    for (int k = 0; k < kU; ++k) {
        if constexpr (RND >= 0)
            save<V, RND == 1>(v[k], live[k], row[k], col[k], f.pitch, f.epitch, rng, codes, exps);
        if constexpr (OP != kSave) {
            if (live[k]) {
                float o[V];
#pragma unroll
                for (int j = 0; j < V; ++j) o[j] = gelu<OP, sizeof(T) == 4>(v[k][j]);
                store<T, V, ALIGN>(h + static_cast<int64_t>(row[k]) * ldh, col[k], f.cols, o);
            }
        }
    }
}

// Codes and exponents -> values (OP = kSave), or with dy: du = dy gelu'(value) and, where h is
// given, h = gelu(value).
template <typename T, int V, int ALIGN, int OP>
__global__ void __launch_bounds__(kT) read_kernel(const int8_t* __restrict__ codes,
                                                  const uint8_t* __restrict__ exps, Flat f,
                                                  uint32_t row0, const T* __restrict__ dy,
                                                  int64_t lddy, T* __restrict__ du, int64_t lddu,
                                                  T* __restrict__ h, int64_t ldh) {
    float v[kU][V], g[kU][V];
    uint32_t row[kU], col[kU];
    bool live[kU];
#pragma unroll
    for (int k = 0; k < kU; ++k) {
        const uint32_t i = (blockIdx.x * kU + k) * kT + threadIdx.x;
        live[k] = i < f.pieces;
        if (!live[k]) continue;
        const uint32_t r = quot(i, f.per_row);
        row[k] = row0 + r;
        col[k] = (i - r * f.per_row.d) * V;
        saved<V>(codes + static_cast<int64_t>(row[k]) * f.pitch,
                 exps + static_cast<int64_t>(row[k]) * f.epitch, col[k], v[k]);
        if constexpr (OP != kSave)
            load<T, V, ALIGN>(dy + static_cast<int64_t>(row[k]) * lddy, col[k], f.cols, g[k]);
    }
#pragma unroll
    for (int k = 0; k < kU; ++k) {
        if (!live[k]) continue;
        if constexpr (OP == kSave) {
            store<T, V, ALIGN>(du + static_cast<int64_t>(row[k]) * lddu, col[k], f.cols, v[k]);
        } else if constexpr (!std::is_same<T, __half>::value) {
            float o[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float u_phi;
                const float p = OP == kGeluErf
                                    ? normal_cdf<sizeof(T) == 4, true>(v[k][j], &u_phi)
                                    : tanh_cdf<true>(v[k][j], &u_phi);
                g[k][j] *= p + u_phi;
                o[j] = v[k][j] * p;
            }
            store<T, V, ALIGN>(du + static_cast<int64_t>(row[k]) * lddu, col[k], f.cols, g[k]);
            if (h) store<T, V, ALIGN>(h + static_cast<int64_t>(row[k]) * ldh, col[k], f.cols, o);
        }
    }
}

// Runs one launch per range of rows whose pieces can be numbered in 31 bits.
template <int V, typename F>
gq_status over_rows(int64_t rows, int64_t cols, F launch) {
    Flat f;
    f.cols = cols;
    f.pitch = code_pitch(cols);
    f.epitch = exp_pitch(cols);
    const int64_t per_row = f.pitch / V;
    f.per_row = make_div(static_cast<uint32_t>(per_row));
    // the last block's numbers pass `pieces` by less than kT * kU
    const int64_t most = (int64_t(1) << 31) - kT * kU;
    const int64_t chunk = most / per_row;  // >= 1: a row has fewer than 2^31 - 32 columns
    if (chunk < 1) return GQ_ERR_INVALID;
    for (int64_t r0 = 0; r0 < rows; r0 += chunk) {
        const int64_t n = rows - r0 < chunk ? rows - r0 : chunk;
        f.pieces = static_cast<uint32_t>(n * per_row);
        launch(static_cast<unsigned>((n * per_row + kT * kU - 1) / (kT * kU)), f,
               static_cast<uint32_t>(r0));
        if (cudaGetLastError() != cudaSuccess) return GQ_ERR_CUDA;
    }
    return GQ_OK;
}

template <typename T, int V, int ALIGN, int OP>
gq_status run_save(const void* x, int64_t ldx, void* h, int64_t ldh, int64_t rows, int64_t cols,
                   int rnd, const Rng& rng, int8_t* codes, uint8_t* exps, cudaStream_t st) {
    const T* xp = static_cast<const T*>(x);
    T* hp = static_cast<T*>(h);
    return over_rows<V>(rows, cols, [&](unsigned grid, const Flat& f, uint32_t row0) {
        if (rnd == GQ_ACT_RANDOM)
            save_kernel<T, V, ALIGN, OP, 1>
                <<<grid, kT, 0, st>>>(xp, ldx, hp, ldh, f, row0, rng, codes, exps);
        else if (rnd == GQ_ACT_NEAREST)
            save_kernel<T, V, ALIGN, OP, 0>
                <<<grid, kT, 0, st>>>(xp, ldx, hp, ldh, f, row0, rng, codes, exps);
        else if constexpr (OP != kSave)
            save_kernel<T, V, ALIGN, OP, -1>
                <<<grid, kT, 0, st>>>(xp, ldx, hp, ldh, f, row0, rng, codes, exps);
    });
}

template <int OP>
gq_status any_save(const void* x, int dtype, int64_t ldx, void* h, int64_t ldh, int64_t rows,
                   int64_t cols, int rnd, const Rng& rng, int8_t* codes, uint8_t* exps,
                   cudaStream_t st) {
    int al = row_align(x, dtype, rows, ldx);
    if (OP != kSave) al = min(al, row_align(h, dtype, rows, ldh));
#define GQA_RUN(T)                                                                               \
    (al == 32 ? run_save<T, 16, 32, OP>(x, ldx, h, ldh, rows, cols, rnd, rng, codes, exps, st)   \
     : al == 16 ? run_save<T, 16, 16, OP>(x, ldx, h, ldh, rows, cols, rnd, rng, codes, exps, st) \
                : run_save<T, 1, 0, OP>(x, ldx, h, ldh, rows, cols, rnd, rng, codes, exps, st))
    return dtype == GQ_F32 ? GQA_RUN(float) : GQA_RUN(bf16);
#undef GQA_RUN
}

template <typename T, int V, int ALIGN, int OP>
gq_status run_read(const int8_t* codes, const uint8_t* exps, int64_t rows, int64_t cols,
                   const void* dy, int64_t lddy, void* du, int64_t lddu, void* h, int64_t ldh,
                   cudaStream_t st) {
    return over_rows<V>(rows, cols, [&](unsigned grid, const Flat& f, uint32_t row0) {
        read_kernel<T, V, ALIGN, OP><<<grid, kT, 0, st>>>(
            codes, exps, f, row0, static_cast<const T*>(dy), lddy, static_cast<T*>(du), lddu,
            static_cast<T*>(h), ldh);
    });
}

template <typename T, int OP>
gq_status any_read(int al, const int8_t* codes, const uint8_t* exps, int64_t rows, int64_t cols,
                   const void* dy, int64_t lddy, void* du, int64_t lddu, void* h, int64_t ldh,
                   cudaStream_t st) {
    return al == 32   ? run_read<T, 16, 32, OP>(codes, exps, rows, cols, dy, lddy, du, lddu, h, ldh, st)
           : al == 16 ? run_read<T, 16, 16, OP>(codes, exps, rows, cols, dy, lddy, du, lddu, h, ldh, st)
                      : run_read<T, 1, 0, OP>(codes, exps, rows, cols, dy, lddy, du, lddu, h, ldh, st);
}

}  // namespace

extern "C" {

int64_t gq_act_exp_pitch(int64_t cols) { return cols < 1 ? 0 : exp_pitch(cols); }

gq_status gq_act_quantize(const void *x, int dtype, int64_t rows, int64_t cols, int64_t ldx,
                          int rounding, uint64_t seed, uint64_t step, int8_t *codes,
                          uint8_t *exps, void *stream) {
    if (!in_type(dtype) || !size_ok(rows, cols)) return GQ_ERR_INVALID;
    if (rounding != GQ_ACT_NEAREST && rounding != GQ_ACT_RANDOM) return GQ_ERR_INVALID;
    if (!matrix_ok(x, dtype, rows, cols, ldx)) return GQ_ERR_INVALID;
    if (rows == 0) return GQ_OK;
    if (!saved_ok(codes, exps)) return GQ_ERR_INVALID;
    return any_save<kSave>(x, dtype, ldx, nullptr, 0, rows, cols, rounding, make_rng(seed, step),
                           codes, exps, static_cast<cudaStream_t>(stream));
}

gq_status gq_act_dequantize(const int8_t *codes, const uint8_t *exps, int64_t rows, int64_t cols,
                            void *out, int out_dtype, int64_t ldout, void *stream) {
    if ((!in_type(out_dtype) && out_dtype != GQ_F16) || !size_ok(rows, cols)) return GQ_ERR_INVALID;
    if (!matrix_ok(out, out_dtype, rows, cols, ldout)) return GQ_ERR_INVALID;
    if (rows == 0) return GQ_OK;
    if (!saved_ok(codes, exps)) return GQ_ERR_INVALID;
    const int al = row_align(out, out_dtype, rows, ldout);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (out_dtype == GQ_F32)
        return any_read<float, kSave>(al, codes, exps, rows, cols, nullptr, 0, out, ldout, nullptr, 0, st);
    if (out_dtype == GQ_BF16)
        return any_read<bf16, kSave>(al, codes, exps, rows, cols, nullptr, 0, out, ldout, nullptr, 0, st);
    return any_read<__half, kSave>(al, codes, exps, rows, cols, nullptr, 0, out, ldout, nullptr, 0, st);
}

gq_status gq_gelu_forward(const void *u, int dtype, int64_t rows, int64_t cols, int64_t ldu,
                          int form, void *h, int64_t ldh, int rounding, uint64_t seed,
                          uint64_t step, int8_t *codes, uint8_t *exps, void *stream) {
    if (!in_type(dtype) || !size_ok(rows, cols)) return GQ_ERR_INVALID;
    if (form != GQ_GELU_ERF && form != GQ_GELU_TANH) return GQ_ERR_INVALID;
    if (rounding != GQ_ACT_NEAREST && rounding != GQ_ACT_RANDOM) return GQ_ERR_INVALID;
    if (!matrix_ok(u, dtype, rows, cols, ldu) || !matrix_ok(h, dtype, rows, cols, ldh))
        return GQ_ERR_INVALID;
    if (rows == 0) return GQ_OK;
    if ((codes || exps) && !saved_ok(codes, exps)) return GQ_ERR_INVALID;
    const int rnd = codes ? rounding : -1;  // no checkpoint asked for
    const Rng rng = make_rng(seed, step);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return form == GQ_GELU_ERF
               ? any_save<kGeluErf>(u, dtype, ldu, h, ldh, rows, cols, rnd, rng, codes, exps, st)
               : any_save<kGeluTanh>(u, dtype, ldu, h, ldh, rows, cols, rnd, rng, codes, exps, st);
}

gq_status gq_gelu_backward(const void *dh, int dtype, int64_t rows, int64_t cols, int64_t lddh,
                           const int8_t *codes, const uint8_t *exps, int form, void *du,
                           int64_t lddu, void *h, int64_t ldh, void *stream) {
    if (!in_type(dtype) || !size_ok(rows, cols)) return GQ_ERR_INVALID;
    if (form != GQ_GELU_ERF && form != GQ_GELU_TANH) return GQ_ERR_INVALID;
    if (!matrix_ok(dh, dtype, rows, cols, lddh) || !matrix_ok(du, dtype, rows, cols, lddu))
        return GQ_ERR_INVALID;
    if (h && !matrix_ok(h, dtype, rows, cols, ldh)) return GQ_ERR_INVALID;
    if (rows == 0) return GQ_OK;
    if (!saved_ok(codes, exps)) return GQ_ERR_INVALID;
    int al = min(row_align(dh, dtype, rows, lddh), row_align(du, dtype, rows, lddu));
    if (h) al = min(al, row_align(h, dtype, rows, ldh));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
#define GQA_READ(T, OP) any_read<T, OP>(al, codes, exps, rows, cols, dh, lddh, du, lddu, h, ldh, st)
    if (dtype == GQ_F32)
        return form == GQ_GELU_ERF ? GQA_READ(float, kGeluErf) : GQA_READ(float, kGeluTanh);
    return form == GQ_GELU_ERF ? GQA_READ(bf16, kGeluErf) : GQA_READ(bf16, kGeluTanh);
#undef GQA_READ
}

}  // extern "C"
