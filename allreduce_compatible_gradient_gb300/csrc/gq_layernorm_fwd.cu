// gq_layernorm_fwd.cu -- layer norm forward, with or without an 8-bit checkpoint of the normalised rows.
#include "gq_layernorm.cuh"

using namespace gqa;

namespace {

// Rows of more columns than the held form takes: a block per row, thread t of its `threads` takes the
// pieces of 8 columns t, t + threads, ...: the first VPT of them in registers.  Warps go on as long as one
// of their lanes has a column, so that all take part in the checkpoint's reductions.  Rows that are not
// aligned take the same pieces by granules (2,730 x 12,289 bf16 with random codes: 85 us, element by
// element 218); two blocks per SM (one, with 84 registers a thread: 111).
template <typename T, bool ALIGNED, int VPT, int RND>
__global__ void __launch_bounds__(512, 2)
    forward_kernel(const T* __restrict__ x, int64_t ldx, Shape s, Affine af, float eps,
                   T* __restrict__ y, int64_t ldy, float* __restrict__ mean_out,
                   float* __restrict__ rstd_out, int8_t* __restrict__ codes,
                   uint8_t* __restrict__ exps, Rng rng) {
    __shared__ float buf[2][32][1];
    __shared__ float squares[ALIGNED ? 1 : 16 * kSquare];
    const int threads = blockDim.x, t = threadIdx.x, lane = t & 31;
    float* const square = squares + (ALIGNED ? 0 : t / 32 * kSquare);
    const int64_t row = blockIdx.x;
    const T* xr = x + row * ldx;
    T* yr = y + row * ldy;
    const int64_t step = static_cast<int64_t>(threads) * 8;
    const int64_t mine = (t - lane) * 8;           // the warp's first column
    const int64_t beyond = step * VPT + mine;  // that of its first piece that is not in registers

    F2 v[VPT][4];
    F2 acc = f2(0.0f);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        load8<T, ALIGNED>(xr, k * step + t * 8, s.cols, v[k]);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc = add2(acc, v[k][i]);
    }
    for (int64_t c0 = beyond; c0 < s.cols; c0 += step) {
        F2 z[4];
        load8<T, ALIGNED>(xr, c0 + lane * 8, s.cols, z);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc = add2(acc, z[i]);
    }
    float sum[1] = {sum2(acc)};
    row_sum(sum, buf[0], threads);
    const float mean = sum[0] * s.inv_cols;

    auto centre = [&](F2 (&z)[4], int64_t c) {
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = add2(z[i], f2(-mean));
        cut8(z, left_of(c, s.cols));
    };
    acc = f2(0.0f);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        centre(v[k], k * step + t * 8);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc = fma2(v[k][i], v[k][i], acc);
    }
    for (int64_t c0 = beyond; c0 < s.cols; c0 += step) {
        F2 z[4];
        load8<T, ALIGNED>(xr, c0 + lane * 8, s.cols, z);
        centre(z, c0 + lane * 8);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc = fma2(z[i], z[i], acc);
    }
    float sq[1] = {sum2(acc)};
    row_sum(sq, buf[1], threads);
    const float rstd = rsqrtf(__fmul_rn(sq[0], s.inv_cols) + eps);  // within 2 units
    if (t == 0) {
        mean_out[row] = mean;
        rstd_out[row] = rstd;
    }

    auto finish = [&](int64_t first, F2 (&z)[4]) {  // z: x - mean
        const int64_t c = first + lane * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = mul2(z[i], f2(rstd));
        if constexpr (RND >= 0)
            save8<RND == 1>(z, c < s.pitch, static_cast<uint32_t>(row), static_cast<uint32_t>(c), s.pitch,
                            s.epitch, rng, codes, exps);
        F2 w[4], b[4];
        vec8(af.w, af.wide, af.aligned, 1.0f, c, s.cols, w);
        vec8(af.b, af.wide, af.aligned, 0.0f, c, s.cols, b);
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = fma2(z[i], w[i], b[i]);
        put_row<T, ALIGNED>(yr, c, first, s.cols, square, z);
    };
#pragma unroll
    for (int k = 0; k < VPT; ++k)
        if (k * step + mine < s.cols) finish(k * step + mine, v[k]);
    for (int64_t c0 = beyond; c0 < s.cols; c0 += step) {
        F2 z[4];
        load8<T, ALIGNED>(xr, c0 + lane * 8, s.cols, z);
        centre(z, c0 + lane * 8);
        finish(c0, z);
    }
}

template <typename T, bool ALIGNED, int VPT, int RND, int W, int MOST>
__global__ void __launch_bounds__(MOST, MOST == 256 ? (VPT == 1 ? 3 : 2) : 1)
    forward_rows(const T* __restrict__ x, HeldArgs a, Affine af, float eps, T* __restrict__ y,
                 float* __restrict__ mean_out, float* __restrict__ rstd_out,
                 int8_t* __restrict__ codes, uint8_t* __restrict__ exps, Rng rng) {
    __shared__ alignas(16) float buf[2][kSlots];
    extern __shared__ __align__(16) uint8_t ring[];
    const int warp = threadIdx.x >> 5;
    const int group = W == kMany ? 0 : warp / a.wpr, wr = warp - group * a.wpr;
    const uint32_t t = wr * 32 + (threadIdx.x & 31), apart = a.wpr * 256;
    for (int i = threadIdx.x; i < 2 * kSlots; i += blockDim.x) (&buf[0][0])[i] = 0.0f;
    __syncthreads();
    uint32_t row = blockIdx.x * a.groups + group;
    if (row >= a.rows) return;  // whole groups
    float* const slots = &buf[0][W == kFour ? group * 4 : 0];
    bool in[VPT], padded[VPT];  // columns of the matrix; of the codes
    uint32_t col[VPT];
    int left[VPT];  // elements of the row from col on, 0 behind the last column
    F2 w[VPT][4], b[VPT][4], mask[VPT][ALIGNED ? 1 : 4];
    gq::PhiloxGroup pg[VPT];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const uint32_t c = k * apart + t * 8;
        in[k] = c < a.cols;
        padded[k] = c < a.pitch;
        col[k] = in[k] ? c : 0u;
        left[k] = in[k] ? static_cast<int>(a.cols - c) : 0;
#pragma unroll
        for (int i = 0; i < (ALIGNED ? 1 : 4); ++i)
            mask[k][i] = f2(c + 2 * i < a.cols ? 1.0f : 0.0f,
                            c + 2 * i + (ALIGNED ? 0 : 1) < a.cols ? 1.0f : 0.0f);
        vec8(af.w, af.wide, af.aligned, 1.0f, c, a.cols, w[k]);
        vec8(af.b, af.wide, af.aligned, 0.0f, c, a.cols, b[k]);
        if constexpr (RND == 1)
            pg[k] = gq::philox_group(c >> 3, rng.step_lo, rng.step_hi, rng.rk);
    }
    using R = Ring<T, ALIGNED>;
    constexpr int P = R::kPieces, D = R::kSlots;
    const uint32_t plane = blockDim.x * 16, slot_bytes = plane * VPT * P;
    const uint32_t base = gq::smem_u32(ring) + threadIdx.x * 16;
    float* square = reinterpret_cast<float*>(ring + D * slot_bytes) + warp * kSquare;
    uint32_t ahead = row, turn = 0;
    auto fetch = [&]() {  // (the last row again where there is none)
        const T* p = row_of(x, min(ahead, a.rows - 1), a.in);
#pragma unroll
        for (int k = 0; k < VPT; ++k)
            R::fetch(base + (turn & (D - 1)) * slot_bytes + k * P * plane, plane, p + col[k], left[k]);
        copy_commit();
        ahead += a.stride;
        ++turn;
    };
#pragma unroll
    for (int d = 0; d < D - 1; ++d) fetch();
    for (; row < a.rows; row += a.stride) {
        F2 v[VPT][4];
        fetch();
        copy_wait<D>();
        F2 sum = f2(0.0f);
        const uint8_t* slot = ring + (turn & (D - 1)) * slot_bytes + threadIdx.x * 16;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            R::read(slot + k * P * plane, plane, row_of(x, row, a.in) + col[k], left[k], v[k]);
#pragma unroll
            for (int i = 0; i < 4; ++i) sum = add2(sum, v[k][i]);
        }
        float m[1] = {sum2(sum)};
        group_sum<W>(m, slots, wr, a.wpr, group);
        const float mean = m[0] * a.inv_cols;
        F2 sq = f2(0.0f);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const F2 less = f2(-mean);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const F2 m1 = mask[k][ALIGNED ? 0 : i];
                v[k][i] = fma2(v[k][i], m1, mul2(m1, less));
                sq = fma2(v[k][i], v[k][i], sq);
            }
        }
        float q[1] = {sum2(sq)};
        group_sum<W>(q, slots + kSlots, wr, a.wpr, group);
        // not contracted with the sum: y is the same with and without a checkpoint
        const float var = __fmul_rn(q[0], a.inv_cols);
        const float rstd = rsqrtf(var + eps);
        if (t == 0) {
            mean_out[row] = mean;
            rstd_out[row] = rstd;
        }
        const F2 rs = f2(rstd);
        T* py = row_of(y, row, a.out);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[k][i] = mul2(v[k][i], rs);
            if constexpr (RND >= 0) {
                const float inf = __uint_as_float(0x7F800000u);
                const uint32_t e = exp_byte(block_top8(v[k], var < inf && rstd < inf));
                uint4 r = make_uint4(0u, 0u, 0u, 0u);
                if constexpr (RND == 1) r = gq::philox_row(pg[k], row, rng.step_lo, rng.rk);
                const uint2 cc = codes8<RND == 1>(v[k], e, r);
                const uint32_t c = k * apart + t * 8;
                if (padded[k]) {
                    *reinterpret_cast<uint2*>(row_of(codes, row, a.pitch) + c) = cc;
                    if ((t & 3) == 0) row_of(exps, row, a.epitch)[c >> 5] = static_cast<uint8_t>(e);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) v[k][i] = fma2(v[k][i], w[k][i], b[k][i]);
            put8<T, ALIGNED>(py, col[k], in[k], k * apart + wr * 256, a.cols, square, v[k]);
        }
    }
    copy_all();
}

// ---- host ----------------------------------------------------------------------------------

template <typename T>
struct ForwardCall {
    const T* x;
    int64_t ldx;
    Shape s;
    Affine af;
    float eps;
    T* y;
    int64_t ldy;
    float *mean, *rstd;
    int8_t* codes;
    uint8_t* exps;
    Rng rng;
    cudaStream_t st;
};

template <typename T, bool ALIGNED, int VPT, int RND>
gq_status forward_generic(const ForwardCall<T>& a) {
    const int threads = threads_for(a.s.cols, 8 * VPT, 128, 512);
    forward_kernel<T, ALIGNED, VPT, RND><<<static_cast<unsigned>(a.s.rows), threads, 0, a.st>>>(
        a.x, a.ldx, a.s, a.af, a.eps, a.y, a.ldy, a.mean, a.rstd, a.codes, a.exps, a.rng);
    return gqh::launch_status();
}
template <typename T, bool ALIGNED, int RND> struct ForwardHeld {
    const ForwardCall<T>& a;
    const Held& h;
    template <int VPT, int W, int MOST> gq_status operator()() const {
        using R = Ring<T, ALIGNED>;
        auto k = forward_rows<T, ALIGNED, VPT, RND, W, MOST>;
        const size_t smem = static_cast<size_t>(R::kSlots) * h.threads * VPT * 16 * R::kPieces +
                            (ALIGNED ? 0 : h.threads / 32 * kSquare * sizeof(float));
        const int grid = wave(resident_blocks(k, h.threads, smem), (a.s.rows + h.groups - 1) / h.groups);
        const HeldArgs ha = held_args(h, grid, a.s, a.ldx * sizeof(T), 0, a.ldy * sizeof(T));
        k<<<grid, h.threads, smem, a.st>>>(a.x, ha, a.af, a.eps, a.y, a.mean, a.rstd, a.codes, a.exps,
                                           a.rng);
        return gqh::launch_status();
    }
};

template <typename T, int RND>
gq_status forward_any(const ForwardCall<T>& a, bool vec) {
    if (!held_ok(a.s.cols, (a.ldx > a.ldy ? a.ldx : a.ldy) * sizeof(T)))
        return vec ? forward_generic<T, true, 4, RND>(a) : forward_generic<T, false, 4, RND>(a);
    const Held h = held_for(a.s.rows, a.s.cols);
    return vec && a.s.cols % 8 == 0 ? held_switch(h, ForwardHeld<T, true, RND>{a, h})
                                    : held_switch(h, ForwardHeld<T, false, RND>{a, h});
}

}  // namespace

extern "C" {

gq_status gq_layernorm_forward(const void *x, int dtype, int64_t rows, int64_t cols, int64_t ldx,
                               const void *weight, const void *bias, int wdtype, float eps, void *y,
                               int64_t ldy, float *mean, float *rstd, int rounding, uint64_t seed,
                               uint64_t step, int8_t *codes, uint8_t *exps, void *stream) {
    if (!in_type(dtype) || !in_type(wdtype) || !size_ok(rows, cols)) return GQ_ERR_INVALID;
    if (!(eps >= 0.0f) || (rounding != GQ_ACT_NEAREST && rounding != GQ_ACT_RANDOM))
        return GQ_ERR_INVALID;
    if (!matrix_ok(x, dtype, rows, cols, ldx) || !matrix_ok(y, dtype, rows, cols, ldy))
        return GQ_ERR_INVALID;
    if (!vector_ok(weight, wdtype) || !vector_ok(bias, wdtype)) return GQ_ERR_INVALID;
    if (rows == 0) return GQ_OK;
    if (!mean || !rstd || !mult(mean, 4) || !mult(rstd, 4)) return GQ_ERR_INVALID;
    if ((codes || exps) && !saved_ok(codes, exps)) return GQ_ERR_INVALID;
    const Affine af{weight, bias, wdtype == GQ_F32, mult(weight, 16) && mult(bias, 16)};
    const bool vec = row_align(x, dtype, rows, ldx) && row_align(y, dtype, rows, ldy) && af.aligned;
    const Shape s = shape_of(rows, cols);
    const Rng rng = make_rng(seed, step);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    auto run = [&](auto elt) {
        using T = decltype(elt);
        const ForwardCall<T> a{static_cast<const T*>(x), ldx, s, af, eps, static_cast<T*>(y), ldy, mean,
                               rstd, codes, exps, rng, st};
        return !codes                         ? forward_any<T, -1>(a, vec)
               : rounding == GQ_ACT_NEAREST ? forward_any<T, 0>(a, vec)
                                            : forward_any<T, 1>(a, vec);
    };
    return dtype == GQ_F32 ? run(float()) : run(bf16());
}

}  // extern "C"
