// gq_layernorm.cu -- layer norm forward and backward (C ABI in include/gq.h), optionally over an
// 8-bit checkpoint of the normalised rows.
//
//   forward   xh = (x - mean) rstd, rstd = 1 / sqrt(var + eps);  y = xh w + b
//   backward  dx = rstd (w dy - mean(w dy) - xh mean(w dy xh));  dw = sum_rows dy xh;
//             db = sum_rows dy
//
// Both are bound by memory.  A row stays in registers between its reductions, so it is read
// once: a warp holds a row of up to 1,024 columns (32 per lane), a block of 128 to 512 threads
// a longer one; what does not fit the registers is read again (from L2, mostly).  The backward
// pass keeps dw and db of its threads' columns in registers over all the rows of a block and
// leaves one partial row per block in the workspace; a second kernel adds those in a fixed order,
// so that results do not depend on timing.  All sums are fp32.
#include "gq_act.cuh"

using namespace gqa;

namespace {

constexpr int kWarpRows = 8;   // rows per block where a warp holds a row
constexpr int kSumRows = 32;   // threads that share a column of the partial rows

// Weights and biases come as fp32 or bf16 vectors, or not at all.
struct Affine {
    const void* w;
    const void* b;
    int wide;  // fp32
};
template <int V>
__device__ __forceinline__ void vec_of(const void* p, int wide, float none, int64_t c,
                                       int64_t cols, float (&v)[V]) {
    if (!p) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = none;
    } else if (wide) {
        load<float, V, 16>(static_cast<const float*>(p), c, cols, v);
    } else {
        load<bf16, V, 16>(static_cast<const bf16*>(p), c, cols, v);
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

// Sums over the threads that hold a row: a warp, or the whole block through shared memory (the
// two buffers alternate, so one barrier per reduction is enough).
template <bool WARP, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float (*buf)[N], int threads) {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = warp_sum(v[k]);
    if constexpr (!WARP) {
        const int warps = threads >> 5, lane = threadIdx.x & 31;
        if (lane == 0) {
#pragma unroll
            for (int k = 0; k < N; ++k) buf[threadIdx.x >> 5][k] = v[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = warp_sum(lane < warps ? buf[lane][k] : 0.0f);
    }
}

struct Shape {
    int64_t rows, cols, pitch, epitch;
    float inv_cols;
};
inline Shape shape_of(int64_t rows, int64_t cols) {
    return Shape{rows, cols, code_pitch(cols), exp_pitch(cols),
                 static_cast<float>(1.0 / static_cast<double>(cols))};
}

// Thread t of a row's `threads` takes the pieces of V columns t, t + threads, ...: the first VPT
// of them in registers.  The loops run to the code pitch, and past it to a whole number of pieces
// per warp, so that every lane takes part in the block reductions of the checkpoint.
template <typename T, int V, int VPT, int RND, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : 512)
    forward_kernel(const T* __restrict__ x, int64_t ldx, Shape s, Affine af, float eps,
                   T* __restrict__ y, int64_t ldy, float* __restrict__ mean_out,
                   float* __restrict__ rstd_out, int8_t* __restrict__ codes,
                   uint8_t* __restrict__ exps, Rng rng) {
    __shared__ float buf[2][32][1];
    const int threads = WARP ? 32 : blockDim.x;
    const int t = WARP ? (threadIdx.x & 31) : threadIdx.x;
    const int64_t row = WARP ? static_cast<int64_t>(blockIdx.x) * kWarpRows + (threadIdx.x >> 5)
                             : static_cast<int64_t>(blockIdx.x);
    if (WARP && row >= s.rows) return;  // whole warps
    const T* xr = x + row * ldx;
    T* yr = y + row * ldy;
    const int64_t step = static_cast<int64_t>(threads) * V;
    const int64_t beyond = step * VPT;  // first column that is not in registers

    float v[VPT][V];
    float sum[1] = {0.0f};
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        load<T, V, 16>(xr, k * step + t * V, s.cols, v[k]);
#pragma unroll
        for (int i = 0; i < V; ++i) sum[0] += v[k][i];
    }
    for (int64_t c = beyond + t * V; c < s.cols; c += step) {
        float z[V];
        load<T, V, 16>(xr, c, s.cols, z);
#pragma unroll
        for (int i = 0; i < V; ++i) sum[0] += z[i];
    }
    row_sum<WARP>(sum, buf[0], threads);
    const float mean = sum[0] * s.inv_cols;

    float sq[1] = {0.0f};
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int64_t c = k * step + t * V;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            v[k][i] = c + i < s.cols ? v[k][i] - mean : 0.0f;
            sq[0] = fmaf(v[k][i], v[k][i], sq[0]);
        }
    }
    for (int64_t c = beyond + t * V; c < s.cols; c += step) {
        float z[V];
        load<T, V, 16>(xr, c, s.cols, z);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float d = c + i < s.cols ? z[i] - mean : 0.0f;
            sq[0] = fmaf(d, d, sq[0]);
        }
    }
    row_sum<WARP>(sq, buf[1], threads);
    const float rstd = 1.0f / sqrtf(sq[0] * s.inv_cols + eps);
    if (t == 0) {
        mean_out[row] = mean;
        rstd_out[row] = rstd;
    }

    auto finish = [&](int64_t c, float (&z)[V]) {  // z: x - mean
#pragma unroll
        for (int i = 0; i < V; ++i) z[i] = z[i] * rstd;
        if constexpr (RND >= 0)
            save<V, RND == 1>(z, c < s.pitch, static_cast<uint32_t>(row), static_cast<uint32_t>(c),
                              s.pitch, s.epitch, rng, codes, exps);
        if (c < s.cols) {
            float w[V], b[V];
            vec_of<V>(af.w, af.wide, 1.0f, c, s.cols, w);
            vec_of<V>(af.b, af.wide, 0.0f, c, s.cols, b);
#pragma unroll
            for (int i = 0; i < V; ++i) z[i] = fmaf(z[i], w[i], b[i]);
            store<T, V, 16>(yr, c, s.cols, z);
        }
    };
#pragma unroll
    for (int k = 0; k < VPT; ++k)
        if (k * step < s.cols) finish(k * step + t * V, v[k]);
    for (int64_t c0 = beyond; c0 < s.cols; c0 += step) {
        const int64_t c = c0 + t * V;
        float z[V];
        load<T, V, 16>(xr, c, s.cols, z);
#pragma unroll
        for (int i = 0; i < V; ++i) z[i] = c + i < s.cols ? z[i] - mean : 0.0f;
        finish(c, z);
    }
}

// What the backward pass reads the normalised row from: its checkpoint, or x with the row's mean
// and rstd.
template <typename T> struct Source {
    const int8_t* codes;
    const uint8_t* exps;
    const T* x;
    int64_t ldx;
    const float* mean;
};

template <typename T, int V, bool CODES>
__device__ __forceinline__ void hat_of(const Source<T>& src, const Shape& s, int64_t row, float mean,
                                       float rstd, int64_t c, float (&v)[V]) {
    if constexpr (CODES) {
        if (c < s.pitch) {
            saved<V>(src.codes + row * s.pitch, src.exps + row * s.epitch, c, v);
            if (c + V > s.cols) {  // a block marked 255 reads as NaN in the padding too
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (c + i >= s.cols) v[i] = 0.0f;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = 0.0f;
        }
    } else {
        load<T, V, 16>(src.x + row * src.ldx, c, s.cols, v);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = c + i < s.cols ? (v[i] - mean) * rstd : 0.0f;
    }
}

// SUMS: the block's rows' sums of dy xh and dy go to partial[block][0 and 1][cols]; the caller
// sees to it that a row fits the registers.  Without SUMS only dx is written.
template <typename T, int V, int VPT, bool CODES, bool WARP, bool SUMS>
__global__ void __launch_bounds__(WARP ? 256 : 512)
    backward_kernel(const T* __restrict__ dy, int64_t lddy, Shape s, const void* w, int wide,
                    const float* __restrict__ rstd_in, Source<T> src, T* __restrict__ dx,
                    int64_t lddx, float* __restrict__ partial) {
    __shared__ float buf[2][32][2];
    extern __shared__ float shared_cols[];  // WARP: 2 x cols
    const int threads = WARP ? 32 : blockDim.x;
    const int t = WARP ? (threadIdx.x & 31) : threadIdx.x;
    const int64_t step = static_cast<int64_t>(threads) * V;
    const int64_t beyond = step * VPT;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * (WARP ? kWarpRows : 1);

    float aw[SUMS ? VPT : 1][V], ab[SUMS ? VPT : 1][V];
    if constexpr (SUMS) {
#pragma unroll
        for (int k = 0; k < VPT; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) aw[k][i] = ab[k][i] = 0.0f;
    }
    int flip = 0;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * (WARP ? kWarpRows : 1) +
                       (WARP ? (threadIdx.x >> 5) : 0);
         row < s.rows; row += stride) {
        const T* dyr = dy + row * lddy;
        T* dxr = dx + row * lddx;
        const float rstd = rstd_in[row];
        const float mean = CODES ? 0.0f : src.mean[row];
        float g[VPT][V], h[VPT][V];
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            load<T, V, 16>(dyr, k * step + t * V, s.cols, g[k]);
            hat_of<T, V, CODES>(src, s, row, mean, rstd, k * step + t * V, h[k]);
        }
        float c[2] = {0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            float wv[V];
            vec_of<V>(w, wide, 1.0f, k * step + t * V, s.cols, wv);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if constexpr (SUMS) {
                    aw[k][i] = fmaf(g[k][i], h[k][i], aw[k][i]);
                    ab[k][i] += g[k][i];
                }
                g[k][i] *= wv[i];
                c[0] += g[k][i];
                c[1] = fmaf(g[k][i], h[k][i], c[1]);
            }
        }
        if constexpr (!SUMS) {
            for (int64_t col = beyond + t * V; col < s.cols; col += step) {
                float a[V], b[V], wv[V];
                load<T, V, 16>(dyr, col, s.cols, a);
                hat_of<T, V, CODES>(src, s, row, mean, rstd, col, b);
                vec_of<V>(w, wide, 1.0f, col, s.cols, wv);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    a[i] *= wv[i];
                    c[0] += a[i];
                    c[1] = fmaf(a[i], b[i], c[1]);
                }
            }
        }
        row_sum<WARP>(c, buf[flip], threads);
        flip ^= 1;
        const float c1 = c[0] * s.inv_cols, c2 = c[1] * s.inv_cols;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int64_t col = k * step + t * V;
            if (col < s.cols) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    g[k][i] = (g[k][i] - fmaf(h[k][i], c2, c1)) * rstd;
                store<T, V, 16>(dxr, col, s.cols, g[k]);
            }
        }
        if constexpr (!SUMS) {
            for (int64_t col = beyond + t * V; col < s.cols; col += step) {
                float a[V], b[V], wv[V];
                load<T, V, 16>(dyr, col, s.cols, a);
                hat_of<T, V, CODES>(src, s, row, mean, rstd, col, b);
                vec_of<V>(w, wide, 1.0f, col, s.cols, wv);
#pragma unroll
                for (int i = 0; i < V; ++i) a[i] = (a[i] * wv[i] - fmaf(b[i], c2, c1)) * rstd;
                store<T, V, 16>(dxr, col, s.cols, a);
            }
        }
    }
    if constexpr (SUMS) {
        float* pw = partial + static_cast<int64_t>(blockIdx.x) * 2 * s.cols;
        float* pb = pw + s.cols;
        if constexpr (WARP) {  // the block's warps add up their columns one after another
            const int warp = threadIdx.x >> 5;
            for (int q = 0; q < kWarpRows; ++q) {
                if (warp == q) {
#pragma unroll
                    for (int k = 0; k < VPT; ++k)
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            const int64_t col = k * step + t * V + i;
                            if (col < s.cols) {
                                float* a = shared_cols + col;
                                float* b = a + s.cols;
                                *a = (q ? *a : 0.0f) + aw[k][i];
                                *b = (q ? *b : 0.0f) + ab[k][i];
                            }
                        }
                }
                __syncthreads();
            }
            for (int64_t i = threadIdx.x; i < 2 * s.cols; i += blockDim.x) pw[i] = shared_cols[i];
        } else {
#pragma unroll
            for (int k = 0; k < VPT; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int64_t col = k * step + t * V + i;
                    if (col < s.cols) {
                        pw[col] = aw[k][i];
                        pb[col] = ab[k][i];
                    }
                }
        }
    }
}

// Column sums for rows that do not fit the registers: thread = column, blockIdx.y = a share of
// the rows; partial[blockIdx.y][0 and 1][cols].
template <typename T, bool CODES>
__global__ void __launch_bounds__(256)
    columns_kernel(const T* __restrict__ dy, int64_t lddy, Shape s,
                   const float* __restrict__ rstd_in, Source<T> src, float* __restrict__ partial) {
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (col >= s.cols) return;
    float aw = 0.0f, ab = 0.0f;
#pragma unroll 4
    for (int64_t row = blockIdx.y; row < s.rows; row += gridDim.y) {
        const float g = up(dy[row * lddy + col]);
        float h[1];
        hat_of<T, 1, CODES>(src, s, row, CODES ? 0.0f : src.mean[row], rstd_in[row], col, h);
        aw = fmaf(g, h[0], aw);
        ab += g;
    }
    float* p = partial + static_cast<int64_t>(blockIdx.y) * 2 * s.cols + col;
    p[0] = aw;
    p[s.cols] = ab;
}

// Adds the partial rows: 32 columns x 32 shares of the rows per block.
template <typename G>
__global__ void __launch_bounds__(1024)
    sum_kernel(const float* __restrict__ partial, int parts, int64_t cols, G* __restrict__ dw,
               G* __restrict__ db) {
    __shared__ float tile[kSumRows][33];
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
    float a = 0.0f;
    if (col < 2 * cols) {
#pragma unroll 8
        for (int p = threadIdx.y; p < parts; p += kSumRows) a += partial[p * 2 * cols + col];
    }
    tile[threadIdx.y][threadIdx.x] = a;
    __syncthreads();
    const float total = warp_sum(tile[threadIdx.x][threadIdx.y]);
    const int64_t out = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.y;
    if (threadIdx.x == 0 && out < 2 * cols) {
        if (out < cols) {
            if (dw) down(total, dw[out]);
        } else if (db) {
            down(total, db[out - cols]);
        }
    }
}

// ---- host ----------------------------------------------------------------------------------

constexpr int64_t kRegCols8 = 8192;  // columns that the backward block holds (V = 8: 512 x 2 x 8)

int threads_for(int64_t cols, int per_thread, int least, int most) {
    int t = least;
    while (t < most && static_cast<int64_t>(t) * per_thread < cols) t *= 2;
    return t;
}

template <typename T, int V, int VPT, bool WARP>
gq_status forward_run(const T* x, int64_t ldx, const Shape& s, const Affine& af, float eps, T* y,
                      int64_t ldy, float* mean, float* rstd, int8_t* codes, uint8_t* exps, int rnd,
                      const Rng& rng, cudaStream_t st) {
    const int threads = WARP ? 256 : threads_for(s.cols, V * VPT, 128, 512);
    const int64_t blocks = WARP ? (s.rows + kWarpRows - 1) / kWarpRows : s.rows;
    const unsigned grid = static_cast<unsigned>(blocks);
    if (rnd == GQ_ACT_RANDOM)
        forward_kernel<T, V, VPT, 1, WARP><<<grid, threads, 0, st>>>(x, ldx, s, af, eps, y, ldy, mean,
                                                                     rstd, codes, exps, rng);
    else if (rnd == GQ_ACT_NEAREST)
        forward_kernel<T, V, VPT, 0, WARP><<<grid, threads, 0, st>>>(x, ldx, s, af, eps, y, ldy, mean,
                                                                     rstd, codes, exps, rng);
    else
        forward_kernel<T, V, VPT, -1, WARP><<<grid, threads, 0, st>>>(x, ldx, s, af, eps, y, ldy, mean,
                                                                      rstd, codes, exps, rng);
    return gqh::launch_status();
}

template <typename T>
gq_status forward_any(const T* x, int64_t ldx, const Shape& s, const Affine& af, float eps, T* y,
                      int64_t ldy, float* mean, float* rstd, int8_t* codes, uint8_t* exps, int rnd,
                      const Rng& rng, bool vec, cudaStream_t st) {
#define GQA_FWD(V, VPT, WARP) \
    forward_run<T, V, VPT, WARP>(x, ldx, s, af, eps, y, ldy, mean, rstd, codes, exps, rnd, rng, st)
    if (vec) {
        if (s.cols <= 256) return GQA_FWD(8, 1, true);
        if (s.cols <= 512) return GQA_FWD(8, 2, true);
        if (s.cols <= 1024) return GQA_FWD(8, 4, true);
        return GQA_FWD(8, 4, false);
    }
    if (s.cols <= 256) return GQA_FWD(1, 8, true);
    return GQA_FWD(1, 8, false);
#undef GQA_FWD
}

// Partial rows of the backward pass: blocks of its main kernel (SUMS), or row shares of the
// column kernel.
struct Plan {
    int parts;
    int threads;   // of the main kernel
    bool warp, sums;
    int vpt;
};

inline Plan backward_plan(int64_t rows, int64_t cols, bool vec) {
    Plan p;
    const int sms = gqh::sm_count();
    if (vec) {
        p.warp = cols <= 1024;
        p.sums = cols <= kRegCols8;
        p.vpt = p.warp ? (cols <= 256 ? 1 : cols <= 512 ? 2 : 4) : 2;
        p.threads = p.warp ? 256 : threads_for(cols, 16, 128, 512);
    } else {
        p.warp = cols <= 256;
        p.sums = cols <= 4096;
        p.vpt = 8;
        p.threads = p.warp ? 256 : threads_for(cols, 8, 128, 512);
    }
    const int64_t units = p.warp ? (rows + kWarpRows - 1) / kWarpRows : rows;
    const int64_t full = static_cast<int64_t>(sms) * (p.threads <= 256 ? 2 : 1);
    p.parts = static_cast<int>(units < full ? units : full);
    if (!p.sums) {
        const int64_t share = (rows + 63) / 64;
        p.parts = static_cast<int>(share < 64 ? share : 64);
    }
    if (p.parts < 1) p.parts = 1;
    return p;
}

template <typename T, int V, int VPT, bool WARP, bool SUMS>
gq_status backward_run(const T* dy, int64_t lddy, const Shape& s, const void* w, int wide,
                       const float* rstd, const Source<T>& src, T* dx, int64_t lddx, float* partial,
                       const Plan& p, cudaStream_t st) {
    const size_t smem = WARP ? 2 * s.cols * sizeof(float) : 0;
    const unsigned grid = static_cast<unsigned>(SUMS ? p.parts : s.rows);
    if (src.codes)
        backward_kernel<T, V, VPT, true, WARP, SUMS><<<grid, p.threads, smem, st>>>(
            dy, lddy, s, w, wide, rstd, src, dx, lddx, partial);
    else
        backward_kernel<T, V, VPT, false, WARP, SUMS><<<grid, p.threads, smem, st>>>(
            dy, lddy, s, w, wide, rstd, src, dx, lddx, partial);
    return gqh::launch_status();
}

template <typename T>
gq_status backward_any(const T* dy, int64_t lddy, const Shape& s, const void* w, int wide,
                       const float* rstd, const Source<T>& src, T* dx, int64_t lddx, void* dw,
                       void* db, int gdtype, float* partial, bool vec, cudaStream_t st) {
    const Plan p = backward_plan(s.rows, s.cols, vec);
    gq_status r;
#define GQA_BWD(V, VPT, WARP, SUMS) \
    backward_run<T, V, VPT, WARP, SUMS>(dy, lddy, s, w, wide, rstd, src, dx, lddx, partial, p, st)
    if (vec)
        r = p.warp ? (p.vpt == 1   ? GQA_BWD(8, 1, true, true)
                      : p.vpt == 2 ? GQA_BWD(8, 2, true, true)
                                   : GQA_BWD(8, 4, true, true))
                   : (p.sums ? GQA_BWD(8, 2, false, true) : GQA_BWD(8, 2, false, false));
    else
        r = p.warp ? GQA_BWD(1, 8, true, true)
                   : (p.sums ? GQA_BWD(1, 8, false, true) : GQA_BWD(1, 8, false, false));
#undef GQA_BWD
    if (r != GQ_OK || (!dw && !db)) return r;
    if (!p.sums) {
        const dim3 grid(static_cast<unsigned>((s.cols + 255) / 256), static_cast<unsigned>(p.parts));
        if (src.codes)
            columns_kernel<T, true><<<grid, 256, 0, st>>>(dy, lddy, s, rstd, src, partial);
        else
            columns_kernel<T, false><<<grid, 256, 0, st>>>(dy, lddy, s, rstd, src, partial);
    }
    const unsigned grid = static_cast<unsigned>((2 * s.cols + 31) / 32);
    if (gdtype == GQ_F32)
        sum_kernel<float><<<grid, dim3(32, kSumRows), 0, st>>>(
            partial, p.parts, s.cols, static_cast<float*>(dw), static_cast<float*>(db));
    else
        sum_kernel<bf16><<<grid, dim3(32, kSumRows), 0, st>>>(
            partial, p.parts, s.cols, static_cast<bf16*>(dw), static_cast<bf16*>(db));
    return gqh::launch_status();
}

bool vector_ok(const void* p, int dtype) { return !p || (mult(p, elt_bytes(dtype))); }

}  // namespace

extern "C" {

size_t gq_layernorm_workspace_bytes(int64_t rows, int64_t cols) {
    if (!size_ok(rows, cols)) return 0;
    if (rows == 0) return 16;
    const int a = backward_plan(rows, cols, true).parts, b = backward_plan(rows, cols, false).parts;
    return static_cast<size_t>(a > b ? a : b) * 2 * static_cast<size_t>(cols) * sizeof(float);
}

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
    const int rnd = codes ? rounding : -1;
    const bool vec = row_align(x, dtype, rows, ldx) && row_align(y, dtype, rows, ldy) &&
                     mult(weight, 16) && mult(bias, 16);
    const Shape s = shape_of(rows, cols);
    const Affine af{weight, bias, wdtype == GQ_F32};
    const Rng rng = make_rng(seed, step);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == GQ_F32)
        return forward_any(static_cast<const float*>(x), ldx, s, af, eps, static_cast<float*>(y), ldy,
                           mean, rstd, codes, exps, rnd, rng, vec, st);
    return forward_any(static_cast<const bf16*>(x), ldx, s, af, eps, static_cast<bf16*>(y), ldy, mean,
                       rstd, codes, exps, rnd, rng, vec, st);
}

gq_status gq_layernorm_backward(const void *dy, int dtype, int64_t rows, int64_t cols, int64_t lddy,
                                const void *weight, int wdtype, const float *rstd,
                                const int8_t *codes, const uint8_t *exps, const void *x,
                                int64_t ldx, const float *mean, void *dx, int64_t lddx,
                                void *dweight, void *dbias, int gdtype, void *ws, size_t ws_bytes,
                                void *stream) {
    if (!in_type(dtype) || !in_type(wdtype) || !in_type(gdtype) || !size_ok(rows, cols))
        return GQ_ERR_INVALID;
    if (!matrix_ok(dy, dtype, rows, cols, lddy) || !matrix_ok(dx, dtype, rows, cols, lddx))
        return GQ_ERR_INVALID;
    if (!vector_ok(weight, wdtype) || !vector_ok(dweight, gdtype) || !vector_ok(dbias, gdtype))
        return GQ_ERR_INVALID;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (rows == 0) {  // sums over no rows
        const size_t n = static_cast<size_t>(cols) * elt_bytes(gdtype);
        if (dweight && cudaMemsetAsync(dweight, 0, n, st) != cudaSuccess) return GQ_ERR_CUDA;
        if (dbias && cudaMemsetAsync(dbias, 0, n, st) != cudaSuccess) return GQ_ERR_CUDA;
        return GQ_OK;
    }
    if (!rstd || !mult(rstd, 4)) return GQ_ERR_INVALID;
    // exactly one source of the normalised rows
    const bool from_codes = codes || exps;
    if (from_codes == (x != nullptr)) return GQ_ERR_INVALID;
    if (from_codes && !saved_ok(codes, exps)) return GQ_ERR_INVALID;
    if (!from_codes && (!mean || !mult(mean, 4) || !matrix_ok(x, dtype, rows, cols, ldx)))
        return GQ_ERR_INVALID;
    if (!ws || !mult(ws, 16) || ws_bytes < gq_layernorm_workspace_bytes(rows, cols))
        return GQ_ERR_WORKSPACE;
    const bool vec = row_align(dy, dtype, rows, lddy) && row_align(dx, dtype, rows, lddx) &&
                     mult(weight, 16) && (from_codes || row_align(x, dtype, rows, ldx));
    const Shape s = shape_of(rows, cols);
    float* partial = static_cast<float*>(ws);
    if (dtype == GQ_F32) {
        const Source<float> src{codes, exps, static_cast<const float*>(x), ldx, mean};
        return backward_any(static_cast<const float*>(dy), lddy, s, weight, wdtype == GQ_F32, rstd, src,
                            static_cast<float*>(dx), lddx, dweight, dbias, gdtype, partial, vec, st);
    }
    const Source<bf16> src{codes, exps, static_cast<const bf16*>(x), ldx, mean};
    return backward_any(static_cast<const bf16*>(dy), lddy, s, weight, wdtype == GQ_F32, rstd, src,
                        static_cast<bf16*>(dx), lddx, dweight, dbias, gdtype, partial, vec, st);
}

}  // extern "C"
