// gq_layernorm.cu -- layer norm forward and backward (C ABI in include/gq.h), optionally over an
// 8-bit checkpoint of the normalised rows.
//
//   forward   xh = (x - mean) rstd, rstd = 1 / sqrt(var + eps);  y = xh w + b
//   backward  dx = rstd (w dy - mean(w dy) - xh mean(w dy xh));  dw = sum_rows dy xh;
//             db = sum_rows dy
//
// Both are bound by memory.  A row stays in registers between its reductions, so it is read
// once (see "rows held by fixed threads"); the generic kernels at the top take unaligned rows and
// rows of more columns than a block holds, and read again what does not fit their registers (from L2,
// mostly).  The backward pass keeps dw and db of its threads' columns in registers over all the
// rows of a block and leaves one partial row per block in the workspace; a second kernel adds
// those in a fixed order, so that results do not depend on timing.  All sums are fp32.
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
    const float rstd = rsqrtf(__fmul_rn(sq[0], s.inv_cols) + eps);  // within 2 units
    if (t == 0) {
        mean_out[row] = mean;
        rstd_out[row] = rstd;
    }

    auto finish = [&](int64_t c, float (&z)[V]) {  // z: x - mean
#pragma unroll
        for (int i = 0; i < V; ++i) z[i] = z[i] * rstd;
        if constexpr (RND >= 0)
        {
            gq::PhiloxGroup pg[1];
            if constexpr (RND == 1)
                pg[0] = gq::philox_group(static_cast<uint32_t>(c >> 3), rng.step_lo, rng.step_hi, rng.rk);
            save<V, RND == 1>(z, c < s.pitch, static_cast<uint32_t>(row), static_cast<uint32_t>(c),
                              s.pitch, s.epitch, rng, pg, codes, exps);
        }
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

// ---- rows held by fixed threads ------------------------------------------------------------
// The form for 16-byte aligned rows of up to 8,192 columns, a multiple of 8.  A group of 32 wpr
// threads (whole warps, 16 columns per thread as two pieces of 8; 8 columns up to 256) walks over
// rows; a thread has the same columns of every row, so that weights, the backward sums and the column
// part of the random words stay in registers, and the next rows are on their way while one is worked
// on.  What bounds it is the number of instructions per row beside its elements' own: 16 columns per
// thread instead of 8 took the backward pass at 65,536 x 1,024 bf16 from 75 to 65 us; no branches
// depend on the thread either: a thread behind the last column works on copies of the first columns
// with weights and masks of 0, and only its stores are left out.

struct Groups {
    int wpr;     // warps per row
    int groups;  // rows at a time per block
};

// Warps per row, as far as the reductions differ by it.
enum Wide { kOne = 1, kFour = 4, kMany = 16 };

// Sums of N values (1 or 2) over a group's threads.  `mine`: the group's slots, N per warp, room for
// 4 warps at least (unused ones hold 0), 16-byte aligned.  They must not be written again before the
// group has passed another barrier: calls alternate between two sets.
template <int W, int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float* mine, int wr, int wpr, int group) {
    const int lane = threadIdx.x & 31;
    if constexpr (N == 2) {  // the halves of the warp take one each after the first exchange
        const bool upper = lane & 16;
        float x = (upper ? v[1] : v[0]) + __shfl_xor_sync(kFull, upper ? v[0] : v[1], 16);
#pragma unroll
        for (int o = 8; o; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
        if constexpr (W == kOne) {
            v[0] = __shfl_sync(kFull, x, 0);
            v[1] = __shfl_sync(kFull, x, 16);
            return;
        }
        if ((lane & 15) == 0) mine[2 * wr + (lane >> 4)] = x;
    } else {
        v[0] = warp_sum(v[0]);
        if constexpr (W == kOne) return;
        if (lane == 0) mine[wr] = v[0];
    }
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(wpr * 32) : "memory");
    if constexpr (W == kFour) {
        const float4 p = reinterpret_cast<const float4*>(mine)[0];
        if constexpr (N == 2) {
            const float4 q = reinterpret_cast<const float4*>(mine)[1];
            v[0] = (p.x + p.z) + (q.x + q.z);
            v[1] = (p.y + p.w) + (q.y + q.w);
        } else {
            v[0] = (p.x + p.y) + (p.z + p.w);
        }
    } else if constexpr (W == kMany) {
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = warp_sum(lane < wpr ? mine[N * lane + k] : 0.0f);
    }
}
constexpr int kSlots = 32;  // per set and value: 8 groups x 4 slots, or 1 group of up to 16 warps

__device__ __forceinline__ void vec8(const void* p, int wide, float none, int64_t c, int64_t cols,
                                     F2 (&v)[4]) {
    float t[8];
    vec_of<8>(p, wide, none, c, cols, t);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f2(t[2 * i], t[2 * i + 1]);
}

// 8 elements of a thread in a slot: planes of 16 bytes per thread.
template <typename T> struct Ring {
    static constexpr int kPieces = sizeof(T) / 2;
    static __device__ __forceinline__ void fetch(uint32_t to, uint32_t plane, const T* p) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
            copy_async<16>(to + i * plane, reinterpret_cast<const uint8_t*>(p) + 16 * i);
    }
    static __device__ __forceinline__ void read(const uint8_t* at, uint32_t plane, F2 (&v)[4]) {
        Raw8<T> r;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const uint4 a = *reinterpret_cast<const uint4*>(at + i * plane);
            r.w[4 * i] = a.x; r.w[4 * i + 1] = a.y; r.w[4 * i + 2] = a.z; r.w[4 * i + 3] = a.w;
        }
        pairs(r, v);
    }
};

// What a launch of the held form is made for.
struct HeldArgs {
    uint32_t rows, stride;  // stride: rows at a time of the whole grid
    uint32_t cols, pitch, epitch;
    uint32_t in, in2, out;  // bytes from one row to the next
    int wpr, groups;
    float inv_cols;
};

template <typename T, int VPT, int RND, int W, int MOST>
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
    F2 w[VPT][4], b[VPT][4], mask[VPT];
    gq::PhiloxGroup pg[VPT];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const uint32_t c = k * apart + t * 8;
        in[k] = c < a.cols;
        padded[k] = c < a.pitch;
        col[k] = in[k] ? c : 0u;
        mask[k] = f2(in[k] ? 1.0f : 0.0f);
        vec8(af.w, af.wide, 1.0f, c, a.cols, w[k]);
        vec8(af.b, af.wide, 0.0f, c, a.cols, b[k]);
        if constexpr (RND == 1)
            pg[k] = gq::philox_group(c >> 3, rng.step_lo, rng.step_hi, rng.rk);
    }
    constexpr int P = Ring<T>::kPieces;
    const uint32_t plane = blockDim.x * 16, slot_bytes = plane * VPT * P;
    const uint32_t base = gq::smem_u32(ring) + threadIdx.x * 16;
    uint32_t ahead = row, turn = 0;
    auto fetch = [&]() {  // (the last row again where there is none)
        const T* p = row_of(x, min(ahead, a.rows - 1), a.in);
#pragma unroll
        for (int k = 0; k < VPT; ++k)
            Ring<T>::fetch(base + (turn & (kDepth - 1)) * slot_bytes + k * P * plane, plane, p + col[k]);
        copy_commit();
        ahead += a.stride;
        ++turn;
    };
#pragma unroll
    for (int d = 0; d < kDepth - 1; ++d) fetch();
    for (; row < a.rows; row += a.stride) {
        F2 v[VPT][4];
        fetch();
        copy_wait();
        F2 sum = f2(0.0f);
        const uint8_t* slot = ring + (turn & (kDepth - 1)) * slot_bytes + threadIdx.x * 16;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            Ring<T>::read(slot + k * P * plane, plane, v[k]);
#pragma unroll
            for (int i = 0; i < 4; ++i) sum = fma2(v[k][i], mask[k], sum);
        }
        float m[1] = {sum2(sum)};
        group_sum<W>(m, slots, wr, a.wpr, group);
        const float mean = m[0] * a.inv_cols;
        F2 sq = f2(0.0f);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const F2 less = mul2(mask[k], f2(-mean));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[k][i] = fma2(v[k][i], mask[k], less);
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
            if (in[k]) store8(py + col[k], 0, 8, v[k]);
        }
    }
    copy_all();
}

// The block's rows' sums of dy xh and dy go to partial[block][0 and 1][cols].
template <typename T, int VPT, bool CODES, int W, int MOST>
__global__ void __launch_bounds__(MOST, MOST == 256 ? (VPT == 1 ? 3 : 2) : 1)
    backward_rows(const T* __restrict__ dy, HeldArgs a, const void* w, int wide,
                  const float* __restrict__ rstd_in, Source<T> src, T* __restrict__ dx,
                  float* __restrict__ partial) {
    __shared__ alignas(16) float buf[2][2 * kSlots];
    extern __shared__ __align__(16) uint8_t ring[];  // afterwards 2 x cols sums, with several groups
    const int warp = threadIdx.x >> 5;
    const int group = W == kMany ? 0 : warp / a.wpr, wr = warp - group * a.wpr;
    const uint32_t t = wr * 32 + (threadIdx.x & 31), apart = a.wpr * 256;
    for (int i = threadIdx.x; i < 4 * kSlots; i += blockDim.x) (&buf[0][0])[i] = 0.0f;
    __syncthreads();
    float* const slots = &buf[0][W == kFour ? group * 8 : 0];
    bool in[VPT];
    uint32_t col[VPT];
    F2 wv[VPT][4], aw[VPT][4], ab[VPT][4];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const uint32_t c = k * apart + t * 8;
        in[k] = c < a.cols;
        col[k] = in[k] ? c : 0u;
        vec8(w, wide, 1.0f, c, a.cols, wv[k]);
        if (!in[k]) {
#pragma unroll
            for (int i = 0; i < 4; ++i) wv[k][i] = f2(0.0f);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) aw[k][i] = ab[k][i] = f2(0.0f);
    }
    // a slot: dy's planes of 16 bytes per thread, then x's or those of 8 and 4 for the checkpoint (4
    // exponent bytes, of which one is this thread's)
    constexpr int P = Ring<T>::kPieces;
    const uint32_t n = blockDim.x, tid = threadIdx.x, plane = n * 16;
    const uint32_t second = plane * VPT * P, third = second + VPT * n * 8;
    const uint32_t slot_bytes = CODES ? third + VPT * n * 4 : 2 * second;
    const uint32_t base = gq::smem_u32(ring);
    uint32_t row = blockIdx.x * a.groups + group, ahead = row, turn = 0;
    auto fetch = [&]() {  // (the last row again where there is none)
        const uint32_t r = min(ahead, a.rows - 1), to = base + (turn & (kDepth - 1)) * slot_bytes;
        const T* p = row_of(dy, r, a.in);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            Ring<T>::fetch(to + k * P * plane + tid * 16, plane, p + col[k]);
            if constexpr (CODES) {
                copy_async<8>(to + second + (k * n + tid) * 8, row_of(src.codes, r, a.pitch) + col[k]);
                copy_async<4>(to + third + (k * n + tid) * 4,
                              row_of(src.exps, r, a.epitch) + col[k] / 128 * 4);
            } else {
                Ring<T>::fetch(to + second + k * P * plane + tid * 16, plane,
                               row_of(src.x, r, a.in2) + col[k]);
            }
        }
        copy_commit();
        ahead += a.stride;
        ++turn;
    };
    float nrstd = 0.0f, nmean = 0.0f;
    if (row < a.rows) {
#pragma unroll
        for (int d = 0; d < kDepth - 1; ++d) fetch();
        nrstd = __ldg(rstd_in + row);
        if constexpr (!CODES) nmean = __ldg(src.mean + row);
    }
    float* set = slots;
    for (; row < a.rows; row += a.stride) {
        F2 gv[VPT][4], h[VPT][4];
        const float rstd = nrstd, mean = nmean;
        const uint32_t next = min(row + a.stride, a.rows - 1);
        nrstd = __ldg(rstd_in + next);
        if constexpr (!CODES) nmean = __ldg(src.mean + next);
        fetch();
        copy_wait();
        const uint8_t* slot = ring + (turn & (kDepth - 1)) * slot_bytes;
        F2 c1 = f2(0.0f), c2 = f2(0.0f);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            Ring<T>::read(slot + k * P * plane + tid * 16, plane, gv[k]);
            if constexpr (CODES) {
                const uint2 q = *reinterpret_cast<const uint2*>(slot + second + (k * n + tid) * 8);
                const uint32_t e4 = *reinterpret_cast<const uint32_t*>(slot + third + (k * n + tid) * 4);
                values8(q, e4 >> (col[k] / 32 % 4 * 8) & 0xFFu, h[k]);
            } else {
                Ring<T>::read(slot + second + k * P * plane + tid * 16, plane, h[k]);
#pragma unroll
                for (int i = 0; i < 4; ++i) h[k][i] = mul2(add2(h[k][i], f2(-mean)), f2(rstd));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                aw[k][i] = fma2(gv[k][i], h[k][i], aw[k][i]);
                ab[k][i] = add2(ab[k][i], gv[k][i]);
                gv[k][i] = mul2(gv[k][i], wv[k][i]);
                c1 = add2(c1, gv[k][i]);
                c2 = fma2(gv[k][i], h[k][i], c2);
            }
        }
        float m[2] = {sum2(c1), sum2(c2)};
        group_sum<W>(m, set, wr, a.wpr, group);
        set = slots + (set == slots ? 2 * kSlots : 0);
        // dx = rstd g - (rstd mean2) xh - rstd mean1
        const float by = -a.inv_cols * rstd;
        const F2 rs = f2(rstd), m1 = f2(m[0] * by), m2 = f2(m[1] * by);
        T* p = row_of(dx, row, a.out);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                gv[k][i] = fma2(gv[k][i], rs, fma2(h[k][i], m2, m1));
            if (in[k]) store8(p + col[k], 0, 8, gv[k]);
        }
    }
    copy_all();
    float* pw = partial + static_cast<int64_t>(blockIdx.x) * 2 * a.cols;
    float* shared_cols = reinterpret_cast<float*>(ring);
    float* out = a.groups > 1 ? shared_cols : pw;
    for (int q = 0; q < a.groups; ++q) {  // the groups add up their columns one after another
        if (a.groups > 1) __syncthreads();
        if (group != q) continue;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            if (!in[k]) continue;
#pragma unroll
            for (int z = 0; z < 4; ++z) {  // 4 columns of dw, 4 more, the same of db
                const F2 lo = z < 2 ? aw[k][2 * z] : ab[k][2 * z - 4];
                const F2 hi = z < 2 ? aw[k][2 * z + 1] : ab[k][2 * z - 3];
                float4 v;
                split(lo, v.x, v.y);
                split(hi, v.z, v.w);
                float4* at = reinterpret_cast<float4*>(out + (z < 2 ? 0u : a.cols) + col[k] + (z & 1) * 4);
                if (q > 0) {
                    const float4 u = *at;
                    v = make_float4(u.x + v.x, u.y + v.y, u.z + v.z, u.w + v.w);
                }
                *at = v;
            }
        }
    }
    if (a.groups > 1) {
        __syncthreads();
        for (uint32_t i = threadIdx.x; i < a.cols / 2; i += blockDim.x)
            reinterpret_cast<float4*>(pw)[i] = reinterpret_cast<const float4*>(shared_cols)[i];
    }
}

// ---- host ----------------------------------------------------------------------------------

constexpr int64_t kHeldCols = 8192;  // columns of the held form: 512 threads x 2 x 8

int threads_for(int64_t cols, int per_thread, int least, int most) {
    int t = least;
    while (t < most && static_cast<int64_t>(t) * per_thread < cols) t *= 2;
    return t;
}

inline bool held_ok(int64_t cols, int64_t ld_bytes) {
    return cols <= kHeldCols && cols % 8 == 0 && ld_bytes < (int64_t(1) << 32);
}

// Threads of the held form: pieces of 8 columns per thread, warps per row, rows per block.  With
// fewer rows than two per SM a block takes one at a time: there is nothing to share, and the sums
// need not be put together within the block.
struct Held {
    int vpt, threads, wpr, groups;
};
inline Held held_for(int64_t rows, int64_t cols) {
    Held h;
    h.vpt = cols <= 256 ? 1 : 2;
    h.wpr = static_cast<int>((cols + 256 * h.vpt - 1) / (256 * h.vpt));
    h.groups = h.wpr <= 4 && rows > 2 * gqh::sm_count() ? 8 / h.wpr : 1;
    h.threads = 32 * h.wpr * h.groups;
    return h;
}
inline HeldArgs held_args(const Held& h, int grid, const Shape& s, int64_t in, int64_t in2, int64_t out) {
    HeldArgs a;
    a.rows = static_cast<uint32_t>(s.rows);
    a.stride = static_cast<uint32_t>(grid * h.groups);
    a.cols = static_cast<uint32_t>(s.cols);
    a.pitch = static_cast<uint32_t>(s.pitch);
    a.epitch = static_cast<uint32_t>(s.epitch);
    a.in = static_cast<uint32_t>(in);
    a.in2 = static_cast<uint32_t>(in2);
    a.out = static_cast<uint32_t>(out);
    a.wpr = h.wpr;
    a.groups = h.groups;
    a.inv_cols = s.inv_cols;
    return a;
}
// run.template operator()<VPT, W, MOST>() for a shape of the held form
template <typename F> auto held_switch(const Held& h, F run) {
    if (h.vpt == 1) return run.template operator()<1, kOne, 256>();
    if (h.wpr == 1) return run.template operator()<2, kOne, 256>();
    if (h.wpr <= 4) return run.template operator()<2, kFour, 256>();
    if (h.wpr <= 8) return run.template operator()<2, kMany, 256>();
    return run.template operator()<2, kMany, 512>();
}

// One wave of resident blocks, or fewer where the rows run out.
int wave(int64_t resident, int64_t units) { return static_cast<int>(units < resident ? units : resident); }

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

template <typename T, int V, int VPT, int RND, bool WARP>
gq_status forward_generic(const ForwardCall<T>& a) {
    const int threads = WARP ? 256 : threads_for(a.s.cols, V * VPT, 128, 512);
    const int64_t blocks = WARP ? (a.s.rows + kWarpRows - 1) / kWarpRows : a.s.rows;
    forward_kernel<T, V, VPT, RND, WARP><<<static_cast<unsigned>(blocks), threads, 0, a.st>>>(
        a.x, a.ldx, a.s, a.af, a.eps, a.y, a.ldy, a.mean, a.rstd, a.codes, a.exps, a.rng);
    return gqh::launch_status();
}
template <typename T, int RND> struct ForwardHeld {
    const ForwardCall<T>& a;
    const Held& h;
    template <int VPT, int W, int MOST> gq_status operator()() const {
        auto k = forward_rows<T, VPT, RND, W, MOST>;
        const size_t smem = static_cast<size_t>(kDepth) * h.threads * VPT * 8 * sizeof(T);
        const int grid = wave(resident_blocks(k, h.threads, smem), (a.s.rows + h.groups - 1) / h.groups);
        const HeldArgs ha = held_args(h, grid, a.s, a.ldx * sizeof(T), 0, a.ldy * sizeof(T));
        k<<<grid, h.threads, smem, a.st>>>(a.x, ha, a.af, a.eps, a.y, a.mean, a.rstd, a.codes, a.exps,
                                           a.rng);
        return gqh::launch_status();
    }
};

template <typename T, int RND>
gq_status forward_any(const ForwardCall<T>& a, bool vec) {
    if (!vec) return a.s.cols <= 256 ? forward_generic<T, 1, 8, RND, true>(a)
                                     : forward_generic<T, 1, 8, RND, false>(a);
    if (!held_ok(a.s.cols, (a.ldx > a.ldy ? a.ldx : a.ldy) * sizeof(T)))
        return forward_generic<T, 8, 4, RND, false>(a);
    const Held h = held_for(a.s.rows, a.s.cols);
    return held_switch(h, ForwardHeld<T, RND>{a, h});
}

// Partial rows of the backward pass: at most one per block of its main kernel, or the row shares
// of the column kernel.
constexpr int kMostParts = 1024;
enum Form { kHeld, kScalarWarp, kScalar, kLong };  // kLong: rows that no block holds
inline Form backward_form(int64_t cols, int64_t ld_bytes, bool vec, size_t elt) {
    // (the ring of fp32 rows of more than 4,096 columns would pass the shared memory)
    if (vec && held_ok(cols, ld_bytes) && (elt == 2 || cols <= kHeldCols / 2)) return kHeld;
    if (vec && cols > kHeldCols / 2) return kLong;
    return cols <= 256 ? kScalarWarp : cols <= 4096 ? kScalar : kLong;
}

template <typename T>
struct BackwardCall {
    const T* dy;
    int64_t lddy;
    Shape s;
    const void* w;
    int wide;
    const float* rstd;
    Source<T> src;
    T* dx;
    int64_t lddx;
    float* partial;
    cudaStream_t st;
};

template <typename T, bool CODES> struct BackwardHeld {
    const BackwardCall<T>& a;
    const Held& h;
    template <int VPT, int W, int MOST> int operator()() const {
        if constexpr (MOST == 512 && sizeof(T) == 4) {
            return 0;  // not reached: backward_form
        } else {
            // (also room for 2 x cols sums: 64 bytes per thread and piece at least)
            const size_t smem = static_cast<size_t>(kDepth) * h.threads * VPT *
                                (CODES ? 8 * sizeof(T) + 12 : 16 * sizeof(T));
            auto k = backward_rows<T, VPT, CODES, W, MOST>;
            int grid = wave(resident_blocks(k, h.threads, smem), (a.s.rows + h.groups - 1) / h.groups);
            if (grid > kMostParts) grid = kMostParts;
            const HeldArgs ha = held_args(h, grid, a.s, a.lddy * sizeof(T), a.src.ldx * sizeof(T),
                                          a.lddx * sizeof(T));
            k<<<grid, h.threads, smem, a.st>>>(a.dy, ha, a.w, a.wide, a.rstd, a.src, a.dx, a.partial);
            return grid;
        }
    }
};
template <typename T, int V, int VPT, bool CODES, bool WARP, bool SUMS>
int backward_generic(const BackwardCall<T>& a) {
    const int threads = WARP ? 256 : threads_for(a.s.cols, V * VPT, 128, 512);
    const size_t smem = WARP ? 2 * a.s.cols * sizeof(float) : 0;
    auto k = backward_kernel<T, V, VPT, CODES, WARP, SUMS>;
    const int64_t units = WARP ? (a.s.rows + kWarpRows - 1) / kWarpRows : a.s.rows;
    int64_t grid = SUMS ? wave(resident_blocks(k, threads, smem), units) : units;
    if (SUMS && grid > kMostParts) grid = kMostParts;
    k<<<static_cast<unsigned>(grid), threads, smem, a.st>>>(a.dy, a.lddy, a.s, a.w, a.wide, a.rstd, a.src,
                                                           a.dx, a.lddx, a.partial);
    return static_cast<int>(grid);
}

template <typename T, bool CODES>
gq_status backward_any(const BackwardCall<T>& a, void* dw, void* db, int gdtype, bool vec) {
    const int64_t cols = a.s.cols;
    int64_t ld = a.lddy > a.lddx ? a.lddy : a.lddx;
    if (a.src.ldx > ld) ld = a.src.ldx;
    const Form form = backward_form(cols, ld * sizeof(T), vec, sizeof(T));
    int parts;
    if (form == kHeld) {
        const Held h = held_for(a.s.rows, cols);
        parts = held_switch(h, BackwardHeld<T, CODES>{a, h});
    } else if (form == kScalarWarp) {
        parts = backward_generic<T, 1, 8, CODES, true, true>(a);
    } else if (form == kScalar) {
        parts = backward_generic<T, 1, 8, CODES, false, true>(a);
    } else {
        if (vec) backward_generic<T, 8, 2, CODES, false, false>(a);
        else backward_generic<T, 1, 8, CODES, false, false>(a);
        parts = static_cast<int>((a.s.rows + 63) / 64 < 64 ? (a.s.rows + 63) / 64 : 64);
        const dim3 grid(static_cast<unsigned>((cols + 255) / 256), static_cast<unsigned>(parts));
        if (dw || db)
            columns_kernel<T, CODES><<<grid, 256, 0, a.st>>>(a.dy, a.lddy, a.s, a.rstd, a.src, a.partial);
    }
    if (dw || db) {
        const unsigned grid = static_cast<unsigned>((2 * cols + 31) / 32);
        if (gdtype == GQ_F32)
            sum_kernel<float><<<grid, dim3(32, kSumRows), 0, a.st>>>(
                a.partial, parts, cols, static_cast<float*>(dw), static_cast<float*>(db));
        else
            sum_kernel<bf16><<<grid, dim3(32, kSumRows), 0, a.st>>>(
                a.partial, parts, cols, static_cast<bf16*>(dw), static_cast<bf16*>(db));
    }
    return gqh::launch_status();
}

bool vector_ok(const void* p, int dtype) { return !p || (mult(p, elt_bytes(dtype))); }

}  // namespace

extern "C" {

size_t gq_layernorm_workspace_bytes(int64_t rows, int64_t cols) {
    if (!size_ok(rows, cols)) return 0;
    if (rows == 0) return 16;
    return static_cast<size_t>(rows < kMostParts ? rows : kMostParts) * 2 *
           static_cast<size_t>(cols) * sizeof(float);
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
    const bool vec = row_align(x, dtype, rows, ldx) && row_align(y, dtype, rows, ldy) &&
                     mult(weight, 16) && mult(bias, 16);
    const Shape s = shape_of(rows, cols);
    const Affine af{weight, bias, wdtype == GQ_F32};
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
    auto run = [&](auto elt) {
        using T = decltype(elt);
        const BackwardCall<T> a{static_cast<const T*>(dy), lddy, s, weight, wdtype == GQ_F32, rstd,
                                Source<T>{codes, exps, static_cast<const T*>(x), ldx, mean},
                                static_cast<T*>(dx), lddx, static_cast<float*>(ws), st};
        return from_codes ? backward_any<T, true>(a, dweight, dbias, gdtype, vec)
                          : backward_any<T, false>(a, dweight, dbias, gdtype, vec);
    };
    return dtype == GQ_F32 ? run(float()) : run(bf16());
}

}  // extern "C"
