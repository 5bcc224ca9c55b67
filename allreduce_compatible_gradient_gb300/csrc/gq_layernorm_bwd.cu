// gq_layernorm_bwd.cu -- layer norm backward, from an 8-bit checkpoint of the normalised rows or from x.
//
// dw and db of a thread's columns stay in its registers over all the rows of its block; every block
// leaves one partial row in the workspace, and a second kernel adds those in a fixed order, so that
// results do not depend on timing.
#include "gq_layernorm.cuh"

using namespace gqa;

namespace {

constexpr int kSumRows = 32;   // threads that share a column of the partial rows

// What the backward pass reads the normalised row from: its checkpoint, or x with the row's mean
// and rstd.
template <typename T> struct Source {
    const int8_t* codes;
    const uint8_t* exps;
    const T* x;
    int64_t ldx;
    const float* mean;
};

template <typename T, bool ALIGNED, bool CODES>
__device__ __forceinline__ void hat_of(const Source<T>& src, const Shape& s, int64_t row, float mean,
                                       float rstd, int64_t c, F2 (&v)[4]) {
    if constexpr (CODES) {
        if (c < s.pitch) {
            const uint2 q = __ldg(reinterpret_cast<const uint2*>(src.codes + row * s.pitch + c));
            values8(q, src.exps[row * s.epitch + (c >> 5)], v);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = f2(0.0f);
        }
    } else {
        load8<T, ALIGNED>(src.x + row * src.ldx, c, s.cols, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = mul2(add2(v[i], f2(-mean)), f2(rstd));
    }
    cut8(v, left_of(c, s.cols));  // a block marked 255 reads as NaN in the padding too
}

// dx of rows of more columns than the held form takes: a block per row, as in the forward pass.  4,092 x
// 8,200 bf16 from codes with the columns' sums below: 129 us with two blocks per SM, 171 with one (84
// registers a thread), 144 with three and nothing kept in registers between the two passes.
template <typename T, bool ALIGNED, int VPT, bool CODES>
__global__ void __launch_bounds__(512, 2)
    backward_kernel(const T* __restrict__ dy, int64_t lddy, Shape s, const void* w, int wide,
                    const float* __restrict__ rstd_in, Source<T> src, T* __restrict__ dx,
                    int64_t lddx) {
    __shared__ float buf[32][2];
    __shared__ float squares[ALIGNED ? 1 : 16 * kSquare];
    const int threads = blockDim.x, t = threadIdx.x, lane = t & 31;
    float* const square = squares + (ALIGNED ? 0 : t / 32 * kSquare);
    const int64_t step = static_cast<int64_t>(threads) * 8, row = blockIdx.x;
    const int64_t mine = (t - lane) * 8, beyond = step * VPT + mine;

    const T* dyr = dy + row * lddy;
    T* dxr = dx + row * lddx;
    const float rstd = rstd_in[row];
    const float mean = CODES ? 0.0f : src.mean[row];
    F2 c1 = f2(0.0f), c2 = f2(0.0f);
    auto fetch = [&](int64_t c, F2 (&g)[4], F2 (&h)[4]) {  // w dy and xh
        load8<T, ALIGNED>(dyr, c, s.cols, g);
        hat_of<T, ALIGNED, CODES>(src, s, row, mean, rstd, c, h);
        F2 wv[4];
        vec8(w, wide & 1, wide >> 1, 1.0f, c, s.cols, wv);
#pragma unroll
        for (int i = 0; i < 4; ++i) g[i] = mul2(g[i], wv[i]);
    };
    auto add = [&](const F2 (&g)[4], const F2 (&h)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            c1 = add2(c1, g[i]);
            c2 = fma2(g[i], h[i], c2);
        }
    };
    F2 g[VPT][4], h[VPT][4];
#pragma unroll
    for (int k = 0; k < VPT; ++k) fetch(k * step + t * 8, g[k], h[k]);
#pragma unroll
    for (int k = 0; k < VPT; ++k) add(g[k], h[k]);
    for (int64_t c0 = beyond; c0 < s.cols; c0 += step) {
        F2 a[4], b[4];
        fetch(c0 + lane * 8, a, b);
        add(a, b);
    }
    float m[2] = {sum2(c1), sum2(c2)};
    row_sum(m, buf, threads);
    const F2 m1 = f2(-m[0] * s.inv_cols), m2 = f2(-m[1] * s.inv_cols), rs = f2(rstd);
    auto finish = [&](int64_t first, F2 (&a)[4], const F2 (&b)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = mul2(add2(a[i], fma2(b[i], m2, m1)), rs);
        put_row<T, ALIGNED>(dxr, first + lane * 8, first, s.cols, square, a);
    };
#pragma unroll
    for (int k = 0; k < VPT; ++k)
        if (k * step + mine < s.cols) finish(k * step + mine, g[k], h[k]);
    for (int64_t c0 = beyond; c0 < s.cols; c0 += step) {
        F2 a[4], b[4];
        fetch(c0 + lane * 8, a, b);
        finish(c0, a, b);
    }
}

// Column sums for rows that do not fit the registers: thread = 8 columns, blockIdx.y = a share of
// the rows; partial[blockIdx.y][0 and 1][cols].
template <typename T, bool ALIGNED, bool CODES>
__global__ void __launch_bounds__(128)
    columns_kernel(const T* __restrict__ dy, int64_t lddy, Shape s,
                   const float* __restrict__ rstd_in, Source<T> src, float* __restrict__ partial) {
    const int64_t c = (static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x) * 8;
    if (c >= s.cols) return;
    F2 aw[4], ab[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) aw[i] = ab[i] = f2(0.0f);
#pragma unroll 2
    for (int64_t row = blockIdx.y; row < s.rows; row += gridDim.y) {
        F2 g[4], h[4];
        load8<T, ALIGNED>(dy + row * lddy, c, s.cols, g);
        hat_of<T, ALIGNED, CODES>(src, s, row, CODES ? 0.0f : src.mean[row], rstd_in[row], c, h);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            aw[i] = fma2(g[i], h[i], aw[i]);
            ab[i] = add2(ab[i], g[i]);
        }
    }
    float* p = partial + static_cast<int64_t>(blockIdx.y) * 2 * s.cols + c;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float u[2], d[2];
        split(aw[i / 2], u[0], u[1]);
        split(ab[i / 2], d[0], d[1]);
        if (c + i < s.cols) {
            p[i] = u[i % 2];
            p[s.cols + i] = d[i % 2];
        }
    }
}

// Adds the partial rows: 32 columns x 32 shares of the rows per block.  (partial is not __restrict__: the
// main kernel may still write it when this one starts, so its loads must be ordinary ones, which stay behind
// the wait.)
template <typename G>
__global__ void __launch_bounds__(1024)
    sum_kernel(const float* partial, int parts, int64_t cols, G* dw, G* db) {
    __shared__ float tile[kSumRows][33];
    gq::pdl_wait();
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

// Slots of a block's ring: 2 for rows of fp32 that take 512 threads, whose 4 would pass the shared memory.
template <typename T, bool ALIGNED, int MOST>
constexpr int slots_of = sizeof(T) == 4 && MOST == 512 ? 2 : Ring<T, ALIGNED>::kSlots;

// The block's rows' sums of dy xh and dy go to partial[block][0 and 1][cols].
template <typename T, bool ALIGNED, int VPT, bool CODES, int W, int MOST>
__global__ void __launch_bounds__(MOST, MOST == 256 ? (VPT == 1 ? 3 : 2) : 1)
    backward_rows(const T* __restrict__ dy, HeldArgs a, const void* w, int wide,
                  const float* __restrict__ rstd_in, Source<T> src, T* __restrict__ dx,
                  float* __restrict__ partial) {
    gq::pdl_launch_dependents();  // sum_kernel, which waits for this one's end before it reads
    __shared__ alignas(16) float buf[2][2 * kSlots];
    extern __shared__ __align__(16) uint8_t ring[];  // afterwards the groups' column sums
    const int warp = threadIdx.x >> 5;
    const int group = W == kMany ? 0 : warp / a.wpr, wr = warp - group * a.wpr;
    const uint32_t t = wr * 32 + (threadIdx.x & 31), apart = a.wpr * 256;
    for (int i = threadIdx.x; i < 4 * kSlots; i += blockDim.x) (&buf[0][0])[i] = 0.0f;
    __syncthreads();
    float* const slots = &buf[0][W == kFour ? group * 8 : 0];
    bool in[VPT];
    uint32_t col[VPT];
    int left[VPT];  // elements of the row from col on, 0 behind the last column
    F2 wv[VPT][4], aw[VPT][4], ab[VPT][4];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const uint32_t c = k * apart + t * 8;
        in[k] = c < a.cols;
        col[k] = in[k] ? c : 0u;
        left[k] = in[k] ? static_cast<int>(a.cols - c) : 0;
        vec8(w, wide & 1, wide >> 1, 1.0f, c, a.cols, wv[k]);
#pragma unroll
        for (int i = 0; i < 4; ++i) aw[k][i] = ab[k][i] = f2(0.0f);
    }
    // a slot: dy's planes of 16 bytes per thread, then x's or those of 8 and 4 for the checkpoint (4
    // exponent bytes, of which one is this thread's)
    using R = Ring<T, ALIGNED>;
    constexpr int P = R::kPieces, D = slots_of<T, ALIGNED, MOST>;
    const uint32_t n = blockDim.x, tid = threadIdx.x, plane = n * 16;
    const uint32_t second = plane * VPT * P, third = second + VPT * n * 8;
    const uint32_t slot_bytes = CODES ? third + VPT * n * 4 : 2 * second;
    const uint32_t base = gq::smem_u32(ring);
    uint32_t row = blockIdx.x * a.groups + group, ahead = row, turn = 0;
    auto fetch = [&]() {  // (the last row again where there is none)
        const uint32_t r = min(ahead, a.rows - 1), to = base + (turn & (D - 1)) * slot_bytes;
        const T* p = row_of(dy, r, a.in);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            R::fetch(to + k * P * plane + tid * 16, plane, p + col[k], left[k]);
            if constexpr (CODES) {
                copy_async<8>(to + second + (k * n + tid) * 8, row_of(src.codes, r, a.pitch) + col[k]);
                copy_async<4>(to + third + (k * n + tid) * 4,
                              row_of(src.exps, r, a.epitch) + col[k] / 128 * 4);
            } else {
                R::fetch(to + second + k * P * plane + tid * 16, plane,
                         row_of(src.x, r, a.in2) + col[k], left[k]);
            }
        }
        copy_commit();
        ahead += a.stride;
        ++turn;
    };
    float* square = reinterpret_cast<float*>(ring + D * slot_bytes) + warp * kSquare;
    float nrstd = 0.0f, nmean = 0.0f;
    if (row < a.rows) {
#pragma unroll
        for (int d = 0; d < D - 1; ++d) fetch();
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
        copy_wait<D>();
        const uint8_t* slot = ring + (turn & (D - 1)) * slot_bytes;
        F2 c1 = f2(0.0f), c2 = f2(0.0f);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            R::read(slot + k * P * plane + tid * 16, plane, row_of(dy, row, a.in) + col[k], left[k], gv[k]);
            if constexpr (CODES) {
                const uint2 q = *reinterpret_cast<const uint2*>(slot + second + (k * n + tid) * 8);
                const uint32_t e4 = *reinterpret_cast<const uint32_t*>(slot + third + (k * n + tid) * 4);
                values8(q, e4 >> (col[k] / 32 % 4 * 8) & 0xFFu, h[k]);
            } else {
                R::read(slot + second + k * P * plane + tid * 16, plane,
                        row_of(src.x, row, a.in2) + col[k], left[k], h[k]);
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
            put8<T, ALIGNED>(p, col[k], in[k], k * apart + wr * 256, a.cols, square, gv[k]);
        }
    }
    copy_all();
    // every group's column sums to shared memory (whole warps' columns, behind the last one too), then
    // the block's to its partial row
    float* const sums = reinterpret_cast<float*>(ring);
    const uint32_t pitch = apart * VPT;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
#pragma unroll
        for (int z = 0; z < 4; ++z) {  // 4 columns of dw, 4 more, the same of db
            const F2* from = z < 2 ? aw[k] : ab[k];
            float4 v;
            split(from[z % 2 * 2], v.x, v.y);
            split(from[z % 2 * 2 + 1], v.z, v.w);
            *reinterpret_cast<float4*>(sums + (2 * group + z / 2) * pitch + k * apart + t * 8 + z % 2 * 4) = v;
        }
    }
    __syncthreads();
    float* pw = partial + static_cast<int64_t>(blockIdx.x) * 2 * a.cols;
    for (uint32_t i = threadIdx.x * (ALIGNED ? 4 : 1); i < 2 * a.cols; i += blockDim.x * (ALIGNED ? 4 : 1)) {
        const float* at = sums + (i < a.cols ? i : pitch + i - a.cols);
        if constexpr (ALIGNED) {
            float4 v = *reinterpret_cast<const float4*>(at);
            for (int q = 1; q < a.groups; ++q) {
                const float4 u = *reinterpret_cast<const float4*>(at + 2 * q * pitch);
                v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
            }
            *reinterpret_cast<float4*>(pw + i) = v;
        } else {
            float v = *at;
            for (int q = 1; q < a.groups; ++q) v += at[2 * q * pitch];
            pw[i] = v;
        }
    }
}

// ---- host ----------------------------------------------------------------------------------

// Partial rows: at most one per block of the main kernel, or the row shares of the column kernel.
constexpr int kMostParts = 1024;
inline int column_parts(int64_t rows) { return static_cast<int>((rows + 7) / 8 < 128 ? (rows + 7) / 8 : 128); }

template <typename T>
struct BackwardCall {
    const T* dy;
    int64_t lddy;
    Shape s;
    const void* w;
    int wide;  // 1: fp32, 2: 16-byte aligned
    const float* rstd;
    Source<T> src;
    T* dx;
    int64_t lddx;
    float* partial;
    cudaStream_t st;
};

template <typename T, bool ALIGNED, bool CODES> struct BackwardHeld {
    const BackwardCall<T>& a;
    const Held& h;
    template <int VPT, int W, int MOST> int operator()() const {
        using R = Ring<T, ALIGNED>;
        // (also room for the column sums, 64 bytes per thread and piece: the slots have 88 at least)
        const size_t smem = static_cast<size_t>(slots_of<T, ALIGNED, MOST>) * h.threads * VPT *
                                (CODES ? 16 * R::kPieces + 12 : 32 * R::kPieces) +
                            (ALIGNED ? 0 : h.threads / 32 * kSquare * sizeof(float));
        auto k = backward_rows<T, ALIGNED, VPT, CODES, W, MOST>;
        int grid = wave(resident_blocks(k, h.threads, smem), (a.s.rows + h.groups - 1) / h.groups);
        if (grid > kMostParts) grid = kMostParts;
        const HeldArgs ha = held_args(h, grid, a.s, a.lddy * sizeof(T), a.src.ldx * sizeof(T),
                                      a.lddx * sizeof(T));
        k<<<grid, h.threads, smem, a.st>>>(a.dy, ha, a.w, a.wide, a.rstd, a.src, a.dx, a.partial);
        return grid;
    }
};
template <typename T, bool ALIGNED, bool CODES>
void backward_generic(const BackwardCall<T>& a, int parts, bool sums) {
    constexpr int VPT = 2;
    const int threads = threads_for(a.s.cols, 8 * VPT, 128, 512);
    backward_kernel<T, ALIGNED, VPT, CODES><<<static_cast<unsigned>(a.s.rows), threads, 0, a.st>>>(
        a.dy, a.lddy, a.s, a.w, a.wide, a.rstd, a.src, a.dx, a.lddx);
    const dim3 grid(static_cast<unsigned>((a.s.cols + 1023) / 1024), static_cast<unsigned>(parts));
    if (sums)
        columns_kernel<T, ALIGNED, CODES><<<grid, 128, 0, a.st>>>(a.dy, a.lddy, a.s, a.rstd, a.src, a.partial);
}

template <typename T, bool CODES>
gq_status backward_any(const BackwardCall<T>& a, void* dw, void* db, int gdtype, bool vec) {
    const int64_t cols = a.s.cols;
    int64_t ld = a.lddy > a.lddx ? a.lddy : a.lddx;
    if (a.src.ldx > ld) ld = a.src.ldx;
    int parts;
    if (held_ok(cols, ld * sizeof(T))) {
        const Held h = held_for(a.s.rows, cols);
        parts = vec && cols % 8 == 0 ? held_switch(h, BackwardHeld<T, true, CODES>{a, h})
                                     : held_switch(h, BackwardHeld<T, false, CODES>{a, h});
    } else {
        parts = column_parts(a.s.rows);
        if (vec) backward_generic<T, true, CODES>(a, parts, dw || db);
        else backward_generic<T, false, CODES>(a, parts, dw || db);
    }
    if (cudaPeekAtLastError() == cudaSuccess && (dw || db)) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>((2 * cols + 31) / 32));
        cfg.blockDim = dim3(32, kSumRows);
        cfg.stream = a.st;
        cudaLaunchAttribute attr;  // its launch overlaps the main kernel's end
        attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr.val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        const float* partial = a.partial;
        const cudaError_t e =
            gdtype == GQ_F32 ? cudaLaunchKernelEx(&cfg, sum_kernel<float>, partial, parts, cols,
                                                  static_cast<float*>(dw), static_cast<float*>(db))
                             : cudaLaunchKernelEx(&cfg, sum_kernel<bf16>, partial, parts, cols,
                                                  static_cast<bf16*>(dw), static_cast<bf16*>(db));
        if (e != cudaSuccess) return gqh::status_of(e);
    }
    return gqh::launch_status();
}

}  // namespace

extern "C" {

size_t gq_layernorm_workspace_bytes(int64_t rows, int64_t cols) {
    if (!size_ok(rows, cols)) return 0;
    if (rows == 0) return 16;
    const int64_t parts = cols > kHeldCols ? column_parts(rows) : rows < kMostParts ? rows : kMostParts;
    return static_cast<size_t>(parts) * 2 * static_cast<size_t>(cols) * sizeof(float);
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
        gq_status r = dweight ? gqh::status_of(cudaMemsetAsync(dweight, 0, n, st)) : GQ_OK;
        if (r == GQ_OK && dbias) r = gqh::status_of(cudaMemsetAsync(dbias, 0, n, st));
        return r;
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
        const BackwardCall<T> a{static_cast<const T*>(dy), lddy, s, weight,
                                (wdtype == GQ_F32) + 2 * mult(weight, 16), rstd,
                                Source<T>{codes, exps, static_cast<const T*>(x), ldx, mean},
                                static_cast<T*>(dx), lddx, static_cast<float*>(ws), st};
        return from_codes ? backward_any<T, true>(a, dweight, dbias, gdtype, vec)
                          : backward_any<T, false>(a, dweight, dbias, gdtype, vec);
    };
    return dtype == GQ_F32 ? run(float()) : run(bf16());
}

}  // extern "C"
