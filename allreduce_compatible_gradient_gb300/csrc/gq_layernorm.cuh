// gq_layernorm.cuh -- what the layer norm kernels share (gq_layernorm_fwd.cu, gq_layernorm_bwd.cu):
// layer norm forward and backward (C ABI in include/gq.h), optionally over an 8-bit checkpoint of the
// normalised rows.
//
//   forward   xh = (x - mean) rstd, rstd = 1 / sqrt(var + eps);  y = xh w + b
//   backward  dx = rstd (w dy - mean(w dy) - xh mean(w dy xh));  dw = sum_rows dy xh;
//             db = sum_rows dy
//
// Both are bound by memory, and next to that by what a row does one after the other with 16 warps per SM
// to overlap it (65,536 x 1,024 bf16, inputs changing from call to call: forward 46 us without a
// checkpoint, 58 with one rounded to nearest, 71 at random, of which the memory needs 40, 50 and 50;
// backward 70 from x and 64 from codes, of which it needs 59 and 50).  A row stays in
// registers between its reductions, so it is read once ("rows held by fixed threads"); the generic
// kernels take rows of more columns than a block holds, and read again what does not fit their registers
// (from L2, mostly).  That form costs more: as many bytes in 4,096 x 8,192 and 4,092 x 8,200 bf16 take 37
// and 69 us forward, 45 and 133 backward from codes (whose columns' sums are a second kernel there).
// All sums are fp32.
#pragma once
#include "gq_act.cuh"

namespace gqa {

// Weights and biases come as fp32 or bf16 vectors, or not at all.
struct Affine {
    const void* w;
    const void* b;
    int wide;     // fp32
    int aligned;  // to 16 bytes
};
template <int V>
__device__ __forceinline__ void vec_of(const void* p, int wide, float none, int64_t c,
                                       int64_t cols, float (&v)[V]) {
    if (!p) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = none;
    } else if (wide) {
        load<float, V>(static_cast<const float*>(p), c, cols, v);
    } else {
        load<bf16, V>(static_cast<const bf16*>(p), c, cols, v);
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

// Sums over the block, which holds a row, through shared memory.
template <int N> __device__ __forceinline__ void row_sum(float (&v)[N], float (*buf)[N], int threads) {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = warp_sum(v[k]);
    const int warps = threads >> 5, lane = threadIdx.x & 31;
    if (lane == 0) {
#pragma unroll
        for (int k = 0; k < N; ++k) buf[threadIdx.x >> 5][k] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = warp_sum(lane < warps ? buf[lane][k] : 0.0f);
}

struct Shape {
    int64_t rows, cols, pitch, epitch;
    float inv_cols;
};
inline Shape shape_of(int64_t rows, int64_t cols) {
    return Shape{rows, cols, code_pitch(cols), exp_pitch(cols),
                 static_cast<float>(1.0 / static_cast<double>(cols))};
}

// ---- rows held by fixed threads ------------------------------------------------------------
// The form for rows of up to 8,192 columns, with a variant for 16-byte aligned rows of a multiple of 8
// columns.  A group of 32 wpr threads (whole warps, 16 columns per thread as two pieces of 8) walks over
// rows; a thread has the same columns of every row, so that weights, the backward sums and the column
// part of the random words stay in registers, and the next rows are on their way while one is worked
// on.  What bounds it is the number of instructions per row beside its elements' own: 16 columns per
// thread instead of 8 took the backward pass at 65,536 x 1,024 bf16 from 75 to 65 us.  No branches
// depend on the thread either (65 -> 59 us): a thread behind the last column works on zeros (and on the
// first columns' codes), and only its stores are left out.  The two pieces lie 256
// columns apart, so that neighbours load neighbours (16 columns side by side: 59 -> 67 us).

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

// 8 entries of a per-column vector, 0 behind the last column.
__device__ __forceinline__ void vec8(const void* p, int wide, int aligned, float none, int64_t c,
                                     int64_t cols, F2 (&v)[4]) {
    float t[8];
    if (aligned) {
        vec_of<8>(p, wide, none, c, cols, t);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float e[1];
            vec_of<1>(p, wide, none, c + i, cols, e);
            t[i] = e[0];
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f2(t[2 * i], t[2 * i + 1]);
}

// 8 elements of a thread in a slot of copies in flight: planes of 16 bytes per thread.  Rows that are
// not 16-byte aligned are copied by the 16-byte granules that hold a byte of them, one more at most, and
// moved into place as they are read; `left` of the elements lie in the row, the others read as 0 (an
// aligned piece lies in the row as a whole, or not at all: left 0).
template <typename T, bool ALIGNED> struct Ring {
    static constexpr int kSlots = ALIGNED ? kDepth : 2;
    static constexpr int kPieces = sizeof(T) / 2 + (ALIGNED ? 0 : 1);
    static __device__ __forceinline__ void fetch(uint32_t to, uint32_t plane, const T* p, int left) {
        const uint8_t* q = reinterpret_cast<const uint8_t*>(p);
        if constexpr (ALIGNED) {
#pragma unroll
            for (int i = 0; i < kPieces; ++i) copy_part(to + i * plane, q + 16 * i, left > 0 ? 16u : 0u);
        } else {
            const int m = static_cast<int>(reinterpret_cast<uintptr_t>(q) & 15u);
            const int bytes = m + min(left, 8) * static_cast<int>(sizeof(T));
#pragma unroll
            for (int i = 0; i < kPieces; ++i)
                if (16 * i < bytes) copy_async<16>(to + i * plane, q - m + 16 * i);
        }
    }
    static __device__ __forceinline__ void read(const uint8_t* at, uint32_t plane, const T* p, int left,
                                                F2 (&v)[4]) {
        uint32_t r[4 * kPieces];
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const uint4 a = *reinterpret_cast<const uint4*>(at + i * plane);
            r[4 * i] = a.x; r[4 * i + 1] = a.y; r[4 * i + 2] = a.z; r[4 * i + 3] = a.w;
        }
        const uint32_t m = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 15u;
        pairs(shifted<T, ALIGNED>(r, m, ALIGNED ? 8 : left), v);
    }
};

// Stores a piece of 8 columns.  Aligned: each lane its own.  Else the warp's 256 columns from `first` on
// go through its square in shared memory, so that neighbours store neighbours.
constexpr int kSquare = 32 * 9;  // floats per warp
template <typename T, bool ALIGNED>
__device__ __forceinline__ void put8(T* row, uint32_t col, bool in, uint32_t first, uint32_t cols,
                                     float* square, const F2 (&v)[4]) {
    if constexpr (ALIGNED) {
        if (in) store8(row + col, v);
    } else {
        const int lane = threadIdx.x & 31;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) split(v[i], square[lane * 9 + 2 * i], square[lane * 9 + 2 * i + 1]);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t c = i * 32 + lane;
            if (first + c < cols) down(square[(c >> 3) * 9 + (c & 7)], row[first + c]);
        }
    }
}

// ---- longer rows: 8 columns straight from memory --------------------------------------------
// How many of the 8 columns from c on lie in the row.
__device__ __forceinline__ int left_of(int64_t c, int64_t cols) {
    return static_cast<int>(min(max(cols - c, int64_t(0)), int64_t(8)));
}
// Sets those behind the row's end to 0.
__device__ __forceinline__ void cut8(F2 (&v)[4], int left) {
    if (left >= 8) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float x, y;
        split(v[i], x, y);
        v[i] = f2(2 * i < left ? x : 0.0f, 2 * i + 1 < left ? y : 0.0f);
    }
}
// 8 columns of a row, 0 behind its end; rows that are not aligned by the 16-byte granules that hold them.
template <typename T, bool ALIGNED>
__device__ __forceinline__ void load8(const T* row, int64_t c, int64_t cols, F2 (&v)[4]) {
    constexpr int P = sizeof(T) / 2 + (ALIGNED ? 0 : 1);
    const int left = left_of(c, cols);
    const uint8_t* q = reinterpret_cast<const uint8_t*>(row + c);
    const uint32_t m = ALIGNED ? 0u : static_cast<uint32_t>(reinterpret_cast<uintptr_t>(q)) & 15u;
    const int bytes = left > 0 ? static_cast<int>(m) + left * static_cast<int>(sizeof(T)) : 0;
    uint32_t r[4 * P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const uint4 g = 16 * i < bytes ? __ldg(reinterpret_cast<const uint4*>(q - m) + i)
                                       : make_uint4(0u, 0u, 0u, 0u);
        r[4 * i] = g.x; r[4 * i + 1] = g.y; r[4 * i + 2] = g.z; r[4 * i + 3] = g.w;
    }
    pairs(shifted<T, ALIGNED>(r, m, left), v);
}
// Stores them; `first` is the warp's first column, the whole warp takes part.
template <typename T, bool ALIGNED>
__device__ __forceinline__ void put_row(T* row, int64_t c, int64_t first, int64_t cols, float* square,
                                        const F2 (&v)[4]) {
    if constexpr (ALIGNED) {
        if (c + 8 <= cols) {
            store8(row + c, v);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float e[2];
                split(v[i / 2], e[0], e[1]);
                if (c + i < cols) down(e[i % 2], row[c + i]);
            }
        }
    } else {
        put8<T, false>(row, 0u, false, static_cast<uint32_t>(first), static_cast<uint32_t>(cols), square, v);
    }
}

// What a launch of the held form is made for.
struct HeldArgs {
    uint32_t rows, stride;  // stride: rows at a time of the whole grid
    uint32_t cols, pitch, epitch;
    uint32_t in, in2, out;  // bytes from one row to the next
    int wpr, groups;
    float inv_cols;
};

// ---- host ----------------------------------------------------------------------------------

constexpr int64_t kHeldCols = 8192;  // columns of the held form: 512 threads x 2 x 8

inline int threads_for(int64_t cols, int per_thread, int least, int most) {
    int t = least;
    while (t < most && static_cast<int64_t>(t) * per_thread < cols) t *= 2;
    return t;
}

inline bool held_ok(int64_t cols, int64_t ld_bytes) {
    return cols <= kHeldCols && ld_bytes < (int64_t(1) << 32);
}

// Threads of the held form: pieces of 8 columns per thread, warps per row, rows per block.  One piece
// per thread up to 256 columns, where one warp holds a row so, and from 513 to 768, where three warps do
// and two of two pieces would idle for a quarter of the time or more (43,690 x 768 bf16, backward from
// codes: 50 us with two pieces, 39 with one; at 1,024 columns two are faster, see above).  From 1,025 to
// 1,152 columns two pieces leave a quarter to a third of three warps idle too; one piece, in five warps
// with a reduction of more steps and one row per block, was not measured there.  Eight warps a block, two blocks per SM: three, with 84
// registers a thread, took the forward pass at 65,536 x 1,024 from 72 to 78 us.  With fewer rows than
// two per SM a block takes one at a time: there is nothing to share, and the sums need not be put
// together within the block.
struct Held {
    int vpt, threads, wpr, groups;
};
inline Held held_for(int64_t rows, int64_t cols) {
    Held h;
    h.vpt = cols <= 256 || (cols > 512 && cols <= 768) ? 1 : 2;
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
    if (h.vpt == 1 && h.wpr == 1) return run.template operator()<1, kOne, 256>();
    if (h.vpt == 1) return run.template operator()<1, kFour, 256>();
    if (h.wpr == 1) return run.template operator()<2, kOne, 256>();
    if (h.wpr <= 4) return run.template operator()<2, kFour, 256>();
    if (h.wpr <= 8) return run.template operator()<2, kMany, 256>();
    return run.template operator()<2, kMany, 512>();
}

// One wave of resident blocks, or fewer where the rows run out.
inline int wave(int64_t resident, int64_t units) { return static_cast<int>(units < resident ? units : resident); }

inline bool vector_ok(const void* p, int dtype) { return !p || (mult(p, elt_bytes(dtype))); }

}  // namespace gqa
