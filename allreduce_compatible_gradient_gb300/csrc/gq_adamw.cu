// gq_adamw.cu -- the AdamW step over many tensors at once, with its two moments in fp32 or in 8 bits, and
// the norm of all gradients that clipping needs (C ABI in include/gq.h).
//
//   g' = g min(1, max_norm / (norm + 1e-6))        (g where no limit is given)
//   m = beta1 m + (1 - beta1) g'       v = beta2 v + (1 - beta2) g'^2
//   p = p (1 - lr decay) - lr / (1 - beta1^t)  m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
//
// States in 8 bits, per 32 elements: the first moment as e4m3 codes with an exponent byte (gq_fp8.cuh's rule),
// the second as its root r = sqrt(v) in unsigned codes of 4 exponent and 4 fraction bits with an exponent
// byte of its own: c < 16 stands for c, others for (16 + c % 16) 2^(c / 16 - 1), times 2^(E - 127).  The root
// halves the range, and what a code rounds is then the step's denominator itself.  A root that is not zero
// keeps a code that is not zero: a moment that survives its rounding where the root does not would be divided
// by eps.  Products and sums of the moments are rounded one by one, so that codes are those of the
// formulas in fp32 on any compiler; the update, which no code depends on, is contracted and divides by a
// reciprocal (2 units in the last place of the update).
//
// Random rounding (seed): an average of 1,000 steps moves by less than half of a code's step at a time, and
// rounding to nearest would leave it where it is.  16-bit numbers of the library's Philox stream.
//
// What bounds it: memory, one pass over everything; 28 bytes an element with fp32 states, 14.1 with 8-bit ones
// and bf16 gradients.  The tensors' addresses are an argument of the kernel (constant memory), so that nothing
// is copied to the device and a captured step keeps its own.
#include "gq_fp8.cuh"

#include <cmath>

using namespace gqa;

namespace {

constexpr int kThreadsA = 256;
constexpr int kRounds = 4;                          // of 8 elements per thread and block
constexpr int kChunk = kThreadsA * 8 * kRounds;     // elements of a block

struct Slot {
    void* p;
    const void* g;
    void* m;            // fp32, or codes
    void* v;
    uint8_t* e;         // exponents of 32 elements: of m, of the root
    int64_t n;
    uint32_t first;     // block of the launch
    uint32_t row;       // the first of the tensor's three rows of random words
    uint8_t wp, wg, wm, wv;  // widest access that each takes: 32 or 16 bytes, else element by element
};
template <int N> struct Table {
    int count;
    Slot s[N];
    // The tensor that a block works on: the last one that begins at or before it.
    __device__ __forceinline__ int of(uint32_t block) const {
        int lo = 0, hi = count;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s[mid].first <= block) lo = mid;
            else hi = mid;
        }
        return lo;
    }
};

struct Step {
    float beta1, rest1, beta2, rest2, keep, size, fix, eps;  // keep = 1 - lr decay; size, fix: host's step
    float lr, log1, log2;        // for a step that the device counts
    const int64_t* step;         // nullable
    const float* norm;           // nullable
    float max_norm;              // negative: no limit
    int random;
    Rng rng;
};

// 8 elements at p + i; `left` of them exist.  Ordinary loads: most of it is written again.
template <typename T>
__device__ __forceinline__ void get8(const void* p, int64_t i, int64_t left, uint32_t wide, F2 (&v)[4]) {
    const T* q = static_cast<const T*>(p) + i;
    if (wide && left >= 8) {
        if constexpr (sizeof(T) == 4) {
            uint32_t w[8];
            if (wide == 32u) {
                asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                             : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]),
                               "=r"(w[7])
                             : "l"(q));
            } else {
                const uint4 a = reinterpret_cast<const uint4*>(q)[0], b = reinterpret_cast<const uint4*>(q)[1];
                w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
                w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = f2(__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1]));
        } else {
            const uint4 a = *reinterpret_cast<const uint4*>(q);
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
                v[k] = f2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u));
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
        v[k] = f2(2 * k < left ? up(q[2 * k]) : 0.0f, 2 * k + 1 < left ? up(q[2 * k + 1]) : 0.0f);
}
template <typename T>
__device__ __forceinline__ void put8(void* p, int64_t i, int64_t left, uint32_t wide, const float (&v)[8]) {
    T* q = static_cast<T*>(p) + i;
    if (wide && left >= 8) {
        if (sizeof(T) == 4 && wide == 32u) store<T, 8, 32>(q, 0, 8, v);
        else store<T, 8, 16>(q, 0, 8, v);
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (k < left) down(v[k], q[k]);
}

// The maximum of 8 fp32 bit patterns over the 4 lanes of a block of 32.
__device__ __forceinline__ uint32_t top32(uint32_t m) {
    m = max(m, __shfl_xor_sync(kFull, m, 1));
    return max(m, __shfl_xor_sync(kFull, m, 2));
}
// bits >> drop, to nearest even or with a 16-bit number.
template <int DROP> __device__ __forceinline__ uint32_t cut(uint32_t bits, bool random, uint32_t h) {
    const uint32_t by = random ? h << (DROP - 16) | 1u << (DROP - 17)
                               : (1u << (DROP - 1)) - 1u + (bits >> DROP & 1u);
    return (bits + by) >> DROP;
}
__device__ __forceinline__ uint32_t half_of(const uint4& w, int k) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    return u[k >> 1] >> (16 * (k & 1)) & 0xFFFFu;
}
// 31 * 2^14 * 2^(E - 127) >= a: with a = 1.f * 2^k iff 1.f <= 31 / 16, a fraction field of at most 0x780000.
__device__ __forceinline__ uint32_t root_exp_byte(uint32_t top) {
    const int e = static_cast<int>((top + 0x7FFFFu) >> 23) - 18;
    return top >= 0x7F800000u ? 255u : static_cast<uint32_t>(max(e, 1));
}
// A code's bits in an fp32 number's exponent and fraction field are its value times 2^-130; this times
// 2^64 is the value again, in units of 2^(E - 127).
__device__ __forceinline__ float root_scale(uint32_t e) {
    return e == 255u ? __uint_as_float(0x7FFFFFFFu) : __uint_as_float((e + 66u) << 23);
}

struct Words {
    uint4 m, r, p;
};

// 8 elements of a step.  first moments, roots (EIGHT) or second moments, in and out.
template <bool EIGHT>
__device__ __forceinline__ void step8(const Step& a, float clip, float size, float fix, const F2 (&g)[4],
                                      F2 (&m)[4], F2 (&v)[4], float (&p)[8]) {
    const F2 b1 = f2(a.beta1), r1 = f2(a.rest1), b2 = f2(a.beta2), r2 = f2(a.rest2);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const F2 c = mul2(g[i], f2(clip));
        m[i] = add2(mul2(m[i], b1), mul2(c, r1));
        if constexpr (EIGHT) v[i] = mul2(v[i], v[i]);
        v[i] = add2(mul2(v[i], b2), mul2(mul2(c, c), r2));
        float x, y, mx, my;
        split(v[i], x, y);
        x = __fsqrt_rn(x);
        y = __fsqrt_rn(y);
        if constexpr (EIGHT) v[i] = f2(x, y);
        split(m[i], mx, my);
        p[2 * i] = fmaf(p[2 * i], a.keep, -size * __fdividef(mx, fmaf(x, fix, a.eps)));
        p[2 * i + 1] = fmaf(p[2 * i + 1], a.keep, -size * __fdividef(my, fmaf(y, fix, a.eps)));
    }
}

template <typename P, typename G, bool EIGHT, int N>
__global__ void __launch_bounds__(kThreadsA)
    adamw_kernel(const __grid_constant__ Table<N> t, const __grid_constant__ Step a) {
    const Slot& s = t.s[t.of(blockIdx.x)];
    float clip = 1.0f, size = a.size, fix = a.fix;
    if (a.norm) {
        const float norm = *a.norm;
        if (!(norm < INFINITY)) return;  // not a number, or infinite: the step is left out
        if (a.max_norm >= 0.0f) clip = fminf(1.0f, __fdiv_rn(a.max_norm, norm + 1e-6f));
    }
    uint32_t step_lo = a.rng.step_lo, step_hi = a.rng.step_hi;
    if (a.step) {
        const int64_t n = *a.step;
        step_lo = static_cast<uint32_t>(n);
        step_hi = static_cast<uint32_t>(n >> 32);
        const float f = static_cast<float>(n);
        size = __fdiv_rn(a.lr, -expm1f(f * a.log1));
        fix = __fdiv_rn(1.0f, __fsqrt_rn(-expm1f(f * a.log2)));
    }
    const int64_t begin = static_cast<int64_t>(blockIdx.x - s.first) * kChunk + threadIdx.x * 8;
#pragma unroll 1
    for (int k = 0; k < kRounds; ++k) {
        const int64_t i = begin + k * (kThreadsA * 8);
        if (i - threadIdx.x * 8 >= s.n) break;  // of the whole block
        const int64_t left = s.n - i;           // may be 0 or less: then only for the others' sake
        F2 g[4], m[4], v[4], q[4];
        float p[8];
        get8<G>(s.g, i, left, s.wg, g);
        get8<P>(s.p, i, left, s.wp, q);
        uint32_t em = 1u, ev = 1u;
        if constexpr (EIGHT) {
            uint2 cm = make_uint2(0u, 0u), cv = make_uint2(0u, 0u);
            if (left > 0) {
                cm = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(s.m) + i);
                cv = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(s.v) + i);
                const uint32_t e = reinterpret_cast<const uint16_t*>(s.e)[i >> 5];
                em = e & 255u;
                ev = e >> 8;
            }
            const uint32_t wm[2] = {cm.x, cm.y}, wv[2] = {cv.x, cv.y};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                m[j] = mul2(fp8_values2(wm[j >> 1] >> (16 * (j & 1))), f2(step_of(em)));
                const uint32_t c = wv[j >> 1] >> (16 * (j & 1));
                v[j] = mul2(mul2(f2(__uint_as_float((c & 255u) << 19), __uint_as_float((c >> 8 & 255u) << 19)),
                                 f2(0x1p64f)), f2(root_scale(ev)));
            }
        } else {
            get8<float>(s.m, i, left, s.wm, m);
            get8<float>(s.v, i, left, s.wv, v);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) split(q[j], p[2 * j], p[2 * j + 1]);
        step8<EIGHT>(a, clip, size, fix, g, m, v, p);

        Words w;
        if (a.random) {
            const gq::PhiloxGroup pg = gq::philox_group(static_cast<uint32_t>(i >> 3), step_lo, step_hi, a.rng.rk);
            if constexpr (EIGHT) {
                w.m = gq::philox_row(pg, s.row, step_lo, a.rng.rk);
                w.r = gq::philox_row(pg, s.row + 1, step_lo, a.rng.rk);
            }
            if constexpr (sizeof(P) == 2) w.p = gq::philox_row(pg, s.row + 2, step_lo, a.rng.rk);
        }
        if constexpr (sizeof(P) == 2) {
            if (a.random) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t b = __float_as_uint(p[j]);
                    if ((b & 0x7F800000u) != 0x7F800000u) p[j] = __uint_as_float((b + half_of(w.p, j)) & 0xFFFF0000u);
                }
            }
        }
        put8<P>(s.p, i, left, s.wp, p);
        if constexpr (EIGHT) {
            float x[8], r[8];
            uint32_t tm = 0u, tr = 0u;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                split(m[j], x[2 * j], x[2 * j + 1]);
                split(v[j], r[2 * j], r[2 * j + 1]);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                tm = max(tm, __float_as_uint(x[j]) & 0x7FFFFFFFu);
                tr = max(tr, __float_as_uint(r[j]) & 0x7FFFFFFFu);
            }
            em = fp8_exp_byte(top32(tm));
            ev = root_exp_byte(top32(tr));
            const float im = inv_step(em), ir = __uint_as_float((188u - min(ev, 187u)) << 23);
            uint32_t cm[2] = {0u, 0u}, cv[2] = {0u, 0u};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                // e4m3's exponent field becomes fp32's
                const uint32_t b = __float_as_uint(__fmul_rn(__fmul_rn(fabsf(x[j]), im), 0x1p-120f));
                uint32_t c = cut<20>(b, a.random != 0, half_of(w.m, j)) | (x[j] < 0.0f ? 128u : 0u);
                cm[j >> 2] |= (em == 255u ? 0u : c) << (8 * (j & 3));
                const uint32_t d = __float_as_uint(__fmul_rn(__fmul_rn(r[j], ir), 0x1p-64f));
                c = max(cut<19>(d, a.random != 0, half_of(w.r, j)), r[j] > 0.0f ? 1u : 0u);
                cv[j >> 2] |= (ev == 255u ? 0u : c) << (8 * (j & 3));
            }
            if (left > 0) {
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(s.m) + i) = make_uint2(cm[0], cm[1]);
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(s.v) + i) = make_uint2(cv[0], cv[1]);
            }
            // a block of 32 belongs to 4 lanes; the first of them has an element of it, or none has
            if ((threadIdx.x & 3) == 0 && left > 0)
                reinterpret_cast<uint16_t*>(s.e)[i >> 5] = static_cast<uint16_t>(em | ev << 8);
            // codes of the block's other lanes, where the tensor ends inside it, are zeros
            if (left <= 0 && (i & ~int64_t(31)) < s.n) {
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(s.m) + i) = make_uint2(0u, 0u);
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(s.v) + i) = make_uint2(0u, 0u);
            }
        } else {
            float x[8], y[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                split(m[j], x[2 * j], x[2 * j + 1]);
                split(v[j], y[2 * j], y[2 * j + 1]);
            }
            put8<float>(s.m, i, left, s.wm, x);
            put8<float>(s.v, i, left, s.wv, y);
        }
    }
}

// The values of 8-bit states: first moments to p, roots to g (the slot's places for two outputs).
template <typename O, int N>
__global__ void __launch_bounds__(kThreadsA) values_kernel(const __grid_constant__ Table<N> t) {
    const Slot& s = t.s[t.of(blockIdx.x)];
    const int64_t begin = static_cast<int64_t>(blockIdx.x - s.first) * kChunk + threadIdx.x * 8;
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
        const int64_t i = begin + k * (kThreadsA * 8), left = s.n - i;
        if (left <= 0) break;
        const uint2 cm = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(s.m) + i));
        const uint2 cv = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(s.v) + i));
        const uint32_t e = __ldg(reinterpret_cast<const uint16_t*>(s.e) + (i >> 5));
        const uint32_t wm[2] = {cm.x, cm.y}, wv[2] = {cv.x, cv.y};
        float x[8], r[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            split(mul2(fp8_values2(wm[j >> 1] >> (16 * (j & 1))), f2(step_of(e & 255u))), x[2 * j], x[2 * j + 1]);
            const uint32_t c = wv[j >> 1] >> (16 * (j & 1));
            split(mul2(mul2(f2(__uint_as_float((c & 255u) << 19), __uint_as_float((c >> 8 & 255u) << 19)),
                            f2(0x1p64f)), f2(root_scale(e >> 8))), r[2 * j], r[2 * j + 1]);
        }
        put8<O>(s.p, i, left, s.wp, x);
        put8<O>(const_cast<void*>(s.g), i, left, s.wg, r);
    }
}

// ---- the norm ------------------------------------------------------------------------------

constexpr int kNormBlocks = 608;   // partial sums per launch: at most
constexpr int kNormChunk = 16384;  // elements

// Sums of squares of the chunks blockIdx.x, blockIdx.x + gridDim.x, ...: fp32 over a thread's 64 elements of
// a chunk, fp64 over chunks and threads.
template <typename G, int N>
__global__ void __launch_bounds__(256)
    squares_kernel(const __grid_constant__ Table<N> t, uint32_t chunks, double* partial) {
    double sum = 0.0;
    for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        const Slot& s = t.s[t.of(c)];
        const int64_t begin = static_cast<int64_t>(c - s.first) * kNormChunk + threadIdx.x * 8;
        F2 part = f2(0.0f);
#pragma unroll
        for (int k = 0; k < kNormChunk / 2048; ++k) {
            const int64_t i = begin + k * 2048;
            F2 g[4];
            if (i < s.n) get8<G>(s.g, i, s.n - i, s.wg, g);
            else g[0] = g[1] = g[2] = g[3] = f2(0.0f);
#pragma unroll
            for (int j = 0; j < 4; ++j) part = fma2(g[j], g[j], part);
        }
        sum += static_cast<double>(sum2(part));
    }
    __shared__ double warps[8];
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        double all = 0.0;
#pragma unroll
        for (int i = 0; i < 8; ++i) all += warps[i];
        partial[blockIdx.x] = all;
    }
}
__global__ void __launch_bounds__(256) root_kernel(const double* partial, int64_t n, float* norm) {
    double sum = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += 256) sum += partial[i];
    __shared__ double warps[8];
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        double all = 0.0;
#pragma unroll
        for (int i = 0; i < 8; ++i) all += warps[i];
        *norm = static_cast<float>(sqrt(all));
    }
}

// ---- host ----------------------------------------------------------------------------------

// Tables of two sizes: a launch copies its arguments, and 2 KB take 1 us less than 14.
constexpr int kFew = 32, kMany = 256;

bool sizes_ok(int64_t count, const int64_t* numel) {
    if (count < 0 || (count > 0 && !numel) || count >= int64_t(1) << 30) return false;
    for (int64_t i = 0; i < count; ++i)
        if (numel[i] < 0 || numel[i] >= int64_t(1) << 34) return false;
    return true;
}

// Calls launch(table, blocks) for runs of up to N tensors (of at most 2^34 elements: a grid holds them).
// fill(slot, i) sets a tensor's places.
template <int N, typename Fill, typename Launch>
gq_status in_runs(int64_t count, const int64_t* numel, int chunk, Fill fill, Launch launch) {
    Table<N> t;
    t.count = 0;
    uint32_t blocks = 0;
    for (int64_t i = 0; i < count; ++i) {
        if (numel[i] > 0) {
            Slot& s = t.s[t.count++];
            s = Slot{};
            s.n = numel[i];
            s.first = blocks;
            fill(s, i);
            blocks += static_cast<uint32_t>((numel[i] + chunk - 1) / chunk);
        }
        if (t.count > 0 && (t.count == N || i + 1 == count)) {
            launch(t, blocks);
            if (cudaGetLastError() != cudaSuccess) return GQ_ERR_CUDA;
            t.count = 0;
            blocks = 0;
        }
    }
    return GQ_OK;
}

// Widest access to 8 elements at a time.
uint8_t wide(const void* p) { return mult(p, 32) ? 32 : mult(p, 16) ? 16 : 0; }

template <typename P, typename G, bool EIGHT>
gq_status adamw(int64_t count, void* const* params, const void* const* grads, void* const* m, void* const* v,
                uint8_t* const* exps, const int64_t* numel, int64_t first, const Step& a, cudaStream_t st) {
    auto fill = [&](Slot& s, int64_t i) {
        s.p = params[i]; s.g = grads[i]; s.m = m[i]; s.v = v[i];
        s.e = EIGHT ? exps[i] : nullptr;
        s.row = static_cast<uint32_t>(3 * (first + i));
        s.wp = wide(s.p); s.wg = wide(s.g); s.wm = wide(s.m); s.wv = wide(s.v);
    };
    if (count <= kFew)
        return in_runs<kFew>(count, numel, kChunk, fill, [&](const Table<kFew>& t, uint32_t blocks) {
            adamw_kernel<P, G, EIGHT, kFew><<<blocks, kThreadsA, 0, st>>>(t, a);
        });
    return in_runs<kMany>(count, numel, kChunk, fill, [&](const Table<kMany>& t, uint32_t blocks) {
        adamw_kernel<P, G, EIGHT, kMany><<<blocks, kThreadsA, 0, st>>>(t, a);
    });
}

}  // namespace

extern "C" {

size_t gq_tensors_norm_workspace_bytes(int64_t count) {
    const int64_t launches = count <= kFew ? 1 : (count + kMany - 1) / kMany;
    return count < 0 ? 0 : static_cast<size_t>(launches) * kNormBlocks * sizeof(double);
}

gq_status gq_tensors_norm(int64_t count, const void *const *tensors, const int64_t *numel, int dtype,
                          float *norm_dev, void *ws, size_t ws_bytes, void *stream) {
    if (!in_type(dtype) || !sizes_ok(count, numel) || (count > 0 && !tensors) || !norm_dev || !mult(norm_dev, 4))
        return GQ_ERR_INVALID;
    for (int64_t i = 0; i < count; ++i)
        if (numel[i] > 0 && (!tensors[i] || !mult(tensors[i], elt_bytes(dtype)))) return GQ_ERR_INVALID;
    if (!ws || !mult(ws, 16) || ws_bytes < gq_tensors_norm_workspace_bytes(count)) return GQ_ERR_WORKSPACE;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    double* partial = static_cast<double*>(ws);
    int64_t parts = 0;
    auto fill = [&](Slot& s, int64_t i) {
        s.g = tensors[i];
        s.wg = wide(s.g);
    };
    const uint32_t most = static_cast<uint32_t>(4 * gqh::sm_count() < kNormBlocks ? 4 * gqh::sm_count() : kNormBlocks);
    auto run = [&](const auto& t, uint32_t chunks) {
        constexpr int N = sizeof(t.s) / sizeof(Slot);
        const uint32_t blocks = chunks < most ? chunks : most;
        if (dtype == GQ_F32) squares_kernel<float, N><<<blocks, 256, 0, st>>>(t, chunks, partial + parts);
        else squares_kernel<bf16, N><<<blocks, 256, 0, st>>>(t, chunks, partial + parts);
        parts += blocks;
    };
    const gq_status r = count <= kFew ? in_runs<kFew>(count, numel, kNormChunk, fill, run)
                                      : in_runs<kMany>(count, numel, kNormChunk, fill, run);
    if (r != GQ_OK) return r;
    root_kernel<<<1, 256, 0, st>>>(partial, parts, norm_dev);
    return gqh::launch_status();
}

gq_status gq_adamw_step(int64_t count, void *const *params, int param_dtype, const void *const *grads,
                        int grad_dtype, void *const *m, void *const *v, uint8_t *const *exps,
                        const int64_t *numel, int64_t step, const int64_t *step_dev, double lr, double beta1,
                        double beta2, double eps, double weight_decay, const float *norm_dev, double max_norm,
                        int rounding, uint64_t seed, int64_t first, void *stream) {
    if (!in_type(param_dtype) || !in_type(grad_dtype) || !sizes_ok(count, numel)) return GQ_ERR_INVALID;
    if (count > 0 && (!params || !grads || !m || !v)) return GQ_ERR_INVALID;
    if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || !(eps >= 0.0) || !std::isfinite(lr) ||
        !std::isfinite(weight_decay) || (!step_dev && step < 1) || !mult(step_dev, 8) || !mult(norm_dev, 4))
        return GQ_ERR_INVALID;
    if ((rounding != GQ_ACT_NEAREST && rounding != GQ_ACT_RANDOM) || first < 0 || first + count > int64_t(1) << 30)
        return GQ_ERR_INVALID;
    for (int64_t i = 0; i < count; ++i) {
        if (numel[i] == 0) continue;
        if (!params[i] || !grads[i] || !m[i] || !v[i] || (exps && !exps[i])) return GQ_ERR_INVALID;
        if (!mult(params[i], elt_bytes(param_dtype)) || !mult(grads[i], elt_bytes(grad_dtype)) ||
            !mult(m[i], exps ? 16 : 4) || !mult(v[i], exps ? 16 : 4) || (exps && !mult(exps[i], 2)))
            return GQ_ERR_INVALID;
    }
    Step a;
    a.beta1 = static_cast<float>(beta1); a.rest1 = static_cast<float>(1.0 - beta1);
    a.beta2 = static_cast<float>(beta2); a.rest2 = static_cast<float>(1.0 - beta2);
    a.keep = static_cast<float>(1.0 - lr * weight_decay);
    a.eps = static_cast<float>(eps);
    a.lr = static_cast<float>(lr);
    a.log1 = static_cast<float>(std::log(beta1)); a.log2 = static_cast<float>(std::log(beta2));
    a.size = a.fix = 0.0f;
    if (!step_dev) {
        a.size = static_cast<float>(lr / -std::expm1(static_cast<double>(step) * std::log(beta1)));
        a.fix = static_cast<float>(1.0 / std::sqrt(-std::expm1(static_cast<double>(step) * std::log(beta2))));
    }
    a.step = step_dev;
    a.norm = norm_dev;
    a.max_norm = max_norm >= 0.0 ? static_cast<float>(max_norm) : -1.0f;
    a.random = rounding == GQ_ACT_RANDOM;
    a.rng = make_rng(seed, static_cast<uint64_t>(step));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
#define GQA_ADAMW(P, G)                                                                                       \
    (exps ? adamw<P, G, true>(count, params, grads, m, v, exps, numel, first, a, st)                            \
          : adamw<P, G, false>(count, params, grads, m, v, exps, numel, first, a, st))
    if (param_dtype == GQ_F32) return grad_dtype == GQ_F32 ? GQA_ADAMW(float, float) : GQA_ADAMW(float, bf16);
    return grad_dtype == GQ_F32 ? GQA_ADAMW(bf16, float) : GQA_ADAMW(bf16, bf16);
#undef GQA_ADAMW
}

gq_status gq_adamw_values(int64_t count, const uint8_t *const *m, const uint8_t *const *v,
                          const uint8_t *const *exps, const int64_t *numel, void *const *moments,
                          void *const *roots, int out_dtype, void *stream) {
    if (!in_type(out_dtype) || !sizes_ok(count, numel)) return GQ_ERR_INVALID;
    if (count > 0 && (!m || !v || !exps || !moments || !roots)) return GQ_ERR_INVALID;
    for (int64_t i = 0; i < count; ++i) {
        if (numel[i] == 0) continue;
        if (!m[i] || !v[i] || !exps[i] || !moments[i] || !roots[i]) return GQ_ERR_INVALID;
        if (!mult(m[i], 16) || !mult(v[i], 16) || !mult(exps[i], 2) || !mult(moments[i], elt_bytes(out_dtype)) ||
            !mult(roots[i], elt_bytes(out_dtype)))
            return GQ_ERR_INVALID;
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    auto fill = [&](Slot& s, int64_t i) {
        s.p = moments[i]; s.g = roots[i];
        s.m = const_cast<uint8_t*>(m[i]); s.v = const_cast<uint8_t*>(v[i]);
        s.e = const_cast<uint8_t*>(exps[i]);
        s.wp = wide(s.p); s.wg = wide(s.g);
    };
    auto run = [&](const auto& t, uint32_t blocks) {
        constexpr int N = sizeof(t.s) / sizeof(Slot);
        if (out_dtype == GQ_F32) values_kernel<float, N><<<blocks, kThreadsA, 0, st>>>(t);
        else values_kernel<bf16, N><<<blocks, kThreadsA, 0, st>>>(t);
    };
    return count <= kFew ? in_runs<kFew>(count, numel, kChunk, fill, run)
                         : in_runs<kMany>(count, numel, kChunk, fill, run);
}

}  // extern "C"
