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
// by eps.  Products and sums of the moments are rounded one by one, so that codes are those of
// the formulas in fp32, whatever computes them; the update, where nothing is rounded at random behind it, takes
// a reciprocal (2 units in the last place of the update).
//
// Random rounding (seed): an average of 1,000 steps moves by less than half of a code's step at a time, and
// rounding to nearest would leave it where it is.  16-bit numbers of the library's Philox stream.
//
// What bounds it: memory, one pass over everything; 28 bytes an element with fp32 states, 14.1 with 8-bit ones
// and bf16 gradients, where the issue slots are 70 % busy beside it (67 instructions an element; 94 took 650 us
// for 201 M elements).  201 M elements: 796 us with fp32 states and gradients (7.1 TB/s), 455 with 8-bit ones
// (6.2); the norm of their gradients 133 in fp32, 72 in bf16.  The tensors' addresses are an argument of the
// kernel (constant memory), so that nothing is copied to the device and a captured step keeps its own.
#include "gq_fp8.cuh"

#include <cmath>

using namespace gqa;

namespace {

constexpr int kThreadsA = 256;
constexpr int kRound = kThreadsA * 8;   // elements of a block's round, 8 per thread

struct Slot {
    void* p;
    const void* g;
    void* m;            // fp32, or codes
    void* v;
    uint8_t* e;         // exponents of 32 elements: of m, of the root
    int64_t n;
    uint32_t first;     // block of the launch
    uint32_t row;       // the first of the tensor's three rows of random words
    uint32_t at;        // of the tensor's number of steps, where the device counts them
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
    const int64_t* step;         // nullable: the device counts, per tensor where slots say so
    const float* norm;           // nullable
    float max_norm;              // negative: no limit
    int rounds;                  // of a block
    Rng rng;
};

// 8 elements at p + i as they lie; `left` of them exist.  Ordinary loads: most of it is written again.
template <typename T>
__device__ __forceinline__ Raw8<T> raw8(const void* p, int64_t i, int64_t left, uint32_t wide) {
    const T* q = static_cast<const T*>(p) + i;
    Raw8<T> r;
    if (wide && left >= 8) {
        if (sizeof(T) == 4 && wide == 32u) {
            asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                         : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[sizeof(T) == 4 ? 4 : 0]),
                           "=r"(r.w[sizeof(T) == 4 ? 5 : 1]), "=r"(r.w[sizeof(T) == 4 ? 6 : 2]),
                           "=r"(r.w[sizeof(T) == 4 ? 7 : 3])
                         : "l"(q));
        } else {
#pragma unroll
            for (int k = 0; k < static_cast<int>(sizeof(T)) / 2; ++k) {
                const uint4 a = reinterpret_cast<const uint4*>(q)[k];
                r.w[4 * k] = a.x; r.w[4 * k + 1] = a.y; r.w[4 * k + 2] = a.z; r.w[4 * k + 3] = a.w;
            }
        }
        return r;
    }
#pragma unroll
    for (int k = 0; k < static_cast<int>(sizeof(T)) * 2; ++k) r.w[k] = 0u;
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (k < left) {
            if constexpr (sizeof(T) == 4) r.w[k] = __float_as_uint(q[k]);
            else r.w[k >> 1] |= static_cast<uint32_t>(__bfloat16_as_ushort(q[k])) << (16 * (k & 1));
        }
    return r;
}
template <typename T>
__device__ __forceinline__ void get8(const void* p, int64_t i, int64_t left, uint32_t wide, F2 (&v)[4]) {
    pairs(raw8<T>(p, i, left, wide), v);
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

// The largest magnitude of 8 numbers as fp32 bits, above infinity's where one is a NaN; over the 4 lanes of a
// block of 32.
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ uint32_t top32(const float (&v)[8]) {
    const float a = max3(max3(v[0], v[1], v[2]), v[3], v[4]);
    uint32_t m = __float_as_uint(max3(a, max3(v[5], v[6], v[7]), 0.0f));
    m = max(m, __shfl_xor_sync(kFull, m, 1));
    return max(m, __shfl_xor_sync(kFull, m, 2));
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
// The values of 8 codes of either kind, as pairs.
__device__ __forceinline__ void moments8(uint2 c, uint32_t e, F2 (&m)[4]) {
    const uint32_t w[2] = {c.x, c.y};
    const F2 s = f2(step_of(e));
#pragma unroll
    for (int j = 0; j < 4; ++j) m[j] = mul2(fp8_values2(w[j >> 1] >> (16 * (j & 1))), s);
}
__device__ __forceinline__ void roots8(uint2 c, uint32_t e, F2 (&r)[4]) {
    const uint32_t w[2] = {c.x, c.y};
    const F2 s = f2(root_scale(e)), up64 = f2(0x1p64f);
    constexpr uint32_t mask = 0xFFu << 19;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        r[2 * j] = f2(__uint_as_float(w[j] << 19 & mask), __uint_as_float(w[j] << 11 & mask));
        r[2 * j + 1] = f2(__uint_as_float(w[j] << 3 & mask), __uint_as_float(w[j] >> 5 & mask));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = mul2(mul2(r[j], up64), s);
}

// Codes of 8 numbers y whose exponent field has been made the code's own (y is below 2^-111): the code ends at
// bit 27 - LEFT of the number and at bit 32 after a shift by LEFT, where what is behind it is rounded off: to
// nearest even, or by the 16-bit numbers of a Philox call, each with a half behind it, H 256 + 128 of 2^24.
template <int LEFT, bool RANDOM>
__device__ __forceinline__ uint2 codes_of(const uint32_t (&y)[8], const uint4& words) {
    const uint32_t h[4] = {words.x, words.y, words.z, words.w};
    uint32_t t[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t by = RANDOM ? __byte_perm(h[j >> 1], 0x80u, j & 1 ? 0x5324 : 0x5104)
                                   : 0x7FFFFFu + (y[j] >> (24 - LEFT) & 1u);
        t[j] = (y[j] << LEFT) + by;
    }
    return make_uint2(gather_bytes<3>(t[0], t[1], t[2], t[3]), gather_bytes<3>(t[4], t[5], t[6], t[7]));
}

__device__ __forceinline__ float rsqrt_fast(float v) {
    float r;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float rcp_fast(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// Roots of 8 numbers >= 0: a reciprocal root y (an approximation), s = v y, and one of Newton's steps for the
// root, s + (v - s^2) y / 2, whose error is a rounding's.  Numbers below fp32's normal ones, which the
// approximation takes for 0, go the long way.
__device__ __forceinline__ void roots(const F2 (&v)[4], F2 (&r)[4]) {
    uint32_t low = 0xFFFFFFFFu;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float a, b;
        split(v[j], a, b);
        low = min(low, min(__float_as_uint(a) - 1u, __float_as_uint(b) - 1u));  // 0 is the largest
        const F2 y = f2(rsqrt_fast(fmaxf(a, 0x1p-126f)), rsqrt_fast(fmaxf(b, 0x1p-126f)));
        const F2 s = mul2(v[j], y), half = mul2(y, f2(0.5f));
        r[j] = fma2(fma2(mul2(s, f2(-1.0f)), s, v[j]), half, s);
    }
    // (infinities and NaN too: s would be NaN for the former)
    uint32_t high = 0u;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float a, b;
        split(v[j], a, b);
        high = max(high, max(__float_as_uint(a), __float_as_uint(b)));
    }
    if (low < 0x7FFFFFu || high >= 0x7F800000u) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float a, b;
            split(v[j], a, b);
            r[j] = f2(__fsqrt_rn(a), __fsqrt_rn(b));
        }
    }
}

// a + b, each rounded by itself: sums of pairs would be contracted with the products that they add, whatever
// the compiler is told.
__device__ __forceinline__ F2 sum_of(F2 a, F2 b) {
    float ax, ay, bx, by;
    split(a, ax, ay);
    split(b, bx, by);
    return f2(__fadd_rn(ax, bx), __fadd_rn(ay, by));
}

// 8 elements of a step: gradients, first moments, second moments and parameters; the roots come back in r.
// EXACT: the update's operations are rounded one by one like the moments', for a parameter that is rounded at
// random behind them.
template <bool EXACT>
__device__ __forceinline__ void step8(const Step& a, float clip, float size, float fix, const F2 (&g)[4],
                                      F2 (&m)[4], F2 (&v)[4], F2 (&p)[4], F2 (&r)[4]) {
    const F2 b1 = f2(a.beta1), r1 = f2(a.rest1), b2 = f2(a.beta2), r2 = f2(a.rest2);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const F2 c = mul2(g[j], f2(clip));
        m[j] = sum_of(mul2(m[j], b1), mul2(c, r1));
        v[j] = sum_of(mul2(v[j], b2), mul2(mul2(c, c), r2));
    }
    roots(v, r);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float x, y;
        if constexpr (EXACT) {
            float mx, my;
            split(sum_of(mul2(r[j], f2(fix)), f2(a.eps)), x, y);
            split(m[j], mx, my);
            p[j] = sum_of(mul2(p[j], f2(a.keep)), mul2(f2(__fdiv_rn(mx, x), __fdiv_rn(my, y)), f2(-size)));
        } else {
            split(fma2(r[j], f2(fix), f2(a.eps)), x, y);
            const F2 u = mul2(m[j], f2(rcp_fast(x), rcp_fast(y)));
            p[j] = fma2(p[j], f2(a.keep), mul2(u, f2(-size)));
        }
    }
}
__device__ __forceinline__ void apart(const F2 (&v)[4], float (&x)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) split(v[j], x[2 * j], x[2 * j + 1]);
}

// What a thread reads of 8 elements with 8-bit states.
template <typename P, typename G> struct Load {
    Raw8<P> p;
    Raw8<G> g;
    uint2 m, v;
    uint32_t e;
    __device__ __forceinline__ void fetch(const Slot& s, int64_t i) {
        const int64_t left = s.n - i;
        g = raw8<G>(s.g, i, left, s.wg);
        p = raw8<P>(s.p, i, left, s.wp);
        m = v = make_uint2(0u, 0u);
        e = 0x0101u;
        if (left > 0) {
            m = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(s.m) + i);
            v = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(s.v) + i);
            e = reinterpret_cast<const uint16_t*>(s.e)[i >> 5];
        }
    }
};

template <typename P, typename G, bool EIGHT, bool RANDOM, int N>
__global__ void __launch_bounds__(kThreadsA)
    adamw_kernel(const __grid_constant__ Table<N> t, const __grid_constant__ Step a) {
    // from the end: the last gradients are what the norm's pass has left in the L2
    const uint32_t block = gridDim.x - 1 - blockIdx.x;
    const Slot& s = t.s[t.of(block)];
    float clip = 1.0f, size = a.size, fix = a.fix;
    gq::pdl_wait();
    if (a.norm) {
        const float norm = *a.norm;
        if (!(norm < INFINITY)) return;  // not a number, or infinite: the step is left out
        if (a.max_norm >= 0.0f) clip = fminf(1.0f, __fdiv_rn(a.max_norm, norm + 1e-6f));
    }
    uint32_t step_lo = a.rng.step_lo, step_hi = a.rng.step_hi;
    if (a.step) {
        const int64_t n = a.step[s.at];
        step_lo = static_cast<uint32_t>(n);
        step_hi = static_cast<uint32_t>(n >> 32);
        const float f = static_cast<float>(n);
        size = __fdiv_rn(a.lr, -expm1f(f * a.log1));
        fix = __fdiv_rn(1.0f, __fsqrt_rn(-expm1f(f * a.log2)));
    }
    const int64_t begin = static_cast<int64_t>(block - s.first) * (a.rounds * kRound);
    // 8-bit states: the next round is on its way while one is computed (the instructions of a round take as
    // long as its bytes)
    Load<P, G> next;
    if constexpr (EIGHT) next.fetch(s, begin + threadIdx.x * 8);
#pragma unroll 1
    for (int k = 0; k < a.rounds; ++k) {
        const int64_t i0 = begin + k * kRound, i = i0 + threadIdx.x * 8;
        if (i0 >= s.n) break;          // of the whole block
        const int64_t left = s.n - i;  // may be 0 or less: then only for the others' sake
        F2 g[4], m[4], v[4], p[4], r[4];
        if constexpr (EIGHT) {
            const Load<P, G> now = next;
            if (k + 1 < a.rounds && i0 + kRound < s.n) next.fetch(s, i + kRound);
            pairs(now.g, g);
            pairs(now.p, p);
            moments8(now.m, now.e & 255u, m);
            roots8(now.v, now.e >> 8, v);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = mul2(v[j], v[j]);
        } else {
            get8<G>(s.g, i, left, s.wg, g);
            get8<P>(s.p, i, left, s.wp, p);
            get8<float>(s.m, i, left, s.wm, m);
            get8<float>(s.v, i, left, s.wv, v);
        }
        step8<RANDOM && sizeof(P) == 2>(a, clip, size, fix, g, m, v, p, r);

        uint4 wm = make_uint4(0u, 0u, 0u, 0u), wr = wm, wp = wm;
        if constexpr (RANDOM) {
            const gq::PhiloxGroup pg = gq::philox_group(static_cast<uint32_t>(i >> 3), step_lo, step_hi, a.rng.rk);
            if constexpr (EIGHT) {
                wm = gq::philox_row(pg, s.row, step_lo, a.rng.rk);
                wr = gq::philox_row(pg, s.row + 1, step_lo, a.rng.rk);
            }
            if constexpr (sizeof(P) == 2) wp = gq::philox_row(pg, s.row + 2, step_lo, a.rng.rk);
        }
        float x[8];
        apart(p, x);
        if constexpr (RANDOM && sizeof(P) == 2) {
            const uint32_t h[4] = {wp.x, wp.y, wp.z, wp.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t b = __float_as_uint(x[j]);
                if ((b & 0x7F800000u) != 0x7F800000u)
                    x[j] = __uint_as_float((b + (h[j >> 1] >> (16 * (j & 1)) & 0xFFFFu)) & 0xFFFF0000u);
            }
        }
        put8<P>(s.p, i, left, s.wp, x);
        if constexpr (EIGHT) {
            uint32_t y[8];
            apart(m, x);
            const uint32_t em = fp8_exp_byte(top32(x));
            uint32_t sign[2] = {gather_bytes<3>(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                                                __float_as_uint(x[3])),
                                gather_bytes<3>(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]),
                                                __float_as_uint(x[7]))};
            F2 im = f2(inv_step(em));
#pragma unroll
            for (int j = 0; j < 4; ++j) m[j] = mul2(mul2(m[j], im), f2(0x1p-120f));  // e4m3's exponent field
            apart(m, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = __float_as_uint(x[j]);
            uint2 cm = codes_of<4, RANDOM>(y, wm);  // (the sign is shifted out)
            cm.x = (cm.x & 0x7F7F7F7Fu) | (sign[0] & 0x80808080u);
            cm.y = (cm.y & 0x7F7F7F7Fu) | (sign[1] & 0x80808080u);
            if (em == 255u) cm = make_uint2(0u, 0u);

            apart(r, x);
            const uint32_t er = root_exp_byte(top32(x));
            im = f2(__uint_as_float((188u - min(er, 187u)) << 23));
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = min(__float_as_uint(x[j]), 1u << 19);  // the least code, or 0
#pragma unroll
            for (int j = 0; j < 4; ++j) r[j] = mul2(mul2(r[j], im), f2(0x1p-64f));
            apart(r, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = max(__float_as_uint(x[j]), y[j]);
            uint2 cr = codes_of<5, RANDOM>(y, wr);
            if (er == 255u) cr = make_uint2(0u, 0u);
            // where the tensor ends inside a block of 32, its other lanes' codes are zeros
            if ((i & ~int64_t(31)) < s.n) {
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(s.m) + i) = cm;
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(s.v) + i) = cr;
                if ((threadIdx.x & 3) == 0) reinterpret_cast<uint16_t*>(s.e)[i >> 5] = static_cast<uint16_t>(em | er << 8);
            }
        } else {
            apart(m, x);
            put8<float>(s.m, i, left, s.wm, x);
            apart(v, x);
            put8<float>(s.v, i, left, s.wv, x);
        }
    }
}

// The values of 8-bit states: first moments to p, roots to g (the slot's places for two outputs).
template <typename O, int N>
__global__ void __launch_bounds__(kThreadsA) values_kernel(const __grid_constant__ Table<N> t, int rounds) {
    const Slot& s = t.s[t.of(blockIdx.x)];
    const int64_t begin = static_cast<int64_t>(blockIdx.x - s.first) * (rounds * kRound) + threadIdx.x * 8;
#pragma unroll 2
    for (int k = 0; k < rounds; ++k) {
        const int64_t i = begin + k * kRound, left = s.n - i;
        if (left <= 0) break;
        const uint2 cm = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(s.m) + i));
        const uint2 cv = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(s.v) + i));
        const uint32_t e = __ldg(reinterpret_cast<const uint16_t*>(s.e) + (i >> 5));
        F2 v[4];
        float x[8];
        moments8(cm, e & 255u, v);
        apart(v, x);
        put8<O>(s.p, i, left, s.wp, x);
        roots8(cv, e >> 8, v);
        apart(v, x);
        put8<O>(const_cast<void*>(s.g), i, left, s.wg, x);
    }
}

// ---- the norm ------------------------------------------------------------------------------

constexpr int kNormBlocks = 1216;  // partial sums per launch: at most

// Sums of squares of the chunks blockIdx.x, blockIdx.x + gridDim.x, ...: fp32 over a thread's elements of a
// chunk (64 at most) and over a warp, with what chunks' sums lose carried along; fp64 over warps and blocks
// (over threads, its few units took 3 us of a pass).  A block whose sums leave fp32's range reads its chunks once
// more and adds in fp64 from the first square on: the norm is no number only where a square is none.
template <typename G, int N>
__global__ void __launch_bounds__(256)
    squares_kernel(const __grid_constant__ Table<N> t, uint32_t chunks, int rounds, double* partial) {
    gq::pdl_wait();
    gq::pdl_launch_dependents();  // the sum of the sums waits before it reads
    float sum = 0.0f, carry = 0.0f;
    for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        const Slot& s = t.s[t.of(c)];
        int64_t i = static_cast<int64_t>(c - s.first) * (rounds * kRound) + threadIdx.x * 8;
        F2 part[2] = {f2(0.0f), f2(0.0f)};
        for (int k = 0; k < rounds; k += 4) {
            Raw8<G> w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j, i += kRound) {
                if (k + j < rounds && i < s.n) {
                    w[j] = raw8<G>(s.g, i, s.n - i, s.wg);
                } else {
#pragma unroll
                    for (int q = 0; q < static_cast<int>(sizeof(G)) * 2; ++q) w[j].w[q] = 0u;
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                F2 g[4];
                pairs(w[j], g);
#pragma unroll
                for (int q = 0; q < 4; ++q) part[q & 1] = fma2(g[q], g[q], part[q & 1]);
            }
        }
        const float more = sum2(add2(part[0], part[1])) - carry, all = sum + more;
        carry = (all - sum) - more;
        sum = all;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    __shared__ float warps[8];
    if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = sum;
    // (an infinity or a NaN among the gradients, or sums above 3.4e38, which leave an infinity or a NaN behind)
    if (__syncthreads_or(!(sum < INFINITY))) {
        double wide = 0.0;
        for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
            const Slot& s = t.s[t.of(c)];
            int64_t i = static_cast<int64_t>(c - s.first) * (rounds * kRound) + threadIdx.x * 8;
#pragma unroll 1
            for (int k = 0; k < rounds && i < s.n; ++k, i += kRound) {
                F2 g[4];
                pairs(raw8<G>(s.g, i, s.n - i, s.wg), g);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float x, y;
                    split(mul2(g[q], g[q]), x, y);
                    wide += static_cast<double>(x);
                    wide += static_cast<double>(y);
                }
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) wide += __shfl_xor_sync(kFull, wide, o);
        __shared__ double wides[8];
        if ((threadIdx.x & 31) == 0) wides[threadIdx.x >> 5] = wide;
        __syncthreads();
        if (threadIdx.x == 0) {
            double all = 0.0;
#pragma unroll
            for (int i = 0; i < 8; ++i) all += wides[i];
            partial[blockIdx.x] = all;
        }
        return;
    }
    if (threadIdx.x == 0) {
        double all = 0.0;
#pragma unroll
        for (int i = 0; i < 8; ++i) all += static_cast<double>(warps[i]);
        partial[blockIdx.x] = all;
    }
}
__global__ void __launch_bounds__(256) root_kernel(const double* partial, int64_t n, float* norm) {
    gq::pdl_launch_dependents();
    gq::pdl_wait();
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

// Rounds of a block, of `most`: fewer where the tensors would not give every SM several blocks.
int rounds_for(int64_t count, const int64_t* numel, int most) {
    int64_t total = 0;
    for (int64_t i = 0; i < count; ++i) total += numel[i];
    const int64_t each = total / (8 * gqh::sm_count()) / kRound;
    return each < 1 ? 1 : each < most ? static_cast<int>(each) : most;
}

// Widest access to 8 elements at a time.
uint8_t wide(const void* p) { return mult(p, 32) ? 32 : mult(p, 16) ? 16 : 0; }

template <typename P, typename G, bool EIGHT, bool RANDOM>
gq_status adamw(int64_t count, void* const* params, const void* const* grads, void* const* m, void* const* v,
                uint8_t* const* exps, const int64_t* numel, int64_t first, const int64_t* places,
                const int64_t* step_places, Step a, cudaStream_t st) {
    auto fill = [&](Slot& s, int64_t i) {
        s.p = params[i]; s.g = grads[i]; s.m = m[i]; s.v = v[i];
        s.e = EIGHT ? exps[i] : nullptr;
        s.row = static_cast<uint32_t>(3 * (first + (places ? places[i] : i)));
        s.at = step_places ? static_cast<uint32_t>(step_places[i]) : 0u;
        s.wp = wide(s.p); s.wg = wide(s.g); s.wm = wide(s.m); s.wv = wide(s.v);
    };
    a.rounds = rounds_for(count, numel, EIGHT ? 16 : 4);
    if (count <= kFew)
        return in_runs<kFew>(count, numel, a.rounds * kRound, fill, [&](const Table<kFew>& t, uint32_t blocks) {
            launch_early(adamw_kernel<P, G, EIGHT, RANDOM, kFew>, blocks, kThreadsA, st, t, a);
        });
    return in_runs<kMany>(count, numel, a.rounds * kRound, fill, [&](const Table<kMany>& t, uint32_t blocks) {
        launch_early(adamw_kernel<P, G, EIGHT, RANDOM, kMany>, blocks, kThreadsA, st, t, a);
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
    const uint32_t most = static_cast<uint32_t>(8 * gqh::sm_count() < kNormBlocks ? 8 * gqh::sm_count() : kNormBlocks);
    const int rounds = rounds_for(count, numel, 8);
    auto run = [&](const auto& t, uint32_t chunks) {
        constexpr int N = sizeof(t.s) / sizeof(Slot);
        const uint32_t blocks = chunks < most ? chunks : most;
        if (dtype == GQ_F32) launch_early(squares_kernel<float, N>, blocks, 256, st, t, chunks, rounds, partial + parts);
        else launch_early(squares_kernel<bf16, N>, blocks, 256, st, t, chunks, rounds, partial + parts);
        parts += blocks;
    };
    const gq_status r = count <= kFew ? in_runs<kFew>(count, numel, rounds * kRound, fill, run)
                                      : in_runs<kMany>(count, numel, rounds * kRound, fill, run);
    if (r != GQ_OK) return r;
    launch_early(root_kernel, 1, kThreadsA, st, static_cast<const double*>(partial), parts, norm_dev);
    return gqh::launch_status();
}

gq_status gq_adamw_step(int64_t count, void *const *params, int param_dtype, const void *const *grads,
                        int grad_dtype, void *const *m, void *const *v, uint8_t *const *exps,
                        const int64_t *numel, int64_t step, const int64_t *step_dev, double lr, double beta1,
                        double beta2, double eps, double weight_decay, const float *norm_dev, double max_norm,
                        int rounding, uint64_t seed, int64_t first, void *stream) {
    return gq_adamw_step_places(count, params, param_dtype, grads, grad_dtype, m, v, exps, numel, step, step_dev, lr,
                                beta1, beta2, eps, weight_decay, norm_dev, max_norm, rounding, seed, first, nullptr,
                                nullptr, stream);
}

gq_status gq_adamw_step_places(int64_t count, void *const *params, int param_dtype, const void *const *grads,
                               int grad_dtype, void *const *m, void *const *v, uint8_t *const *exps,
                               const int64_t *numel, int64_t step, const int64_t *step_dev, double lr, double beta1,
                               double beta2, double eps, double weight_decay, const float *norm_dev, double max_norm,
                               int rounding, uint64_t seed, int64_t first, const int64_t *places,
                               const int64_t *step_places, void *stream) {
    if (!in_type(param_dtype) || !in_type(grad_dtype) || !sizes_ok(count, numel)) return GQ_ERR_INVALID;
    if (count > 0 && (!params || !grads || !m || !v)) return GQ_ERR_INVALID;
    if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || !(eps >= 0.0) || !std::isfinite(lr) ||
        !std::isfinite(weight_decay) || (!step_dev && step < 1) || !mult(step_dev, 8) || !mult(norm_dev, 4))
        return GQ_ERR_INVALID;
    if ((rounding != GQ_ACT_NEAREST && rounding != GQ_ACT_RANDOM) || first < 0 || first > (int64_t(1) << 30) - count)
        return GQ_ERR_INVALID;
    for (int64_t i = 0; places && i < count; ++i)
        if (places[i] < (i > 0 ? places[i - 1] + 1 : 0) || places[i] >= (int64_t(1) << 30) - first) return GQ_ERR_INVALID;
    if (step_places && !step_dev) return GQ_ERR_INVALID;
    for (int64_t i = 0; step_places && i < count; ++i)
        if (step_places[i] < 0 || step_places[i] >= int64_t(1) << 31) return GQ_ERR_INVALID;
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
    a.rng = make_rng(seed, static_cast<uint64_t>(step));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool random = rounding == GQ_ACT_RANDOM;
#define GQA_ADAMW(P, G, EIGHT, RANDOM) \
    adamw<P, G, EIGHT, RANDOM>(count, params, grads, m, v, exps, numel, first, places, step_places, a, st)
#define GQA_STATE(P, G)                                                                     \
    (exps ? random ? GQA_ADAMW(P, G, true, true) : GQA_ADAMW(P, G, true, false)              \
          : random && sizeof(P) == 2 ? GQA_ADAMW(P, G, false, (sizeof(P) == 2)) : GQA_ADAMW(P, G, false, false))
    if (param_dtype == GQ_F32) return grad_dtype == GQ_F32 ? GQA_STATE(float, float) : GQA_STATE(float, bf16);
    return grad_dtype == GQ_F32 ? GQA_STATE(bf16, float) : GQA_STATE(bf16, bf16);
#undef GQA_STATE
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
    const int rounds = rounds_for(count, numel, 4);
    auto fill = [&](Slot& s, int64_t i) {
        s.p = moments[i]; s.g = roots[i];
        s.m = const_cast<uint8_t*>(m[i]); s.v = const_cast<uint8_t*>(v[i]);
        s.e = const_cast<uint8_t*>(exps[i]);
        s.wp = wide(s.p); s.wg = wide(s.g);
    };
    auto run = [&](const auto& t, uint32_t blocks) {
        constexpr int N = sizeof(t.s) / sizeof(Slot);
        if (out_dtype == GQ_F32) values_kernel<float, N><<<blocks, kThreadsA, 0, st>>>(t, rounds);
        else values_kernel<bf16, N><<<blocks, kThreadsA, 0, st>>>(t, rounds);
    };
    return count <= kFew ? in_runs<kFew>(count, numel, rounds * kRound, fill, run)
                         : in_runs<kMany>(count, numel, rounds * kRound, fill, run);
}

}  // extern "C"
