// gq_act.cu -- 8-bit activation checkpoints and GELU over them (C ABI in include/gq.h).
//
// Every kernel here reads each input once and writes each output once: it is bound by memory, and
// next to that by the instructions it issues (random rounding above all: a Philox call per 8
// elements).  A thread owns a piece of 16 columns (half a block of the format; the other half is its
// neighbour's) and walks down the rows, so that the column part of the random words is computed once
// and the next rows' copies are in flight meanwhile.  At 32,768 x 4,096 bf16 (268 MB), call after call with
// inputs that change, saving takes 69 us rounding to nearest (5.9 TB/s) and 78 at random (its issue slots
// 69 % busy), reading back 73 (5.6 TB/s), GELU forward 92 without a checkpoint, 121 with one rounded to
// nearest (5.6 TB/s) and 137 at random, backward 121 and with the output 155 (6.1 TB/s).
#include "gq_act.cuh"

#include <type_traits>

using namespace gqa;

namespace {

constexpr int kT = 256;  // threads per block

// ---- GELU ----------------------------------------------------------------------------------
// Normal distribution function at -|u|: q(|u|) = t P(t) exp(-u^2 / 2), t = 1 / (1 + p |u|), the form of
// Hastings' approximations (1955).  The polynomials are least-maximum fits of erfc(z) exp(z^2) / 2, z =
// u / sqrt 2, over 0 <= u <= 14 (computed for this file by iteratively reweighted least squares on
// Chebyshev nodes); the fit's relative error is below 1.7e-7 (8 coefficients, fp32 outputs) or 4.7e-6 (6
// coefficients, bf16 outputs, whose own rounding is 2e-3).  GELU as computed for fp32 outputs is within
// 2.7e-7 |u| of its value everywhere, and within 5.4e-7 of it for |u| < 1, 2.1e-6 down to u = -6 and 8.1e-6
// down to -13, where the rounding of u^2 / 2 enters through the exponential.  One exponential serves the
// distribution and the density.  Two elements are worked on at a time (pairs of fp32): instructions, not
// memory, bounded the first form of the backward pass (32,768 x 4,096 bf16 with the output: 239 us one at a
// time, 150 so, of which the memory needs 139).
template <bool WIDE> struct Tail;
template <> struct Tail<true> {
    static constexpr float p = 0.30f;
    static constexpr int n = 8;
    static __device__ __forceinline__ float c(int i) {
        const float k[n] = {0.03567477688193321f, -0.15720310807228088f, 0.20635353028774261f,
                            -0.05368367210030556f, 0.12856164574623108f, 0.09991348534822464f,
                            0.12075395882129669f, 0.11962930113077164f};
        return k[i];
    }
};
template <> struct Tail<false> {
    static constexpr float p = 0.31f;
    static constexpr int n = 6;
    static __device__ __forceinline__ float c(int i) {
        const float k[n] = {-0.07392916828393936f, 0.1804504245519638f, 0.01574462652206421f,
                            0.13342982530593872f, 0.1204412654042244f, 0.1238607019186019f};
        return k[i];
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
__device__ __forceinline__ F2 exp2_fast(F2 a) {
    float x, y;
    split(a, x, y);
    return f2(exp2_fast(x), exp2_fast(y));
}
__device__ __forceinline__ F2 rcp_fast(F2 a) {
    float x, y;
    split(a, x, y);
    return f2(rcp_fast(x), rcp_fast(y));
}
__device__ __forceinline__ F2 abs2(F2 a) { return F2{a.v & 0x7FFFFFFF7FFFFFFFull}; }

// Phi(u), and with DENSITY u phi(u) too.
template <bool WIDE, bool DENSITY>
__device__ __forceinline__ F2 normal_cdf(F2 u, F2* u_phi) {
    const F2 t = rcp_fast(fma2(abs2(u), f2(Tail<WIDE>::p), f2(1.0f)));
    const F2 g = exp2_fast(mul2(mul2(u, f2(-0.72134752044448170f)), u));  // exp(-u^2 / 2)
    F2 q = f2(Tail<WIDE>::c(0));
#pragma unroll
    for (int i = 1; i < Tail<WIDE>::n; ++i) q = fma2(q, t, f2(Tail<WIDE>::c(i)));
    q = mul2(mul2(q, t), g);
    if constexpr (DENSITY) *u_phi = mul2(u, mul2(g, f2(0.39894228040143268f)));
    float u0, u1, q0, q1;
    split(u, u0, u1);
    split(q, q0, q1);
    return f2(u0 < 0.0f ? q0 : 1.0f - q0, u1 < 0.0f ? q1 : 1.0f - q1);
}

// 1 / (1 + exp(-2 z)) with z = sqrt(2/pi) (u + 0.044715 u^3), which is (1 + tanh z) / 2; u is
// held to +-16, where it is 0 or 1 already and u^3 cannot overflow.
template <bool DENSITY>
__device__ __forceinline__ F2 tanh_cdf(F2 u, F2* u_phi) {
    constexpr float k = 0.79788456080286536f, b = 0.044715f, l = -2.8853900817779268f;  // -2 / ln 2
    float x, y;
    split(u, x, y);
    const F2 c = f2(fminf(fmaxf(x, -16.0f), 16.0f), fminf(fmaxf(y, -16.0f), 16.0f));
    const F2 c2 = mul2(c, c);
    const F2 z = mul2(c, fma2(c2, f2(k * b * l), f2(k * l)));
    const F2 p = rcp_fast(add2(exp2_fast(z), f2(1.0f)));
    if constexpr (DENSITY) {
        const F2 d = mul2(mul2(p, fma2(p, f2(-2.0f), f2(2.0f))), fma2(c2, f2(3.0f * k * b), f2(k)));
        *u_phi = mul2(u, d);
    }
    return p;
}

enum Op { kSave = 0, kGeluErf = GQ_GELU_ERF + 1, kGeluTanh = GQ_GELU_TANH + 1 };

template <int OP, bool WIDE, bool DENSITY>
__device__ __forceinline__ F2 cdf(F2 u, F2* u_phi) {
    if constexpr (OP == kGeluErf) return normal_cdf<WIDE, DENSITY>(u, u_phi);
    else return tanh_cdf<DENSITY>(u, u_phi);
}

// Threads numbered along the pieces of a row, then along `lanes` rows; each goes on with every
// `lanes`-th row.  All make the same number of turns: neighbours may sit in different rows, and reduce
// over the warp.
struct Walk {
    uint32_t lanes, turns, rows, cols, pitch, epitch;
    Div per_row;
};

// Slots of a ring: kDepth, or 2 where 64 + 16 bytes per thread and row would leave room for one block.
template <typename T, bool ALIGNED> constexpr int kRing = sizeof(T) == 4 && !ALIGNED ? 2 : kDepth;

// 16 elements of type T of a thread, in words of 32 bits.
template <typename T> constexpr int kWords = 4 * sizeof(T);

// Brings the 16 elements at p (column c) into planes of 16 bytes per thread.  With ALIGNED rows the
// part behind the last column arrives as zeros.  Otherwise the 16-byte granules that hold a byte of
// them are copied, one more at most.
template <typename T, bool ALIGNED>
__device__ __forceinline__ void fetch16(uint32_t to, uint32_t plane, const T* p, int left) {
    const uint8_t* q = reinterpret_cast<const uint8_t*>(p);
    constexpr int N = sizeof(T);  // granules of 16 aligned elements
    if constexpr (ALIGNED) {
        if (left >= 16) {
#pragma unroll
            for (int i = 0; i < N; ++i) copy_async<16>(to + i * plane, q + 16 * i);
        } else if (left > 0) {
            const int bytes = left * static_cast<int>(sizeof(T));
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int n = max(0, min(16, bytes - 16 * i));
                copy_part(to + i * plane, n ? q + 16 * i : q, n);
            }
        }
    } else {
        const int m = static_cast<int>(reinterpret_cast<uintptr_t>(q) & 15u);
        const int bytes = m + min(left, 16) * static_cast<int>(sizeof(T));
#pragma unroll
        for (int i = 0; i <= N; ++i)
            if (left > 0 && 16 * i < bytes) copy_async<16>(to + i * plane, q - m + 16 * i);
    }
}
template <typename T, bool ALIGNED>
__device__ __forceinline__ void read16(const uint8_t* at, uint32_t plane, const T* p, int left,
                                       uint32_t (&w)[kWords<T>]) {
    constexpr int N = sizeof(T), W = kWords<T>;
    uint32_t r[W + 4];
#pragma unroll
    for (int i = 0; i < (ALIGNED ? N : N + 1); ++i) {
        const uint4 a = *reinterpret_cast<const uint4*>(at + i * plane);
        r[4 * i] = a.x; r[4 * i + 1] = a.y; r[4 * i + 2] = a.z; r[4 * i + 3] = a.w;
    }
    if (ALIGNED && left <= 0) {  // padding: nothing was copied
#pragma unroll
        for (int i = 0; i < W; ++i) r[i] = 0u;
    }
    if constexpr (!ALIGNED) {  // moves the words down by the row's offset in its granule
        const uint32_t m = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 15u;
#pragma unroll
        for (int i = 0; i < W + 2; ++i) r[i] = (m & 8u) ? r[i + 2] : r[i];
#pragma unroll
        for (int i = 0; i < W + 1; ++i) r[i] = (m & 4u) ? r[i + 1] : r[i];
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < W; ++i) r[i] = __funnelshift_r(r[i], r[i + 1], (m & 2u) * 8u);
        }
        if (left < 16) {
#pragma unroll
            for (int i = 0; i < W; ++i) {
                if constexpr (sizeof(T) == 4) {
                    if (i >= left) r[i] = 0u;
                } else {
                    if (2 * i >= left) r[i] = 0u;
                    else if (2 * i + 1 >= left) r[i] &= 0xFFFFu;
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = r[i];
}
template <typename T>
__device__ __forceinline__ void pairs16(const uint32_t (&w)[kWords<T>], F2 (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (sizeof(T) == 4)
            v[i] = f2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        else
            v[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    }
}

// Largest magnitude of 16 elements as fp32 bits, a NaN above all.
template <typename T> __device__ __forceinline__ uint32_t top16(const uint32_t (&w)[kWords<T>]) {
    if constexpr (sizeof(T) == 2) {  // two at a time; the sign that comes out is not used
        uint32_t m = w[0];
#pragma unroll
        for (int i = 1; i < 8; ++i)
            asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(w[i]));
        m &= 0x7FFF7FFFu;
        return max(m << 16, m & 0xFFFF0000u);
    } else {
        uint32_t m = w[0] & 0x7FFFFFFFu;
#pragma unroll
        for (int i = 1; i < 16; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
        return m;
    }
}

// Stores a lane's 16 elements of a row that is not 16-byte aligned, of which `left` lie in the row.
// adjoins: the lane before holds what is in front of them.  16-byte granules are put together from two neighbours' words; only where a neighbour is missing, and at the row's end, are elements
// stored one by one.  The whole warp takes part.
template <typename T>
__device__ __forceinline__ void put_words(T* p, int left, bool adjoins, const uint32_t (&w)[kWords<T>]) {
    constexpr int E = sizeof(T), NW = kWords<T>, N = 16, G = 16 / E;  // words, elements, those of a granule
    const int lane = threadIdx.x & 31;
    const uint32_t m = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 15u;
    const int full = left >= N;
    const int before = __shfl_up_sync(kFull, full, 1);
    const int joined = full && before && adjoins && lane > 0;
    const int after = __shfl_down_sync(kFull, joined, 1);
    uint32_t r[NW + 4];
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __shfl_up_sync(kFull, w[NW - 4 + i], 1);
#pragma unroll
    for (int i = 0; i < NW; ++i) r[4 + i] = w[i];
    const uint32_t d = 16u - m;  // the first granule's start in r
#pragma unroll
    for (int i = 0; i < NW; ++i) r[i] = (d & 16u) ? r[i + 4] : r[i];
#pragma unroll
    for (int i = 0; i < NW + 2; ++i) r[i] = (d & 8u) ? r[i + 2] : r[i];
#pragma unroll
    for (int i = 0; i < NW + 1; ++i) r[i] = (d & 4u) ? r[i + 1] : r[i];
    if constexpr (E == 2) {
#pragma unroll
        for (int i = 0; i < NW; ++i) r[i] = __funnelshift_r(r[i], r[i + 1], (d & 2u) * 8u);
    }
    auto one = [&](int i) {
        if constexpr (E == 4) reinterpret_cast<uint32_t*>(p)[i] = w[i];
        else reinterpret_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(w[i / 2] >> i % 2 * 16);
    };
    if (full) {
        uint4* q = reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(p) - m);
#pragma unroll
        for (int j = 0; j < NW / 4; ++j)
            if (j > 0 || joined || m == 0u)
                q[j] = make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
        if (m != 0u && !joined) {  // up to the first granule's end
#pragma unroll
            for (int i = 0; i < G; ++i)
                if (E * i < static_cast<int>(d)) one(i);
        }
        if (m != 0u && (!after || lane == 31)) {  // the next granule's part
#pragma unroll
            for (int i = 0; i < G; ++i)
                if (E * (G - i) <= static_cast<int>(m)) one(N - G + i);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < left) one(i);
    }
}
// The other way, for fp32 values that were read from codes: a piece's 16 values go to shared memory, and
// 16 lanes each store those of one piece after the other, neighbours to neighbours.  (13,860 x 1,922
// fp32: read from codes in 28 us so, in 33 by granules; GELU forward with random codes 55 so, 51 by
// granules.  32,046 x 1,317 bf16: read from codes in 42 so, in 29 by granules.)
struct Stage {
    float v[32][17];
    void* to[32];
    int left[32];
};
template <typename T, bool GRANULES>
__device__ __forceinline__ void put16(T* p, bool live, bool adjoins, int left, int align, Stage* st,
                                      const F2 (&v)[8]) {
    float o[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) split(v[i], o[2 * i], o[2 * i + 1]);
    if (align == 0) {
        if constexpr (GRANULES) {
            uint32_t w[kWords<T>];
#pragma unroll
            for (int i = 0; i < kWords<T>; ++i) {
                if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(o[i]);
                else w[i] = pack2(o[2 * i], o[2 * i + 1], T());
            }
            put_words(p, live ? left : 0, adjoins, w);
        } else {
            const int lane = threadIdx.x & 31;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 16; ++i) st->v[lane][i] = o[i];
            st->to[lane] = p;
            st->left[lane] = live ? left : 0;
            __syncwarp();
#pragma unroll 4
            for (int i = 0; i < 16; ++i) {
                const int k = 2 * i + (lane >> 4), j = lane & 15;
                if (j < st->left[k]) static_cast<T*>(st->to[k])[j] = st->v[k][j];
            }
        }
    } else if (live) {
        if (align == 32) store<T, 16, 32>(p, 0, left, o);
        else store<T, 16, 16>(p, 0, left, o);
    }
}

// x -> codes and exponents (OP = kSave), or h = gelu(x) with or without them.
template <typename T, bool ALIGNED, int OP, int RND>
__global__ void __launch_bounds__(kT, 4)
    save_kernel(const T* __restrict__ x, int64_t ldx, T* __restrict__ h, int64_t ldh, int align,
                Walk a, Rng rng, int8_t* __restrict__ codes, uint8_t* __restrict__ exps) {
    extern __shared__ __align__(16) uint8_t ring[];
    constexpr int N = sizeof(T) + (ALIGNED ? 0 : 1), D = kRing<T, ALIGNED>;
    constexpr uint32_t plane = kT * 16, slot = plane * N;
    const uint32_t id = blockIdx.x * kT + threadIdx.x, first = quot(id, a.per_row);
    const uint32_t piece = id - first * a.per_row.d, c = piece * 16;
    const int left = static_cast<int>(a.cols) - static_cast<int>(c);
    const bool mine = first < a.lanes;
    const uint32_t base = gq::smem_u32(ring) + threadIdx.x * 16;
    gq::PhiloxGroup pg[2];
    if constexpr (RND == 1) {
        pg[0] = gq::philox_group(2 * piece, rng.step_lo, rng.step_hi, rng.rk);
        pg[1] = gq::philox_group(2 * piece + 1, rng.step_lo, rng.step_hi, rng.rk);
    }
    uint32_t ahead = first, turn = 0;
    auto fetch = [&]() {
        if (mine && ahead < a.rows)
            fetch16<T, ALIGNED>(base + (turn & (D - 1)) * slot, plane,
                                x + static_cast<int64_t>(ahead) * ldx + c, left);
        copy_commit();
        ahead += a.lanes;
        ++turn;
    };
#pragma unroll
    for (int d = 0; d < D - 1; ++d) fetch();
    uint32_t row = first;
    for (uint32_t k = 0; k < a.turns; ++k, row += a.lanes) {
        fetch();
        copy_wait<D>();
        const bool live = mine && row < a.rows;
        uint32_t w[kWords<T>];
        F2 v[8];
        read16<T, ALIGNED>(ring + threadIdx.x * 16 + (turn & (D - 1)) * slot, plane,
                           x + static_cast<int64_t>(row) * ldx + c, left, w);
        pairs16<T>(w, v);
        if constexpr (RND >= 0) {
            uint32_t m = top16<T>(w);
            m = max(m, __shfl_xor_sync(kFull, m, 1));
            const uint32_t e = exp_byte(m);
            uint2 q[2];
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const F2 half[4] = {v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]};
                uint4 r = make_uint4(0u, 0u, 0u, 0u);
                if constexpr (RND == 1) r = gq::philox_row(pg[g], row, rng.step_lo, rng.rk);
                q[g] = codes8<RND == 1>(half, e, r);
            }
            if (live) {
                *reinterpret_cast<uint4*>(row_of(codes, row, a.pitch) + c) =
                    make_uint4(q[0].x, q[0].y, q[1].x, q[1].y);
                if ((piece & 1) == 0) row_of(exps, row, a.epitch)[piece >> 1] = static_cast<uint8_t>(e);
            }
        }
        if constexpr (OP != kSave) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = mul2(v[i], cdf<OP, sizeof(T) == 4, false>(v[i], nullptr));
            put16<T, true>(h + static_cast<int64_t>(row) * ldh + c, live, piece > 0, left, align, nullptr, v);
        }
    }
    copy_all();
}

// Codes and exponents -> values (OP = kSave), or with dy: du = dy gelu'(value) and, where h is
// given, h = gelu(value).
template <typename T, bool ALIGNED, int OP>
__global__ void __launch_bounds__(kT, 4)
    read_kernel(const int8_t* __restrict__ codes, const uint8_t* __restrict__ exps, Walk a,
                const T* __restrict__ dy, int64_t lddy, T* __restrict__ du, int64_t lddu,
                T* __restrict__ h, int64_t ldh, int align) {
    extern __shared__ __align__(16) uint8_t ring[];
    constexpr int N = OP == kSave ? 0 : sizeof(T) + (ALIGNED ? 0 : 1), D = kRing<T, ALIGNED>;
    // a slot: dy's planes, one of 16 codes per thread, one of the 4 exponent bytes with its own
    constexpr uint32_t plane = kT * 16, slot = plane * (N + 1) + kT * 4;
    const uint32_t id = blockIdx.x * kT + threadIdx.x, first = quot(id, a.per_row);
    const uint32_t piece = id - first * a.per_row.d, c = piece * 16;
    const int left = static_cast<int>(a.cols) - static_cast<int>(c);
    const bool mine = first < a.lanes;
    Stage* st = reinterpret_cast<Stage*>(ring + D * slot) + (threadIdx.x >> 5);
    const uint32_t base = gq::smem_u32(ring), tid = threadIdx.x;
    uint32_t ahead = first, turn = 0;
    auto fetch = [&]() {
        if (mine && ahead < a.rows) {
            const uint32_t to = base + (turn & (D - 1)) * slot;
            if constexpr (OP != kSave)
                fetch16<T, ALIGNED>(to + tid * 16, plane, dy + static_cast<int64_t>(ahead) * lddy + c, left);
            copy_async<16>(to + N * plane + tid * 16, row_of(codes, ahead, a.pitch) + c);
            copy_async<4>(to + (N + 1) * plane + tid * 4, row_of(exps, ahead, a.epitch) + (piece >> 3) * 4);
        }
        copy_commit();
        ahead += a.lanes;
        ++turn;
    };
#pragma unroll
    for (int d = 0; d < D - 1; ++d) fetch();
    uint32_t row = first;
    for (uint32_t k = 0; k < a.turns; ++k, row += a.lanes) {
        fetch();
        copy_wait<D>();
        const bool live = mine && row < a.rows;
        const uint8_t* at = ring + (turn & (D - 1)) * slot;
        const uint4 q = *reinterpret_cast<const uint4*>(at + N * plane + tid * 16);
        const uint32_t e4 = *reinterpret_cast<const uint32_t*>(at + (N + 1) * plane + tid * 4);
        const uint32_t e = e4 >> (piece / 2 % 4 * 8) & 0xFFu;
        F2 v[8], lo[4], hi[4];
        values8(make_uint2(q.x, q.y), e, lo);
        values8(make_uint2(q.z, q.w), e, hi);
#pragma unroll
        for (int i = 0; i < 4; ++i) { v[i] = lo[i]; v[4 + i] = hi[i]; }
        T* out = du + static_cast<int64_t>(row) * lddu + c;
        if constexpr (OP == kSave) {
            put16<T, sizeof(T) == 2>(out, live, piece > 0, left, align, st, v);
        } else {
            uint32_t w[kWords<T>];
            F2 g[8];
            read16<T, ALIGNED>(at + tid * 16, plane, dy + static_cast<int64_t>(row) * lddy + c, left, w);
            pairs16<T>(w, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                F2 u_phi;
                const F2 p = cdf<OP, sizeof(T) == 4, true>(v[i], &u_phi);
                g[i] = mul2(g[i], add2(p, u_phi));
                v[i] = mul2(v[i], p);
            }
            put16<T, sizeof(T) == 2>(out, live, piece > 0, left, align, st, g);
            if (h) put16<T, sizeof(T) == 2>(h + static_cast<int64_t>(row) * ldh + c, live, piece > 0, left, align, st, v);
        }
    }
    copy_all();
}

// Threads for a matrix: as many rows at a time as one wave of resident blocks holds, spread evenly
// over the turns.
template <typename K>
unsigned plan_walk(K kernel, size_t smem, int64_t rows, int64_t cols, Walk& a) {
    const int64_t pieces = code_pitch(cols) / 16;
    const int64_t most = resident_blocks(kernel, kT, smem) * kT / pieces;
    const int64_t lanes = most < 1 ? 1 : most < rows ? most : rows;
    a.turns = static_cast<uint32_t>((rows + lanes - 1) / lanes);
    a.lanes = static_cast<uint32_t>((rows + a.turns - 1) / a.turns);
    a.rows = static_cast<uint32_t>(rows);
    a.cols = static_cast<uint32_t>(cols);
    a.pitch = static_cast<uint32_t>(code_pitch(cols));
    a.epitch = static_cast<uint32_t>(exp_pitch(cols));
    a.per_row = make_div(static_cast<uint32_t>(pieces));
    return static_cast<unsigned>((a.lanes * pieces + kT - 1) / kT);
}
template <typename T> constexpr size_t stage_bytes(int align) {
    return align || sizeof(T) == 2 ? 0 : kT / 32 * sizeof(Stage);
}

// What a call is made of; rows 32-, 16- or 0-byte aligned.
struct SaveCall {
    const void* x;
    int64_t ldx;
    void* h;
    int64_t ldh, rows, cols;
    int in, out;
    Rng rng;
    int8_t* codes;
    uint8_t* exps;
    cudaStream_t st;
};
template <typename T, bool ALIGNED, int OP, int RND> gq_status run_save(const SaveCall& s) {
    auto k = save_kernel<T, ALIGNED, OP, RND>;
    const size_t smem = kRing<T, ALIGNED> * kT * 16 * (sizeof(T) + (ALIGNED ? 0 : 1));
    Walk a;
    const unsigned grid = plan_walk(k, smem, s.rows, s.cols, a);
    k<<<grid, kT, smem, s.st>>>(static_cast<const T*>(s.x), s.ldx, static_cast<T*>(s.h), s.ldh, s.out, a,
                                s.rng, s.codes, s.exps);
    return gqh::launch_status();
}
template <typename T, int OP> gq_status any_save(const SaveCall& s, int rnd) {
#define GQA_SAVE(RND) (s.in ? run_save<T, true, OP, RND>(s) : run_save<T, false, OP, RND>(s))
    if (rnd == GQ_ACT_RANDOM) return GQA_SAVE(1);
    if constexpr (OP != kSave) {
        if (!s.codes) return GQA_SAVE(-1);
    }
    return GQA_SAVE(0);
#undef GQA_SAVE
}

struct ReadCall {
    const int8_t* codes;
    const uint8_t* exps;
    int64_t rows, cols;
    const void* dy;
    int64_t lddy;
    void* du;
    int64_t lddu;
    void* h;
    int64_t ldh;
    int in, out;
    cudaStream_t st;
};
template <typename T, bool ALIGNED, int OP> gq_status run_read(const ReadCall& s) {
    auto k = read_kernel<T, ALIGNED, OP>;
    const size_t n = OP == kSave ? 0 : sizeof(T) + (ALIGNED ? 0 : 1);
    const size_t smem = kRing<T, ALIGNED> * (kT * 16 * (n + 1) + kT * 4) + stage_bytes<T>(s.out);
    Walk a;
    const unsigned grid = plan_walk(k, smem, s.rows, s.cols, a);
    k<<<grid, kT, smem, s.st>>>(s.codes, s.exps, a, static_cast<const T*>(s.dy), s.lddy,
                                static_cast<T*>(s.du), s.lddu, static_cast<T*>(s.h), s.ldh, s.out);
    return gqh::launch_status();
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
    const SaveCall s{x, ldx, nullptr, 0, rows, cols, row_align(x, dtype, rows, ldx), 0,
                     make_rng(seed, step), codes, exps, static_cast<cudaStream_t>(stream)};
    return dtype == GQ_F32 ? any_save<float, kSave>(s, rounding) : any_save<bf16, kSave>(s, rounding);
}

gq_status gq_act_dequantize(const int8_t *codes, const uint8_t *exps, int64_t rows, int64_t cols,
                            void *out, int out_dtype, int64_t ldout, void *stream) {
    if ((!in_type(out_dtype) && out_dtype != GQ_F16) || !size_ok(rows, cols)) return GQ_ERR_INVALID;
    if (!matrix_ok(out, out_dtype, rows, cols, ldout)) return GQ_ERR_INVALID;
    if (rows == 0) return GQ_OK;
    if (!saved_ok(codes, exps)) return GQ_ERR_INVALID;
    const ReadCall s{codes, exps, rows, cols, nullptr, 0, out, ldout, nullptr, 0, 0,
                     row_align(out, out_dtype, rows, ldout), static_cast<cudaStream_t>(stream)};
    if (out_dtype == GQ_F32) return run_read<float, true, kSave>(s);
    return out_dtype == GQ_BF16 ? run_read<bf16, true, kSave>(s) : run_read<__half, true, kSave>(s);
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
    const SaveCall s{u, ldu, h, ldh, rows, cols, row_align(u, dtype, rows, ldu),
                     row_align(h, dtype, rows, ldh), make_rng(seed, step), codes, exps,
                     static_cast<cudaStream_t>(stream)};
    const int rnd = codes ? rounding : GQ_ACT_NEAREST;
    if (dtype == GQ_F32)
        return form == GQ_GELU_ERF ? any_save<float, kGeluErf>(s, rnd) : any_save<float, kGeluTanh>(s, rnd);
    return form == GQ_GELU_ERF ? any_save<bf16, kGeluErf>(s, rnd) : any_save<bf16, kGeluTanh>(s, rnd);
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
    int out = row_align(du, dtype, rows, lddu);
    if (h) out = min(out, row_align(h, dtype, rows, ldh));
    const ReadCall s{codes, exps, rows, cols, dh, lddh, du, lddu, h, ldh,
                     row_align(dh, dtype, rows, lddh), out, static_cast<cudaStream_t>(stream)};
#define GQA_READ(T, OP) (s.in ? run_read<T, true, OP>(s) : run_read<T, false, OP>(s))
    if (dtype == GQ_F32)
        return form == GQ_GELU_ERF ? GQA_READ(float, kGeluErf) : GQA_READ(float, kGeluTanh);
    return form == GQ_GELU_ERF ? GQA_READ(bf16, kGeluErf) : GQA_READ(bf16, kGeluTanh);
#undef GQA_READ
}

}  // extern "C"
