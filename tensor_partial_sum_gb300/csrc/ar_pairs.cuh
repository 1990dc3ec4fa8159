// Pairs of floats in the packed float arithmetic of sm_100 and later, whose
// results are those of the scalar instructions, and the widening and rounding
// of vectors into them.
#pragma once

#include "ar_kernels.cuh"

namespace tps {

using pair_t = unsigned long long;  // the first float in the low half

__device__ __forceinline__ pair_t make_pair(float lo, float hi) {
    pair_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ float2 halves(pair_t v) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
}
__device__ __forceinline__ pair_t both(float x) { return make_pair(x, x); }
__device__ __forceinline__ pair_t add2(pair_t a, pair_t b) {
    pair_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ pair_t sub2(pair_t a, pair_t b) {
    pair_t d;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ pair_t mul2(pair_t a, pair_t b) {
    pair_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ pair_t fma2(pair_t a, pair_t b, pair_t c) {
    pair_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// Columns in W words, and their pairs.
template <int T, int W>
constexpr int kCols = 4 * W / Elem<T>::bytes;

template <int T, int W>
__device__ __forceinline__ void widen_pairs(const uint32_t (&w)[W], pair_t (&v)[kCols<T, W> / 2]) {
#pragma unroll
    for (int k = 0; k < kCols<T, W> / 2; ++k) {
        if constexpr (T == kF32) {
            v[k] = make_pair(__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1]));
        } else {
            float lo, hi;
            widen2<T>(w[k], lo, hi);
            v[k] = make_pair(lo, hi);
        }
    }
}
template <int T, int W>
__device__ __forceinline__ void round_pairs(const pair_t (&v)[kCols<T, W> / 2], uint32_t (&w)[W]) {
#pragma unroll
    for (int k = 0; k < kCols<T, W> / 2; ++k) {
        const float2 f = halves(v[k]);
        if constexpr (T == kF32) {
            w[2 * k] = __float_as_uint(f.x);
            w[2 * k + 1] = __float_as_uint(f.y);
        } else {
            w[k] = narrow2<T>(f.x, f.y);
        }
    }
}
// Rounding through a wire type chosen at run time (kF32: none) of operands held as T.
template <int T, int N>
__device__ __forceinline__ void wire_pairs(int wire, pair_t (&v)[N]) {
    auto through = [&](auto round) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            float2 f = halves(v[k]);
            round(f.x, f.y);
            v[k] = make_pair(f.x, f.y);
        }
    };
    if (wire == kF16) through([](float &a, float &b) { wire2<T, kF16>(a, b); });
    if (wire == kBF16) through([](float &a, float &b) { wire2<T, kBF16>(a, b); });
}
// a + b, and in `lost` what its rounding left off of it (Knuth's two-sum: exact unless it overflows).
__device__ __forceinline__ float exact_add(float a, float b, float &lost) {
    const float s = __fadd_rn(a, b), z = __fsub_rn(s, a);
    lost = __fadd_rn(__fsub_rn(a, __fsub_rn(s, z)), __fsub_rn(b, z));
    return s;
}
// Sums of many terms that may cancel, with what their additions lose.  No bits get lost but those below the losses'
// own sum.
struct LongSum {
    float sum = 0.0f, lost = 0.0f;
    __device__ __forceinline__ void add(float v) {
        float e;
        sum = exact_add(sum, v, e);
        lost += e;
    }
    __device__ __forceinline__ void join(float other_sum, float other_lost) {  // the same bits whichever of the two is *this
        float e;
        sum = exact_add(sum, other_sum, e);
        lost = (lost + other_lost) + e;
    }
    __device__ __forceinline__ float value() const { return lost == lost ? sum + lost : sum; }  // an infinite sum loses NaN
};
struct PairSum {
    pair_t sum = 0, lost = 0;
    __device__ __forceinline__ void add(pair_t v) {
        const pair_t s = add2(sum, v), z = sub2(s, sum);
        lost = add2(lost, add2(sub2(sum, sub2(s, z)), sub2(v, z)));
        sum = s;
    }
    __device__ __forceinline__ LongSum joined() const {
        const float2 s = halves(sum), l = halves(lost);
        LongSum t;
        t.sum = s.x, t.lost = l.x;
        t.join(s.y, l.y);
        return t;
    }
};
// The sum of 2 N columns of type T added to `total`.  Floats keep what every addition loses.  16-bit elements are added
// plainly first: with their 8 or 11 bits in a float's 24, few of those additions lose anything, and none more than 2^-24
// of the columns' magnitudes at each of its levels (keeping it took 20% of the forward pass of bf16 [4096, 4096]).
template <int T, int N>
__device__ __forceinline__ void add_columns(const pair_t (&v)[N], LongSum &total) {
    if constexpr (T == kF32) {
        PairSum s;
        s.sum = v[0];
#pragma unroll
        for (int k = 1; k < N; ++k) s.add(v[k]);
        const LongSum j = s.joined();
        total.join(j.sum, j.lost);
    } else {
        pair_t s[N];
#pragma unroll
        for (int k = 0; k < N; ++k) s[k] = v[k];
#pragma unroll
        for (int n = N / 2; n > 0; n /= 2)
#pragma unroll
            for (int k = 0; k < n; ++k) s[k] = add2(s[k], s[k + n]);
        const float2 f = halves(s[0]);
        total.add(f.x + f.y);
    }
}
// Set the columns from `n` on to +0.
template <int N>
__device__ __forceinline__ void first_pairs(pair_t (&v)[N], int n) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const float2 f = halves(v[k]);
        v[k] = make_pair(2 * k < n ? f.x : 0.0f, 2 * k + 1 < n ? f.y : 0.0f);
    }
}

}  // namespace tps
