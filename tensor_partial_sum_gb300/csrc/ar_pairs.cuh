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
// Their sum, in pairs of pairs.
template <int N>
__device__ __forceinline__ float sum_pairs(const pair_t (&v)[N]) {
    pair_t s[N];
#pragma unroll
    for (int k = 0; k < N; ++k) s[k] = v[k];
#pragma unroll
    for (int n = N / 2; n > 0; n /= 2)
#pragma unroll
        for (int k = 0; k < n; ++k) s[k] = add2(s[k], s[k + n]);
    const float2 f = halves(s[0]);
    return f.x + f.y;
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
