// Eight adjacent columns of a row as one thread holds them: one 16- or 32-byte
// vector wherever the row starts in memory.
#pragma once

#include "ar_kernels.cuh"

namespace tps {

template <int T>
constexpr int kWords8 = 2 * Elem<T>::bytes;  // 32-bit words of eight elements: 8 or 4

// Eight elements as read: the words of the vector, or of the aligned vectors around it.
template <int T, bool ALIGNED>
struct Raw8 {
    uint32_t w[kWords8<T> + (ALIGNED ? 0 : 4)];
};

// words[k] = the word `bytes` (0..15, whole elements) further on in s.
template <int NW>
__device__ __forceinline__ void shift_words(const uint32_t (&s)[NW + 4], unsigned bytes, uint32_t (&out)[NW]) {
    uint32_t a[NW + 2], b[NW + 1];
#pragma unroll
    for (int k = 0; k < NW + 2; ++k) a[k] = (bytes & 8) ? s[k + 2] : s[k];
#pragma unroll
    for (int k = 0; k < NW + 1; ++k) b[k] = (bytes & 4) ? a[k + 1] : a[k];
#pragma unroll
    for (int k = 0; k < NW; ++k) out[k] = __funnelshift_r(b[k], b[k + 1], (bytes & 3) * 8);
}

// Ask for the eight elements at `at`, the columns from `col` of a row of ne0 (whole: all eight exist).
template <int T, bool ALIGNED>
__device__ __forceinline__ void load8(const char *at, unsigned long long col, unsigned long long ne0, bool whole,
                                      Raw8<T, ALIGNED> &r) {
    constexpr int NW = kWords8<T>, es = Elem<T>::bytes;
    const unsigned off = ALIGNED ? 0 : static_cast<unsigned>(reinterpret_cast<uintptr_t>(at) & 15);
    if (off == 0 && whole) {
        if constexpr (ALIGNED) {
            load_words<4 * NW, false>(at, reinterpret_cast<uint32_t(&)[NW]>(r.w));
        } else {
#pragma unroll
            for (int k = 0; k < NW; k += 4) {
                const uint4 q = *reinterpret_cast<const uint4 *>(at + 4 * k);
                r.w[k] = q.x, r.w[k + 1] = q.y, r.w[k + 2] = q.z, r.w[k + 3] = q.w;
            }
        }
        return;
    }
    if constexpr (!ALIGNED) {
        // the aligned vectors around the eight elements, where they lie inside the row
        if (whole && col > 0 && (ne0 - col - 8) * es >= 16 - off) {
            const char *base = at - off;
#pragma unroll
            for (int k = 0; k < NW + 4; k += 4) {
                const uint4 q = *reinterpret_cast<const uint4 *>(base + 4 * k);
                r.w[k] = q.x, r.w[k + 1] = q.y, r.w[k + 2] = q.z, r.w[k + 3] = q.w;
            }
            return;
        }
    }
    // the row's ends: one element after another, put where raw8_words will look for them
    uint32_t w[NW] = {};
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (col + k < ne0) {
            if constexpr (T == kF32) {
                w[k] = *reinterpret_cast<const uint32_t *>(at + 4 * k);
            } else {
                w[k / 2] |= static_cast<uint32_t>(*reinterpret_cast<const unsigned short *>(at + 2 * k)) << (16 * (k & 1));
            }
        }
    if constexpr (ALIGNED) {
#pragma unroll
        for (int k = 0; k < NW; ++k) r.w[k] = w[k];
    } else {
        // moved up by `off` bytes
        uint32_t s[NW + 4], b[NW + 5];
#pragma unroll
        for (int k = 0; k < NW + 4; ++k) s[k] = k < NW ? w[k] : 0u;
        b[0] = 0u;
#pragma unroll
        for (int k = 0; k < NW + 4; ++k) b[k + 1] = s[k];
        uint32_t c[NW + 4], d[NW + 4];
#pragma unroll
        for (int k = 0; k < NW + 4; ++k) c[k] = __funnelshift_l(b[k], b[k + 1], (off & 3) * 8);
#pragma unroll
        for (int k = 0; k < NW + 4; ++k) d[k] = (off & 4) ? (k ? c[k - 1] : 0u) : c[k];
#pragma unroll
        for (int k = 0; k < NW + 4; ++k) r.w[k] = (off & 8) ? (k > 1 ? d[k - 2] : 0u) : d[k];
    }
}

// The words of the eight elements that load8 asked for at `at`.
template <int T, bool ALIGNED>
__device__ __forceinline__ void raw8_words(const Raw8<T, ALIGNED> &r, const char *at, uint32_t (&w)[kWords8<T>]) {
    if constexpr (ALIGNED) {
#pragma unroll
        for (int k = 0; k < kWords8<T>; ++k) w[k] = r.w[k];
    } else {
        shift_words<kWords8<T>>(r.w, static_cast<unsigned>(reinterpret_cast<uintptr_t>(at) & 15), w);
    }
}

// Store eight elements (those below ne0) at `at`.  Off a 16-byte boundary, a lane writes the aligned
// vectors that start with the last bytes of the lane before; `prev` / `next`: the lane before / after
// holds the eight columns before / after of the same row, all of them inside it.  The whole warp calls.
template <int T, bool ALIGNED>
__device__ __forceinline__ void store8(char *at, const uint32_t (&w)[kWords8<T>], unsigned long long col,
                                       unsigned long long ne0, bool whole, bool active, bool prev, bool next) {
    constexpr int NW = kWords8<T>, es = Elem<T>::bytes;
    auto element = [&](int k) {
        if constexpr (T == kF32) {
            *reinterpret_cast<uint32_t *>(at + 4 * k) = w[k];
        } else {
            *reinterpret_cast<unsigned short *>(at + 2 * k) = static_cast<unsigned short>(w[k / 2] >> (16 * (k & 1)));
        }
    };
    if constexpr (ALIGNED) {
        if (active && whole) {
            store_words<4 * NW>(at, w);
        } else if (active) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (col + k < ne0) element(k);
        }
    } else {
        const unsigned off = static_cast<unsigned>(reinterpret_cast<uintptr_t>(at) & 15);
        uint32_t s[NW + 4];
#pragma unroll
        for (int k = 0; k < 4; ++k) s[k] = __shfl_up_sync(~0u, w[NW - 4 + k], 1);
#pragma unroll
        for (int k = 0; k < NW; ++k) s[k + 4] = w[k];
        if (!active) return;
        if (!whole) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (col + k < ne0) element(k);
            return;
        }
        if (off == 0) {
#pragma unroll
            for (int k = 0; k < NW; k += 4)
                *reinterpret_cast<uint4 *>(at + 4 * k) = make_uint4(w[k], w[k + 1], w[k + 2], w[k + 3]);
            return;
        }
        uint32_t o[NW];
        shift_words<NW>(s, 16 - off, o);  // from 16 - off bytes into [previous, own]: what belongs at at - off
        char *base = at - off;
#pragma unroll
        for (int k = 0; k < NW; k += 4)
            if (k > 0 || prev) *reinterpret_cast<uint4 *>(base + 4 * k) = make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const unsigned from = static_cast<unsigned>(k * es);  // bytes into the eight elements
            if ((!prev && from < 16 - off) || (!next && from >= 4 * NW - off)) element(k);
        }
    }
}

// Widened values of eight elements' words (no rounding).
template <int T>
__device__ __forceinline__ void widen8(const uint32_t (&w)[kWords8<T>], float (&x)[8]) {
    word_operands<T, T, kWords8<T>>(w, x);
}

}  // namespace tps
