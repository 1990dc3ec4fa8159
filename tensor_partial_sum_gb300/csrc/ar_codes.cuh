// The 8-bit codes of checkpoints: block scales that are powers of two, and the
// codes themselves.  Multiplying by the scale or its inverse is exact, so an
// element is rounded once, and the same inputs give the same codes everywhere.
#pragma once

#include "ar_pairs.cuh"

namespace tps {

constexpr int kE4M3 = 0;
constexpr int kInt8 = 1;
constexpr int kCodeBlock = 32;  // adjacent elements that share a scale

// A checkpoint as kernels see it.
struct CodeRows {
    uint8_t *codes;  // nullptr: none
    long long code_row;
    uint8_t *scales;
    long long scale_row;
    int format;
};

// The scale byte (e + 127) of a block whose largest magnitude has these bits.  With M = 1.75 * 2^8 (e4m3) or
// 1.984375 * 2^6 (int8) the largest code, 2^e >= amax / M raises amax's exponent by one exactly where its
// fraction is above M's: a carry out of the fraction.
__device__ __forceinline__ unsigned scale_byte(int format, uint32_t amax_bits) {
    if (amax_bits >= 0x7F800000u) return 255u;  // infinities and NaN
    const int e = format == kE4M3 ? static_cast<int>((amax_bits + 0x1FFFFFu) >> 23) - 8
                                  : static_cast<int>((amax_bits + 0x01FFFFu) >> 23) - 6;
    return e > 0 ? static_cast<unsigned>(e) : 0u;
}
// 2^-e for the scale byte of finite elements, at most 249 (int8, next to the largest floats).
__device__ __forceinline__ float scale_inverse(unsigned byte) { return __uint_as_float((254u - byte) << 23); }
// 2^e, NaN for 255 and the subnormal 2^-127 for 0.
__device__ __forceinline__ float scale_value(unsigned byte) {
    return __uint_as_float(byte == 255u ? 0x7FC00000u : byte ? byte << 23 : 0x00400000u);
}

// Codes of two elements times 2^-e, the first in the low byte.
__device__ __forceinline__ uint32_t encode2(int format, float lo, float hi) {
    if (format == kE4M3) {
        unsigned short d;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
        return d;
    }
    return (static_cast<uint32_t>(__float2int_rn(lo)) & 0xFFu) | ((static_cast<uint32_t>(__float2int_rn(hi)) & 0xFFu) << 8);
}
// What the codes in the low two bytes of v stand for, without the scale.
__device__ __forceinline__ void decode2(int format, uint32_t v, float &lo, float &hi) {
    if (format == kE4M3) {
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<unsigned short>(v & 0xFFFFu)));
        lo = f16_lo(h);
        hi = f16_hi(h);
    } else {
        lo = static_cast<float>(static_cast<int8_t>(v & 0xFFu));
        hi = static_cast<float>(static_cast<int8_t>((v >> 8) & 0xFFu));
    }
}

// Codes of 2 N values times 2^-e, four to a word.  int8: adding 1.5 * 2^23 rounds to a whole number, ties to even,
// in the low bits.
template <int N>
__device__ __forceinline__ void encode_pairs(int format, const pair_t (&v)[N], pair_t inv, uint32_t (&w)[N / 2]) {
#pragma unroll
    for (int k = 0; k < N; k += 2) {
        const pair_t a = mul2(v[k], inv), b = mul2(v[k + 1], inv);
        if (format == kE4M3) {
            const float2 f = halves(a), g = halves(b);
            w[k / 2] = encode2(kE4M3, f.x, f.y) | encode2(kE4M3, g.x, g.y) << 16;
        } else {
            const pair_t magic = both(12582912.0f);
            const float2 f = halves(add2(a, magic)), g = halves(add2(b, magic));
            const uint32_t lo = __byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x0040);
            const uint32_t hi = __byte_perm(__float_as_uint(g.x), __float_as_uint(g.y), 0x0040);
            w[k / 2] = __byte_perm(lo, hi, 0x5410);
        }
    }
}
// What they stand for.  int8: the byte plus 128 in the low bits of 2^23.
template <int N>
__device__ __forceinline__ void decode_pairs(int format, const uint32_t (&w)[N / 2], float scale, pair_t (&v)[N]) {
    const pair_t s = both(scale);
#pragma unroll
    for (int k = 0; k < N; k += 2) {
        float a, b, c, d;
        if (format == kE4M3) {
            decode2(kE4M3, w[k / 2], a, b);
            decode2(kE4M3, w[k / 2] >> 16, c, d);
            v[k] = mul2(make_pair(a, b), s);
            v[k + 1] = mul2(make_pair(c, d), s);
        } else {
            const uint32_t x = w[k / 2] ^ 0x80808080u;
            const pair_t bias = both(-8388736.0f);
            v[k] = mul2(add2(make_pair(__uint_as_float(__byte_perm(x, 0x4B000000u, 0x7440)),
                                       __uint_as_float(__byte_perm(x, 0x4B000000u, 0x7441))), bias), s);
            v[k + 1] = mul2(add2(make_pair(__uint_as_float(__byte_perm(x, 0x4B000000u, 0x7442)),
                                           __uint_as_float(__byte_perm(x, 0x4B000000u, 0x7443))), bias), s);
        }
    }
}

__device__ __forceinline__ float decode_elem(const CodeRows &c, size_t row, size_t i) {
    const unsigned b = c.scales[static_cast<long long>(row) * c.scale_row + static_cast<long long>(i / kCodeBlock)];
    float lo, hi;
    decode2(c.format, c.codes[static_cast<long long>(row) * c.code_row + static_cast<long long>(i)], lo, hi);
    return lo * scale_value(b);
}

// One element a lane, the warp's 32 adjacent elements from a multiple of 32 on: a block.  The whole warp calls;
// a lane behind the row (inside false) adds nothing to the scale.
__device__ __forceinline__ void encode_block(const CodeRows &c, size_t row, size_t i, float x, bool inside) {
    const uint32_t bits = inside ? __float_as_uint(x) & 0x7FFFFFFFu : 0u;
    const unsigned byte = scale_byte(c.format, __reduce_max_sync(~0u, bits));
    if (!inside) return;
    const float v = byte == 255u ? 0.0f : x * scale_inverse(byte);
    c.codes[static_cast<long long>(row) * c.code_row + static_cast<long long>(i)] =
        static_cast<uint8_t>(encode2(c.format, v, v) & 0xFFu);
    if (i % kCodeBlock == 0)
        c.scales[static_cast<long long>(row) * c.scale_row + static_cast<long long>(i / kCodeBlock)] =
            static_cast<uint8_t>(byte);
}

}  // namespace tps
