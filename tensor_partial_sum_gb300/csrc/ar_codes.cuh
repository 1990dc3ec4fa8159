// The 8-bit codes of checkpoints: block scales that are powers of two, and the
// codes themselves.  Multiplying by the scale or its inverse is exact, so an
// element is rounded once, and the same inputs give the same codes everywhere.
#pragma once

#include "ar_kernels.cuh"

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
// 2^-e for the scale byte of finite elements, at most 248.
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
