// Philox4x32-10, the counter-based generator of Salmon, Moraes, Dror and Shaw,
// "Parallel random numbers: as easy as 1, 2, 3" (SC 2011): ten rounds of two
// 32x32-bit products whose halves are crossed and keyed.  A word depends on
// the key and the counter alone, so any thread can make any element's word.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace tps {

// The ten round keys: key + round * Weyl constant, the same for every thread,
// so the host makes them once per launch.
struct PhiloxKeys {
    uint32_t k0[10];
    uint32_t k1[10];
};

inline PhiloxKeys philox_keys(uint64_t seed) {
    PhiloxKeys k;
    uint32_t a = static_cast<uint32_t>(seed), b = static_cast<uint32_t>(seed >> 32);
    for (int r = 0; r < 10; ++r, a += 0x9E3779B9u, b += 0xBB67AE85u) k.k0[r] = a, k.k1[r] = b;
    return k;
}

__device__ __forceinline__ void philox4(const PhiloxKeys &k, uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3,
                                        uint32_t (&w)[4]) {
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = static_cast<uint64_t>(c0) * 0xD2511F53u;
        const uint64_t b = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
        c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ k.k0[r];
        c1 = static_cast<uint32_t>(b);
        c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ k.k1[r];
        c3 = static_cast<uint32_t>(a);
    }
    w[0] = c0, w[1] = c1, w[2] = c2, w[3] = c3;
}

}  // namespace tps
