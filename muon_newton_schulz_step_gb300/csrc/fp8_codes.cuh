// Power-of-two scales of blocks of E4M3 codes.
#pragma once

#include <cstdint>

namespace muon {

// The block's exponent from the bits of its largest finite magnitude.
// 448 = 1.75 * 2^8: with max = m * 2^q, 1 <= m < 2, e = q - 8 where m <= 1.75, else q - 7.
__device__ __forceinline__ int scale_exponent(uint32_t top) {
    if (top == 0u) return 0;
    int q = static_cast<int>(top >> 23) - 127;
    uint32_t frac = top & 0x7fffffu;
    if (q == -127) {                                     // subnormal: normalise
        const int up = __clz(frac) - 8;
        q = -126 - up;
        frac = (frac << up) & 0x7fffffu;
    }
    const int e = frac <= 0x600000u ? q - 8 : q - 7;
    return e < -127 ? -127 : e;
}

// 2^-e for e in [-127, 127]
__device__ __forceinline__ float inverse_scale(int e) {
    return e == 127 ? __uint_as_float(0x00400000u) : __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
}

// 2^e for e in [-126, 127]
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

}  // namespace muon
