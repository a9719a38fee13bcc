// E4M3 codes of blocks with power-of-two scales.
#pragma once

#include <cstdint>

#include "ptx.cuh"

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

// Eight consecutive elements as loaded: bf16 in a, fp32 in a and b.
struct Raw {
    uint4 a, b;
};

__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

template <bool BF16>
__device__ __forceinline__ float element(const Raw& r, int j) {
    if (BF16) {
        const uint32_t w = word(r.a, j >> 1);
        return __uint_as_float((j & 1) ? (w & 0xffff0000u) : (w << 16));
    }
    return __uint_as_float(j < 4 ? word(r.a, j) : word(r.b, j - 4));
}

constexpr uint32_t kInf = 0x7f800000u;

// Largest magnitude of eight elements, as fp32 bits (NaN and infinity at or above kInf).
template <bool BF16>
__device__ __forceinline__ uint32_t row_max(const Raw& r) {
    if (BF16) {
        const uint32_t k = 0x7fff7fffu;
        const uint32_t v = __vmaxu2(__vmaxu2(r.a.x & k, r.a.y & k), __vmaxu2(r.a.z & k, r.a.w & k));
        return max(v & 0xffff0000u, v << 16);
    }
    const uint32_t k = 0x7fffffffu;
    return max(max(max(r.a.x & k, r.a.y & k), max(r.a.z & k, r.a.w & k)),
               max(max(r.b.x & k, r.b.y & k), max(r.b.z & k, r.b.w & k)));
}

// Elements that are not finite: NaN in their place (infinities would saturate in
// the conversion), zero for the maxima.
template <bool BF16>
__device__ __noinline__ Raw replace_odd(Raw r, bool zero) {
    uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
    for (int i = 0; i < (BF16 ? 4 : 8); ++i) {
        if (BF16) {
            if ((w[i] & 0x7f800000u) == 0x7f800000u) w[i] = zero ? w[i] & 0x0000ffffu : w[i] | 0x7fff0000u;
            if ((w[i] & 0x7f80u) == 0x7f80u) w[i] = zero ? w[i] & 0xffff0000u : w[i] | 0x7fffu;
        } else if ((w[i] & kInf) == kInf) {
            w[i] = zero ? 0u : w[i] | 0x7fffffffu;
        }
    }
    r.a = make_uint4(w[0], w[1], w[2], w[3]);
    r.b = make_uint4(w[4], w[5], w[6], w[7]);
    return r;
}

template <bool BF16>
__device__ __forceinline__ uint2 codes_of(const Raw& r, const float (&by)[8]) {
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        q[i] = ptx::cvt_e4m3x2(__fmul_rn(element<BF16>(r, 2 * i + 1), by[2 * i + 1]),
                               __fmul_rn(element<BF16>(r, 2 * i), by[2 * i]));
    return make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
}

template <bool BF16>
__device__ __forceinline__ uint2 codes_of(const Raw& r, float by) {
    const float b[8] = {by, by, by, by, by, by, by, by};
    return codes_of<BF16>(r, b);
}

}  // namespace muon
