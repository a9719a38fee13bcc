// Weights of 4 bits with a scale for each `block` columns of a row (32, 64 or 128).
//
// w[n, k] = code[n, k] * scale[k / block, n]; codes are whole numbers from -8 to 7, two to
// a byte, the even column in the low half; rows end on a multiple of 128 columns.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

namespace muon {

// The reduction is worked off in blocks of 128 columns, each in four steps of 32: in step m
// lane j of the four that share a row holds the word of eight codes (and the eight elements
// of x) from column 32 m + 8 j on.  A matrix fragment wants 2 + 2 codes from each lane; which
// columns they are is free, as long as both operands agree.

// Eight codes as bf16, 2^-11 times their number: element i of pair p is column 4 i + p, exactly.
// A code with its sign bit turned over is code + 8, and bf16's numbers from 0 to 255 smallest steps
// (2^-133 each) are spaced evenly: four bits at either end of a byte are a number as they lie, and one
// fused multiply-add brings them up and takes the 8 off.  With 2^-11 the sum of 128 products is at
// most half of the largest |x|, so no x overflows before its scale has been applied; kCodeUnit, at the
// end, takes it back.  Nine instructions for eight codes; eleven with a shift for each pair and
// their offset as a larger number's last bits.
constexpr float kCodeUnit = 2048.0f;

struct EightCodes {
    uint32_t pair[4];
};

__device__ __forceinline__ EightCodes decode(uint32_t w) {
    EightCodes d;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const bool up = p & 1;                             // the upper half of the bytes
        uint32_t u;                                        // (a & b) ^ c
        asm("lop3.b32 %0, %1, %2, %3, 0x6a;"
            : "=r"(u)
            : "r"(p < 2 ? w : w >> 8), "r"(up ? 0x00f000f0u : 0x000f000fu), "r"(up ? 0x00800080u : 0x00080008u));
        // times 2^118 or 2^122, less 2^-8
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d.pair[p]) : "r"(u), "r"(up ? 0x7a807a80u : 0x7c807c80u), "r"(0xbb80bb80u));
    }
    return d;
}

// Eight elements of x in the order that decode() gives codes: pair p is (p, 4 + p).
__device__ __forceinline__ uint4 in_pairs(uint32_t a01, uint32_t a23, uint32_t a45, uint32_t a67) {
    return make_uint4(__byte_perm(a01, a45, 0x5410), __byte_perm(a01, a45, 0x7632), __byte_perm(a23, a67, 0x5410),
                      __byte_perm(a23, a67, 0x7632));
}

// fp32 as three bf16 whose sum it is: 8 bits of the significand each, cut and not rounded, so
// that the largest numbers stay finite.  Infinities and NaN stay in the first.
__device__ __noinline__ float3 split_odd(float v) {
    const uint32_t u = __float_as_uint(v);
    if ((u & 0x7f800000u) == 0x7f800000u)
        return make_float3(__uint_as_float((u & 0xffff0000u) | ((u & 0x007fffffu) != 0u ? 0x00400000u : 0u)), 0.0f, 0.0f);
    const float rest = v - __uint_as_float(u & 0xffff0000u);
    return make_float3(v, rest, rest - __uint_as_float(__float_as_uint(rest) & 0xffff0000u));
}

// Eight consecutive elements of x as `PARTS` fragments in decode()'s order; zero past column k.
template <int PARTS>
struct EightOfX {
    uint4 v[PARTS];
};

template <int PARTS>
struct RawOfX {
    uint4 v[PARTS == 1 ? 1 : 2];
};

template <int PARTS>
__device__ __forceinline__ RawOfX<PARTS> load_x(const char* at) {
    RawOfX<PARTS> r;
    r.v[0] = __ldg(reinterpret_cast<const uint4*>(at));
    if constexpr (PARTS != 1) r.v[1] = __ldg(reinterpret_cast<const uint4*>(at) + 1);
    return r;
}

// The same of elements that lie on no vector, or of which only `left` are there (zeros past them):
// eight whole ones by the words around them, as far as those lie in x ([begin, end)).
template <int PARTS>
__device__ __forceinline__ RawOfX<PARTS> load_x_edge(const char* at, int left, const char* begin, const char* end) {
    constexpr int kWords = PARTS == 1 ? 4 : 8;
    uint32_t w[kWords + 1] = {};
    const int off = PARTS == 1 ? static_cast<int>(reinterpret_cast<uintptr_t>(at) & 2) : 0;
    const uint32_t* q = reinterpret_cast<const uint32_t*>(at - off);
    if (left >= 8 && at - off >= begin && at + 4 * kWords + off <= end) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = __ldg(q + i);
        if (PARTS == 1) {
            if (off != 0) w[kWords] = __ldg(q + kWords);
#pragma unroll
            for (int i = 0; i < kWords; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 8 * off);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i >= left) continue;
            if (PARTS == 1) w[i / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(at)[i]) << (16 * (i & 1));
            else w[i] = reinterpret_cast<const uint32_t*>(at)[i];
        }
    }
    RawOfX<PARTS> r;
    r.v[0] = make_uint4(w[0], w[1], w[2], w[3]);
    if constexpr (PARTS != 1) r.v[1] = make_uint4(w[4], w[5], w[6], w[7]);
    return r;
}

// Apart from the kernel where its registers are few.
template <int PARTS>
__device__ __noinline__ RawOfX<PARTS> call_x_edge(const char* at, int left, const char* begin, const char* end) {
    return load_x_edge<PARTS>(at, left, begin, end);
}

template <int PARTS>
__device__ __forceinline__ EightOfX<PARTS> fragments(const RawOfX<PARTS>& r) {
    EightOfX<PARTS> f;
    if constexpr (PARTS == 1) {
        f.v[0] = in_pairs(r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w);
    } else {
        const uint32_t w[8] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w, r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
        float3 t[8];                                       // the upper halves of each are the parts
        float zero = 0.0f;                                 // NaN if one of the eight is not finite
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            t[i].x = __uint_as_float(w[i]);
            t[i].y = t[i].x - __uint_as_float(w[i] & 0xffff0000u);
            t[i].z = t[i].y - __uint_as_float(__float_as_uint(t[i].y) & 0xffff0000u);
            zero = fmaf(t[i].x, 0.0f, zero);
        }
        if (zero != 0.0f) {
#pragma unroll
            for (int i = 0; i < 8; ++i) t[i] = split_odd(__uint_as_float(w[i]));
        }
        auto upper = [](float lo, float hi) { return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632); };
        f.v[0] = make_uint4(upper(t[0].x, t[4].x), upper(t[1].x, t[5].x), upper(t[2].x, t[6].x), upper(t[3].x, t[7].x));
        f.v[1] = make_uint4(upper(t[0].y, t[4].y), upper(t[1].y, t[5].y), upper(t[2].y, t[6].y), upper(t[3].y, t[7].y));
        f.v[2] = make_uint4(upper(t[0].z, t[4].z), upper(t[1].z, t[5].z), upper(t[2].z, t[6].z), upper(t[3].z, t[7].z));
    }
    return f;
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], const float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

// A step of 32 columns: two products of 16; `first`: of a scale's columns, so that the sum begins.
__device__ __forceinline__ void mma_step(float (&c)[4], bool first, const EightCodes& lo, const EightCodes& hi,
                                         const uint4& b) {
    const float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (first) mma_bf16(c, zero, lo.pair[0], hi.pair[0], lo.pair[1], hi.pair[1], b.x, b.y);
    else mma_bf16(c, c, lo.pair[0], hi.pair[0], lo.pair[1], hi.pair[1], b.x, b.y);
    mma_bf16(c, c, lo.pair[2], hi.pair[2], lo.pair[3], hi.pair[3], b.z, b.w);
}

}  // namespace muon
