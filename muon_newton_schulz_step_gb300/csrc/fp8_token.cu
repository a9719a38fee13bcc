// The forward product for few tokens: y[t, n] = sum_k q(x)[t, k] W_g[n, k], with
// the rounding of x to E4M3 in the same launch.
//
// Serving makes this product for one token at a time (or a few per expert): its
// time is the weight's bytes, read once, and the launch.  The tiled product would
// load 128 rows per CTA on a third of the SMs and needs the codes of x from a
// launch before it (24 us for one token and 6144 x 6144; here @@).
//
// A block takes 16 rows of one weight, its eight warps take the reduction's
// blocks of 128 in turn.  A lane reads 16 consecutive bytes of a row at a time (the
// matrix fragments want 4 here and 4 there: the reduction index is permuted within
// 64, the same way for both operands), so a warp has several KB on their way, and
// the products of a block of 128 run on mma.sync: 16 rows x 8 tokens cost no more
// than one token.  (tcgen05 has nothing to add: the tensor core idles either way,
// and its operands would take a trip through shared memory.)  A warp rounds the
// part of x that it multiplies, in the layout of the fragment, as it needs it.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fp8_codes.cuh"
#include "groups.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = 8;
constexpr int kRows = 16;            // weight rows per block
constexpr int kTokens = 8;           // tokens per pass over the weight

__device__ __forceinline__ uint4 load_stream(const uint8_t* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Weight codes of one block of 128 for a 16-row fragment: rows lane / 4 and + 8,
// bytes 16 (lane % 4) of either half.
struct WeightBlock {
    uint4 v[2][2];
    __device__ __forceinline__ void load(const uint8_t* lo, const uint8_t* hi, int kb) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            v[0][h] = load_stream(lo + kb * 128 + 64 * h);
            v[1][h] = load_stream(hi + kb * 128 + 64 * h);
        }
    }
};

// 16 consecutive elements of a token from column col on; zero past the last.
template <bool BF16>
__device__ __forceinline__ void load16(const Fp8TokenParams& p, long long row, int col, float (&f)[16]) {
    if (p.vec && col + 16 <= p.k) {
        if (BF16) {
            const uint4* s = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.x) + row * p.ld_x + col);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint4 r = s[h];
                const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f[8 * h + 2 * i] = __uint_as_float(w[i] << 16);
                    f[8 * h + 2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
                }
            }
        } else {
            const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(p.x) + row * p.ld_x + col);
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const float4 r = s[h];
                f[4 * h] = r.x; f[4 * h + 1] = r.y; f[4 * h + 2] = r.z; f[4 * h + 3] = r.w;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            f[i] = 0.0f;
            if (col + i < p.k) {
                const long long at = row * p.ld_x + col + i;
                f[i] = BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.x)[at])
                            : static_cast<const float*>(p.x)[at];
            }
        }
    }
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) k_fp8_token(const __grid_constant__ Fp8TokenParams p) {
    __shared__ float part[kWarps][kTokens][kRows];
    __shared__ int span[2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = blockIdx.y;
    if (p.offsets == nullptr) {
        if (threadIdx.x == 0) {
            span[0] = 0;
            span[1] = p.tokens;
        }
    } else if (warp == 0) {
        int low = 0;
        for (int g0 = 0; g0 <= g; g0 += 32) {
            const GroupSpan s = warp_group_spans(p.offsets, p.groups, p.tokens, g0, low);
            if (g0 + lane == g) {
                span[0] = s.lo;
                span[1] = s.cnt;
            }
        }
    }
    const int n0 = blockIdx.x * kRows;
    const int r = lane >> 2, j = lane & 3;
    // rows past the last read the last one's codes; their results are not stored
    const uint8_t* w = p.w + (static_cast<long long>(g) * p.n) * p.ldk + 16 * j;
    const uint8_t* lo = w + static_cast<long long>(min(n0 + r, p.n - 1)) * p.ldk;
    const uint8_t* hi = w + static_cast<long long>(min(n0 + r + 8, p.n - 1)) * p.ldk;
    const int blocks = static_cast<int>(p.ldk >> 7);
    const uint8_t* ws = p.w_scale + (static_cast<long long>(g) * ((p.n + 127) >> 7) + (n0 >> 7)) * blocks;
    __syncthreads();
    const int first = span[0], count = span[1];

    for (int t0 = 0; t0 < count; t0 += kTokens) {
        float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        const bool mine = t0 + r < count;                // as B fragment: this lane's token
        const long long row = first + t0 + r;
        auto multiply = [&](const WeightBlock& wb, int kb) {
            float f[2][16];
            uint32_t top = 0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (mine) {
                    load16<BF16>(p, row, kb * 128 + 64 * h + 16 * j, f[h]);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) f[h][i] = 0.0f;
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const uint32_t m = __float_as_uint(f[h][i]) & 0x7fffffffu;
                    top = max(top, m >= 0x7f800000u ? 0u : m);
                }
            }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int e = scale_exponent(top);
            const float by = inverse_scale(e);
            float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float v[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float x = f[h][4 * i + q];
                        v[q] = isinf(x) ? __uint_as_float(0x7fffffffu) : __fmul_rn(x, by);
                    }
                    b[i] = ptx::cvt_e4m3x2(v[1], v[0]) | (static_cast<uint32_t>(ptx::cvt_e4m3x2(v[3], v[2])) << 16);
                }
                mma_e4m3(c, wb.v[0][h].x, wb.v[1][h].x, wb.v[0][h].y, wb.v[1][h].y, b[0], b[1]);
                mma_e4m3(c, wb.v[0][h].z, wb.v[1][h].z, wb.v[0][h].w, wb.v[1][h].w, b[2], b[3]);
            }
            // both scales as one exponent, in two factors that cannot leave fp32 on their own
            const int ew = static_cast<int>(ws[kb]) - 127;
            const int e0 = __shfl_sync(0xffffffffu, e, 8 * j) + ew, e1 = __shfl_sync(0xffffffffu, e, 8 * j + 4) + ew;
            const float a0 = power_of_two(e0 >> 1), b0 = power_of_two(e0 - (e0 >> 1));
            const float a1 = power_of_two(e1 >> 1), b1 = power_of_two(e1 - (e1 >> 1));
            acc[0] = fmaf(c[0] * a0, b0, acc[0]);
            acc[1] = fmaf(c[1] * a1, b1, acc[1]);
            acc[2] = fmaf(c[2] * a0, b0, acc[2]);
            acc[3] = fmaf(c[3] * a1, b1, acc[3]);
        };
        int kb = warp;
        for (; kb + 2 * kWarps < blocks; kb += 3 * kWarps) {
            WeightBlock wb[3];
#pragma unroll
            for (int i = 0; i < 3; ++i) wb[i].load(lo, hi, kb + i * kWarps);
#pragma unroll
            for (int i = 0; i < 3; ++i) multiply(wb[i], kb + i * kWarps);
        }
        for (; kb < blocks; kb += kWarps) {
            WeightBlock wb;
            wb.load(lo, hi, kb);
            multiply(wb, kb);
        }
        // accumulator: rows r, r + 8; tokens 2 j, 2 j + 1
        part[warp][2 * j][r] = acc[0];
        part[warp][2 * j + 1][r] = acc[1];
        part[warp][2 * j][r + 8] = acc[2];
        part[warp][2 * j + 1][r + 8] = acc[3];
        __syncthreads();
        if (threadIdx.x < kTokens * kRows) {
            const int t = threadIdx.x / kRows, n = threadIdx.x % kRows;
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) s += part[i][t][n];
            if (t0 + t < count && n0 + n < p.n) {
                const long long at = static_cast<long long>(first + t0 + t) * p.ld_out + n0 + n;
                if (p.out_f32) static_cast<float*>(p.out)[at] = s;
                else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(s);
            }
        }
        __syncthreads();                                 // `part` is written anew
    }
}

}  // namespace

cudaError_t launch_fp8_token(const Fp8TokenParams& p, cudaStream_t s) {
    const dim3 grid((p.n + kRows - 1) / kRows, p.groups);
    if (p.bf16) k_fp8_token<true><<<grid, kThreads, 0, s>>>(p);
    else k_fp8_token<false><<<grid, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace muon
