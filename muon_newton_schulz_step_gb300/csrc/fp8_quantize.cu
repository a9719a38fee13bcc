// Matrices to E4M3 codes with one power-of-two scale for each block of 128.
//
//   e    = the smallest integer with max|x| <= 448 * 2^e over the block (finite
//          elements; 0 for a zero block), kept within [-127, 127]; byte e + 127
//   code = E4M3(x * 2^-e), rounded to nearest even (the scaling is exact)
//   a NaN or an infinity becomes E4M3's NaN: it reaches the products it is in
//
// Three kinds of block, in the layout of the input (row-major, rows of 128-byte
// multiples, zero codes past the last column):
//   row    128 columns of one row          scale[column block][row]
//   col    128 rows of one column          scale[row block][column]
//   block  128 x 128                       scale[row block][column block]
// Row blocks feed the products that reduce over columns, col blocks those that
// reduce over rows (the weight gradient); there the rows are tokens sorted by
// expert, so blocks start anew at each group's first row and each group's codes
// are padded with zero rows to a multiple of 128.  128 x 128 blocks serve the
// weights: the same codes and scales read along either dimension.
//
// Bound by HBM: one read of x and one write per code.  A 256-thread block takes
// a 128 x 128 tile: a warp two rows at a time, 16 lanes x 8 consecutive columns
// a row, so a lane's 64 values stay in registers between the maximum and the
// codes, row maxima meet in four shuffles and column maxima in one shuffle and
// one exchange through shared memory, and the row and the col codes of one
// matrix come from a single read.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "groups.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsPerThread = 8;

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

__device__ __forceinline__ uint32_t magnitude(float v) {
    const uint32_t b = __float_as_uint(v) & 0x7fffffffu;
    return b >= 0x7f800000u ? 0u : b;                    // not finite: no part in the maximum
}

__device__ __forceinline__ uint2 codes(const float (&v)[8], const float (&by)[8]) {
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // infinities saturate in the conversion: make them NaN (inf * 0 + ...) first
        float lo = v[2 * i], hi = v[2 * i + 1];
        lo = __fmul_rn(lo, by[2 * i]);
        hi = __fmul_rn(hi, by[2 * i + 1]);
        if (isinf(v[2 * i])) lo = __uint_as_float(0x7fffffffu);
        if (isinf(v[2 * i + 1])) hi = __uint_as_float(0x7fffffffu);
        q[i] = ptx::cvt_e4m3x2(hi, lo);
    }
    return make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
}

struct RowBlock {
    long long row0;       // first row in x
    int rows;             // rows of it, 0..128
    long long padded0;    // first row among the padded col codes
    bool valid;
};

// Row block `rb` of the groups' padded row blocks (one group: rb itself).  Warp 0
// adds up the groups' blocks; offsets outside [0, rows] or descending are clamped.
__device__ __forceinline__ void find_row_block(const QuantParams& p, long long rb, RowBlock* out) {
    if (p.groups == 0) {
        if (threadIdx.x == 0) {
            out->row0 = rb * 128;
            const long long left = p.rows - rb * 128;
            out->rows = static_cast<int>(left < 128 ? left : 128);
            out->padded0 = rb * 128;
            out->valid = left > 0;
        }
        return;
    }
    if (threadIdx.x >= 32) return;
    if (threadIdx.x == 0) out->valid = false;
    __syncwarp();
    int before = 0, low = 0;                             // row blocks of the groups so far; their last row
    for (int g0 = 0; g0 < p.groups; g0 += 32) {
        const GroupSpan span = warp_group_spans(p.offsets, p.groups, static_cast<int>(p.rows), g0, low);
        const int nb = (span.cnt + 127) >> 7;
        const int inc = warp_inclusive_sum(nb);
        const int k = static_cast<int>(rb) - (before + inc - nb);
        if (k >= 0 && k < nb) {
            out->row0 = static_cast<long long>(span.lo) + 128 * k;
            out->rows = span.cnt - 128 * k < 128 ? span.cnt - 128 * k : 128;
            out->padded0 = rb * 128;
            out->valid = true;
        }
        before += __shfl_sync(0xffffffffu, inc, 31);
        if (rb < before) break;
    }
}

template <bool BF16>
__device__ __forceinline__ void load8(const QuantParams& p, const char* base, long long row, long long col, float (&v)[8]) {
    const long long off = row * p.ld + col;
    if (p.vec && col + 8 <= p.cols) {
        if (BF16) {
            const uint4 r = *reinterpret_cast<const uint4*>(base + off * 2);
            const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        } else {
            const float4* s = reinterpret_cast<const float4*>(base + off * 4);
            const float4 a = s[0], b = s[1];
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] = 0.0f;
            if (col + i < p.cols)
                v[i] = BF16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(base)[off + i])
                            : reinterpret_cast<const float*>(base)[off + i];
        }
    }
}

template <bool BF16, bool ROW, bool COL, bool BLK>
__global__ void __launch_bounds__(kThreads) k_fp8_quantize(const __grid_constant__ QuantParams p) {
    __shared__ uint32_t part[8][128];
    __shared__ RowBlock rb;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int cg = lane & 15, half = lane >> 4;
    const long long cb = blockIdx.x;
    const long long batch = blockIdx.z;
    const char* base = static_cast<const char*>(p.x) + batch * p.ldb * (BF16 ? 2 : 4);

    for (long long y = blockIdx.y; y < p.row_blocks; y += gridDim.y) {
        find_row_block(p, y, &rb);
        __syncthreads();
        const RowBlock r = rb;
        if (!r.valid) return;                            // the blocks past the last one
        const long long col = cb * 128 + cg * 8;
        float v[kRowsPerThread][8];
#pragma unroll
        for (int i = 0; i < kRowsPerThread; ++i) {
            const int lr = i * 16 + warp * 2 + half;
            if (lr < r.rows) {
                load8<BF16>(p, base, r.row0 + lr, col, v[i]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
            }
        }
        if (ROW) {
#pragma unroll
            for (int i = 0; i < kRowsPerThread; ++i) {
                const int lr = i * 16 + warp * 2 + half;
                uint32_t top = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) top = max(top, magnitude(v[i][j]));
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                const int e = scale_exponent(top);
                float by[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) by[j] = inverse_scale(e);
                if (lr < r.rows) {
                    *reinterpret_cast<uint2*>(p.row_q + (r.row0 + lr) * p.ldq + col) = codes(v[i], by);
                    if (cg == 0) p.row_scale[cb * p.rows + r.row0 + lr] = static_cast<uint8_t>(e + 127);
                }
            }
        }
        if (COL || BLK) {
            uint32_t top[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                top[j] = 0;
#pragma unroll
                for (int i = 0; i < kRowsPerThread; ++i) top[j] = max(top[j], magnitude(v[i][j]));
                top[j] = max(top[j], __shfl_xor_sync(0xffffffffu, top[j], 16));
            }
            if (half == 0) {
#pragma unroll
                for (int j = 0; j < 8; ++j) part[warp][cg * 8 + j] = top[j];
            }
            __syncthreads();
            if (threadIdx.x < 128) {
                uint32_t t = 0;
#pragma unroll
                for (int w = 0; w < 8; ++w) t = max(t, part[w][threadIdx.x]);
                part[0][threadIdx.x] = t;
            }
            __syncthreads();
            if (COL) {
                float by[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) by[j] = inverse_scale(scale_exponent(part[0][cg * 8 + j]));
#pragma unroll
                for (int i = 0; i < kRowsPerThread; ++i) {
                    const int lr = i * 16 + warp * 2 + half;
                    *reinterpret_cast<uint2*>(p.col_q + (r.padded0 + lr) * p.ldq + col) = codes(v[i], by);
                }
                if (threadIdx.x < 128)
                    p.col_scale[(r.padded0 >> 7) * p.ldq + cb * 128 + threadIdx.x] =
                        static_cast<uint8_t>(scale_exponent(part[0][threadIdx.x]) + 127);
            }
            if (BLK) {
                uint32_t t = max(max(part[0][lane], part[0][lane + 32]), max(part[0][lane + 64], part[0][lane + 96]));
                t = __reduce_max_sync(0xffffffffu, t);
                const int e = scale_exponent(t);
                float by[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) by[j] = inverse_scale(e);
                uint8_t* q = p.blk_q + batch * p.rows * p.ldq;
#pragma unroll
                for (int i = 0; i < kRowsPerThread; ++i) {
                    const int lr = i * 16 + warp * 2 + half;
                    if (lr < r.rows) *reinterpret_cast<uint2*>(q + (r.row0 + lr) * p.ldq + col) = codes(v[i], by);
                }
                if (threadIdx.x == 0)
                    p.blk_scale[(batch * ((p.rows + 127) >> 7) + (r.row0 >> 7)) * gridDim.x + cb] =
                        static_cast<uint8_t>(e + 127);
            }
        }
        __syncthreads();                                 // rb and part are written anew
    }
}

template <bool BF16>
cudaError_t run(const QuantParams& p, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>(p.ldq / 128),
                    static_cast<unsigned>(p.row_blocks < 65535 ? p.row_blocks : 65535),
                    static_cast<unsigned>(p.batch));
    if (p.blk_q != nullptr) k_fp8_quantize<BF16, false, false, true><<<grid, kThreads, 0, s>>>(p);
    else if (p.row_q != nullptr && p.col_q != nullptr) k_fp8_quantize<BF16, true, true, false><<<grid, kThreads, 0, s>>>(p);
    else if (p.row_q != nullptr) k_fp8_quantize<BF16, true, false, false><<<grid, kThreads, 0, s>>>(p);
    else k_fp8_quantize<BF16, false, true, false><<<grid, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fp8_quantize(const QuantParams& p, cudaStream_t s) {
    return p.bf16 ? run<true>(p, s) : run<false>(p, s);
}

}  // namespace muon
