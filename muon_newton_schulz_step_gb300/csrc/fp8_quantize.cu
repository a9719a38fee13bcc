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
// 128 x 128 tiles of one row block: a warp two rows at a time, 16 lanes x 8
// consecutive columns a row.  All of a thread's eight vectors are loaded before
// the first is looked at (a conditional load per vector would make eight DRAM
// latencies of one) and stay in registers in their own type between the maximum
// and the codes: bf16 magnitudes are compared two at a time as integers, row
// maxima meet in four shuffles, column maxima in one shuffle and one exchange
// through shared memory, and the row and the col codes come from a single read.
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

// Largest magnitudes of columns over rows, as fp32 bits (bf16: two packed).
template <bool BF16>
struct Maxima {
    uint32_t m[BF16 ? 4 : 8];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (uint32_t& v : m) v = 0;
    }
    __device__ __forceinline__ void add(const Raw& r) {
        if (BF16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) m[i] = __vmaxu2(m[i], word(r.a, i) & 0x7fff7fffu);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                m[i] = max(m[i], word(r.a, i) & 0x7fffffffu);
                m[i + (BF16 ? 0 : 4)] = max(m[i + (BF16 ? 0 : 4)], word(r.b, i) & 0x7fffffffu);
            }
        }
    }
    // of elements that are not finite: nothing
    __device__ __forceinline__ void add_finite(const Raw& r) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint32_t v = __float_as_uint(element<BF16>(r, j)) & 0x7fffffffu;
            if (v >= kInf) v = 0;
            if (BF16) {
                const uint32_t h = v >> 16;
                m[j >> 1] = __vmaxu2(m[j >> 1], (j & 1) ? h << 16 : h);
            } else {
                m[BF16 ? 0 : j] = max(m[BF16 ? 0 : j], v);
            }
        }
    }
    __device__ __forceinline__ uint32_t column(int j) const {
        if (BF16) return (j & 1) ? (m[j >> 1] & 0xffff0000u) : (m[j >> 1] << 16);
        return m[BF16 ? 0 : j];
    }
    __device__ __forceinline__ uint32_t all() const {
        if (BF16) {
            const uint32_t v = __vmaxu2(__vmaxu2(m[0], m[1]), __vmaxu2(m[2], m[3]));
            return max(v & 0xffff0000u, v << 16);
        }
        uint32_t v = 0;
#pragma unroll
        for (uint32_t x : m) v = max(v, x);
        return v;
    }
};

// Codes of eight elements; ODD: infinities among them (the conversion would
// saturate them) become NaN.
template <bool BF16, bool ODD>
__device__ __forceinline__ uint2 codes(const Raw& r, const float (&by)[8]) {
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo = __fmul_rn(element<BF16>(r, 2 * i), by[2 * i]), hi = __fmul_rn(element<BF16>(r, 2 * i + 1), by[2 * i + 1]);
        if (ODD) {
            if (isinf(element<BF16>(r, 2 * i))) lo = __uint_as_float(0x7fffffffu);
            if (isinf(element<BF16>(r, 2 * i + 1))) hi = __uint_as_float(0x7fffffffu);
        }
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
__device__ __forceinline__ void find_row_block(const QuantParams& p, const int* offsets, long long rb, RowBlock* out) {
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
        const GroupSpan span = warp_group_spans(offsets, p.groups, static_cast<int>(p.rows), g0, low);
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

// Eight elements at the matrix's edge, or without the alignment for vectors.
template <bool BF16>
__device__ __forceinline__ Raw load_edge(const QuantParams& p, const char* base, long long row, long long col) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        w[i] = 0;
        if (col + i < p.cols) {
            const long long at = row * p.ld + col + i;
            w[i] = BF16 ? static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(base)[at])
                        : reinterpret_cast<const uint32_t*>(base)[at];
        }
    }
    Raw r;
    if (BF16) {
        r.a = make_uint4(w[0] | (w[1] << 16), w[2] | (w[3] << 16), w[4] | (w[5] << 16), w[6] | (w[7] << 16));
        r.b = r.a;
    } else {
        r.a = make_uint4(w[0], w[1], w[2], w[3]);
        r.b = make_uint4(w[4], w[5], w[6], w[7]);
    }
    return r;
}

// One tile's maxima, scales and codes.  ODD: some element is not finite.
template <bool BF16, bool ROW, bool COL, bool BLK, bool ODD>
__device__ __forceinline__ void tile(const QuantParams& p, const RowBlock& r, const Raw (&v)[kRowsPerThread],
                                     uint32_t (&part)[8][128], long long cb, long long batch) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int cg = lane & 15, half = lane >> 4;
    const long long col = cb * 128 + cg * 8;
    if (ROW) {
#pragma unroll
        for (int i = 0; i < kRowsPerThread; ++i) {
            const int lr = i * 16 + warp * 2 + half;
            Maxima<BF16> m;
            m.clear();
            if (ODD) m.add_finite(v[i]); else m.add(v[i]);
            uint32_t top = m.all();
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            const int e = scale_exponent(top);
            float by[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) by[j] = inverse_scale(e);
            if (lr < r.rows) {
                *reinterpret_cast<uint2*>(p.row_q + (r.row0 + lr) * p.ldq + col) = codes<BF16, ODD>(v[i], by);
                if (cg == 0) p.row_scale[cb * p.rows + r.row0 + lr] = static_cast<uint8_t>(e + 127);
            }
        }
    }
    if (COL || BLK) {
        Maxima<BF16> m;
        m.clear();
#pragma unroll
        for (int i = 0; i < kRowsPerThread; ++i) {
            if (ODD) m.add_finite(v[i]); else m.add(v[i]);
        }
        uint32_t top[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            top[j] = m.column(j);
            top[j] = max(top[j], __shfl_xor_sync(0xffffffffu, top[j], 16));
        }
        __syncthreads();                                 // part's last readers are done
        if (half == 0) {
            uint4* dst = reinterpret_cast<uint4*>(&part[warp][cg * 8]);
            dst[0] = make_uint4(top[0], top[1], top[2], top[3]);
            dst[1] = make_uint4(top[4], top[5], top[6], top[7]);
        }
        __syncthreads();
        if (COL) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint4 t = *reinterpret_cast<const uint4*>(&part[0][cg * 8 + 4 * h]);
#pragma unroll
                for (int w = 1; w < 8; ++w) {
                    const uint4 u = *reinterpret_cast<const uint4*>(&part[w][cg * 8 + 4 * h]);
                    t = make_uint4(max(t.x, u.x), max(t.y, u.y), max(t.z, u.z), max(t.w, u.w));
                }
                top[4 * h] = t.x;
                top[4 * h + 1] = t.y;
                top[4 * h + 2] = t.z;
                top[4 * h + 3] = t.w;
            }
            float by[8];
            uint32_t sc[2] = {0, 0};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int e = scale_exponent(top[j]);
                by[j] = inverse_scale(e);
                sc[j >> 2] |= static_cast<uint32_t>(e + 127) << (8 * (j & 3));
            }
#pragma unroll
            for (int i = 0; i < kRowsPerThread; ++i) {
                const int lr = i * 16 + warp * 2 + half;
                *reinterpret_cast<uint2*>(p.col_q + (r.padded0 + lr) * p.ldq + col) = codes<BF16, ODD>(v[i], by);
            }
            if (threadIdx.x < 16)
                *reinterpret_cast<uint2*>(p.col_scale + (r.padded0 >> 7) * p.ldq + col) = make_uint2(sc[0], sc[1]);
        }
        if (BLK) {
            uint32_t t = 0;
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                const uint4 u = *reinterpret_cast<const uint4*>(&part[w][lane * 4]);
                t = max(max(t, max(u.x, u.y)), max(u.z, u.w));
            }
            t = __reduce_max_sync(0xffffffffu, t);
            const int e = scale_exponent(t);
            float by[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) by[j] = inverse_scale(e);
            uint8_t* q = p.blk_q + batch * p.rows * p.ldq;
#pragma unroll
            for (int i = 0; i < kRowsPerThread; ++i) {
                const int lr = i * 16 + warp * 2 + half;
                if (lr < r.rows) *reinterpret_cast<uint2*>(q + (r.row0 + lr) * p.ldq + col) = codes<BF16, ODD>(v[i], by);
            }
            if (threadIdx.x == 0)
                p.blk_scale[(batch * ((p.rows + 127) >> 7) + (r.row0 >> 7)) * (p.ldq >> 7) + cb] =
                    static_cast<uint8_t>(e + 127);
        }
    }
}

template <bool BF16, bool ROW, bool COL, bool BLK>
__global__ void __launch_bounds__(kThreads) k_fp8_quantize(const __grid_constant__ QuantParams p) {
    __shared__ uint32_t part[8][128];
    __shared__ RowBlock rb;
    __shared__ int offsets[COL ? kFp8MaxGroups + 1 : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int cg = lane & 15, half = lane >> 4;
    const long long batch = blockIdx.z, colblocks = p.ldq >> 7;
    const char* base = static_cast<const char*>(p.x) + batch * p.ldb * (BF16 ? 2 : 4);
    if (COL && p.groups > 0) {
        for (int g = threadIdx.x; g <= p.groups; g += kThreads) offsets[g] = p.offsets[g];
        __syncthreads();
    }

    for (long long y = blockIdx.y; y < p.row_blocks; y += gridDim.y) {
        find_row_block(p, offsets, y, &rb);
        __syncthreads();
        const RowBlock r = rb;
        if (!r.valid) return;                            // the blocks past the last one
        for (long long cb = blockIdx.x; cb < colblocks; cb += gridDim.x) {
            const long long col = cb * 128 + cg * 8;
            Raw v[kRowsPerThread];
            if (p.vec && cb * 128 + 128 <= p.cols && r.rows == 128) {
                const char* src = base + ((r.row0 + warp * 2 + half) * p.ld + col) * (BF16 ? 2 : 4);
                const long long step = 16 * p.ld * (BF16 ? 2 : 4);
#pragma unroll
                for (int i = 0; i < kRowsPerThread; ++i) {
                    v[i].a = *reinterpret_cast<const uint4*>(src + i * step);
                    v[i].b = BF16 ? v[i].a : *reinterpret_cast<const uint4*>(src + i * step + 16);
                }
            } else if (p.vec && cb * 128 + 128 <= p.cols) {
                // a group's last rows
                const char* src = base + ((r.row0 + warp * 2 + half) * p.ld + col) * (BF16 ? 2 : 4);
                const long long step = 16 * p.ld * (BF16 ? 2 : 4);
#pragma unroll
                for (int i = 0; i < kRowsPerThread; ++i) {
                    v[i].a = v[i].b = make_uint4(0, 0, 0, 0);
                    if (i * 16 + warp * 2 + half < r.rows) {
                        v[i].a = *reinterpret_cast<const uint4*>(src + i * step);
                        if (!BF16) v[i].b = *reinterpret_cast<const uint4*>(src + i * step + 16);
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < kRowsPerThread; ++i) {
                    const int lr = i * 16 + warp * 2 + half;
                    v[i].a = v[i].b = make_uint4(0, 0, 0, 0);
                    if (lr < r.rows) v[i] = load_edge<BF16>(p, base, r.row0 + lr, col);
                }
            }
            Maxima<BF16> m;
            m.clear();
#pragma unroll
            for (int i = 0; i < kRowsPerThread; ++i) m.add(v[i]);
            if (__syncthreads_or(m.all() >= kInf)) tile<BF16, ROW, COL, BLK, true>(p, r, v, part, cb, batch);
            else tile<BF16, ROW, COL, BLK, false>(p, r, v, part, cb, batch);
        }
        __syncthreads();                                 // rb is written anew
    }
}

template <bool BF16>
cudaError_t run(const QuantParams& p, cudaStream_t s) {
    // several tiles of a row block per block of threads where there are enough of
    // both: finding a group's row block costs about as much as half a tile
    const long long colblocks = p.ldq / 128;
    const long long share = p.groups > 0 && colblocks * p.row_blocks > 4096 ? 4 : 1;
    const dim3 grid(static_cast<unsigned>((colblocks + share - 1) / share),
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
