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

#include "fp8_codes.cuh"
#include "groups.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsPerThread = 8;

// Largest magnitudes of eight columns over rows: bf16 two to a word, fp32 bits one.
template <bool BF16>
struct ColMax {
    uint32_t m[BF16 ? 4 : 8];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (uint32_t& v : m) v = 0;
    }
    __device__ __forceinline__ void add(const Raw& r) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (BF16) {
                m[i] = __vmaxu2(m[i], word(r.a, i) & 0x7fff7fffu);
            } else {
                m[i] = max(m[i], word(r.a, i) & 0x7fffffffu);
                m[i + 4] = max(m[i + 4], word(r.b, i) & 0x7fffffffu);
            }
        }
    }
    __device__ __forceinline__ void meet(int lane_mask) {
#pragma unroll
        for (uint32_t& v : m) {
            const uint32_t o = __shfl_xor_sync(0xffffffffu, v, lane_mask);
            v = BF16 ? __vmaxu2(v, o) : max(v, o);
        }
    }
    __device__ __forceinline__ uint32_t column(int j) const {
        if constexpr (BF16) return (j & 1) ? (m[j >> 1] & 0xffff0000u) : (m[j >> 1] << 16);
        else return m[j];
    }
    __device__ __forceinline__ uint32_t all() const {
        uint32_t v = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) v = max(v, column(j));
        return v;
    }
};

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

// The first `left` of eight elements, zero in the places of the others.
template <bool BF16>
__device__ __forceinline__ Raw first_of(const Raw& r, int left) {
    if (left >= 8) return r;
    uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (i >= left) {
            if (BF16) w[i >> 1] &= (i & 1) ? 0x0000ffffu : 0xffff0000u;
            else w[i] = 0;
        }
    }
    Raw o;
    o.a = make_uint4(w[0], w[1], w[2], w[3]);
    o.b = BF16 ? o.a : make_uint4(w[4], w[5], w[6], w[7]);
    return o;
}

// Eight elements from any element on: the 16-byte vectors that hold them, shifted
// into place (rows of odd length start anywhere; element by element they loaded at
// a quarter of the rate).
template <bool BF16>
struct Shifted {
    static constexpr int kSize = BF16 ? 2 : 4, kVecs = BF16 ? 2 : 3;
    uint4 v[kVecs];
    static __device__ __forceinline__ const char* from(const char* s) {
        return reinterpret_cast<const char*>(reinterpret_cast<uintptr_t>(s) & ~static_cast<uintptr_t>(15));
    }
    __device__ __forceinline__ void load(const char* s) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) v[i] = *reinterpret_cast<const uint4*>(from(s) + 16 * i);
    }
    // the elements at s, `left` of them
    __device__ __forceinline__ Raw take(const char* s, int left) const {
        constexpr int kWords = 8 * kSize / 4;            // result words; one more for the odd half
        uint32_t w[12];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            w[4 * i] = v[i].x; w[4 * i + 1] = v[i].y; w[4 * i + 2] = v[i].z; w[4 * i + 3] = v[i].w;
        }
        const unsigned shift = static_cast<unsigned>(reinterpret_cast<uintptr_t>(s)) & 15u;
        const bool one = shift & 4, two = shift & 8;
#pragma unroll
        for (int i = 0; i <= kWords + 2; ++i) w[i] = one && i + 1 < 4 * kVecs ? w[i + 1] : w[i];
#pragma unroll
        for (int i = 0; i <= kWords; ++i) w[i] = two && i + 2 < 4 * kVecs ? w[i + 2] : w[i];
        if (BF16) {
            const unsigned bits = 8 * (shift & 2);
#pragma unroll
            for (int i = 0; i < kWords; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], bits);
        }
        Raw r;
        r.a = make_uint4(w[0], w[1], w[2], w[3]);
        r.b = BF16 ? r.a : make_uint4(w[4], w[5], w[6], w[7]);
        return first_of<BF16>(r, left);
    }
};

// Eight elements one by one: for the few whose vectors reach beyond the tensor.
template <bool BF16>
__device__ __noinline__ Raw load_last(const QuantParams& p, const char* base, long long row, long long col) {
    const char* s = base + (row * p.ld + col) * (BF16 ? 2 : 4);
    const int left = static_cast<int>(p.cols - col < 8 ? p.cols - col : 8);
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (i < left) {
            if (BF16) w[i >> 1] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(s)[i]) << (16 * (i & 1));
            else w[i] = reinterpret_cast<const uint32_t*>(s)[i];
        }
    }
    Raw r;
    r.a = make_uint4(w[0], w[1], w[2], w[3]);
    r.b = BF16 ? r.a : make_uint4(w[4], w[5], w[6], w[7]);
    return r;
}

// Shared memory of a block of threads.
struct Tile {
    uint32_t part[8][128];       // column maxima of each warp's rows
    float by[128];               // col blocks: 2^-e of each column
};

// One tile's maxima, scales and codes.
template <bool BF16, bool ROW, bool COL, bool BLK>
__device__ __forceinline__ void tile(const QuantParams& p, const RowBlock& r, Raw (&v)[kRowsPerThread], Tile& sh,
                                     long long cb, long long batch) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int cg = lane & 15, half = lane >> 4;
    const long long col = cb * 128 + cg * 8;
    uint32_t rm[kRowsPerThread];
    ColMax<BF16> cm;
    cm.clear();
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kRowsPerThread; ++i) {
        if (ROW) top = max(top, rm[i] = row_max<BF16>(v[i]));
        if (COL || BLK) cm.add(v[i]);
    }
    if (!ROW) top = cm.all();
    if (ROW && !COL ? __any_sync(0xffffffffu, top >= kInf) : __syncthreads_or(top >= kInf)) {
        cm.clear();
#pragma unroll
        for (int i = 0; i < kRowsPerThread; ++i) {
            const Raw f = replace_odd<BF16>(v[i], true);
            v[i] = replace_odd<BF16>(v[i], false);
            if (ROW) rm[i] = row_max<BF16>(f);
            if (COL || BLK) cm.add(f);
        }
    }
    if (COL || BLK) {
        cm.meet(16);
        if (half == 0) {
            uint4* dst = reinterpret_cast<uint4*>(&sh.part[warp][cg * 8]);
            dst[0] = make_uint4(cm.column(0), cm.column(1), cm.column(2), cm.column(3));
            dst[1] = make_uint4(cm.column(4), cm.column(5), cm.column(6), cm.column(7));
        }
        __syncthreads();
    }
    if (ROW) {
        // eight rows' maxima over 16 lanes: halve the rows a lane keeps at each
        // exchange; lane pair k of a half ends up with row k
        const bool b3 = cg & 8, b2 = cg & 4, b1 = cg & 2;
        uint32_t q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            q[i] = max(b3 ? rm[i + 4] : rm[i], __shfl_xor_sync(0xffffffffu, b3 ? rm[i] : rm[i + 4], 8));
#pragma unroll
        for (int i = 0; i < 2; ++i) q[i] = max(b2 ? q[i + 2] : q[i], __shfl_xor_sync(0xffffffffu, b2 ? q[i] : q[i + 2], 4));
        uint32_t m = max(b1 ? q[1] : q[0], __shfl_xor_sync(0xffffffffu, b1 ? q[0] : q[1], 2));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        const int e = scale_exponent(m);
        const float inv = inverse_scale(e);
        const int mine = (cg >> 1) * 16 + warp * 2 + half;
        if ((cg & 1) == 0 && mine < r.rows) p.row_scale[cb * p.rows + r.row0 + mine] = static_cast<uint8_t>(e + 127);
        uint8_t* dst = p.row_q + (r.row0 + warp * 2 + half) * p.ldq + col;
#pragma unroll
        for (int i = 0; i < kRowsPerThread; ++i) {
            const float by = __shfl_sync(0xffffffffu, inv, (lane & 16) + 2 * i);
            if (i * 16 + warp * 2 + half < r.rows)
                *reinterpret_cast<uint2*>(dst + i * 16 * p.ldq) = codes_of<BF16>(v[i], by);
        }
    }
    if (COL) {
        if (threadIdx.x < 128) {
            uint32_t t = 0;
#pragma unroll
            for (int w = 0; w < 8; ++w) t = max(t, sh.part[w][threadIdx.x]);
            const int e = scale_exponent(t);
            sh.by[threadIdx.x] = inverse_scale(e);
            p.col_scale[(r.padded0 >> 7) * p.ldq + cb * 128 + threadIdx.x] = static_cast<uint8_t>(e + 127);
        }
        __syncthreads();
        float by[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4 f = *reinterpret_cast<const float4*>(&sh.by[cg * 8 + 4 * h]);
            by[4 * h] = f.x;
            by[4 * h + 1] = f.y;
            by[4 * h + 2] = f.z;
            by[4 * h + 3] = f.w;
        }
        uint8_t* dst = p.col_q + (r.padded0 + warp * 2 + half) * p.ldq + col;
#pragma unroll
        for (int i = 0; i < kRowsPerThread; ++i) *reinterpret_cast<uint2*>(dst + i * 16 * p.ldq) = codes_of<BF16>(v[i], by);
    }
    if (BLK) {
        uint32_t t = 0;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            const uint4 u = *reinterpret_cast<const uint4*>(&sh.part[w][lane * 4]);
            t = max(max(t, max(u.x, u.y)), max(u.z, u.w));
        }
        t = __reduce_max_sync(0xffffffffu, t);
        const int e = scale_exponent(t);
        const float by = inverse_scale(e);
        uint8_t* dst = p.blk_q + (batch * p.rows + r.row0 + warp * 2 + half) * p.ldq + col;
#pragma unroll
        for (int i = 0; i < kRowsPerThread; ++i)
            if (i * 16 + warp * 2 + half < r.rows)
                *reinterpret_cast<uint2*>(dst + i * 16 * p.ldq) = codes_of<BF16>(v[i], by);
        if (threadIdx.x == 0)
            p.blk_scale[(batch * ((p.rows + 127) >> 7) + (r.row0 >> 7)) * (p.ldq >> 7) + cb] = static_cast<uint8_t>(e + 127);
    }
    // the next tile writes `part` after its vote, a barrier that follows every
    // thread's last read here
}

// The tiles of one block of threads.  VEC: rows start on 16 bytes.
template <bool BF16, bool ROW, bool COL, bool BLK, bool VEC>
__device__ __forceinline__ void quantize(const QuantParams& p, Tile& sh, RowBlock& rb, int* offsets, long long batch) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int cg = lane & 15, half = lane >> 4;
    const long long colblocks = p.ldq >> 7;
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
            if (VEC && cb * 128 + 128 <= p.cols) {
                const char* src = base + ((r.row0 + warp * 2 + half) * p.ld + col) * (BF16 ? 2 : 4);
                const long long step = 16 * p.ld * (BF16 ? 2 : 4);
                const int rows = r.rows - warp * 2 - half;
#pragma unroll
                for (int i = 0; i < kRowsPerThread; ++i) {
                    v[i].a = v[i].b = make_uint4(0, 0, 0, 0);
                    if (i * 16 < rows) {
                        v[i].a = *reinterpret_cast<const uint4*>(src + i * step);
                        if (!BF16) v[i].b = *reinterpret_cast<const uint4*>(src + i * step + 16);
                    }
                }
            } else {
                // All of a warp's vectors are loaded ahead here, too.  One that is not all
                // the tensor's own (its first or last) is marked, and made of elements after.
                // With the edge tiles' rows loaded one after the other, 1001 x 1300 in bf16
                // took 7.8 us for row codes; 5.4 so.
                constexpr int kSize = BF16 ? 2 : 4;
                const char* const first = static_cast<const char*>(p.x);
                const char* src = base + ((r.row0 + warp * 2 + half) * p.ld + col) * kSize;
                const long long step = 16 * p.ld * kSize;
                const int rows = r.rows - warp * 2 - half;
                const int left = static_cast<int>(p.cols - col < 8 ? (p.cols > col ? p.cols - col : 0) : 8);
                uint32_t odd = 0;
                constexpr int kAt = VEC ? kRowsPerThread : BF16 ? 4 : 2;   // rows at a time
                constexpr int kEdge = VEC ? kRowsPerThread : 2;   // at the edges (fewer registers: 4000 x 6150 bf16 23.8 -> 20.5 us)
                bool inner = false;                      // nothing to ask of any vector
                if constexpr (!VEC) {
                    inner = __all_sync(0xffffffffu,
                                       rows > 16 * (kRowsPerThread - 1) && left > 0 && Shifted<BF16>::from(src) >= first &&
                                           Shifted<BF16>::from(src + (kRowsPerThread - 1) * step) +
                                                   16 * Shifted<BF16>::kVecs <= p.x_end);
                    if (inner) {
#pragma unroll
                        for (int i = 0; i < kRowsPerThread; i += kAt) {
                            Shifted<BF16> x[kAt];
#pragma unroll
                            for (int u = 0; u < kAt; ++u) x[u].load(src + (i + u) * step);
#pragma unroll
                            for (int u = 0; u < kAt; ++u) v[i + u] = x[u].take(src + (i + u) * step, left);
                        }
                    }
                }
#pragma unroll
                for (int i0 = 0; i0 < kRowsPerThread && !inner; i0 += kEdge) {
                    if constexpr (VEC) {
#pragma unroll
                        for (int i = 0; i < kRowsPerThread; ++i) {
                            v[i].a = v[i].b = make_uint4(0, 0, 0, 0);
                            const char* a = src + i * step;
                            const bool want = i * 16 < rows && left > 0, more = !BF16 && want && left > 4;
                            if (want && a + 16 <= p.x_end) v[i].a = *reinterpret_cast<const uint4*>(a);
                            if (more && a + 32 <= p.x_end) v[i].b = *reinterpret_cast<const uint4*>(a + 16);
                            odd |= (want && a + (more ? 32 : 16) > p.x_end ? 1u : 0u) << i;
                        }
#pragma unroll
                        for (int i = 0; i < kRowsPerThread; ++i) v[i] = first_of<BF16>(v[i], left);
                    } else {
                        Shifted<BF16> x[kEdge];
#pragma unroll
                        for (int u = 0; u < kEdge; ++u) {
                            const char* a = src + (i0 + u) * step;
#pragma unroll
                            for (int k = 0; k < Shifted<BF16>::kVecs; ++k) {
                                const char* q = Shifted<BF16>::from(a) + 16 * k;
                                const bool want = (i0 + u) * 16 < rows && q < a + left * kSize;
                                const bool own = q >= first && q + 16 <= p.x_end;
                                x[u].v[k] = make_uint4(0, 0, 0, 0);
                                if (want && own) x[u].v[k] = *reinterpret_cast<const uint4*>(q);
                                odd |= (want && !own ? 1u : 0u) << (i0 + u);
                            }
                        }
#pragma unroll
                        for (int u = 0; u < kEdge; ++u) v[i0 + u] = x[u].take(src + (i0 + u) * step, left);
                    }
                }
                if (odd != 0) {
#pragma unroll
                    for (int i = 0; i < kRowsPerThread; ++i)
                        if (odd >> i & 1u) v[i] = load_last<BF16>(p, base, r.row0 + i * 16 + warp * 2 + half, col);
                }
            }
            tile<BF16, ROW, COL, BLK>(p, r, v, sh, cb, batch);
        }
        __syncthreads();                                 // rb is written anew
    }
}

template <bool BF16, bool ROW, bool COL, bool BLK, bool VEC>
__global__ void __launch_bounds__(kThreads, BF16 ? 3 : 2) k_fp8_quantize(const __grid_constant__ QuantParams p) {
    __shared__ Tile sh;
    __shared__ RowBlock rb;
    __shared__ int offsets[COL ? kFp8MaxGroups + 1 : 1];
    asm volatile("griddepcontrol.launch_dependents;");   // the product's set-up may overlap; it waits for the codes
    quantize<BF16, ROW, COL, BLK, VEC>(p, sh, rb, offsets, blockIdx.z);
}

// Two matrices: blockIdx.z 0 takes the first (row and col codes, or col codes
// alone), 1 the second's col codes.
template <bool BF16, bool ROW, bool VEC>
__global__ void __launch_bounds__(kThreads, BF16 ? 3 : 2)
    k_fp8_quantize_pair(const __grid_constant__ QuantParams p, const __grid_constant__ QuantParams q) {
    __shared__ Tile sh;
    __shared__ RowBlock rb;
    __shared__ int offsets[kFp8MaxGroups + 1];
    asm volatile("griddepcontrol.launch_dependents;");
    if (blockIdx.z == 0) quantize<BF16, ROW, true, false, VEC>(p, sh, rb, offsets, 0);
    else quantize<BF16, false, true, false, VEC>(q, sh, rb, offsets, 0);
}

// Several tiles of a row block per block of threads where there are enough of
// both: finding a group's row block costs about as much as half a tile.
dim3 quantize_grid(const QuantParams& p) {
    const long long colblocks = p.ldq / 128;
    const long long share = p.groups > 0 && colblocks * p.row_blocks > 4096 ? 4 : 1;
    return dim3(static_cast<unsigned>((colblocks + share - 1) / share),
                static_cast<unsigned>(p.row_blocks < 65535 ? p.row_blocks : 65535), static_cast<unsigned>(p.batch));
}

template <bool BF16, bool VEC>
cudaError_t run_pair(const QuantParams& p, const QuantParams& q, cudaStream_t s) {
    const dim3 a = quantize_grid(p), b = quantize_grid(q);
    const dim3 grid(a.x > b.x ? a.x : b.x, a.y > b.y ? a.y : b.y, 2);
    if (p.row_q != nullptr) k_fp8_quantize_pair<BF16, true, VEC><<<grid, kThreads, 0, s>>>(p, q);
    else k_fp8_quantize_pair<BF16, false, VEC><<<grid, kThreads, 0, s>>>(p, q);
    return cudaGetLastError();
}

template <bool BF16, bool VEC>
cudaError_t run(const QuantParams& p, cudaStream_t s) {
    const dim3 grid = quantize_grid(p);
    if (p.blk_q != nullptr) k_fp8_quantize<BF16, false, false, true, VEC><<<grid, kThreads, 0, s>>>(p);
    else if (p.row_q != nullptr && p.col_q != nullptr)
        k_fp8_quantize<BF16, true, true, false, VEC><<<grid, kThreads, 0, s>>>(p);
    else if (p.row_q != nullptr) k_fp8_quantize<BF16, true, false, false, VEC><<<grid, kThreads, 0, s>>>(p);
    else k_fp8_quantize<BF16, false, true, false, VEC><<<grid, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fp8_quantize(const QuantParams& p, cudaStream_t s) {
    if (p.bf16) return p.vec ? run<true, true>(p, s) : run<true, false>(p, s);
    return p.vec ? run<false, true>(p, s) : run<false, false>(p, s);
}

bool fp8_quantize_pairs(const QuantParams& p, const QuantParams& q) {
    return p.bf16 == q.bf16 && p.vec == q.vec && p.col_q != nullptr && q.col_q != nullptr && q.row_q == nullptr;
}

cudaError_t launch_fp8_quantize_pair(const QuantParams& p, const QuantParams& q, cudaStream_t s) {
    if (p.bf16) return p.vec ? run_pair<true, true>(p, q, s) : run_pair<true, false>(p, q, s);
    return p.vec ? run_pair<false, true>(p, q, s) : run_pair<false, false>(p, q, s);
}

}  // namespace muon
