// Products with weights of 4 bits: y[t, n] = sum_k x[t, k] code[n, k] scale[k / block, n].
//
// Serving makes these products for one token, or a few for each expert: their time is the
// weights' bytes, a quarter of bf16's.  Codes become bf16 exactly, x is bf16 (fp32 is
// taken as the sum of three bf16), products of 16 columns run on mma.sync with fp32 sums, and
// a scale multiplies the sum over its columns, so nothing is rounded before the result.
//
// A weight code costs half an instruction to take out and half one to turn into bf16
// (two at a time); a vector unit's product would cost another per code and token, a
// matrix fragment of 16 rows x 8 tokens a sixteenth.  (tcgen05 has nothing to add: its
// operands would take a trip through shared memory, and the tensor core idles either way.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "groups.cuh"
#include "int4.cuh"
#include "internal.h"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// -------------------------------------------------------------- rounding --
// scale = max|w| / 7 rounded to bf16, code = w / scale rounded to the nearest whole number
// (ties to even) between -7 and 7.  A scale that rounds to zero has zero codes; one of
// columns with an infinity or a NaN is NaN, so that their products show it.  A warp takes 128
// columns of a row, four a lane.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_int4_quantize(const Int4QuantParams p) {
    const int lane = threadIdx.x & 31;
    const long long item = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const long long row = item / p.kblocks;                 // over all matrices
    if (row >= p.rows * p.batch) return;
    const int kb = static_cast<int>(item - row * p.kblocks);
    const int col = kb * 128 + 4 * lane;
    const T* w = static_cast<const T*>(p.w) + row * p.cols;
    float v[4];
    float top = 0.0f;
    bool odd = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = col + i < p.cols ? static_cast<float>(w[col + i]) : 0.0f;
        odd |= !(fabsf(v[i]) <= 3.402823466e+38f);
        top = fmaxf(top, fabsf(v[i]));
    }
    const int lanes = p.block / 4;
    for (int o = 1; o < lanes; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const unsigned group = (lanes == 32 ? 0xffffffffu : ((1u << lanes) - 1u) << (lane & ~(lanes - 1)));
    odd = (__ballot_sync(0xffffffffu, odd) & group) != 0u;
    const __nv_bfloat16 scale = __float2bfloat16_rn(odd ? __int_as_float(0x7fc00000) : __fdiv_rn(top, 7.0f));
    const float by = __bfloat162float(scale);
    uint32_t code = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float q = by > 0.0f ? fminf(fmaxf(rintf(__fdiv_rn(v[i], by)), -7.0f), 7.0f) : 0.0f;
        code |= (static_cast<uint32_t>(static_cast<int>(q)) & 15u) << (4 * i);
    }
    reinterpret_cast<uint16_t*>(p.codes)[(row * p.kblocks + kb) * 32 + lane] = static_cast<uint16_t>(code);
    if (lane % lanes == 0) {
        const long long b = row / p.rows, n = row - b * p.rows;
        const long long per = 128 / p.block;
        p.scale[(b * p.kblocks * per + kb * per + lane / lanes) * p.rows + n] = scale;
    }
}

// --------------------------------------------------------------- groups --
// The column tiles of all groups, TILE tokens each: made by every block for itself.
struct GroupTable {
    int tile0[kFp8MaxGroups + 1];                          // first column tile of each group
    int lo[kFp8MaxGroups], cnt[kFp8MaxGroups];
    int first, last;                                       // rows of any group
};

template <int TILE>
__device__ __forceinline__ void make_table(const Int4Params& p, GroupTable& t) {
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int low = 0, tiles = 0, first = p.tokens;
        for (int g0 = 0; g0 < p.groups; g0 += 32) {
            const GroupSpan s = warp_group_spans(p.offsets, p.groups, p.tokens, g0, low);
            const int mine = (s.cnt + TILE - 1) / TILE;
            const int sum = warp_inclusive_sum(mine);
            if (g0 + lane < p.groups) {
                t.tile0[g0 + lane] = tiles + sum - mine;
                t.lo[g0 + lane] = s.lo;
                t.cnt[g0 + lane] = s.cnt;
            }
            tiles += __shfl_sync(0xffffffffu, sum, 31);
            const unsigned some = __ballot_sync(0xffffffffu, s.cnt > 0);
            if (some != 0u && first == p.tokens) first = __shfl_sync(0xffffffffu, s.lo, __ffs(some) - 1);
        }
        if (lane == 0) {
            t.tile0[p.groups] = tiles;
            t.first = first;
            t.last = first == p.tokens ? p.tokens : low;
        }
    }
    __syncthreads();
}

// The group of a column tile: the last whose first tile is not past it (empty groups share
// their first tile with the next).
__device__ __forceinline__ int group_of(const GroupTable& t, int groups, int tile) {
    int lo = 0, hi = groups - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.tile0[mid] <= tile) lo = mid; else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ void store_out(const Int4Params& p, long long at, float v) {
    if (p.out_f32) static_cast<float*>(p.out)[at] = v;
    else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(v);
}

// Rows of no group become zero: those before the first group's and after the last's.
__device__ __forceinline__ void zero_rest(const Int4Params& p, const GroupTable& t) {
    const long long lead = t.first, rest = lead + p.tokens - t.last;
    if (rest == 0) return;
    const long long total = rest * p.n;
    for (long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; i < total;
         i += static_cast<long long>(gridDim.x) * kThreads) {
        const long long r = i / p.n;
        store_out(p, (r < lead ? r : r - lead + t.last) * p.ld_out + (i - r * p.n), 0.0f);
    }
}

// ------------------------------------------------------------ few tokens --
// A block takes 16 rows of a weight and up to eight tokens; its warps take the reduction's
// blocks of 128 in turn and add their sums up in shared memory at the end, in a fixed order.
// Codes of kAhead blocks are under way for each warp, the first of the next item's before
// the sums of this one are added.  x comes through the first level, which the items of a
// block share.
constexpr int kRows = 16;
constexpr int kTokens = 8;
constexpr int kAhead = 4;

template <int BLOCK, int PARTS>
__global__ void __launch_bounds__(kThreads, 2) k_int4_few(const Int4Params p) {
    constexpr int kScales = 128 / BLOCK;
    __shared__ GroupTable table;
    __shared__ float part[kWarps][kTokens][kRows + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = lane >> 2, j = lane & 3;
    make_table<kTokens>(p, table);
    const int row_tiles = (p.n + kRows - 1) / kRows;
    const long long items = static_cast<long long>(table.tile0[p.groups]) * row_tiles;

    uint4 codes[kAhead][2];
    const uint8_t *w_lo = nullptr, *w_hi = nullptr;
    auto aim = [&](long long item) {
        const int tile = static_cast<int>(item / row_tiles), n0 = static_cast<int>(item - static_cast<long long>(tile) * row_tiles) * kRows;
        const uint8_t* w = p.w + group_of(table, p.groups, tile) * p.w_batch;
        // rows past the last read the last one's codes; their results are not stored
        w_lo = w + min(n0 + r, p.n - 1) * p.ldw;
        w_hi = w + min(n0 + r + 8, p.n - 1) * p.ldw;
    };
    auto fetch = [&](int kb0) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (kb0 + i * kWarps < p.kblocks) {
                codes[i][0] = load_codes<BLOCK>(w_lo, kb0 + i * kWarps, j);
                codes[i][1] = load_codes<BLOCK>(w_hi, kb0 + i * kWarps, j);
            }
        }
    };
    long long item = blockIdx.x;
    if (item < items) {
        aim(item);
        fetch(warp);
    }
    for (; item < items; item += gridDim.x) {
        const int tile = static_cast<int>(item / row_tiles), n0 = static_cast<int>(item - static_cast<long long>(tile) * row_tiles) * kRows;
        const int g = group_of(table, p.groups, tile);
        const int t0 = table.lo[g] + (tile - table.tile0[g]) * kTokens;
        const int tokens = min(kTokens, table.lo[g] + table.cnt[g] - t0);
        const __nv_bfloat16* s = p.scale + g * p.scale_batch;
        const __nv_bfloat16 *s_lo = s + min(n0 + r, p.n - 1), *s_hi = s + min(n0 + r + 8, p.n - 1);
        // as B fragment a lane holds token r; as accumulator tokens 2 j and 2 j + 1
        const bool have = r < tokens;
        const char* x = static_cast<const char*>(p.x) + (t0 + (have ? r : 0)) * p.ld_x * (PARTS == 1 ? 2 : 4);

        float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int kb0 = warp; kb0 < p.kblocks; kb0 += kAhead * kWarps) {
            if (kb0 != warp) fetch(kb0);
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int kb = kb0 + i * kWarps;
                if (kb >= p.kblocks) break;
                float by[kScales][2];
#pragma unroll
                for (int q = 0; q < kScales; ++q) {
                    by[q][0] = __bfloat162float(s_lo[static_cast<long long>(kb * kScales + q) * p.n]);
                    by[q][1] = __bfloat162float(s_hi[static_cast<long long>(kb * kScales + q) * p.n]);
                }
                RawOfX<PARTS> raw[4];
#pragma unroll
                for (int m = 0; m < 4; ++m) {
#pragma unroll
                    for (int v = 0; v < (PARTS == 1 ? 1 : 2); ++v) raw[m].v[v] = make_uint4(0, 0, 0, 0);
                    if (have) raw[m] = load_x<PARTS>(x, kb * 128 + chunk_of<BLOCK>(m, j) * 8, p.k, p.vec);
                }
                float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const EightCodes lo = decode(word_of(codes[i][0], m)), hi = decode(word_of(codes[i][1], m));
                    const EightOfX<PARTS> b = fragments<PARTS>(raw[m]);
#pragma unroll
                    for (int q = PARTS - 1; q >= 0; --q) mma_step(c, lo, hi, b.v[q]);
                    if ((m + 1) % (4 / kScales) == 0) {
                        const int q = m / (4 / kScales);
                        acc[0] = fmaf(c[0], by[q][0], acc[0]);
                        acc[1] = fmaf(c[1], by[q][0], acc[1]);
                        acc[2] = fmaf(c[2], by[q][1], acc[2]);
                        acc[3] = fmaf(c[3], by[q][1], acc[3]);
                        c[0] = c[1] = c[2] = c[3] = 0.0f;
                    }
                }
            }
        }
        if (item + gridDim.x < items) {
            aim(item + gridDim.x);
            fetch(warp);
        }
        __syncthreads();                                   // the sums of the item before have been read
        part[warp][2 * j][r] = acc[0];
        part[warp][2 * j + 1][r] = acc[1];
        part[warp][2 * j][r + 8] = acc[2];
        part[warp][2 * j + 1][r + 8] = acc[3];
        __syncthreads();
        if (threadIdx.x < kTokens * kRows) {
            const int t = threadIdx.x / kRows, n = threadIdx.x % kRows;
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) sum += part[i][t][n];
            if (t < tokens && n0 + n < p.n) store_out(p, (t0 + t) * p.ld_out + n0 + n, sum * kCodeUnit);
        }
    }
    if (p.offsets != nullptr) zero_rest(p, table);
}

template <int BLOCK>
cudaError_t few(const Int4Params& p, int sms, cudaStream_t s) {
    const long long tiles = p.tokens / kTokens + (p.groups < p.tokens ? p.groups : p.tokens);
    const long long items = tiles * ((p.n + kRows - 1) / kRows);
    const long long most = 2ll * sms;
    const unsigned grid = static_cast<unsigned>(items < most ? items : most);
    if (p.x_bf16) k_int4_few<BLOCK, 1><<<grid, kThreads, 0, s>>>(p);
    else k_int4_few<BLOCK, 3><<<grid, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_int4_quantize(const Int4QuantParams& p, cudaStream_t s) {
    const long long blocks = (p.rows * p.batch * p.kblocks + kWarps - 1) / kWarps;
    if (p.bf16) k_int4_quantize<__nv_bfloat16><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(p);
    else k_int4_quantize<float><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_int4_linear(const Int4Params& p, int sms, cudaStream_t s) {
    switch (p.block) {
        case 32: return few<32>(p, sms, s);
        case 64: return few<64>(p, sms, s);
        default: return few<128>(p, sms, s);
    }
}

}  // namespace muon
