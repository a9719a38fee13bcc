// Products with weights of 4 bits: y[t, n] = sum_k x[t, k] code[n, k] scale[k / block, n].
//
// Serving makes these products for one token, or a few for each expert: their time is the
// weights' bytes, a quarter of bf16's.  Codes become bf16 exactly, x is bf16 (fp32 is
// taken as the sum of three bf16), products of 16 columns run on mma.sync with fp32 sums, and
// a scale multiplies the sum over its columns, so no operand is rounded.
//
// A lane's word of eight codes costs 9 instructions to take out and turn into bf16 (two codes at a
// time: mask and offset in one three-way operation, one fused multiply-add).  A unit of 32 rows x 128
// columns is 16 words a lane, 144 instructions of 307 in all with scales of 128 columns, of 328 with 64
// and 361 with 32, and 16 products of 16 x 16 x 8; one of 16 rows, scales of 128, 278 with its share of
// the launch's.  On the vector units each word and token would cost eight more.
//
// Device time, bf16 x: one token x 6144 x 6144 8.4 us (weights of 19.5 MB, 2.9 us at the rate of a
// copy; 9.0 from memory; 12.7 with loads through registers and no ring), 8 tokens 9.1.  A fixed part
// bounds it: one token takes 4.2 us for 16 rows of k = 6144, 4.7 for 2048, and from 8192 rows (9.2) on 0.69 us
// for 1024 more (4.7 TB/s); its instructions alone would take 4.4 us of the SMs' issue slots.
// 256 rows over 96 experts of 2048 x 6144, of which 75 have rows: 122 us, with scales of 32 columns 129
// (534 MB read, 4.1 TB/s); bound by the copies, which alone, without products, take 99 and 104, with issue slots
// 57 - 62 % busy beside them.  Past 16 tokens of a weight the time goes with the tokens, 18 us for 32, 32 for
// 64, 195 for 512: every 16 tokens take the codes out again.  (Below that tcgen05 would add a trip
// of its operands through shared memory, and the tensor core is 12 - 22 % busy.)  fp32 x, three times the
// products and its split: 15 us for one token.  Two warps to a row's reduction instead of eight gained 1 % for
// the experts, shifts by multiplication lost 10: not kept.
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

// -------------------------------------------------------------- products --
// An item is 16 RT rows of a weight and up to 8 NT tokens of one group; a block takes
// consecutive items, all its warps together: each the reduction's blocks of 128 in turn (a
// unit), and at an item's end they add their sums up in shared memory, in a fixed order.  So
// a single token's product fills the SMs (one token x 6144 x 6144 is 384 items), and any
// number of tokens or groups runs the same way.
//
// Codes and scales of kStages - 1 units are under way for each warp by asynchronous copies
// into a ring of its own, over the ends of items, with no wait between warps.  A row's 64
// bytes lie there in 16-byte pieces that ldmatrix reads without bank conflicts; it hands lane
// (r, j) the word of 8 codes that its fragment wants.  Fragment rows r and r + 8 are the
// weight's rows 2 r and 2 r + 1, whose scales are neighbours.  x comes from L2 through the
// first level, a unit ahead.
template <int RT>
struct Unit {
    uint4 codes[RT * 64];                                  // 16 RT rows of 64 bytes, even rows first
    uint32_t scale[RT * 8][4];                             // bf16 pairs of a pair of rows, the unit's scales
};

// Units under way and the sums of one or two items.  Two blocks per SM, three where RT and PARTS are
// 1 (by registers: the tiles of 16 tokens fill the 128 of two blocks, and keep 16 to 64 bytes of a lane in
// local memory for scales of 32 and 64 columns, with fp32 x of 64 and 128; those of 8 tokens at most 8).  With six
// units (RT 1) the start of a block costs more than it gains, one token x 6144 x 6144 9.5 us against 8.4 with
// three and 8.1 with two (10.1, 9.1 and 9.1 with the weight from memory; a third as many rows 6.6, 6.0 and 6.9).
template <int PARTS, int RT, int NT>
struct Shape {
    static constexpr int kStages = 3;
    static constexpr int kTurns = NT == 1 ? 2 : 1;
    static constexpr bool kAheadX = PARTS * NT <= 3;       // else registers do not last
    static constexpr size_t kRing = sizeof(Unit<RT>) * kStages * kWarps;
};

__device__ __forceinline__ uint32_t shared_address(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// Piece m of row `slot` of a unit, in 16 bytes: eight rows' pieces m lie in eight different places modulo 128.
__device__ __forceinline__ int piece(int slot, int m) { return slot * 4 + (m ^ ((slot >> 1) & 3)); }

template <int BLOCK, int PARTS, int RT, int NT>
__global__ void __launch_bounds__(kThreads, RT == 1 && PARTS == 1 ? 3 : 2) k_int4_linear(const Int4Params p) {
    using S = Shape<PARTS, RT, NT>;
    constexpr int kScales = 128 / BLOCK, kSteps = 4 / kScales;
    constexpr int kRows = 16 * RT, kTokens = 8 * NT, kSize = PARTS == 1 ? 2 : 4;
    constexpr int kStages = S::kStages, kUnit = static_cast<int>(sizeof(Unit<RT>));
    extern __shared__ uint4 dynamic[];
    __shared__ GroupTable table;
    __shared__ float part[S::kTurns][kWarps][kTokens][kRows + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = lane >> 2, j = lane & 3;
    Unit<RT>* const ring = reinterpret_cast<Unit<RT>*>(dynamic) + warp * kStages;
    const uint32_t ring_at = shared_address(ring);
    const unsigned row_tiles = (p.n + kRows - 1) / kRows;
    unsigned tiles = (p.tokens + kTokens - 1) / kTokens;
    if (p.offsets != nullptr) {
        make_table<kTokens>(p, table);
        tiles = table.tile0[p.groups];
    }
    // this block's items: an equal share, in a row
    const unsigned items = tiles * row_tiles, share = items / gridDim.x, over = items - share * gridDim.x;
    const unsigned begin = blockIdx.x * share + min(blockIdx.x, over);
    const int mine = static_cast<int>(share + (blockIdx.x < over ? 1u : 0u));
    const unsigned first_tile = begin / row_tiles, first_row = begin - first_tile * row_tiles;

    // ---- the copies: items left, block of the reduction, this lane's sources and places
    int c_left = warp < p.kblocks ? mine : 0, ckb = warp;
    unsigned c_tile = first_tile, c_row = first_row;
    const uint8_t* codes[2 * RT] = {};
    const __nv_bfloat16* scales = nullptr;
    bool scaled = false;                                   // this lane copies scales of the item
    int c_group = 0;
    const long long scale_hop = static_cast<long long>(kWarps) * kScales * p.n;
    // rows 8 i + lane / 4, even ones before odd ones; 16 rows on is 16 slots on
    const int row0 = lane >> 2, slot0 = (row0 & 1) * 8 + (row0 >> 1);
    const int put[2] = {piece(slot0, lane & 3) * 16, piece(slot0 + 4, lane & 3) * 16};
    const int q0 = lane / (8 * RT), at0 = lane % (8 * RT), put_scale = RT * 1024 + (at0 * 4 + q0) * 4;
    if (p.offsets != nullptr && mine > 0) c_group = group_of(table, p.groups, first_tile);
    auto aim = [&] {
        const int n0 = static_cast<int>(c_row) * kRows;
        const uint8_t* w = p.w + c_group * p.w_batch + warp * 64 + (lane & 3) * 16;
        // rows past the last are the last one again; their results are not stored
#pragma unroll
        for (int i = 0; i < 2 * RT; ++i) codes[i] = w + min(n0 + i * 8 + row0, p.n - 1) * p.ldw;
        const int at = n0 + 2 * at0;
        scaled = p.pairs && q0 < kScales && at < p.n;
        scales = p.scale + c_group * p.scale_batch + static_cast<long long>(warp * kScales + q0) * p.n + at;
    };
    auto copy = [&](uint32_t to) {
        if (c_left > 0) {
#pragma unroll
            for (int i = 0; i < 2 * RT; ++i) {
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + put[i & 1] + (i >> 1) * 1024), "l"(codes[i]));
                codes[i] += kWarps * 64;
            }
            if (scaled) {                                  // a lane's pair, and those that 32 lanes do not reach
#pragma unroll
                for (int i = 0; i < kScales * RT; i += 4)
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to + put_scale + (i / RT) * 4),
                                 "l"(scales + static_cast<long long>(i / RT) * p.n));
                scales += scale_hop;
            }
            ckb += kWarps;
            if (ckb >= p.kblocks) {
                ckb = warp;
                if (--c_left > 0) {
                    if (++c_row == row_tiles) {
                        c_row = 0;
                        ++c_tile;
                        if (p.offsets != nullptr) c_group = group_of(table, p.groups, c_tile);
                    }
                    aim();
                }
            }
        }
        asm volatile("cp.async.commit_group;");
    };
    if (c_left > 0) aim();
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) copy(ring_at + i * kUnit);
    int stage = 0, turn = 0;
    // ldmatrix: lane 8 m + i names piece m of row i; eight rows on, the pieces lie alike
    const uint32_t get = ring_at + piece(lane & 7, lane >> 3) * 16;

    // ---- the items: group, tokens, and where this lane's tokens lie.  As B fragment a lane
    // holds tokens r, r + 8, ..; as accumulator tokens 2 j and 2 j + 1 of each eight
    unsigned tile = first_tile, row_tile = first_row;
    int g = 0, t0 = 0, tokens = 0;
    const char* x[NT];
    auto look = [&] {                                      // at a new column tile
        t0 = static_cast<int>(tile) * kTokens;
        int end = p.tokens;
        if (p.offsets != nullptr) {
            g = group_of(table, p.groups, tile);
            t0 = table.lo[g] + (static_cast<int>(tile) - table.tile0[g]) * kTokens;
            end = table.lo[g] + table.cnt[g];
        }
        tokens = min(kTokens, end - t0);
        // tokens past the last are the last one again; their results are not stored
#pragma unroll
        for (int t = 0; t < NT; ++t)
            x[t] = static_cast<const char*>(p.x) + ((t0 + min(8 * t + r, tokens - 1)) * p.ld_x + 8 * j) * kSize;
    };
    const int whole = p.vec ? p.k / 128 : 0;               // units whose x loads as vectors
    const char* const x_begin = static_cast<const char*>(p.x);
    const char* const x_end = x_begin + ((p.tokens - 1) * p.ld_x + p.k) * kSize;
    constexpr int kHeld = S::kAheadX ? 4 : 1;              // steps whose x is in registers
    RawOfX<PARTS> raw[kHeld][NT];
    auto load = [&](int kb, int m0) {                      // kHeld steps of unit kb from m0 on
        if (kb < whole) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const char* at = x[t] + kb * (128 * kSize);
#pragma unroll
                for (int m = 0; m < kHeld; ++m) raw[m][t] = load_x<PARTS>(at + 32 * kSize * (m0 + m));
            }
            return;
        }
#pragma unroll
        for (int m = 0; m < kHeld; ++m) {
            const int col = kb * 128 + 32 * (m0 + m);      // of lane 0
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const char* at = x[t] + static_cast<long long>(col) * kSize;
                raw[m][t] = S::kAheadX ? load_x_edge<PARTS>(at, p.k - col - 8 * j, x_begin, x_end)
                                       : call_x_edge<PARTS>(at, p.k - col - 8 * j, x_begin, x_end);
            }
        }
    };
    if (mine > 0) look();
    if (S::kAheadX && mine > 0 && warp < p.kblocks) load(warp, 0);
    for (int left = mine; left > 0; --left) {
        const int n0 = static_cast<int>(row_tile) * kRows, out_row = t0, out_rows = tokens, group = g;
        const bool on = row_tile + 1 == row_tiles;         // the next item is of another column tile
        float acc[RT][NT][4] = {};
        for (int kb = warp; kb < p.kblocks; kb += kWarps) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
            __syncwarp();
            const uint32_t from = get + stage * kUnit;
            uint32_t w[RT][2][4];
#pragma unroll
            for (int a = 0; a < RT; ++a)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(w[a][h][0]), "=r"(w[a][h][1]), "=r"(w[a][h][2]), "=r"(w[a][h][3])
                                 : "r"(from + a * 1024 + h * 512));
            uint32_t by[RT][4];
#pragma unroll
            for (int a = 0; a < RT; ++a) {
                if (p.pairs) {
                    const uint32_t* s = ring[stage].scale[a * 8 + r];
                    if (kScales == 4) {
                        const uint4 v = *reinterpret_cast<const uint4*>(s);
                        by[a][0] = v.x, by[a][1] = v.y, by[a][2] = v.z, by[a][3] = v.w;
                    } else {
#pragma unroll
                        for (int q = 0; q < kScales; ++q) by[a][q] = s[q];
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < kScales; ++q) {
                        const uint16_t* s = reinterpret_cast<const uint16_t*>(p.scale) + group * p.scale_batch +
                                            static_cast<long long>(kb * kScales + q) * p.n;
                        const int row = n0 + a * 16 + 2 * r;
                        by[a][q] = s[min(row, p.n - 1)] | (static_cast<uint32_t>(s[min(row + 1, p.n - 1)]) << 16);
                    }
                }
            }
            // into the place of the unit before this one, which every lane has read
            copy(ring_at + (stage == 0 ? kStages - 1 : stage - 1) * kUnit);
            stage = stage == kStages - 1 ? 0 : stage + 1;

            float c[RT][NT][4];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                if (!S::kAheadX) load(kb, m);
                EightCodes lo[RT], hi[RT];
#pragma unroll
                for (int a = 0; a < RT; ++a) {
                    lo[a] = decode(w[a][0][m]);
                    hi[a] = decode(w[a][1][m]);
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const EightOfX<PARTS> b = fragments<PARTS>(raw[m % kHeld][t]);
#pragma unroll
                    for (int a = 0; a < RT; ++a)
#pragma unroll
                        for (int q = PARTS - 1; q >= 0; --q)
                            mma_step(c[a][t], q == PARTS - 1 && m % kSteps == 0, lo[a], hi[a], b.v[q]);
                }
                if ((m + 1) % kSteps == 0) {
#pragma unroll
                    for (int a = 0; a < RT; ++a) {
                        const uint32_t s = by[a][m / kSteps];
                        const float s_lo = __uint_as_float(s << 16), s_hi = __uint_as_float(s & 0xffff0000u);
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            acc[a][t][0] = fmaf(c[a][t][0], s_lo, acc[a][t][0]);
                            acc[a][t][1] = fmaf(c[a][t][1], s_lo, acc[a][t][1]);
                            acc[a][t][2] = fmaf(c[a][t][2], s_hi, acc[a][t][2]);
                            acc[a][t][3] = fmaf(c[a][t][3], s_hi, acc[a][t][3]);
                        }
                    }
                }
            }
            if (S::kAheadX) {                              // x of the next unit (at the very end, one more of this item)
                const bool done = kb + kWarps >= p.kblocks;
                if (done && on && left > 1) {
                    ++tile;
                    look();
                }
                load(done ? warp : kb + kWarps, 0);
            }
        }
        // with room for two items' sums, those of the item before the last have been read by now
        if (S::kTurns == 1) __syncthreads();
#pragma unroll
        for (int a = 0; a < RT; ++a)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) part[turn][warp][8 * t + 2 * j + (i & 1)][16 * a + 2 * r + (i >> 1)] = acc[a][t][i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kTokens * kRows; i += kThreads) {
            const int t = (i + static_cast<int>(threadIdx.x)) / kRows, n = (i + static_cast<int>(threadIdx.x)) % kRows;
            if (t < out_rows && n0 + n < p.n) {
                float sum = 0.0f;
#pragma unroll
                for (int k = 0; k < kWarps; ++k) sum += part[turn][k][t][n];
                store_out(p, (out_row + t) * p.ld_out + n0 + n, sum * kCodeUnit);
            }
        }
        turn = S::kTurns - 1 - turn;
        if (on && left > 1 && !(S::kAheadX && warp < p.kblocks)) {     // those that have not looked ahead
            ++tile;
            look();
        }
        row_tile = on ? 0 : row_tile + 1;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (p.offsets != nullptr) zero_rest(p, table);
}

// Blocks that the SMs hold at once.
template <int PARTS, int RT>
long long resident(int sms) {
    return (RT == 1 && PARTS == 1 ? 3ll : 2ll) * sms;
}

template <int BLOCK, int PARTS, int RT, int NT>
cudaError_t run(const Int4Params& p, int sms, cudaStream_t s) {
    const auto kernel = k_int4_linear<BLOCK, PARTS, RT, NT>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(Shape<PARTS, RT, NT>::kRing));
    if (e != cudaSuccess) return e;
    const long long tiles = p.offsets == nullptr ? (p.tokens + 8 * NT - 1) / (8 * NT)
                                                 : p.tokens / (8 * NT) + (p.groups < p.tokens ? p.groups : p.tokens);
    const long long items = tiles * ((p.n + 16 * RT - 1) / (16 * RT)), most = resident<PARTS, RT>(sms);
    kernel<<<static_cast<unsigned>(items < most ? items : most), kThreads, Shape<PARTS, RT, NT>::kRing, s>>>(p);
    return cudaGetLastError();
}

// Tokens of a tile by what a group has on average; two fragments of rows (x read once for both,
// and half the epilogues) unless items of one fit on the SMs at once.  6144 x 6144: 16 tokens 13.5 us
// in a tile of 16, 17.1 in two of 8; 512 tokens 203 and 355 (207 in tiles of 32, whose registers do
// not last).  One fragment and two, rows of k = 6144: 2048 4.6 us and 5.9, 6144 8.6 and 9.2, 8192 10.3
// and 9.2, 12288 14.6 and 12.2; 8 experts of 2048 with a row each 17.5 and 16.4, 30 of them 56 and 46.
template <int BLOCK, int PARTS>
cudaError_t by_shape(const Int4Params& p, int sms, cudaStream_t s) {
    const long long groups = p.groups < p.tokens ? p.groups : p.tokens;
    if (p.tokens / groups > 8) return run<BLOCK, PARTS, 2, 2>(p, sms, s);
    if (groups * ((p.n + 15) / 16) > resident<PARTS, 1>(sms)) return run<BLOCK, PARTS, 2, 1>(p, sms, s);
    return run<BLOCK, PARTS, 1, 1>(p, sms, s);
}

template <int BLOCK>
cudaError_t by_type(const Int4Params& p, int sms, cudaStream_t s) {
    return p.x_bf16 ? by_shape<BLOCK, 1>(p, sms, s) : by_shape<BLOCK, 3>(p, sms, s);
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
        case 32: return by_type<32>(p, sms, s);
        case 64: return by_type<64>(p, sms, s);
        default: return by_type<128>(p, sms, s);
    }
}

}  // namespace muon
