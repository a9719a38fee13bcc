// Products of E4M3 matrices with one power-of-two scale for each block of 128
// along the reduction, on pairs of SMs (tcgen05 cta_group::2, block scaling in
// the tensor core).
//
//   forward       y[t, n]    = sum_k  x[t, k]  W_g[n, k]     tokens t of group g
//   grad input    dx[t, k]   = sum_n dy[t, n]  W_g[n, k]
//   grad weight   dW_g[n, k] = sum_t dy[t, n]   x[t, k]      t over group g
//
// The experts' products of the pages' model (384 experts, 96 whole ones on a
// rank; 8-bit products for expert matrices are the open question of "Domyn is
// training a 1T-parameter MoE on Europe's Jupiter supercomputer, and published
// the recipe", section "What moved the number").
//
// Scales are powers of two (E8M0), the form that tcgen05.mma takes itself: the
// accumulators stay in TMEM over the whole reduction and no register ever
// rescales them.  One scale covers 128 elements, four K = 32 instructions; the
// scale words hold four reduction blocks' bytes, so one 32 x 16-byte copy per
// 128 rows feeds sixteen instructions, each naming its byte.
//
// Layout of a tile: forward and grad input put tokens on the MMA's columns, and
// the weight's other dimension on its 256 rows (128 per CTA).  So a group's tile
// is as wide as the group needs (a multiple of 32 up to 256): an expert with 40
// tokens costs a 64-column tile and not 256 rows.  The weight gradient has n on
// the rows and k on the columns.
//
// Codes keep one layout: the weight is read along either dimension (K-major or
// MN-major operand descriptors), so nothing is transposed.
//
// Per CTA: warp 0 TMA producer (stages of 32 KB), warp 1 MMA issuer (leader
// only), warps 2-3 scale words, warps 4-11 epilogue.  Two accumulators of 256
// columns and the scales do not fit in 512 TMEM columns: the second accumulator
// starts at column 224, and the 32 columns that both own are drained first, so
// the next tile's products wait for an eighth of the epilogue.  Every wait is
// bounded.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "groups.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace muon {

// Device-side status word of this kernel: 0, or MUON_ERR_TIMEOUT (5).
__device__ int g_muon_fp8_error = 0;

namespace {

constexpr int kThreads = 384;
constexpr int kTile = 256;
constexpr int kHalf = 128;
constexpr int kMaxStages = 6;
constexpr int kScaleStages = 4;
constexpr uint32_t kStageA = kHalf * kFp8Block;        // 16 KB
constexpr uint32_t kStageB = kHalf * kFp8Block;       // 16 KB
constexpr uint32_t kBoxRows = 32;                       // B operand, K-major: rows per TMA box
constexpr uint32_t kScaleBytes = 3 * 512;               // A 128 rows, B 2 x 128 columns
constexpr uint32_t kAcc1 = 224;                         // second accumulator's first TMEM column
constexpr uint32_t kScaleCol = 480;                     // scale words' first TMEM column
constexpr uint32_t kScaleBuf = 16;                      // columns per scale buffer (4 A + 8 B)
constexpr uint32_t kTmemCols = 512;
constexpr int kPanel = 8;                               // column tiles per panel of the tile order
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr uint64_t kDrainLimitNs = 20000000ull;
constexpr int kErrTimeout = 5;

// Pipeline stages, and bytes of the block of results that an epilogue warp has on
// its way out (32 rows of 64 bytes; of 128 bytes for the weight gradient, whose
// reductions are short).  What a second block per warp would take is better spent
// on the sixth stage: 32768 tokens of 96 experts, 2048 x 6144, forward 332 -> 322 us,
// input gradient 351 -> 339.  8192 x 6144 x 6144: 178 us (3470 TFLOP/s).
template <int MODE>
struct Ring {
    static constexpr int stages = MODE == kFp8GradWeight ? kMaxStages - 1 : kMaxStages;
    static constexpr uint32_t block = MODE == kFp8GradWeight ? 32 * 128 : 32 * 64;   // one per epilogue warp
    static constexpr size_t bytes = 1024 + stages * (kStageA + kStageB) + 8 * block + kScaleStages * kScaleBytes;
};

struct Barriers {
    uint64_t full[kMaxStages];          // both CTAs' loads -> MMA (the leader's are used)
    uint64_t empty[kMaxStages];         // MMA -> this CTA's producer
    uint64_t sfull[kScaleStages];    // both CTAs' scale words -> MMA (the leader's are used)
    uint64_t sempty[kScaleStages];   // MMA -> this CTA's scale warp
    uint64_t tfull[2];               // MMA -> this CTA's epilogue
    uint64_t tempty[2];              // both epilogues -> MMA: accumulator drained
    uint64_t shared_free[2];         // both epilogues -> MMA: its part of the common columns drained
    uint32_t tmem;
    int abort;
    int tiles;                       // of the launch
};

// Group table: first row, rows, first tile, first padded reduction block.
struct Groups {
    int lo[kFp8MaxGroups];
    int cnt[kFp8MaxGroups];
    int tile0[kFp8MaxGroups + 4];    // groups + 1 used
    int block0[kFp8MaxGroups];
    int width[kFp8MaxGroups];        // columns of the group's tiles
};

// a / d for 0 <= a < 2^31, with inv = 1 / d in fp32: the estimate is off by at
// most one while the quotient stays below 2^22.
__device__ __forceinline__ int quotient(int a, int d, float inv) {
    int q = __float2int_rz(__int2float_rn(a) * inv);
    const int r = a - q * d;
    if (r < 0) --q;
    else if (r >= d) ++q;
    return q;
}

struct Tile {
    int g;
    int m0;          // first MMA row of the pair's tile
    int c0;          // first MMA column
    int cols;        // MMA columns that are in use
    int width;       // MMA columns: cols rounded up
    int kb0, nkb;    // reduction blocks
};

// n columns in equal tiles of at most 256 (2^shift: 256, 128 or 64), in multiples of
// `unit`: 32, or the 64 columns of the weight gradient's result blocks.
__device__ __forceinline__ int column_tiles(int n, int shift) { return (n + (1 << shift) - 1) >> shift; }

__device__ __forceinline__ void split_columns(int n, int shift, int unit, int& tiles, int& width) {
    tiles = column_tiles(n, shift);
    width = tiles > 0 ? ((n + tiles - 1) / tiles + unit - 1) / unit * unit : unit;
}

// Tile t of the launch; `g` only moves forward.  Integer divisions are avoided:
// four of them took 900 cycles of every tile in every role.
template <int SK>
__device__ __forceinline__ Tile decode_tile(const Fp8GemmParams& p, const Groups& gs, int t, int& g, int pp) {
    while (t >= gs.tile0[g + 1]) ++g;
    const int mt = (p.m_ext + kTile - 1) / kTile;
    const bool gw = p.mode == kFp8GradWeight;
    const int n = gw ? p.n_ext : gs.cnt[g];
    const int nt = column_tiles(n, p.col_shift), width = gs.width[g];
    int l = t - gs.tile0[g];
    const int full = nt / kPanel * kPanel;
    int m, c;
    if (l < full * mt) {
        const int per = kPanel * mt;
        const int panel = quotient(l, per, __frcp_rn(__int2float_rn(per))), r = l - panel * per;
        m = r / kPanel;
        c = panel * kPanel + r % kPanel;
    } else {
        l -= full * mt;
        const int w = nt - full;
        m = quotient(l, w, __frcp_rn(__int2float_rn(w)));
        c = full + l - m * w;
    }
    Tile x;
    x.g = g;
    x.m0 = m * kTile;
    const int off = c * width;
    // A tile has a column, so neither bound takes effect; without them the compiler's
    // schedule costs the experts' forward 4 % (443 against 427 us).
    x.cols = max(0, n - off < width ? n - off : width);
    const int unit = gw ? 64 : 32;
    x.width = max(unit, (x.cols + unit - 1) / unit * unit);
    x.c0 = gw ? off : gs.lo[g] + off;
    x.kb0 = gw ? gs.block0[g] : 0;
    x.nkb = gw ? (gs.cnt[g] + kFp8Block - 1) / kFp8Block : p.kblocks;
    if (SK > 1) {                    // this pair's slice, in whole groups of four blocks
        const int quads = (x.nkb + 3) / 4, last = min(x.nkb, quads * (pp + 1) / SK * 4);
        x.kb0 = quads * pp / SK * 4;
        x.nkb = last - x.kb0;
    }
    return x;
}

__device__ __forceinline__ void record_failure(volatile int* abort) {
    atomicCAS(&g_muon_fp8_error, 0, kErrTimeout);
    *abort = 1;
}

// The scale bytes of four reduction blocks of N x 32 indices, this lane's every
// 32nd from idx on, for blocks kb0 .. kb0 + 3 below kb1.  Indices and blocks past
// the end take the last one's bytes: their products are zero or are not stored.
// No load depends on another or on a branch, so all are in flight at once, and
// nothing here looks at a byte: the caller packs them when it needs them.
template <int N>
struct ScaleBytes {
    uint32_t v[N][4];
    __device__ __forceinline__ void load(const Fp8Scale& s, long long base, int idx, int kb0, int kb1, int width) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int kb = min(kb0 + i, kb1 - 1);
            const uint8_t* q = s.p + base + static_cast<long long>(kb) * s.red;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                v[j][i] = 0x7f;
                if (32 * j < width)
                    v[j][i] = q[static_cast<long long>(min(idx + 32 * j, s.limit - 1) >> s.shift) * s.idx];
            }
        }
    }
    __device__ __forceinline__ uint32_t word(int j) const {
        return v[j][0] | (v[j][1] << 8) | (v[j][2] << 16) | (v[j][3] << 24);
    }
};

// The scale words of one group of four reduction blocks on their way to shared
// memory: A's 128 rows, B's 256 columns.
template <int MODE>
struct ScaleGroup {
    ScaleBytes<1> a;                 // 128 x 128 blocks: one scale for the CTA's 128 rows
    ScaleBytes<8> b;
    __device__ __forceinline__ void load(const Fp8GemmParams& p, const Tile& x, int m, int kb, int lane) {
        const int kb1 = x.kb0 + x.nkb;
        a.load(p.s_a, x.g * p.s_a.batch, m, kb, kb1, 32);
        b.load(p.s_b, 0, x.c0 + lane, kb, kb1, x.width);
    }
    __device__ __forceinline__ void store(uint8_t* dst, int lane) const {
        const uint32_t w = a.word(0);
        uint4* d = reinterpret_cast<uint4*>(dst + lane * 16);
        d[0] = make_uint4(w, w, w, w);
        d[32] = make_uint4(b.word(0), b.word(1), b.word(2), b.word(3));
        d[64] = make_uint4(b.word(4), b.word(5), b.word(6), b.word(7));
    }
};

// Weight gradient: both operands' bytes lie along the index, four to a load, and
// become words by a 4 x 4 transpose (48 byte loads a group kept a warp busy for
// longer than the group's products).
template <>
struct ScaleGroup<kFp8GradWeight> {
    uint32_t v[3][4];                // A's rows, B's columns 0-127, 128-255; this lane's four of block kb + i
    __device__ __forceinline__ void load(const Fp8GemmParams& p, const Tile& x, int m, int kb, int lane) {
        const int kb1 = x.kb0 + x.nkb;
        // rows and columns past the end: the last whole word (s_a, s_b hold multiples of 128)
        const int ia = min(m + 4 * lane, p.s_a.limit - 4);
        const int ib0 = min(x.c0 + 4 * lane, p.s_b.limit - 4), ib1 = min(x.c0 + 128 + 4 * lane, p.s_b.limit - 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const long long r = min(kb + i, kb1 - 1);
            const uint8_t* qa = p.s_a.p + r * p.s_a.red;
            const uint8_t* qb = p.s_b.p + r * p.s_b.red;
            v[0][i] = *reinterpret_cast<const uint32_t*>(qa + ia);
            v[1][i] = *reinterpret_cast<const uint32_t*>(qb + ib0);
            v[2][i] = *reinterpret_cast<const uint32_t*>(qb + ib1);
        }
    }
    __device__ __forceinline__ void store(uint8_t* dst, int lane) const {
#pragma unroll
        for (int o = 0; o < 3; ++o) {
            const uint32_t lo0 = __byte_perm(v[o][0], v[o][1], 0x5140), hi0 = __byte_perm(v[o][0], v[o][1], 0x7362);
            const uint32_t lo1 = __byte_perm(v[o][2], v[o][3], 0x5140), hi1 = __byte_perm(v[o][2], v[o][3], 0x7362);
            const uint32_t w[4] = {__byte_perm(lo0, lo1, 0x5410), __byte_perm(lo0, lo1, 0x7632),
                                   __byte_perm(hi0, hi1, 0x5410), __byte_perm(hi0, hi1, 0x7632)};
            // index 4 lane + i: word (4 lane + i) / 32 of 16-byte row (4 lane + i) % 32
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<uint32_t*>(dst + 512 * o + ((4 * lane + i) & 31) * 16 + (lane >> 3) * 4) = w[i];
        }
    }
};

// SK: pairs of a cluster that share one tile's reduction, each a slice of it (one tile
// per cluster); 1: a cluster is one pair.
template <int MODE, bool F32, int SK>
__global__ void __launch_bounds__(kThreads, 1) k_fp8_gemm(const __grid_constant__ Fp8GemmParams p) {
    constexpr int kStages = Ring<MODE>::stages;
    constexpr uint32_t kEpiBytes = Ring<MODE>::block;
    constexpr bool kAMn = MODE != kFp8Forward;          // A operand MN-major
    constexpr bool kBMn = MODE == kFp8GradWeight;      // B operand MN-major
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint8_t* sm_a = smem;
    uint8_t* sm_b = sm_a + kStages * kStageA;
    uint8_t* s_epi = sm_b + kStages * kStageB;
    uint8_t* s_sc = s_epi + 8 * kEpiBytes;
    Barriers& b = *reinterpret_cast<Barriers*>(s_sc + kScaleStages * kScaleBytes);
    Groups& gs = *reinterpret_cast<Groups*>(s_sc + kScaleStages * kScaleBytes + 512);
    volatile int* abort = &b.abort;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t crank = ptx::cluster_ctarank();
    const uint32_t rank = crank & 1u, lead = crank & ~1u;   // in the pair; cluster rank of the pair's leader
    const int pp = static_cast<int>(crank >> 1);            // pair in the cluster
    const bool leader = rank == 0;
    const int pair = static_cast<int>(ptx::cluster_id_x());     // the tiles are dealt to clusters
    const int npairs = static_cast<int>(ptx::num_clusters_x());
    const uint64_t limit = p.wait_ns != 0 ? p.wait_ns : kWaitLimitNs;

    if (threadIdx.x == 32) {
        for (int s = 0; s < kStages; ++s) {
            ptx::mbar_init(ptx::smem_addr(&b.full[s]), 1);
            ptx::mbar_init(ptx::smem_addr(&b.empty[s]), 1);
        }
        for (int s = 0; s < kScaleStages; ++s) {
            ptx::mbar_init(ptx::smem_addr(&b.sfull[s]), 2);
            ptx::mbar_init(ptx::smem_addr(&b.sempty[s]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            ptx::mbar_init(ptx::smem_addr(&b.tfull[a]), 1);
            ptx::mbar_init(ptx::smem_addr(&b.tempty[a]), 16);       // 8 epilogue warps of both CTAs
            ptx::mbar_init(ptx::smem_addr(&b.shared_free[a]), 8);   // 4 of them
        }
        b.abort = 0;
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&p.tm_a);
        ptx::prefetch_tmap(&p.tm_b);
        if (!kBMn) ptx::prefetch_tmap(&p.tm_part);
        if (MODE != kFp8GradWeight && p.vec) ptx::prefetch_tmap(&p.tm_res);
    }
    if (warp == 0) {
        const int mt = (p.m_ext + kTile - 1) / kTile;
        int low = 0, tiles = 0, blocks = 0;
        const int rows = MODE == kFp8GradWeight ? p.rows : p.n_ext;
        for (int g0 = 0; g0 < p.groups; g0 += 32) {
            const GroupSpan sp = warp_group_spans(p.offsets, p.groups, rows, g0, low);
            const int g = g0 + lane;
            int nt, width;
            split_columns(MODE == kFp8GradWeight ? p.n_ext : sp.cnt, p.col_shift, MODE == kFp8GradWeight ? 64 : 32, nt, width);
            const int n = g < p.groups ? nt * mt : 0;
            const int nb = (sp.cnt + kFp8Block - 1) / kFp8Block;
            const int it = warp_inclusive_sum(n), ib = warp_inclusive_sum(nb);
            if (g < p.groups) {
                gs.lo[g] = sp.lo;
                gs.cnt[g] = sp.cnt;
                gs.tile0[g] = tiles + it - n;
                gs.block0[g] = blocks + ib - nb;
                gs.width[g] = width;
            }
            tiles += __shfl_sync(0xffffffffu, it, 31);
            blocks += __shfl_sync(0xffffffffu, ib, 31);
        }
        if (lane == 0) {
            gs.tile0[p.groups] = tiles;
            b.tiles = tiles;
        }
    }
    if (warp == 1) {
        ptx::tmem_alloc_pair(ptx::smem_addr(&b.tmem), kTmemCols);
        ptx::tmem_relinquish_pair();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::cluster_sync();   // barriers of both CTAs initialised, TMEM allocated, group table written
    ptx::tc_fence_after();
    const uint32_t tmem = b.tmem;
    const int tiles = b.tiles;
    // Everything so far may run while the launch before drains.  It wrote the codes, and
    // they are read from here on; or (kSyncLate) it is the layer's other product, which
    // itself began after the codes were complete and let this launch start only then:
    // both run side by side, and this one ends after the other.
    if (p.sync != kSyncLate) asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");

    if (warp == 0) {
        // ------------------------------------------------------ producer --
        {
            int stage = 0, g = 0;
            uint32_t phase = 0, armed = 0, armed_parity = 0;
            bool ok = true;
            for (int t = pair; ok && t < tiles; t += npairs) {
                const Tile x = decode_tile<SK>(p, gs, t, g, pp);
                const int m = x.m0 + static_cast<int>(rank) * kHalf;
                const int half = x.width / 2;
                const int c = x.c0 + static_cast<int>(rank) * half;
                const int boxes = kBMn ? 4 : (half + static_cast<int>(kBoxRows) - 1) / static_cast<int>(kBoxRows);
                const bool whole = boxes == kHalf / static_cast<int>(kBoxRows);
                const uint32_t bytes = 2 * (kStageA + boxes * kBoxRows * kFp8Block);
                const int gb = MODE == kFp8GradWeight ? 0 : x.g;
                for (int kb = x.kb0; kb < x.kb0 + x.nkb; ++kb) {
                    if (!ptx::wait_parity_cluster(ptx::smem_addr(&b.empty[stage]), phase ^ 1u, abort, limit)) {
                        record_failure(abort);
                        ok = false;
                        break;
                    }
                    const uint32_t local = ptx::smem_addr(&b.full[stage]);
                    const uint32_t fb = ptx::mapa_shared(local, lead);
                    if (leader) {
                        armed |= 1u << stage;
                        armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
                    }
                    if (ptx::elect_one()) {
                        if (leader) ptx::mbar_arrive_expect_tx(local, bytes);
                        const uint32_t di = ptx::smem_addr(sm_a + stage * kStageA);
                        const uint32_t d_o = ptx::smem_addr(sm_b + stage * kStageB);
                        if (kAMn) {
                            ptx::tma_load_3d_pair(di, &p.tm_a, fb, m, kb * kFp8Block, gb);
                        } else {
                            ptx::tma_load_3d_pair(di, &p.tm_a, fb, kb * kFp8Block, m, gb);
                        }
                        if (kBMn) {
                            ptx::tma_load_3d_pair(d_o, &p.tm_b, fb, c & ~15, kb * kFp8Block, 0);
                        } else if (whole) {
                            ptx::tma_load_3d_pair(d_o, &p.tm_b, fb, kb * kFp8Block, c, 0);
                        } else {
                            for (int i = 0; i < boxes; ++i)
                                ptx::tma_load_3d_pair(d_o + i * kBoxRows * kFp8Block, &p.tm_part, fb, kb * kFp8Block,
                                                      c + i * static_cast<int>(kBoxRows), 0);
                        }
                    }
                    __syncwarp();
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (leader && (!ok || *abort)) {
                // loads in flight land before the CTAs leave
                for (int s = 0; s < kStages; ++s)
                    if ((armed >> s) & 1u)
                        ptx::wait_parity_cluster(ptx::smem_addr(&b.full[s]), (armed_parity >> s) & 1u, nullptr,
                                                 kDrainLimitNs);
            }
        }
    } else if (warp == 1) {
        // ----------------------------------------------------------- MMA --
        // The whole warp runs the loop and one elected lane issues: descriptors stay
        // warp-uniform, which a loop under `lane == 0` would not let the compiler see.
        if (leader) {
            const uint64_t ad0 = ptx::sdesc_sw128(ptx::smem_addr(sm_a), 16, 1024);
            const uint64_t bd0 = ptx::sdesc_sw128(ptx::smem_addr(sm_b), 16, 1024);
            // next 32 elements of K: 32 bytes of a row (K-major) or 32 rows of 128 bytes (MN-major)
            constexpr uint64_t a_k = (kAMn ? 4096 : 32) >> 4;
            constexpr uint64_t b_k = (kBMn ? 4096 : 32) >> 4;
            const uint16_t mine = static_cast<uint16_t>(0x3u << lead);
            int stage = 0, sstage = 0, it = 0, g = 0;
            uint32_t phase = 0, sphase = 0;
            bool ok = true;
            for (int t = pair; ok && t < tiles; t += npairs, ++it) {
                const Tile x = decode_tile<SK>(p, gs, t, g, pp);
                const int acc = it & 1;
                const uint32_t use = static_cast<uint32_t>(it >> 1) & 1u;
                // The copy of four blocks' scale words is issued a block before the first
                // of them, into the other of two buffers: the copies run in order with the
                // products, and one that its products wait for leaves the tensor core idle
                // for a copy's latency (155 cycles of 2048, measured).
                auto copy_scales = [&](int i) -> bool {
                    if (!ptx::wait_parity_cluster(ptx::smem_addr(&b.sfull[sstage]), sphase, abort, limit)) return false;
                    ptx::tc_fence_after();
                    const uint32_t src = ptx::smem_addr(s_sc + sstage * kScaleBytes);
                    const uint32_t dst = tmem + kScaleCol + static_cast<uint32_t>((i >> 2) & 1) * kScaleBuf;
                    if (ptx::elect_one()) {
                        ptx::tmem_copy_scales_pair(dst, ptx::sdesc_rows16(src));
                        ptx::tmem_copy_scales_pair(dst + 4, ptx::sdesc_rows16(src + 512));
                        if (x.width > 128) ptx::tmem_copy_scales_pair(dst + 8, ptx::sdesc_rows16(src + 1024));
                        ptx::mma_commit_pair(ptx::smem_addr(&b.sempty[sstage]), mine);
                    }
                    __syncwarp();
                    if (++sstage == kScaleStages) {
                        sstage = 0;
                        sphase ^= 1u;
                    }
                    return true;
                };
                if ((x.nkb > 0 && !copy_scales(0)) ||
                    !ptx::wait_parity_cluster(ptx::smem_addr(&b.tempty[acc]), use ^ 1u, abort, limit) ||
                    (it > 0 && !ptx::wait_parity_cluster(ptx::smem_addr(&b.shared_free[acc ^ 1]),
                                                         static_cast<uint32_t>((it - 1) >> 1) & 1u, abort, limit))) {
                    record_failure(abort);
                    break;
                }
                ptx::tc_fence_after();
                const uint32_t d = tmem + (acc ? kAcc1 : 0u);
                const uint32_t idesc0 = ptx::idesc_mxf8(kTile, x.width, kAMn, kBMn, 0);
                const int kb1 = x.kb0 + x.nkb;
                for (int kb = x.kb0; kb < kb1; ++kb) {
                    const int i = kb - x.kb0;
                    if ((i & 3) == 3 && kb + 1 < kb1 && !copy_scales(i + 1)) {
                        record_failure(abort);
                        ok = false;
                        break;
                    }
                    if (!ptx::wait_parity_cluster(ptx::smem_addr(&b.full[stage]), phase, abort, limit)) {
                        record_failure(abort);
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after();
                    const uint64_t ad = ad0 + static_cast<uint64_t>(stage) * (kStageA >> 4);
                    const uint64_t bd = bd0 + static_cast<uint64_t>(stage) * (kStageB >> 4);
                    const uint32_t sf = static_cast<uint32_t>(i & 3);
                    const uint32_t idesc = idesc0 | (sf << 4) | (sf << 29);
                    const uint32_t sfa = tmem + kScaleCol + static_cast<uint32_t>((i >> 2) & 1) * kScaleBuf;
                    if (ptx::elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            ptx::mma_mxf8_pair(d, ad + kk * a_k, bd + kk * b_k, idesc, sfa, sfa + 4,
                                               (kk != 0 || kb != x.kb0) ? 1u : 0u);
                        ptx::mma_commit_pair(ptx::smem_addr(&b.empty[stage]), mine);
                    }
                    __syncwarp();
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
                if (ptx::elect_one()) ptx::mma_commit_pair(ptx::smem_addr(&b.tfull[acc]), mine);
                __syncwarp();
            }
        }
    } else if (warp < 4) {
        // --------------------------------------------------------- scales --
        // Warps 2 and 3 take turns by groups of four reduction blocks; each loads
        // its next group's bytes before it stores the current one's, so that four
        // groups are on their way: one load latency per group, waited for group by
        // group, is longer than the products of a group of a narrow tile.
        ScaleGroup<MODE> v[2];
        int seq = 0, waiting = -1, g = 0;
        bool ok = true;
        auto store = [&](const ScaleGroup<MODE>& w, int n) -> bool {
            const int st = n % kScaleStages;
            const uint32_t use = static_cast<uint32_t>(n / kScaleStages) & 1u;
            if (!ptx::wait_parity_cluster(ptx::smem_addr(&b.sempty[st]), use ^ 1u, abort, limit)) {
                record_failure(abort);
                return false;
            }
            w.store(s_sc + st * kScaleBytes, lane);
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive_cluster(ptx::mapa_shared(ptx::smem_addr(&b.sfull[st]), lead));
            return true;
        };
        for (int t = pair; ok && t < tiles; t += npairs) {
            const Tile x = decode_tile<SK>(p, gs, t, g, pp);
            const int m = x.m0 + static_cast<int>(rank) * kHalf;
            for (int i = 0; ok && i < x.nkb; i += 4, ++seq) {
                if ((seq & 1) != warp - 2) continue;
                if ((seq >> 1) & 1) {                    // which of the two register sets
                    v[1].load(p, x, m, x.kb0 + i, lane);
                    if (waiting >= 0) ok = store(v[0], waiting);
                } else {
                    v[0].load(p, x, m, x.kb0 + i, lane);
                    if (waiting >= 0) ok = store(v[1], waiting);
                }
                waiting = seq;
            }
        }
        if (ok && waiting >= 0) {
            if ((waiting >> 1) & 1) store(v[1], waiting);
            else store(v[0], waiting);
        }
    } else if (warp >= 4) {
        // ------------------------------------------------------ epilogue --
        //   weight gradient: a lane holds consecutive results of one row; blocks of 32
        //   rows of 128 bytes go through shared memory and leave in whole lines.  These
        //   tiles are nearly all epilogue, and their stores are the warps' own: TMA
        //   stores wait behind the loads that the producer has asked for ahead (2500
        //   cycles; in 128-byte blocks they brought the weights of 96 experts to 784 us, the
        //   rest of the tile as it is now to 532);
        //   else: lanes run along the row; where rows start on 16 bytes, 8 x 8 blocks of
        //   bf16 go through shared memory transposed and leave by TMA, 32 rows of 64
        //   bytes at a time.
        const int q = warp & 3;
        const int half = (warp - 4) >> 2;                // even or odd 32-column chunks
        uint8_t* const stage = s_epi + (warp - 4) * kEpiBytes;
        int it = 0, g = 0;
        bool met = false;                                // SK > 1: the pairs have exchanged their sums
        for (int t = pair; t < tiles; t += npairs, ++it) {
            const Tile x = decode_tile<SK>(p, gs, t, g, pp);
            const int acc = it & 1;
            const uint32_t use = static_cast<uint32_t>(it >> 1) & 1u;
            const int m0 = x.m0 + static_cast<int>(rank) * kHalf + q * 32;
            const int batch = MODE == kFp8GradWeight ? x.g : 0;
            const int chunks = x.width / 32;
            const uint32_t src = tmem + (acc ? kAcc1 : 0u) + (static_cast<uint32_t>(q * 32) << 16);
            // the accumulators' common columns (of the first its last 32, second half; of the
            // second its first 32, first half) are read first
            const bool owner = (acc == 0) == (half == 1);
            auto release_shared = [&] {
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive_cluster_relaxed(ptx::mapa_shared(ptx::smem_addr(&b.shared_free[acc]), lead));
            };
            auto release = [&] {
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive_cluster_relaxed(ptx::mapa_shared(ptx::smem_addr(&b.tempty[acc]), lead));
            };
            // no sleep between polls: the next tile's products wait for the first chunk
            if (!ptx::wait_parity_cluster(ptx::smem_addr(&b.tfull[acc]), use, abort, limit)) {
                record_failure(abort);
                break;
            }
            ptx::tc_fence_after();
            // SK > 1: each pair finishes some 32-column chunks.  The others leave their sums of
            // those in their own shared memory (the ring is idle: the tile's products have read
            // it), and after all have met it adds them to its own in the order of the slices.
            auto leave = [&](int ch, const uint32_t (&r)[32]) {
                uint4* o = reinterpret_cast<uint4*>(smem) + (ch * 4 + q) * 256 + lane;
#pragma unroll
                for (int v = 0; v < 8; ++v) o[v * 32] = make_uint4(r[4 * v], r[4 * v + 1], r[4 * v + 2], r[4 * v + 3]);
            };
            auto meet = [&] {
                __syncwarp();
                ptx::cluster_sync();
                met = true;
            };
            auto join = [&](int ch, uint32_t (&r)[32]) {
                const uint32_t at = ptx::smem_addr(smem) + ((ch * 4 + q) * 256 + lane) * 16;
                float sum[32];
#pragma unroll
                for (int s = 0; s < SK; ++s) {
                    const uint32_t from = ptx::mapa_shared(at, static_cast<uint32_t>(2 * s) + rank);
#pragma unroll
                    for (int v = 0; v < 8; ++v) {
                        uint4 w = make_uint4(r[4 * v], r[4 * v + 1], r[4 * v + 2], r[4 * v + 3]);
                        if (s != pp) w = ptx::ld_cluster_v4(from + v * 512);
                        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            sum[4 * v + e] = s == 0 ? __uint_as_float(u[e]) : sum[4 * v + e] + __uint_as_float(u[e]);
                    }
                }
#pragma unroll
                for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(sum[j]);
            };
            if constexpr (MODE == kFp8GradWeight) {
                // groups of 64 columns: 0, 2 and 1, 3; the second half of the first accumulator from its end
                uint32_t r[2][32];
                if constexpr (SK > 1) {                  // group half + 2 i is pair i's to finish
#pragma unroll 1
                    for (int i = 0; i < 2; ++i) {
                        if (i == pp) continue;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int ch = 2 * half + 4 * i + h;
                            if (ch >= chunks) continue;
                            ptx::tmem_ld_32x32b_x32(src + static_cast<uint32_t>(32 * ch), r[h]);
                            ptx::tmem_wait_ld();
                            leave(ch, r[h]);
                        }
                    }
                    meet();
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (SK > 1 && i != pp) continue;
                    const int pr = SK == 1 && acc == 0 && half == 1 ? 3 - 2 * i : half + 2 * i;
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (2 * pr + h < chunks) ptx::tmem_ld_32x32b_x32(src + static_cast<uint32_t>(64 * pr + 32 * h), r[h]);
                    ptx::tmem_wait_ld();
                    if constexpr (SK > 1) {
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            if (2 * pr + h < chunks) join(2 * pr + h, r[h]);
                    } else {
                        if (i == 0 && owner) release_shared();
                        if (i == 1) release();
                    }
                    if (x.nkb == 0) {
#pragma unroll
                        for (int j = 0; j < 64; ++j) r[j >> 5][j & 31] = 0u;
                    }
                    if (2 * pr >= chunks) continue;
#pragma unroll
                    for (int h = 0; h < (F32 ? 2 : 1); ++h) {
                        uint8_t* const row = stage + lane * 128;
                        __syncwarp();                    // the last block has been read
#pragma unroll
                        for (int u = 0; u < 8; ++u) {
                            uint4 v;
                            if (F32) {
                                v = make_uint4(r[h][4 * u], r[h][4 * u + 1], r[h][4 * u + 2], r[h][4 * u + 3]);
                            } else {
                                uint32_t w[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const int j = 8 * u + 2 * e;
                                    const __nv_bfloat162 f = __floats2bfloat162_rn(__uint_as_float(r[j >> 5][j & 31]),
                                                                                   __uint_as_float(r[j >> 5][(j & 31) + 1]));
                                    w[e] = *reinterpret_cast<const uint32_t*>(&f);
                                }
                                v = make_uint4(w[0], w[1], w[2], w[3]);
                            }
                            *reinterpret_cast<uint4*>(row + ((u ^ (lane & 7)) << 4)) = v;
                        }
                        __syncwarp();
                        constexpr int kPer = F32 ? 4 : 8, kSize = F32 ? 4 : 2;   // elements per 16 bytes
                        const int col0 = x.c0 + 64 * pr + 32 * h;
                        char* const out0 = static_cast<char*>(p.out) +
                                           (batch * p.out_batch + static_cast<long long>(m0) * p.ld + col0) * kSize;
                        if (p.vec) {
                            const int col = col0 + kPer * (lane & 7);
                            char* o = out0 + ((lane >> 3) * p.ld + kPer * (lane & 7)) * kSize;
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                const int rr = 4 * k + (lane >> 3);
                                const uint4 v = *reinterpret_cast<const uint4*>(
                                    stage + rr * 128 + (((lane & 7) ^ (rr & 7)) << 4));
                                if (m0 + rr < p.m_ext) {
                                    if (col + kPer <= p.n_ext) {
                                        *reinterpret_cast<uint4*>(o) = v;
                                    } else {
                                        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                                        for (int e = 0; e < kPer; ++e) {
                                            if (col + e >= p.n_ext) continue;
                                            if (F32) reinterpret_cast<uint32_t*>(o)[e] = w[e];
                                            else reinterpret_cast<uint16_t*>(o)[e] =
                                                static_cast<uint16_t>(w[e >> 1] >> (16 * (e & 1)));
                                        }
                                    }
                                }
                                o += 4 * p.ld * kSize;
                            }
                        } else {
                            // rows that start anywhere: one row per instruction, four bytes a lane where they are aligned
                            const int rows = min(32, p.m_ext - m0);
                            const int col = col0 + (F32 ? lane : 2 * lane);
                            for (int rr = 0; rr < rows; ++rr) {
                                const uint32_t v = *reinterpret_cast<const uint32_t*>(
                                    stage + rr * 128 + (((lane >> 2) ^ (rr & 7)) << 4) + (lane & 3) * 4);
                                char* o = out0 + rr * p.ld * kSize + 4 * lane;
                                if (F32) {
                                    if (col < p.n_ext) *reinterpret_cast<uint32_t*>(o) = v;
                                } else if ((reinterpret_cast<uintptr_t>(o) & 3u) == 0 && col + 1 < p.n_ext) {
                                    *reinterpret_cast<uint32_t*>(o) = v;
                                } else {
                                    if (col < p.n_ext) *reinterpret_cast<uint16_t*>(o) = static_cast<uint16_t>(v);
                                    if (col + 1 < p.n_ext) reinterpret_cast<uint16_t*>(o)[1] = static_cast<uint16_t>(v >> 16);
                                }
                            }
                        }
                    }
                }
                continue;
            }
            auto chunk = [&](int i) { return acc == 0 && half == 1 ? 7 - 2 * i : half + 2 * i; };
            auto read = [&](int ch, uint32_t (&r)[2][16]) {
                if (ch >= chunks) return;
                if (!F32 && p.vec) {
                    ptx::tmem_ld_16x256b_x4(src + static_cast<uint32_t>(ch * 32), r[0]);
                    ptx::tmem_ld_16x256b_x4(src + static_cast<uint32_t>(ch * 32) + (16u << 16), r[1]);
                } else {
                    ptx::tmem_ld_32x32b_x32(src + static_cast<uint32_t>(ch * 32), reinterpret_cast<uint32_t(&)[32]>(r));
                }
            };
            auto write = [&](int ch, uint32_t (&r)[2][16]) {
                if (ch >= chunks) return;
                const int left = x.cols - ch * 32;
                const int c = x.c0 + ch * 32;
                if (!F32 && p.vec) {
                    const uint32_t buf_addr = ptx::smem_addr(stage);
                    if (lane == 0) ptx::bulk_wait_group_read<0>();   // its last store has read it
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t w[4];
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            const __nv_bfloat162 v =
                                __floats2bfloat162_rn(__uint_as_float(r[h >> 1][4 * j + 2 * (h & 1)]),
                                                      __uint_as_float(r[h >> 1][4 * j + 2 * (h & 1) + 1]));
                            w[h] = *reinterpret_cast<const uint32_t*>(&v);
                        }
                        const int row = 8 * j + (lane & 7);
                        ptx::stmatrix_x4_trans(buf_addr + row * 64 + (((lane >> 3) ^ ((row >> 1) & 3)) << 4), w[0], w[1],
                                               w[2], w[3]);
                    }
                    // a TMA store ends rows on 16 bytes: the last odd columns are the warp's own to write
                    if (left >= 32 && (m0 + 32 <= p.m_ext || p.m_ext % 8 == 0)) {
                        ptx::fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            if (m0 < p.m_ext) ptx::tma_store_3d(&p.tm_res, buf_addr, m0, c, 0);
                            ptx::bulk_commit_group();
                        }
                    } else {
                        // or a group's last rows: the next group's lie behind them
                        __syncwarp();
                        const int mm = m0 + 8 * (lane & 3);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int row = 8 * i + (lane >> 2);
                            const uint4 v =
                                *reinterpret_cast<const uint4*>(stage + row * 64 + (((lane & 3) ^ ((row >> 1) & 3)) << 4));
                            if (row < left) {
                                __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + static_cast<long long>(c + row) * p.ld + mm;
                                if (mm + 8 <= p.m_ext) {
                                    *reinterpret_cast<uint4*>(o) = v;
                                } else {
                                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                                    for (int e = 0; e < 8; ++e)
                                        if (mm + e < p.m_ext)
                                            o[e] = __ushort_as_bfloat16(static_cast<unsigned short>(w[e >> 1] >> (16 * (e & 1))));
                                }
                            }
                        }
                    }
                } else if (m0 + lane < p.m_ext) {
                    const long long at = static_cast<long long>(c) * p.ld + m0 + lane;
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const float v = __uint_as_float(r[j >> 4][j & 15]);
                        if (j < left) {
                            if (F32) static_cast<float*>(p.out)[at + j * p.ld] = v;
                            else static_cast<__nv_bfloat16*>(p.out)[at + j * p.ld] = __float2bfloat16_rn(v);
                        }
                    }
                }
            };
            if constexpr (SK > 1) {
                // chunk 2 i + half is pair i % SK's to finish
                uint32_t r[2][16];
#pragma unroll 1
                for (int i = 0; half + 2 * i < chunks; ++i) {
                    if (i % SK == pp) continue;
                    read(half + 2 * i, r);
                    ptx::tmem_wait_ld();
                    leave(half + 2 * i, reinterpret_cast<uint32_t(&)[32]>(r));
                }
                meet();
#pragma unroll 1
                for (int i = pp; half + 2 * i < chunks; i += SK) {
                    read(half + 2 * i, r);
                    ptx::tmem_wait_ld();
                    join(half + 2 * i, reinterpret_cast<uint32_t(&)[32]>(r));
                    write(half + 2 * i, r);
                }
                break;
            }
            // each chunk is read while the one before it is written
            uint32_t ra[2][16], rb[2][16];
            read(chunk(0), ra);
            ptx::tmem_wait_ld();
            if (owner) release_shared();
            read(chunk(1), rb);
            write(chunk(0), ra);
            ptx::tmem_wait_ld();
            read(chunk(2), ra);
            write(chunk(1), rb);
            ptx::tmem_wait_ld();
            read(chunk(3), rb);
            write(chunk(2), ra);
            ptx::tmem_wait_ld();
            release();
            write(chunk(3), rb);
        }
        if (SK > 1 && !met) {                            // after a failure: the other warps wait there
            __syncwarp();
            ptx::cluster_sync();
        }
        if (SK == 1 && MODE != kFp8GradWeight && p.zero_rest) {
            // rows of no group: before the first group's and behind the last one's
            const int head = gs.lo[0], tail = gs.lo[p.groups - 1] + gs.cnt[p.groups - 1];
            const int rest = head + p.n_ext - tail;
            for (int i = static_cast<int>(blockIdx.x) * 8 + warp - 4; i < rest; i += static_cast<int>(gridDim.x) * 8) {
                const long long row = i < head ? i : tail + i - head;
                for (int m = lane; m < p.m_ext; m += 32) {
                    if (F32) static_cast<float*>(p.out)[row * p.ld + m] = 0.0f;
                    else static_cast<__nv_bfloat16*>(p.out)[row * p.ld + m] = __float2bfloat16_rn(0.0f);
                }
            }
        }
        if (lane == 0) ptx::bulk_wait_group_all();       // every block written
        __syncwarp();
    }
    if (SK > 1 && warp < 4) {
        __syncwarp();
        ptx::cluster_sync();                             // the epilogue's exchange
    }

    if (p.sync == kSyncLate) asm volatile("griddepcontrol.wait;" ::: "memory");
    ptx::tc_fence_before();
    __syncthreads();
    ptx::cluster_sync();   // no CTA leaves while its peer may still signal its barriers
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc_pair(tmem, kTmemCols);
    }
}

static_assert(sizeof(Barriers) <= 512, "barrier block");
template <int MODE>
constexpr size_t smem_bytes() {
    return Ring<MODE>::bytes + 512 + sizeof(Groups);
}
static_assert(smem_bytes<kFp8Forward>() <= 232448 && smem_bytes<kFp8GradWeight>() <= 232448, "shared memory");

template <int MODE, bool F32, int SK>
cudaError_t run(const Fp8GemmParams& p, int clusters, cudaStream_t s) {
    const cudaError_t e = cudaFuncSetAttribute(k_fp8_gemm<MODE, F32, SK>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem_bytes<MODE>()));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * SK * clusters);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem_bytes<MODE>();
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2 * SK;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = p.sync != kSyncNone ? 2 : 1;
    const cudaError_t l = cudaLaunchKernelEx(&cfg, k_fp8_gemm<MODE, F32, SK>, p);
    return l != cudaSuccess ? l : cudaGetLastError();
}

template <int MODE, int SK>
cudaError_t run(const Fp8GemmParams& p, int clusters, cudaStream_t s) {
    return p.out_f32 ? run<MODE, true, SK>(p, clusters, s) : run<MODE, false, SK>(p, clusters, s);
}

template <int SK>
cudaError_t run_slices(const Fp8GemmParams& p, int tiles, cudaStream_t s) {
    switch (p.mode) {
        case kFp8Forward: return run<kFp8Forward, SK>(p, tiles, s);
        case kFp8GradInput: return run<kFp8GradInput, SK>(p, tiles, s);
        default: return run<kFp8GradWeight, SK>(p, tiles, s);
    }
}

}  // namespace

cudaError_t launch_fp8_gemm(const Fp8GemmParams& p, int sms, cudaStream_t s) {
    const long long mt = (p.m_ext + kTile - 1) / kTile;
    const long long columns = (p.n_ext + (1 << p.col_shift) - 1) >> p.col_shift;
    const long long nt = p.mode == kFp8GradWeight ? p.groups * columns
                                                  : (p.groups == 1 ? columns : p.n_ext / kTile + p.groups);
    const long long most = mt * nt;
    if (p.slices > 1) {
        const int tiles = static_cast<int>(mt * columns);
        return p.slices == 2 ? run_slices<2>(p, tiles, s)
               : p.slices == 3 ? run_slices<3>(p, tiles, s)
                               : run_slices<4>(p, tiles, s);
    }
    const int pairs = static_cast<int>(most < sms / 2 ? (most > 0 ? most : 1) : sms / 2);
    switch (p.mode) {
        case kFp8Forward: return run<kFp8Forward, 1>(p, pairs, s);
        case kFp8GradInput: return run<kFp8GradInput, 1>(p, pairs, s);
        default: return run<kFp8GradWeight, 1>(p, pairs, s);
    }
}

// Clusters of 4, 6 and 8 CTAs that the current device holds at once (0: none).
void fp8_gemm_clusters(int (&n)[3]) {
    auto ask = [](auto* kernel, int size) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(size);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = smem_bytes<kFp8Forward>();
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = size;
        at[0].val.clusterDim.y = 1;
        at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        int most = 0;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(smem_bytes<kFp8Forward>())) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&most, kernel, &cfg) != cudaSuccess) {
            cudaGetLastError();
            most = 0;
        }
        return most;
    };
    n[0] = ask(k_fp8_gemm<kFp8Forward, false, 2>, 4);
    n[1] = ask(k_fp8_gemm<kFp8Forward, false, 3>, 6);
    n[2] = ask(k_fp8_gemm<kFp8Forward, false, 4>, 8);
}

// How a product of one weight is cut where 256 x 256 tiles leave SMs idle: into narrower
// column tiles, and the reduction into slices, which up to four pairs of a cluster take
// and add up through shared memory.  All of it has to fit at once, or a second wave
// starts.  Forward, by what was measured: a block of 128 of the reduction takes a pair
// 0.2 us in a tile of 64 columns or fewer (its ring waits for the weight) and 0.27 in one
// of 256 (the tensor core's rate), all pairs together load 11 MB in a microsecond (8.4 in
// narrow tiles), a full tile's results take 1.1 us, and a meeting 0.5 to 3.
// One pair and 256 columns -> this, tokens x n x k: 9 x 6144 x 6144 16.4 us -> 12.4 (three
// slices, in two waves, 20.6), 9 x 2048 x 6144 16.5 -> 10.1, 256 x 2048 x 6144 20.3 -> 13.2,
// 1024 x 2048 x 6144 20.7 -> 18.1, 512 x 1024 x 1024 9.5 -> 8.0, 512 x 300 x 500 10.9 -> 7.6.
// Gradients: the layer's other product wants the idle SMs too, and a slice pays from
// sixteen blocks on (2048 tokens of 520 x 1300, backward: 30.3 us, 39.0 with slices of
// eight blocks; 8192 tokens 75.2 -> 65).
void fp8_gemm_cut(Fp8GemmParams& p, int sms, const int (&clusters)[3]) {
    p.col_shift = 8;
    p.slices = 1;
    if (p.offsets != nullptr || p.groups != 1) return;
    auto up = [](long long a, long long b) { return (a + b - 1) / b; };
    const long long mt = up(p.m_ext, kTile), pairs = sms / 2, whole = mt * up(p.n_ext, kTile);
    const long long blocks = p.mode == kFp8GradWeight ? up(p.rows, kFp8Block) : p.kblocks;
    if (p.mode != kFp8Forward) {
        for (int s = 2; s <= 4; ++s)
            if (blocks >= 16 * s && whole <= clusters[s - 2]) p.slices = s;
        return;
    }
    float best = 0.0f;
    for (int shift = 8; shift >= 6; --shift) {
        const long long tiles = mt * up(p.n_ext, 1 << shift);
        const float width = static_cast<float>(up(up(p.n_ext, up(p.n_ext, 1 << shift)), 32) * 32) / 256.0f;
        const float loads = tiles * blocks * (1.0f + width) * 32.768e-3f / (width > 0.5f ? 11.0f : 8.4f);
        for (int s = 1; s <= 4; ++s) {
            if (tiles * s > pairs || (s > 1 && (blocks < 4 * s || tiles > clusters[s - 2]))) continue;
            const float ring = up(up(blocks, 4), s) * 4 * (0.2f + 0.093f * fmaxf(0.0f, width - 0.25f));
            const float t = 6.2f + 1.1f * width + fmaxf(ring, loads) + (s > 1 ? 0.5f + width * (s == 2 ? 1.3f : 2.6f) : 0.0f);
            if (best == 0.0f || t < 0.98f * best) {
                best = t;
                p.col_shift = shift;
                p.slices = s;
            }
        }
    }
}

cudaError_t read_and_clear_fp8_error(int* code) {
    int v = 0;
    const cudaError_t e = cudaMemcpyFromSymbol(&v, g_muon_fp8_error, sizeof(int));
    if (e != cudaSuccess) return e;
    *code = v;
    const int zero = 0;
    return cudaMemcpyToSymbol(g_muon_fp8_error, &zero, sizeof(int));
}

}  // namespace muon
