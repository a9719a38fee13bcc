// Internal structures shared by the host code and the kernels of the Muon
// library.  Nothing here crosses the C ABI.
#pragma once

#include <cmath>
#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime_api.h>

#include <functional>

namespace muon {

// ------------------------------------------------------------ elementwise --
// The momentum / normalisation / packing / update kernels walk 64 x 64 tiles
// of one matrix at a time; a launch covers up to kEwMaxMats matrices whose
// descriptors travel as a kernel parameter (no host->device copy per call).
constexpr int kEwTile = 64;
constexpr int kEwThreads = 256;
constexpr int kEwMaxMats = 224;

enum EwSrc : int { kSrcBf16 = 0, kSrcF32 = 1 };

struct EwMat {
    const void* src;          // G (muon_step) or the input matrix (ns only)
    float* mom;               // fp32 momentum (muon_step) or nullptr
    void* dst;                // W (muon_step) or the input matrix (ns only, output)
    __nv_bfloat16* x;         // oriented, padded bf16 iterate X0 (pack) / O (unpack)
    __nv_bfloat16* oout;      // optional copy of O, rows x cols (unpack, weight update)
    long long part;           // first norm partial of this matrix
    int rows, cols;           // m, n as stored
    int ldx;                  // row length of the oriented, padded iterate
    int xrows_pad;            // rows of the oriented, padded iterate
    int trans;                // 1 when m > n (the iterate holds the transpose)
    int vec;                  // 1 when 8-element vector access is legal for this matrix
    int tile0;                // first tile of this matrix in this launch
    uint8_t* x8;              // pack with the FP8 Gram: E4M3 copy of X0 * 2^8, layout of x (or nullptr)
    float dcy, s;             // weight-update scalars (muon_step)
};

struct EwParams {
    int nmats;
    int total_tiles;
    int src_dtype;            // EwSrc of src
    int dst_dtype;            // EwSrc of dst (W)
    int nesterov;
    int g_count;              // stacked gradients per matrix, summed in fp32 in order
    float mu;
    double eps;               // normalisation epsilon
    double* partials;         // per-tile sums of squares (pass 1 writes, finalize reads)
    float* sigma;             // per-matrix 1/(|U|_F + eps), indexed by sigma_base + i
    int sigma_base;
    int fp8;                  // pack: some matrices also get the E4M3 copy of X0 (EwMat::x8)
    EwMat m[kEwMaxMats];
};

// ----------------------------------------------------------------- FP8 Gram --
// FP8 variant of the Gram product: its operands are X * 2^8 rounded to E4M3
// (an exact scaling; every iterate's elements stay below its largest singular
// value, which the quintic keeps under 1.21, and 1.21 * 2^8 < 448, E4M3's
// largest finite value); the product's fp32 sums are unscaled by 2^-16 before
// the bf16 rounding.  The E4M3 copy is written beside X by the kernel that
// writes X: the pack for X0, the update's epilogue for the later iterates.
constexpr int kFp8ScaleExp = 8;

// ------------------------------------------------------------------- GEMM --
// One persistent, warp-specialised tcgen05 kernel runs the three products of
// a Newton-Schulz iteration over every matrix of every shape bucket.
constexpr int kBN = 256;      // accumulator columns per tile
constexpr int kBK = 64;       // bf16 elements of K per stage (one 128-byte swizzle row)
constexpr int kMaxBuckets = 8;

enum GemmMode : int {
    kGram = 0,                // out = bf16(X X^T)                  (symmetric)
    kPoly = 1,                // out = bf16(b*A + c*A A)            (symmetric)
    kUpdate = 2               // out = bf16(a*X + B X)
};

struct GemmBucket {
    CUtensorMap tmA;          // A operand, box {64, 128, 1}, K-major
    CUtensorMap tmB;          // B operand: K-major box {64, 256, 1} or MN-major box {64, 64, 1}
    __nv_bfloat16* out;       // output, nmat x rows x ld
    const __nv_bfloat16* epi; // epilogue input with the same layout as out (Poly: A, Update: X)
    long long mat_stride;     // elements between matrices of out / epi
    int ld;                   // row length of out / epi
    int mt, nt;               // tiles along M and N of one matrix
    int kblocks;              // K / kBK
    int tiles_per_mat;
    int nmat;
    int tile0;                // first global tile of this bucket
    int fin0;                 // first entry of this bucket's matrices in FinalParams (final update)
    CUtensorMap tmE;          // update: the iterate X as epilogue input, box {32, 32, 1}, 64-byte swizzle
    CUtensorMap tmO;          // update: the output X', box {32, 32, 1}, 64-byte swizzle
    CUtensorMap tmT;          // upper-only symmetric operand (polynomial: A, update: B): box {64, 64, 1}
                              // over its rows, read as MN-major blocks of the transpose
    CUtensorMap tmQ;          // update before an FP8 Gram: E4M3 copy of X' * 2^8, bytes, box {32, 32, 1}
};

struct GemmParams {
    GemmBucket b[kMaxBuckets];
    int nbuckets;
    int total_tiles;
    int mode;
    float a, bcoef, c;
    unsigned long long wait_ns;   // limit of every wait of the launch; 0: the default (2 s)
    int stall;                    // test hook (pair kernel): no MMA is issued, so the waits expire
    int fp8;                      // Gram: E4M3 operands (tmA / tmB over the E4M3 copy, kblocks of 128)
    int fp8_next;                 // update (TMA epilogue): also writes the E4M3 copy of X' through tmQ
    // 1: the symmetric products (Gram, polynomial) store only their tiles with
    // tm <= tn (diagonal tiles in full), and their consumers (polynomial,
    // update) read the K blocks left of a row tile's diagonal as MN-major
    // blocks of the stored transpose (tmT); 0: full storage, K-major reads only
    int upper_only;
};

// Last update of the iteration fused with what follows it: the epilogue rounds
// O = bf16(a X + B X) and writes it straight to the caller's matrix in its
// stored orientation -- the weight update W <- dcy*W - s*O (muon_step) or the
// store of O into the input (Newton-Schulz only) -- so O never makes a round
// trip through HBM.  One table entry per matrix of the launch.
constexpr int kFinalMaxMats = 448;

enum FinalKind : int {
    kFinNone = 0,             // plain update: X' to the workspace
    kFinStore = 1,            // O (bf16) into the caller's bf16 matrix
    kFinWBf16 = 2,            // weight update of a bf16 W
    kFinWF32 = 3              // weight update of an fp32 W
};

struct FinalMat {
    void* w;                  // W (weight update) or the input matrix (store), rows x cols as stored
    __nv_bfloat16* oout;      // optional copy of O, rows x cols, or nullptr
    float dcy, s;             // weight-update scalars
    int rows, cols;           // as stored
    int trans;                // 1 when rows > cols (the iterate holds the transpose)
    int vec;                  // 1 when cols % 8 == 0 (16-byte vector access along a stored row)
};

struct FinalParams {
    FinalMat m[kFinalMaxMats];
};

// ------------------------------------------------------------ small path --
// Matrices whose iterate, A and B fit in shared memory run every
// Newton-Schulz iteration in one CTA (ns_small.cu).
constexpr int kSmallMaxMats = 512;
constexpr size_t kSmallMaxSmem = 200 * 1024;

struct SmallMat {
    __nv_bfloat16* x;         // oriented iterate (r x k, row stride ldx), updated in place
    int r, k, ldx, pad_;
};

constexpr int kMaxNsSteps = 64;

struct SmallParams {
    int nmats;
    int steps;
    float coef[3 * kMaxNsSteps];   // (a, b, c) of every iteration
    SmallMat m[kSmallMaxMats];
};

// ------------------------------------------------------------------ AdamW --
constexpr int kAdamMaxTensors = 256;

struct AdamWTensor {
    void* p;                  // parameter (bf16 or fp32), updated in place
    const void* g;            // gradient (bf16 or fp32)
    float* m;                 // first moment, fp32
    float* v;                 // second moment, fp32
    long long n;              // elements
    long long tile0;          // first tile of this tensor in this launch
};

struct AdamWParams {
    int ntensors;
    int p_bf16, g_bf16;
    long long total_tiles;
    float beta1, beta2, eps, b1c, b2c, dcy, step_size, inv_sqrt_bc2;
    AdamWTensor t[kAdamMaxTensors];
};

cudaError_t launch_adamw(const AdamWParams& p, int sms, cudaStream_t s);
long long adamw_tile_elems();

// ----------------------------------------------------------- gradient norm --
// One descriptor per tensor of a launch; tiles of kNormTileBytes of one tensor.
constexpr int kNormTileBytes = 32768;
constexpr int kNormMaxTensors = 640;
constexpr int kNormFewTensors = 40;      // launches of up to this many take the small parameter block
constexpr int kNormMaxBlocks = 1216;     // partial sums per launch

struct NormTensor {
    const void* g;            // gradient (bf16 or fp32)
    void* out;                // clip: where the scaled gradient goes (may be g)
    long long n;              // elements
    int tile0;                // first tile of this tensor in this launch
    int bf16;                 // 1: bf16, 0: fp32
};

struct NormHead {
    int ntensors;
    int total_tiles;
    int npartials;            // clip / finish: partial sums of the whole list
    int in_place;             // clip: out is g for every tensor
    float max_norm;
    double* partials;         // norm: this launch's; clip / finish: the whole list's
    float* norm;              // the norm, written by the finishing launch (clip: its first block)
};

template <int N>
struct NormParams {
    NormHead h;
    NormTensor t[N];
};

int norm_grid(int total_tiles, int sms);
template <int N>
cudaError_t launch_grad_norm(const NormParams<N>& p, int grid, cudaStream_t s);
template <int N>
cudaError_t launch_grad_clip(const NormParams<N>& p, int grid, bool first, cudaStream_t s);
cudaError_t launch_grad_norm_finish(const NormHead& h, cudaStream_t s);

// ----------------------------------------------------------------- routing --
constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxTopK = 32;
constexpr int kRouteMaxPerLane = 32;

struct RouteParams {
    const void* logits;       // tokens x experts, row stride ld
    const float* bias;        // experts, or nullptr
    float* weights;           // tokens x top_k
    int* chosen;              // tokens x top_k
    int* counts;              // experts
    const float* d_weights;   // backward: tokens x top_k
    void* d_logits;           // backward: tokens x experts, row stride ld_d
    long long tokens, ld, ld_d;
    int experts, top_k, groups, top_groups;
    int group_size;           // experts / groups
    int lanes;                // lanes per group (a power of two)
    int per_lane;             // experts per lane, consecutive
    int sigmoid, renormalize;
    int bf16;
    int vec;                  // 1: four consecutive experts of a lane load as one vector
    float scale;
};

cudaError_t launch_route(const RouteParams& p, int sms, cudaStream_t s);
cudaError_t launch_route_backward(const RouteParams& p, int sms, cudaStream_t s);

// ------------------------------------------------------ 8-bit block products --
constexpr int kFp8Block = 128;           // elements per scale along the reduction
constexpr int kFp8MaxGroups = 512;

struct QuantParams {
    const void* x;            // rows x cols of `batch` matrices, row stride ld, matrix stride ldb
    const char* x_end;        // one past the last element
    long long rows, cols, ld, ldb;
    int batch;
    int bf16;
    int vec;                  // 16-byte loads are legal
    int groups;               // col blocks start anew at each group's first row (0: one group, all rows)
    const int* offsets;       // groups + 1 row offsets on the device
    uint8_t* row_q;           // rows x ldq E4M3 codes (row blocks), or nullptr
    uint8_t* row_scale;       // col blocks x rows
    uint8_t* col_q;           // padded rows x ldq codes (col blocks), or nullptr
    uint8_t* col_scale;       // padded row blocks x ldq
    uint8_t* blk_q;           // batch x rows x ldq codes (128 x 128 blocks), or nullptr
    uint8_t* blk_scale;       // batch x row blocks x col blocks
    long long ldq;            // cols rounded up to 128
    long long row_blocks;     // grid bound of 128-row blocks (per matrix)
};

// Two matrices with the same element type and row alignment in one launch: p as
// launch_fp8_quantize, q's col blocks only.
bool fp8_quantize_pairs(const QuantParams& p, const QuantParams& q);
cudaError_t launch_fp8_quantize_pair(const QuantParams& p, const QuantParams& q, cudaStream_t s);
cudaError_t launch_fp8_quantize(const QuantParams& p, cudaStream_t s);

enum Fp8Mode : int {
    kFp8Forward = 0,          // tokens grouped; the weight of group g K-major
    kFp8GradInput = 1,        // tokens grouped; the weight of group g MN-major
    kFp8GradWeight = 2        // reduction grouped; both operands MN-major
};

// How a product's launch follows the one before it on the stream.
enum Fp8Sync : int {
    kSyncNone = 0,            // when that has ended
    kSyncEarly = 1,           // set-up overlaps it, then waits: it wrote the operands
    kSyncLate = 2             // beside it: it is a product that began after the operands were complete
};

// Scale bytes of one operand: byte (index, reduction block) of batch g at
// p + g * batch + (index >> shift) * idx + block * red.
struct Fp8Scale {
    const uint8_t* p;
    long long batch, idx, red;
    int shift;
    int limit;                // number of indices
};

struct Fp8GemmParams {
    CUtensorMap tm_a;         // MMA rows' operand: the weight (forward, grad input), dy (grad weight)
    CUtensorMap tm_b;         // MMA columns' operand: the tokens, x (grad weight); 128 indices at a time
    CUtensorMap tm_part;      // forward, grad input: the tokens 32 rows at a time (narrow tiles)
    CUtensorMap tm_res;       // vec, forward and grad input: the output in 32 x 32 blocks
    Fp8Scale s_a, s_b;
    void* out;                // row stride ld
    long long ld;
    long long out_batch;      // grad weight: elements between groups' outputs
    int mode;
    int sync;                 // Fp8Sync
    int col_shift;            // column tiles of at most 2^col_shift: 8, 7 or 6
    int slices;               // pairs of a cluster that share each tile's reduction; 1: none
    int out_f32;
    int vec;                  // output rows start on 16 bytes (forward, grad input: bf16 only)
    int m_ext;                // extent along the MMA's rows: n (forward, grad weight), k (grad input)
    int n_ext;                // extent along its columns: tokens; k (grad weight)
    int kblocks;              // reduction blocks (forward, grad input)
    int groups;               // >= 1
    const int* offsets;       // groups + 1 row offsets, or nullptr: one group of all rows
    int rows;                 // grad weight: tokens
    int zero_rest;            // forward, grad input: rows of no group become zero
    unsigned long long wait_ns;
};

cudaError_t launch_fp8_gemm(const Fp8GemmParams& p, int sms, cudaStream_t s);
void fp8_gemm_clusters(int (&n)[3]);
void fp8_gemm_cut(Fp8GemmParams& p, int sms, const int (&clusters)[3]);

// The forward product of few tokens and one weight, x rounded on the way.
struct Fp8TokenParams {
    const void* x;            // tokens x k, row stride ld_x
    const uint8_t* w;         // n x ldk codes
    const uint8_t* w_scale;   // n blocks x k blocks
    void* out;                // tokens x n, row stride ld_out
    long long ld_x, ldk, ld_out;
    int tokens, n, k;
    int bf16;                 // x
    int vec;                  // 16-byte loads of x are legal
    int out_f32;
};

bool fp8_token_serves(long long tokens, long long n, long long k);
cudaError_t launch_fp8_token(const Fp8TokenParams& p, cudaStream_t s);
cudaError_t read_and_clear_fp8_error(int* code);

// ------------------------------------------------- experts' rows (token_*.cu) --
constexpr int kSortMaxExperts = 1024;
constexpr int kRowsMaxTopK = 32;

struct SortParams {
    const int* chosen;        // entries
    int* order;               // entries
    int* place;               // entries
    int* offsets;             // experts + 1
    int* table;               // blocks x (experts + 1) counts
    int entries, first, experts;
    int blocks, run;          // of the two launches: how many, entries of each
    int bits;                 // of a bucket's number
};

int token_sort_blocks(long long entries);
cudaError_t launch_token_sort(SortParams p, cudaStream_t s);

// dispatch: x tokens' rows, out sorted rows; combine and its gradient: x sorted rows (y).
struct RowsParams {
    const void* x;
    const void* d;            // gradient of combine's result (tokens)
    void* out;                // gradient: dy, or nullptr
    float* dw;                // tokens x top_k, or nullptr
    const float* weights;     // tokens x top_k, or nullptr: all 1
    const int* place;         // tokens x top_k
    const int* offsets;       // groups + 1
    long long ld_x, ld_d, ld_out;
    long long tokens, cols;
    int top_k, groups, rows;  // rows = tokens * top_k
    int x_bf16, d_bf16, out_bf16;
    int runs, parts;          // whole runs of a row; warps for a row
};

cudaError_t launch_dispatch(const RowsParams& p, cudaStream_t s);
cudaError_t launch_combine(const RowsParams& p, cudaStream_t s);
cudaError_t launch_combine_backward(const RowsParams& p, cudaStream_t s);

// ------------------------------------------------------- gated activation --
struct SwigluParams {
    const void *gate, *up;
    const void* d;            // gradient of the result; nullptr: forward
    void* out;
    void *d_gate, *d_up;
    long long ld_gate, ld_up, ld_d, ld_out, ld_dgate, ld_dup;
    long long rows, cols;
    unsigned long long by_runs;   // 2^64 / runs, rounded up
    unsigned runs, total;     // vectors of a row, of the launch
    int rest;                 // elements past the last vector (one row alone)
    int bf16;
};

cudaError_t launch_swiglu(SwigluParams p, cudaStream_t s);

// ------------------------------------------------------ weights of 4 bits --
struct Int4QuantParams {
    const void* w;            // batch x rows x cols
    uint8_t* codes;           // batch x rows x 64 kblocks
    __nv_bfloat16* scale;     // batch x (128 / block kblocks) x rows
    long long batch, rows, cols, kblocks;
    int block, bf16;
};

cudaError_t launch_int4_quantize(const Int4QuantParams& p, cudaStream_t s);

struct Int4Params {
    const void* x;            // tokens x k, row stride ld_x
    const uint8_t* w;         // groups x n x ldw bytes
    const __nv_bfloat16* scale;
    void* out;                // tokens x n, row stride ld_out
    const int* offsets;       // groups + 1, or nullptr: one group
    long long ld_x, ldw, ld_out;
    long long w_batch, scale_batch;
    int tokens, n, k, kblocks, groups;
    int block;                // columns of a scale
    int x_bf16, out_f32;
    int vec;                  // 16-byte loads of x are legal
    int pairs;                // scales of rows 2 i and 2 i + 1 load as one
};

cudaError_t launch_int4_linear(const Int4Params& p, int sms, cudaStream_t s);

// Launch helpers implemented in the .cu files.
// `sms`: the grid is one CTA per resident slot on every SM (capped by the tiles).
cudaError_t launch_momentum_norm(const EwParams& p, int sms, cudaStream_t s);
cudaError_t launch_input_norm(const EwParams& p, int sms, cudaStream_t s);
cudaError_t launch_norm_finalize(const EwParams& p, cudaStream_t s);
cudaError_t launch_pack(const EwParams& p, int sms, bool from_momentum, cudaStream_t s);
cudaError_t launch_unpack(const EwParams& p, int sms, bool weight_update, cudaStream_t s);
// Pair-CTA variant (ns_gemm_pair.cu): 256 x 256 tiles on clusters of two CTAs.
// `sms` bounds the grid.
// `tma_epilogue`: the update moves its epilogue input and output by TMA
// (the buckets' tmE / tmO must be set).
cudaError_t launch_gemm_pair(const GemmParams& p, int sms, bool tma_epilogue, cudaStream_t s);
// The same kernel with the fused final epilogue (p.mode must be kUpdate).
cudaError_t launch_gemm_pair_final(const GemmParams& p, const FinalParams& f, int kind, int sms, cudaStream_t s);
size_t gemm_pair_smem_bytes();
cudaError_t read_and_clear_pair_error(int* code);

// ------------------------------------------------------------ debug guard --
// MUON_DEBUG_GUARD=1: guard regions around every workspace region (guard.cu).
constexpr size_t kGuardBytes = 4096;
constexpr unsigned kGuardWord = 0xA5A5A5A5u;   // every byte 0xA5
constexpr int kMaxGuards = 480;

struct GuardParams {
    const char* base;          // workspace base
    int n;                     // guard regions in this launch
    unsigned long long off[kMaxGuards];   // their offsets from base
};

cudaError_t launch_guard_check(const GuardParams& p, cudaStream_t s);
cudaError_t read_and_clear_guard_error(int* code);

// Host helpers of muon_abi.cu used by other entry points.
int ns5_batched_on_workspace(void* const* ptrs, const int* rows, const int* cols, int count, int steps,
                             const float* coeffs, void* ws, size_t ws_bytes, cudaStream_t stream);
int set_last_error(int status, const char* msg);

// What the operators around the step (train_abi.cu) share with it.
enum OpKind : int { kOpGradNorm = 10, kOpGradClip, kOpRoute, kOpRouteGrad, kOpFp8Quantize, kOpFp8Gemm, kOpFp8Token,
                    kOpTokenSort, kOpDispatch, kOpCombine, kOpCombineGrad, kOpSwiglu, kOpSwigluGrad, kOpInt4Quantize,
                    kOpInt4Linear, kOpEnd };
// The current device, checked; its SMs, and how many clusters of 4, 6 and 8 CTAs of fp8_gemm it holds.
int op_device(int* sms, int (*clusters)[3] = nullptr);
int op_launch(int kind, double flops, double bytes, cudaStream_t s, const std::function<cudaError_t()>& f);
int op_encode_bytes(CUtensorMap* map, const void* base, long long inner, long long outer, long long batch,
                    int box_inner, int box_outer);
int op_encode_result(CUtensorMap* map, const void* base, long long cols, long long rows, long long ld);
cudaError_t launch_ns_small(const SmallParams& p, size_t smem, cudaStream_t s);
size_t ns_small_smem_bytes(int r, int k);

}  // namespace muon
