// C ABI of the operators around the optimizer step (include/muon.h): routing
// and its gradient, 8-bit block products, the global gradient norm and
// clipping.  Validation, launch parameters and tensor maps only; nothing here
// allocates, keeps state or synchronises.
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstring>
#include <memory>

#include "abi_checks.h"
#include "internal.h"
#include "muon.h"

namespace muon {
namespace {

// ----------------------------------------------------------- gradient norm --
int check_grads(const void* const* G, const long long* numel, const int* dtypes, int count, const char* what) {
    for (int i = 0; i < count; ++i) {
        if (numel[i] < 0) return fail(MUON_ERR_INVALID_ARG, "numel[%d] is negative", i);
        if (numel[i] == 0) continue;
        int rc = check_dtype(dtypes[i], what);
        if (rc != MUON_OK) return rc;
        if (G[i] == nullptr) return fail(MUON_ERR_INVALID_ARG, "%s[%d] is NULL", what, i);
        if (reinterpret_cast<uintptr_t>(G[i]) % dtype_size(dtypes[i]) != 0)
            return fail(MUON_ERR_INVALID_ARG, "%s[%d] is not aligned to its elements", what, i);
    }
    return MUON_OK;
}

long long grad_tiles(long long n, int dtype) {
    const long long tile = kNormTileBytes / static_cast<long long>(dtype_size(dtype));
    return (n + tile - 1) / tile;
}

// Launches that a list takes: up to kNormMaxTensors non-empty tensors each and
// tiles that an int counts.
int norm_launches(const long long* numel, int count) {
    int n = 0, in = 0;
    long long tiles = 0;
    for (int i = 0; i < count; ++i) {
        if (numel[i] == 0) continue;
        const long long t = grad_tiles(numel[i], MUON_F32);
        if (n == 0 || in == kNormMaxTensors || tiles + t > INT_MAX / 2) {
            ++n;
            in = 0;
            tiles = 0;
        }
        ++in;
        tiles += t;
    }
    return n;
}

// The list in launches: f(params, first launch of the list).
template <int N, class F>
int for_each_launch(const void* const* G, void* const* out, const long long* numel, const int* dtypes, int count,
                    NormParams<N>& p, F&& f) {
    int i = 0, at = 0;
    while (i < count) {
        long long tiles = 0, counted = 0;
        double bytes = 0.0;
        p.h.ntensors = 0;
        for (; i < count; ++i) {
            if (numel[i] == 0) continue;
            const long long t = grad_tiles(numel[i], dtypes[i]), tf = grad_tiles(numel[i], MUON_F32);
            if (p.h.ntensors == (N < kNormMaxTensors ? N : kNormMaxTensors) ||
                (p.h.ntensors > 0 && counted + tf > INT_MAX / 2))
                break;
            NormTensor& T = p.t[p.h.ntensors++];
            T.g = G[i];
            T.out = out != nullptr ? out[i] : const_cast<void*>(G[i]);
            T.n = numel[i];
            T.tile0 = static_cast<int>(tiles);
            T.bf16 = dtypes[i] == MUON_BF16;
            tiles += t;
            counted += tf;
            bytes += static_cast<double>(numel[i]) * dtype_size(dtypes[i]);
        }
        if (p.h.ntensors == 0) break;
        p.h.total_tiles = static_cast<int>(tiles);
        const int rc = f(p, at, bytes);
        if (rc != MUON_OK) return rc;
        ++at;
    }
    return MUON_OK;
}

template <int N>
int run_norm(const void* const* G, void* const* out, const long long* numel, const int* dtypes, int count, bool clip,
             float max_norm, double* partials, float* norm, int sms, cudaStream_t stream) {
    std::unique_ptr<NormParams<N>> p(new NormParams<N>());
    std::memset(p.get(), 0, sizeof *p);
    int total = 0;
    int rc = for_each_launch<N>(G, nullptr, numel, dtypes, count, *p, [&](NormParams<N>& q, int, double bytes) {
        const int grid = norm_grid(q.h.total_tiles, sms);
        q.h.partials = partials + total;
        total += grid;
        return op_launch(kOpGradNorm, 0.0, bytes, stream, [&] { return launch_grad_norm<N>(q, grid, stream); });
    });
    if (rc != MUON_OK) return rc;
    if (!clip) {
        NormHead h = {};
        h.npartials = total;
        h.partials = partials;
        h.norm = norm;
        return op_launch(kOpGradNorm, 0.0, 8.0 * total, stream, [&] { return launch_grad_norm_finish(h, stream); });
    }
    bool in_place = out == nullptr;
    p->h.max_norm = max_norm;
    return for_each_launch<N>(G, out, numel, dtypes, count, *p, [&](NormParams<N>& q, int at, double bytes) {
        q.h.partials = partials;
        q.h.npartials = total;
        q.h.norm = at == 0 ? norm : nullptr;
        q.h.in_place = in_place ? 1 : 0;
        const int grid = norm_grid(q.h.total_tiles, sms);
        return op_launch(kOpGradClip, 0.0, 2.0 * bytes, stream,
                         [&] { return launch_grad_clip<N>(q, grid, at == 0, stream); });
    });
}

int norm_or_clip(const void* const* G, void* const* out, const long long* numel, const int* dtypes, int count, bool clip,
                 float max_norm, void* workspace, size_t workspace_bytes, float* norm, cudaStream_t stream) {
    if (count < 0) return fail(MUON_ERR_INVALID_ARG, "count is negative");
    if (count > 0 && (G == nullptr || numel == nullptr || dtypes == nullptr))
        return fail(MUON_ERR_INVALID_ARG, "a host array is NULL");
    int rc = check_align(norm, 4, "norm");
    if (rc != MUON_OK) return rc;
    if ((rc = check_grads(G, numel, dtypes, count, "G")) != MUON_OK) return rc;
    if (out != nullptr && (rc = check_grads(const_cast<const void* const*>(out), numel, dtypes, count, "out")) != MUON_OK)
        return rc;
    if (clip && !(max_norm >= 0.0f && std::isfinite(max_norm)))
        return fail(MUON_ERR_INVALID_ARG, "max_norm must be finite and >= 0");
    int used = 0;
    for (int i = 0; i < count; ++i) used += numel[i] > 0;
    int sms = 0;
    if (used == 0) {
        if ((rc = op_device(&sms)) != MUON_OK) return rc;
        const cudaError_t e = cudaMemsetAsync(norm, 0, sizeof(float), stream);
        if (e != cudaSuccess) return fail(MUON_ERR_CUDA, "cudaMemsetAsync: %s", cudaGetErrorString(e));
        return MUON_OK;
    }
    if ((rc = check_align(workspace, 16, "workspace")) != MUON_OK) return rc;
    const size_t need = muon_grad_norm_workspace_bytes(numel, count);
    if (workspace_bytes < need)
        return fail(MUON_ERR_OOM, "workspace has %zu bytes; muon_grad_norm_workspace_bytes gives %zu", workspace_bytes, need);
    if ((rc = op_device(&sms)) != MUON_OK) return rc;
    double* partials = static_cast<double*>(workspace);
    if (used <= kNormFewTensors)
        return run_norm<kNormFewTensors>(G, out, numel, dtypes, count, clip, max_norm, partials, norm, sms, stream);
    return run_norm<kNormMaxTensors>(G, out, numel, dtypes, count, clip, max_norm, partials, norm, sms, stream);
}

// ----------------------------------------------------------------- routing --
int fill_route(RouteParams& p, const void* logits, int dtype, long long tokens, int experts, long long ld,
               const muon_route_opts* o) {
    int rc = check_dtype(dtype, "logits");
    if (rc != MUON_OK) return rc;
    if (o == nullptr) return fail(MUON_ERR_INVALID_ARG, "opts is NULL");
    if (tokens < 0) return fail(MUON_ERR_INVALID_ARG, "tokens is negative");
    if (experts < 1 || experts > kRouteMaxExperts)
        return fail(MUON_ERR_UNSUPPORTED, "experts is %d (1 to %d)", experts, kRouteMaxExperts);
    if (o->top_k < 1 || o->top_k > kRouteMaxTopK || o->top_k > experts)
        return fail(MUON_ERR_INVALID_ARG, "top_k is %d (1 to min(%d, experts))", o->top_k, kRouteMaxTopK);
    if (o->groups < 1 || o->groups > 32 || experts % o->groups != 0)
        return fail(MUON_ERR_INVALID_ARG, "groups is %d (1 to 32, a divisor of experts)", o->groups);
    if (o->top_groups < 1 || o->top_groups > o->groups)
        return fail(MUON_ERR_INVALID_ARG, "top_groups is %d (1 to groups)", o->top_groups);
    if (static_cast<long long>(experts / o->groups) * o->top_groups < o->top_k)
        return fail(MUON_ERR_INVALID_ARG, "top_groups * (experts / groups) is below top_k");
    if (o->score != MUON_SCORE_SOFTMAX && o->score != MUON_SCORE_SIGMOID)
        return fail(MUON_ERR_INVALID_ARG, "unknown score %d", o->score);
    if ((o->renormalize != 0 && o->renormalize != 1) || !std::isfinite(o->scale))
        return fail(MUON_ERR_INVALID_ARG, "renormalize must be 0 or 1 and scale finite");
    if (ld < experts) return fail(MUON_ERR_INVALID_ARG, "the logits' row stride is below experts");
    if (tokens > 0 && (rc = check_align(logits, dtype_size(dtype), "logits")) != MUON_OK) return rc;
    p.logits = logits;
    p.tokens = tokens;
    p.ld = ld;
    p.experts = experts;
    p.top_k = o->top_k;
    p.groups = o->groups;
    p.top_groups = o->top_groups;
    p.group_size = experts / o->groups;
    p.lanes = 1;
    while (p.lanes * 2 * o->groups <= 32) p.lanes *= 2;
    p.per_lane = (p.group_size + p.lanes - 1) / p.lanes;
    if (p.per_lane > kRouteMaxPerLane)
        return fail(MUON_ERR_UNSUPPORTED, "%d groups of %d experts: at most %d experts per group of this number", o->groups,
                    p.group_size, p.lanes * kRouteMaxPerLane);
    // a lane's experts as vectors of four: rounded up, so that every lane starts on one
    const size_t sz = dtype_size(dtype);
    p.vec = p.group_size % 4 == 0 && ld % 4 == 0 && reinterpret_cast<uintptr_t>(logits) % (4 * sz) == 0;
    if (p.vec) p.per_lane = (p.per_lane + 3) / 4 * 4;
    p.sigmoid = o->score == MUON_SCORE_SIGMOID;
    p.renormalize = o->renormalize;
    p.bf16 = dtype == MUON_BF16;
    p.scale = o->scale;
    return MUON_OK;
}

// --------------------------------------------------------------- 8 bits --
QuantParams quantize_params(const void* x, int dtype, long long rows, long long cols, long long ld, int groups,
                            const int* offsets, void* row_codes, void* row_scale, void* col_codes, void* col_scale) {
    QuantParams p = {};
    p.x = x;
    p.rows = rows;
    p.cols = cols;
    p.ld = ld;
    p.x_end = static_cast<const char*>(x) + ((rows - 1) * ld + cols) * static_cast<long long>(dtype_size(dtype));
    p.batch = 1;
    p.bf16 = dtype == MUON_BF16;
    p.vec = reinterpret_cast<uintptr_t>(x) % 16 == 0 && ld * static_cast<long long>(dtype_size(dtype)) % 16 == 0;
    p.row_q = static_cast<uint8_t*>(row_codes);
    p.row_scale = static_cast<uint8_t*>(row_scale);
    p.col_q = static_cast<uint8_t*>(col_codes);
    p.col_scale = static_cast<uint8_t*>(col_scale);
    p.ldq = up128(cols);
    // groups matter to the col blocks alone
    const bool grouped = offsets != nullptr && col_codes != nullptr;
    p.groups = grouped ? groups : 0;
    p.offsets = grouped ? offsets : nullptr;
    p.row_blocks = grouped ? muon_fp8_padded_rows(rows, groups) / 128 : (rows + 127) / 128;
    return p;
}

// Codes of one matrix in a workspace: codes, then scales, each from a multiple of 256 bytes on.
size_t up256(long long n) { return static_cast<size_t>((n + 255) / 256 * 256); }

struct RowCodes {
    size_t code_bytes, scale_bytes;
    char *codes, *scale;
    RowCodes(void* at, long long rows, long long cols)
        : code_bytes(up256(rows * up128(cols))), scale_bytes(up256(rows * (up128(cols) / 128))),
          codes(static_cast<char*>(at)), scale(at != nullptr ? codes + code_bytes : nullptr) {}
    size_t bytes() const { return code_bytes + scale_bytes; }
};

struct ColCodes {
    size_t code_bytes, scale_bytes;
    char *codes, *scale;
    ColCodes(void* at, long long rows, long long cols, int groups)
        : code_bytes(up256(muon_fp8_padded_rows(rows, groups) * up128(cols))),
          scale_bytes(up256(muon_fp8_padded_rows(rows, groups) / 128 * up128(cols))),
          codes(static_cast<char*>(at)), scale(at != nullptr ? codes + code_bytes : nullptr) {}
    size_t bytes() const { return code_bytes + scale_bytes; }
};

int check_linear(int dtype, const char* what, long long tokens, long long ld, int cols, int n, int k, int groups,
                 const int* offsets, const void* w_codes, const void* w_scale) {
    int rc = check_dtype(dtype, what);
    if (rc != MUON_OK) return rc;
    if ((rc = check_groups(tokens, groups, offsets)) != MUON_OK) return rc;
    if ((rc = check_dim(n, "n")) != MUON_OK || (rc = check_dim(k, "k")) != MUON_OK) return rc;
    if (ld < cols) return fail(MUON_ERR_INVALID_ARG, "%s's row stride is below its columns", what);
    if ((rc = check_align(w_codes, 16, "w_codes")) != MUON_OK) return rc;
    if (w_scale == nullptr) return fail(MUON_ERR_INVALID_ARG, "w_scale is NULL");
    return MUON_OK;
}

// `sync` (Fp8Sync) other than none: one of a whole layer's calls; rows of no group become zero.
int fp8_product(int product, const void* a_codes, const void* a_scale, const void* b_codes, const void* b_scale,
                long long tokens, int n, int k, int groups, const int* offsets, void* out, int out_dtype,
                long long ld_out, int sync, cudaStream_t stream) {
    int rc = check_dtype(out_dtype, "out");
    if (rc != MUON_OK) return rc;
    if (product != MUON_FP8_FORWARD && product != MUON_FP8_GRAD_INPUT && product != MUON_FP8_GRAD_WEIGHT)
        return fail(MUON_ERR_INVALID_ARG, "unknown product %d", product);
    if ((rc = check_groups(tokens, groups, offsets)) != MUON_OK) return rc;
    if ((rc = check_dim(n, "n")) != MUON_OK || (rc = check_dim(k, "k")) != MUON_OK) return rc;
    const bool gw = product == MUON_FP8_GRAD_WEIGHT;
    const int inner = product == MUON_FP8_FORWARD ? n : k;
    if (ld_out < inner) return fail(MUON_ERR_INVALID_ARG, "the output's row stride is below its columns");
    if (tokens == 0 && !gw) return MUON_OK;
    if ((rc = check_align(out, dtype_size(out_dtype), "out")) != MUON_OK) return rc;
    if (tokens > 0 && ((rc = check_align(a_codes, 16, "a_codes")) != MUON_OK ||
                       (rc = check_align(b_codes, 16, "b_codes")) != MUON_OK))
        return rc;
    const size_t scale_align = gw ? 4 : 1;               // col blocks' bytes are read four at a time
    if (tokens > 0 && ((rc = check_align(a_scale, scale_align, "a_scale")) != MUON_OK ||
                       (rc = check_align(b_scale, scale_align, "b_scale")) != MUON_OK))
        return rc;
    int sms = 0, clusters[3] = {};
    if ((rc = op_device(&sms, &clusters)) != MUON_OK) return rc;
    if (gw && tokens == 0) {
        const size_t sz = dtype_size(out_dtype);
        const cudaError_t e = cudaMemset2DAsync(out, ld_out * sz, 0, inner * sz, static_cast<size_t>(groups) * n, stream);
        if (e != cudaSuccess) return fail(MUON_ERR_CUDA, "cudaMemset2DAsync: %s", cudaGetErrorString(e));
        return MUON_OK;
    }
    Fp8GemmParams p = {};
    const long long ldn = up128(n), ldk = up128(k), nb = ldn / 128, kb = ldk / 128;
    const uint8_t* as = static_cast<const uint8_t*>(a_scale);
    const uint8_t* bs = static_cast<const uint8_t*>(b_scale);
    p.mode = product;
    p.out = out;
    p.ld = ld_out;
    p.out_f32 = out_dtype == MUON_F32;
    const bool rows16 = reinterpret_cast<uintptr_t>(out) % 16 == 0 &&
                        ld_out * static_cast<long long>(dtype_size(out_dtype)) % 16 == 0;
    p.vec = rows16 && (gw || out_dtype == MUON_BF16);
    p.m_ext = gw ? n : inner;
    p.groups = groups;
    p.offsets = offsets;
    p.rows = static_cast<int>(tokens);
    p.sync = sync;
    p.zero_rest = sync != kSyncNone && !gw;
    if (gw) {
        // a: dy's col codes (padded tokens x ldn); b: x's col codes (padded tokens x ldk)
        const long long padded = muon_fp8_padded_rows(tokens, groups);
        p.n_ext = k;
        p.out_batch = static_cast<long long>(n) * ld_out;
        fp8_gemm_cut(p, sms, clusters);
        p.s_a = {as, 0, 1, ldn, 0, static_cast<int>(ldn)};
        p.s_b = {bs, 0, 1, ldk, 0, static_cast<int>(ldk)};
        if ((rc = op_encode_bytes(&p.tm_a, a_codes, ldn, padded, 1, 128, 128)) != MUON_OK) return rc;
        if ((rc = op_encode_bytes(&p.tm_b, b_codes, ldk, padded, 1, 128, 128)) != MUON_OK) return rc;
    } else {
        // a: x's or dy's row codes (tokens x ld); b: the weight's codes (groups x n x ldk)
        const bool fwd = product == MUON_FP8_FORWARD;
        const long long lda = fwd ? ldk : ldn;
        p.n_ext = static_cast<int>(tokens);
        p.kblocks = static_cast<int>(fwd ? kb : nb);
        p.s_a = fwd ? Fp8Scale{bs, nb * kb, kb, 1, 7, static_cast<int>(ldn)}
                     : Fp8Scale{bs, nb * kb, 1, kb, 7, static_cast<int>(ldk)};
        p.s_b = {as, 0, 1, tokens, 0, static_cast<int>(tokens)};
        fp8_gemm_cut(p, sms, clusters);
        if ((rc = op_encode_bytes(&p.tm_a, b_codes, ldk, n, groups, 128, 128)) != MUON_OK) return rc;
        if ((rc = op_encode_bytes(&p.tm_b, a_codes, lda, tokens, 1, 128, 128)) != MUON_OK) return rc;
        if ((rc = op_encode_bytes(&p.tm_part, a_codes, lda, tokens, 1, 128, 32)) != MUON_OK) return rc;
    }
    if (p.vec && !gw && (rc = op_encode_result(&p.tm_res, out, inner, tokens, ld_out)) != MUON_OK) return rc;
    const double t = static_cast<double>(tokens), flops = 2.0 * t * n * k;
    const double bytes = t * (gw ? n + k : fmax(n, k)) + static_cast<double>(groups) * n * k * (gw ? dtype_size(out_dtype) : 1);
    return op_launch(kOpFp8Gemm, flops, bytes, stream, [&] { return launch_fp8_gemm(p, sms, stream); });
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

size_t muon_grad_norm_workspace_bytes(const long long* numel, int count) {
    if (count <= 0 || numel == nullptr) return 16;
    for (int i = 0; i < count; ++i)
        if (numel[i] < 0) return 0;
    return sizeof(double) * kNormMaxBlocks * static_cast<size_t>(norm_launches(numel, count)) + 16;
}

int muon_grad_norm(const void* const* G, const long long* numel, const int* dtypes, int count, void* workspace,
                   size_t workspace_bytes, float* norm, cudaStream_t stream) {
    return norm_or_clip(G, nullptr, numel, dtypes, count, false, 0.0f, workspace, workspace_bytes, norm, stream);
}

int muon_grad_clip(void* const* G, void* const* out, const long long* numel, const int* dtypes, int count, float max_norm,
                   void* workspace, size_t workspace_bytes, float* norm, cudaStream_t stream) {
    return norm_or_clip(const_cast<const void* const*>(G), out, numel, dtypes, count, true, max_norm, workspace,
                        workspace_bytes, norm, stream);
}

void muon_route_opts_init(muon_route_opts* o) {
    if (o == nullptr) return;
    o->top_k = 1;
    o->groups = 1;
    o->top_groups = 1;
    o->score = MUON_SCORE_SOFTMAX;
    o->renormalize = 1;
    o->scale = 1.0f;
}

int muon_route(const void* logits, int dtype, long long tokens, int experts, long long ld, const float* bias,
               const muon_route_opts* opts, float* weights, int* chosen, int* counts, cudaStream_t stream) {
    RouteParams p = {};
    int rc = fill_route(p, logits, dtype, tokens, experts, ld, opts);
    if (rc != MUON_OK) return rc;
    if (bias != nullptr && (rc = check_align(bias, 4, "bias")) != MUON_OK) return rc;
    if (tokens > 0 && ((rc = check_align(weights, 4, "weights")) != MUON_OK || (rc = check_align(chosen, 4, "chosen")) != MUON_OK))
        return rc;
    if ((rc = check_align(counts, 4, "counts")) != MUON_OK) return rc;
    int sms = 0;
    if ((rc = op_device(&sms)) != MUON_OK) return rc;
    if (tokens == 0) {
        const cudaError_t e = cudaMemsetAsync(counts, 0, sizeof(int) * experts, stream);
        if (e != cudaSuccess) return fail(MUON_ERR_CUDA, "cudaMemsetAsync: %s", cudaGetErrorString(e));
        return MUON_OK;
    }
    p.bias = bias;
    p.weights = weights;
    p.chosen = chosen;
    p.counts = counts;
    const double bytes = static_cast<double>(tokens) * (experts * dtype_size(dtype) + 8.0 * opts->top_k);
    return op_launch(kOpRoute, 0.0, bytes, stream, [&] { return launch_route(p, sms, stream); });
}

int muon_route_backward(const float* d_weights, const void* logits, int dtype, long long tokens, int experts,
                        long long ld, const int* chosen, const muon_route_opts* opts, void* d_logits, long long ld_d,
                        cudaStream_t stream) {
    RouteParams p = {};
    int rc = fill_route(p, logits, dtype, tokens, experts, ld, opts);
    if (rc != MUON_OK) return rc;
    if (ld_d < experts) return fail(MUON_ERR_INVALID_ARG, "the gradient's row stride is below experts");
    if (tokens == 0) return MUON_OK;
    if ((rc = check_align(d_weights, 4, "d_weights")) != MUON_OK) return rc;
    if ((rc = check_align(chosen, 4, "chosen")) != MUON_OK) return rc;
    if ((rc = check_align(d_logits, dtype_size(dtype), "d_logits")) != MUON_OK) return rc;
    if (d_logits == logits) return fail(MUON_ERR_INVALID_ARG, "d_logits must not be the logits");
    int sms = 0;
    if ((rc = op_device(&sms)) != MUON_OK) return rc;
    p.d_weights = d_weights;
    p.chosen = const_cast<int*>(chosen);
    p.d_logits = d_logits;
    p.ld_d = ld_d;
    const size_t four = 4 * dtype_size(dtype);           // four consecutive elements as one vector
    p.vec = experts % 4 == 0 && ld % 4 == 0 && ld_d % 4 == 0 && reinterpret_cast<uintptr_t>(logits) % four == 0 &&
            reinterpret_cast<uintptr_t>(d_logits) % four == 0;
    const double bytes = static_cast<double>(tokens) * (2.0 * experts * dtype_size(dtype) + 8.0 * opts->top_k);
    return op_launch(kOpRouteGrad, 0.0, bytes, stream, [&] { return launch_route_backward(p, sms, stream); });
}

long long muon_fp8_padded_rows(long long rows, int groups) {
    if (rows < 0 || groups < 1) return 0;
    return 128 * (rows / 128 + (rows < groups ? rows : groups));
}

int muon_fp8_quantize(const void* x, int dtype, long long rows, long long cols, long long ld, int groups,
                      const int* offsets, void* row_codes, void* row_scale, void* col_codes, void* col_scale,
                      cudaStream_t stream) {
    int rc = check_dtype(dtype, "x");
    if (rc != MUON_OK) return rc;
    if ((rc = check_groups(rows, groups, offsets)) != MUON_OK) return rc;
    if ((rc = check_dim(cols, "cols")) != MUON_OK) return rc;
    if (ld < cols) return fail(MUON_ERR_INVALID_ARG, "the row stride is below cols");
    if (rows == 0) return MUON_OK;
    if ((row_codes == nullptr) != (row_scale == nullptr) || (col_codes == nullptr) != (col_scale == nullptr))
        return fail(MUON_ERR_INVALID_ARG, "codes and scale come in pairs");
    if (row_codes == nullptr && col_codes == nullptr) return fail(MUON_ERR_INVALID_ARG, "no output is asked for");
    if ((rc = check_align(x, dtype_size(dtype), "x")) != MUON_OK) return rc;
    if (row_codes != nullptr && (rc = check_align(row_codes, 16, "row_codes")) != MUON_OK) return rc;
    if (col_codes != nullptr && (rc = check_align(col_codes, 16, "col_codes")) != MUON_OK) return rc;
    int sms = 0;
    if ((rc = op_device(&sms)) != MUON_OK) return rc;
    const QuantParams p = quantize_params(x, dtype, rows, cols, ld, groups, offsets, row_codes, row_scale, col_codes, col_scale);
    const double n = static_cast<double>(rows) * cols;
    const double bytes = n * (dtype_size(dtype) + (row_codes != nullptr) + (col_codes != nullptr));
    return op_launch(kOpFp8Quantize, 0.0, bytes, stream, [&] { return launch_fp8_quantize(p, stream); });
}

int muon_fp8_quantize_weight(const void* w, int dtype, int batch, long long rows, long long cols, void* codes, void* scale,
                             cudaStream_t stream) {
    int rc = check_dtype(dtype, "w");
    if (rc != MUON_OK) return rc;
    if (batch < 0 || batch > kFp8MaxGroups) return fail(MUON_ERR_INVALID_ARG, "batch is %d (0 to %d)", batch, kFp8MaxGroups);
    if ((rc = check_dim(rows, "rows")) != MUON_OK || (rc = check_dim(cols, "cols")) != MUON_OK) return rc;
    if (batch == 0) return MUON_OK;
    if ((rc = check_align(w, dtype_size(dtype), "w")) != MUON_OK) return rc;
    if ((rc = check_align(codes, 16, "codes")) != MUON_OK) return rc;
    if (scale == nullptr) return fail(MUON_ERR_INVALID_ARG, "scale is NULL");
    int sms = 0;
    if ((rc = op_device(&sms)) != MUON_OK) return rc;
    QuantParams p = {};
    p.x = w;
    p.rows = rows;
    p.cols = cols;
    p.ld = cols;
    p.ldb = rows * cols;
    p.x_end = static_cast<const char*>(w) + batch * rows * cols * static_cast<long long>(dtype_size(dtype));
    p.batch = batch;
    p.bf16 = dtype == MUON_BF16;
    const long long sz = static_cast<long long>(dtype_size(dtype));
    p.vec = reinterpret_cast<uintptr_t>(w) % 16 == 0 && cols * sz % 16 == 0;
    p.blk_q = static_cast<uint8_t*>(codes);
    p.blk_scale = static_cast<uint8_t*>(scale);
    p.ldq = up128(cols);
    p.row_blocks = (rows + 127) / 128;
    const double bytes = static_cast<double>(batch) * rows * cols * (dtype_size(dtype) + 1.0);
    return op_launch(kOpFp8Quantize, 0.0, bytes, stream, [&] { return launch_fp8_quantize(p, stream); });
}

int muon_fp8_product(int product, const void* a_codes, const void* a_scale, const void* b_codes, const void* b_scale,
                     long long tokens, int n, int k, int groups, const int* offsets, void* out, int out_dtype,
                     long long ld_out, cudaStream_t stream) {
    return fp8_product(product, a_codes, a_scale, b_codes, b_scale, tokens, n, k, groups, offsets, out, out_dtype, ld_out,
                       kSyncNone, stream);
}

size_t muon_fp8_linear_workspace_bytes(long long tokens, int n, int k, int grouped) {
    if (tokens <= 0 || n < 1 || k < 1 || (!grouped && fp8_token_serves(tokens, n, k))) return 0;
    return RowCodes(nullptr, tokens, k).bytes();
}

int muon_fp8_linear(const void* x, int x_dtype, long long tokens, long long ld_x, const void* w_codes,
                    const void* w_scale, int n, int k, int groups, const int* offsets, void* workspace,
                    size_t workspace_bytes, void* out, int out_dtype, long long ld_out, cudaStream_t stream) {
    int rc = check_linear(x_dtype, "x", tokens, ld_x, k, n, k, groups, offsets, w_codes, w_scale);
    if (rc != MUON_OK) return rc;
    if ((rc = check_dtype(out_dtype, "out")) != MUON_OK) return rc;
    if (ld_out < n) return fail(MUON_ERR_INVALID_ARG, "the output's row stride is below its columns");
    if (tokens == 0) return MUON_OK;
    if ((rc = check_align(x, dtype_size(x_dtype), "x")) != MUON_OK) return rc;
    if ((rc = check_align(out, dtype_size(out_dtype), "out")) != MUON_OK) return rc;
    if (offsets == nullptr && fp8_token_serves(tokens, n, k)) {
        int sms = 0;
        if ((rc = op_device(&sms)) != MUON_OK) return rc;
        Fp8TokenParams p = {};
        p.x = x;
        p.w = static_cast<const uint8_t*>(w_codes);
        p.w_scale = static_cast<const uint8_t*>(w_scale);
        p.out = out;
        p.ld_x = ld_x;
        p.ldk = up128(k);
        p.ld_out = ld_out;
        p.tokens = static_cast<int>(tokens);
        p.n = n;
        p.k = k;
        p.bf16 = x_dtype == MUON_BF16;
        p.vec = reinterpret_cast<uintptr_t>(x) % 16 == 0 && ld_x * static_cast<long long>(dtype_size(x_dtype)) % 16 == 0;
        p.out_f32 = out_dtype == MUON_F32;
        const double bytes = static_cast<double>(n) * k;
        return op_launch(kOpFp8Token, 2.0 * tokens * n * k, bytes, stream, [&] { return launch_fp8_token(p, stream); });
    }
    if ((rc = check_workspace(workspace, workspace_bytes, muon_fp8_linear_workspace_bytes(tokens, n, k, offsets != nullptr))) != MUON_OK) return rc;
    const RowCodes q(workspace, tokens, k);
    rc = muon_fp8_quantize(x, x_dtype, tokens, k, ld_x, 1, nullptr, q.codes, q.scale, nullptr, nullptr, stream);
    if (rc != MUON_OK) return rc;
    return fp8_product(MUON_FP8_FORWARD, q.codes, q.scale, w_codes, w_scale, tokens, n, k, groups, offsets, out, out_dtype,
                       ld_out, kSyncEarly, stream);
}

size_t muon_fp8_linear_backward_workspace_bytes(long long tokens, int n, int k, int groups, int need_dx, int need_dw) {
    if (tokens <= 0 || n < 1 || k < 1 || groups < 1) return 0;
    size_t bytes = 0;
    if (need_dx) bytes += RowCodes(nullptr, tokens, n).bytes();
    if (need_dw) bytes += ColCodes(nullptr, tokens, n, groups).bytes() + ColCodes(nullptr, tokens, k, groups).bytes();
    return bytes;
}

int muon_fp8_linear_backward(const void* dy, int dy_dtype, long long ld_dy, const void* x, int x_dtype, long long ld_x,
                             long long tokens, const void* w_codes, const void* w_scale, int n, int k, int groups,
                             const int* offsets, void* workspace, size_t workspace_bytes, void* dx, int dx_dtype,
                             long long ld_dx, void* dw, int dw_dtype, cudaStream_t stream) {
    int rc = check_linear(dy_dtype, "dy", tokens, ld_dy, n, n, k, groups, offsets, w_codes, w_scale);
    if (rc != MUON_OK) return rc;
    if (dx == nullptr && dw == nullptr && tokens > 0) return MUON_OK;
    if (dx != nullptr) {
        if ((rc = check_dtype(dx_dtype, "dx")) != MUON_OK) return rc;
        if (ld_dx < k) return fail(MUON_ERR_INVALID_ARG, "dx's row stride is below its columns");
        if ((rc = check_align(dx, dtype_size(dx_dtype), "dx")) != MUON_OK) return rc;
    }
    if (dw != nullptr) {
        if ((rc = check_dtype(dw_dtype, "dw")) != MUON_OK || (rc = check_dtype(x_dtype, "x")) != MUON_OK) return rc;
        if (ld_x < k) return fail(MUON_ERR_INVALID_ARG, "x's row stride is below its columns");
        if ((rc = check_align(dw, dtype_size(dw_dtype), "dw")) != MUON_OK) return rc;
        if (tokens > 0 && (rc = check_align(x, dtype_size(x_dtype), "x")) != MUON_OK) return rc;
    }
    if (tokens == 0) {
        if (dw == nullptr) return MUON_OK;
        return fp8_product(MUON_FP8_GRAD_WEIGHT, nullptr, nullptr, nullptr, nullptr, 0, n, k, groups, offsets, dw, dw_dtype,
                           k, kSyncNone, stream);
    }
    if ((rc = check_align(dy, dtype_size(dy_dtype), "dy")) != MUON_OK) return rc;
    int sms = 0;
    if ((rc = op_device(&sms)) != MUON_OK) return rc;
    const size_t need = muon_fp8_linear_backward_workspace_bytes(tokens, n, k, groups, dx != nullptr, dw != nullptr);
    if ((rc = check_workspace(workspace, workspace_bytes, need)) != MUON_OK) return rc;
    char* at = static_cast<char*>(workspace);
    const RowCodes r(dx != nullptr ? at : nullptr, tokens, n);
    if (dx != nullptr) at += r.bytes();
    const ColCodes c(dw != nullptr ? at : nullptr, tokens, n, groups);
    if (dw != nullptr) at += c.bytes();
    if (dw == nullptr) {
        rc = muon_fp8_quantize(dy, dy_dtype, tokens, n, ld_dy, groups, offsets, r.codes, r.scale, nullptr, nullptr, stream);
        if (rc != MUON_OK) return rc;
        return fp8_product(MUON_FP8_GRAD_INPUT, r.codes, r.scale, w_codes, w_scale, tokens, n, k, groups, offsets, dx,
                           dx_dtype, ld_dx, kSyncEarly, stream);
    }
    const ColCodes xc(at, tokens, k, groups);
    const QuantParams pd = quantize_params(dy, dy_dtype, tokens, n, ld_dy, groups, offsets, r.codes, r.scale, c.codes, c.scale);
    const QuantParams px = quantize_params(x, x_dtype, tokens, k, ld_x, groups, offsets, nullptr, nullptr, xc.codes, xc.scale);
    const double t = static_cast<double>(tokens);
    const double dy_bytes = t * n * (dtype_size(dy_dtype) + 1.0 + (dx != nullptr)), x_bytes = t * k * (dtype_size(x_dtype) + 1.0);
    if (fp8_quantize_pairs(pd, px)) {
        rc = op_launch(kOpFp8Quantize, 0.0, dy_bytes + x_bytes, stream,
                       [&] { return launch_fp8_quantize_pair(pd, px, stream); });
    } else {
        rc = op_launch(kOpFp8Quantize, 0.0, dy_bytes, stream, [&] { return launch_fp8_quantize(pd, stream); });
        if (rc == MUON_OK)
            rc = op_launch(kOpFp8Quantize, 0.0, x_bytes, stream, [&] { return launch_fp8_quantize(px, stream); });
    }
    if (rc != MUON_OK) return rc;
    // both products need the codes alone: the second may run beside the first
    if (dx != nullptr) {
        rc = fp8_product(MUON_FP8_GRAD_INPUT, r.codes, r.scale, w_codes, w_scale, tokens, n, k, groups, offsets, dx, dx_dtype,
                         ld_dx, kSyncEarly, stream);
        if (rc != MUON_OK) return rc;
    }
    return fp8_product(MUON_FP8_GRAD_WEIGHT, c.codes, c.scale, xc.codes, xc.scale, tokens, n, k, groups, offsets, dw, dw_dtype,
                       k, dx != nullptr ? kSyncLate : kSyncEarly, stream);
}

}  // extern "C"
