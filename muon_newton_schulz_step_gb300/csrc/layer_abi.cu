// C ABI of the operators between an expert layer's routing and its result, and of
// the products with weights of 4 bits (include/muon.h).  Validation and launch
// parameters only; nothing here allocates, keeps state or synchronises.
#include <cuda_runtime.h>

#include "abi_checks.h"
#include "internal.h"
#include "muon.h"

namespace muon {
namespace {

// The order of `tokens` x `top_k` entries over `groups` experts.
int check_order(RowsParams& p, long long tokens, int top_k, const int* place, const int* offsets, int groups) {
    if (tokens < 0 || top_k < 1 || top_k > kRowsMaxTopK)
        return fail(MUON_ERR_INVALID_ARG, "tokens is %lld, top_k is %d (1 to %d)", tokens, top_k, kRowsMaxTopK);
    if (tokens > kMaxRows / top_k) return fail(MUON_ERR_INVALID_ARG, "%lld tokens x %d exceed 2^30 rows", tokens, top_k);
    if (groups < 1 || groups > kSortMaxExperts)
        return fail(MUON_ERR_INVALID_ARG, "groups is %d (1 to %d)", groups, kSortMaxExperts);
    p.tokens = tokens;
    p.top_k = top_k;
    p.rows = static_cast<int>(tokens * top_k);
    p.groups = groups;
    p.place = place;
    p.offsets = offsets;
    if (tokens == 0) return MUON_OK;
    const int rc = check_align(place, 4, "place");
    return rc != MUON_OK ? rc : check_align(offsets, 4, "offsets");
}

int check_matrix(const void* p, int dtype, long long ld, long long cols, const char* what) {
    int rc = check_dtype(dtype, what);
    if (rc != MUON_OK) return rc;
    if (ld < cols) return fail(MUON_ERR_INVALID_ARG, "%s's row stride is below its columns", what);
    return check_align(p, dtype_size(dtype), what);
}

int check_block(int block) {
    if (block != 32 && block != 64 && block != 128) return fail(MUON_ERR_INVALID_ARG, "block is %d (32, 64 or 128)", block);
    return MUON_OK;
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

size_t muon_sort_tokens_workspace_bytes(long long entries, int experts) {
    if (entries < 0 || entries > kMaxRows || experts < 1 || experts > kSortMaxExperts) return 0;
    return static_cast<size_t>(token_sort_blocks(entries)) * (experts + 1) * sizeof(int);
}

int muon_sort_tokens(const int* chosen, long long entries, int first, int experts, void* workspace, size_t workspace_bytes,
                     int* order, int* place, int* offsets, cudaStream_t stream) {
    if (entries < 0 || entries > kMaxRows) return fail(MUON_ERR_INVALID_ARG, "entries is %lld (0 to 2^30)", entries);
    if (experts < 1 || experts > kSortMaxExperts)
        return fail(MUON_ERR_UNSUPPORTED, "experts is %d (1 to %d)", experts, kSortMaxExperts);
    if (first < 0 || first > (1 << 30)) return fail(MUON_ERR_INVALID_ARG, "first is %d (0 to 2^30)", first);
    int rc = check_align(offsets, 4, "offsets");
    if (rc != MUON_OK) return rc;
    if (entries > 0) {
        if ((rc = check_align(chosen, 4, "chosen")) != MUON_OK || (rc = check_align(order, 4, "order")) != MUON_OK ||
            (rc = check_align(place, 4, "place")) != MUON_OK)
            return rc;
    }
    if ((rc = check_workspace(workspace, workspace_bytes, muon_sort_tokens_workspace_bytes(entries, experts))) != MUON_OK)
        return rc;
    int sms = 0;
    if ((rc = op_device(&sms)) != MUON_OK) return rc;
    SortParams p = {};
    p.chosen = chosen;
    p.order = order;
    p.place = place;
    p.offsets = offsets;
    p.table = static_cast<int*>(workspace);
    p.entries = static_cast<int>(entries);
    p.first = first;
    p.experts = experts;
    return op_launch(kOpTokenSort, 0.0, 12.0 * entries, stream, [&] { return launch_token_sort(p, stream); });
}

int muon_dispatch_tokens(const void* x, int dtype, long long tokens, long long cols, long long ld_x, int top_k,
                         const int* place, const int* offsets, int groups, void* out, long long ld_out,
                         cudaStream_t stream) {
    RowsParams p = {};
    int rc = check_dtype(dtype, "x");
    if (rc != MUON_OK) return rc;
    if ((rc = check_order(p, tokens, top_k, place, offsets, groups)) != MUON_OK) return rc;
    if ((rc = check_dim(cols, "cols")) != MUON_OK) return rc;
    if (tokens == 0) return MUON_OK;
    if ((rc = check_matrix(x, dtype, ld_x, cols, "x")) != MUON_OK) return rc;
    if ((rc = check_matrix(out, dtype, ld_out, cols, "out")) != MUON_OK) return rc;
    int sms = 0;
    if ((rc = op_device(&sms)) != MUON_OK) return rc;
    p.x = x;
    p.out = out;
    p.ld_x = ld_x;
    p.ld_out = ld_out;
    p.cols = cols;
    p.x_bf16 = dtype == MUON_BF16;
    const double bytes = static_cast<double>(tokens) * (1 + top_k) * cols * dtype_size(dtype);
    return op_launch(kOpDispatch, 0.0, bytes, stream, [&] { return launch_dispatch(p, stream); });
}

int muon_combine_tokens(const void* y, int y_dtype, long long ld_y, long long tokens, long long cols, int top_k,
                        const int* place, const int* offsets, int groups, const float* weights, void* out, int out_dtype,
                        long long ld_out, cudaStream_t stream) {
    RowsParams p = {};
    int rc = check_dtype(y_dtype, "y");
    if (rc != MUON_OK) return rc;
    if ((rc = check_order(p, tokens, top_k, place, offsets, groups)) != MUON_OK) return rc;
    if ((rc = check_dim(cols, "cols")) != MUON_OK) return rc;
    if (tokens == 0) return check_dtype(out_dtype, "out");
    if ((rc = check_matrix(y, y_dtype, ld_y, cols, "y")) != MUON_OK) return rc;
    if ((rc = check_matrix(out, out_dtype, ld_out, cols, "out")) != MUON_OK) return rc;
    if (weights != nullptr && (rc = check_align(weights, 4, "weights")) != MUON_OK) return rc;
    int sms = 0;
    if ((rc = op_device(&sms)) != MUON_OK) return rc;
    p.x = y;
    p.out = out;
    p.weights = weights;
    p.ld_x = ld_y;
    p.ld_out = ld_out;
    p.cols = cols;
    p.x_bf16 = y_dtype == MUON_BF16;
    p.out_bf16 = out_dtype == MUON_BF16;
    const double n = static_cast<double>(tokens) * cols;
    return op_launch(kOpCombine, 2.0 * top_k * n, n * (top_k * dtype_size(y_dtype) + dtype_size(out_dtype)), stream,
                     [&] { return launch_combine(p, stream); });
}

int muon_combine_tokens_backward(const void* d, int d_dtype, long long ld_d, const void* y, int y_dtype, long long ld_y,
                                 long long tokens, long long cols, int top_k, const int* place, const int* offsets,
                                 int groups, const float* weights, void* dy, long long ld_dy, float* d_weights,
                                 cudaStream_t stream) {
    RowsParams p = {};
    int rc = check_dtype(d_dtype, "d");
    if (rc != MUON_OK) return rc;
    if ((rc = check_dtype(y_dtype, "y")) != MUON_OK) return rc;
    if ((rc = check_order(p, tokens, top_k, place, offsets, groups)) != MUON_OK) return rc;
    if ((rc = check_dim(cols, "cols")) != MUON_OK) return rc;
    if (tokens == 0 || (dy == nullptr && d_weights == nullptr)) return MUON_OK;
    if ((rc = check_matrix(d, d_dtype, ld_d, cols, "d")) != MUON_OK) return rc;
    if (dy != nullptr && (rc = check_matrix(dy, y_dtype, ld_dy, cols, "dy")) != MUON_OK) return rc;
    if (d_weights != nullptr) {
        if ((rc = check_align(d_weights, 4, "d_weights")) != MUON_OK) return rc;
        if ((rc = check_matrix(y, y_dtype, ld_y, cols, "y")) != MUON_OK) return rc;
        if (dy == y) return fail(MUON_ERR_INVALID_ARG, "dy must not be y");
    }
    if (weights != nullptr && (rc = check_align(weights, 4, "weights")) != MUON_OK) return rc;
    int sms = 0;
    if ((rc = op_device(&sms)) != MUON_OK) return rc;
    p.x = y;
    p.d = d;
    p.out = dy;
    p.dw = d_weights;
    p.weights = weights;
    p.ld_x = ld_y;
    p.ld_d = ld_d;
    p.ld_out = ld_dy;
    p.cols = cols;
    p.x_bf16 = y_dtype == MUON_BF16;
    p.d_bf16 = d_dtype == MUON_BF16;
    const double n = static_cast<double>(tokens) * cols;
    const double bytes = n * (dtype_size(d_dtype) + ((dy != nullptr) + (d_weights != nullptr)) * top_k * dtype_size(y_dtype));
    return op_launch(kOpCombineGrad, 3.0 * top_k * n, bytes, stream, [&] { return launch_combine_backward(p, stream); });
}

int muon_swiglu(const void* gate, long long ld_gate, const void* up, long long ld_up, int dtype, long long rows,
                long long cols, void* out, long long ld_out, cudaStream_t stream) {
    int rc = check_dtype(dtype, "gate");
    if (rc != MUON_OK) return rc;
    if (rows < 0 || rows > kMaxRows) return fail(MUON_ERR_INVALID_ARG, "rows is %lld (0 to 2^30)", rows);
    if ((rc = check_dim(cols, "cols")) != MUON_OK) return rc;
    if (rows == 0) return MUON_OK;
    if ((rc = check_matrix(gate, dtype, ld_gate, cols, "gate")) != MUON_OK) return rc;
    if ((rc = check_matrix(up, dtype, ld_up, cols, "up")) != MUON_OK) return rc;
    if ((rc = check_matrix(out, dtype, ld_out, cols, "out")) != MUON_OK) return rc;
    int sms = 0;
    if ((rc = op_device(&sms)) != MUON_OK) return rc;
    SwigluParams p = {};
    p.gate = gate;
    p.up = up;
    p.out = out;
    p.ld_gate = ld_gate;
    p.ld_up = ld_up;
    p.ld_out = ld_out;
    p.rows = rows;
    p.cols = cols;
    p.bf16 = dtype == MUON_BF16;
    const double n = static_cast<double>(rows) * cols;
    return op_launch(kOpSwiglu, 5.0 * n, 3.0 * n * dtype_size(dtype), stream, [&] { return launch_swiglu(p, stream); });
}

int muon_swiglu_backward(const void* d, long long ld_d, const void* gate, long long ld_gate, const void* up, long long ld_up,
                         int dtype, long long rows, long long cols, void* d_gate, long long ld_dgate, void* d_up,
                         long long ld_dup, cudaStream_t stream) {
    int rc = check_dtype(dtype, "gate");
    if (rc != MUON_OK) return rc;
    if (rows < 0 || rows > kMaxRows) return fail(MUON_ERR_INVALID_ARG, "rows is %lld (0 to 2^30)", rows);
    if ((rc = check_dim(cols, "cols")) != MUON_OK) return rc;
    if (rows == 0) return MUON_OK;
    if ((rc = check_matrix(d, dtype, ld_d, cols, "d")) != MUON_OK) return rc;
    if ((rc = check_matrix(gate, dtype, ld_gate, cols, "gate")) != MUON_OK) return rc;
    if ((rc = check_matrix(up, dtype, ld_up, cols, "up")) != MUON_OK) return rc;
    if ((rc = check_matrix(d_gate, dtype, ld_dgate, cols, "d_gate")) != MUON_OK) return rc;
    if ((rc = check_matrix(d_up, dtype, ld_dup, cols, "d_up")) != MUON_OK) return rc;
    int sms = 0;
    if ((rc = op_device(&sms)) != MUON_OK) return rc;
    SwigluParams p = {};
    p.gate = gate;
    p.up = up;
    p.d = d;
    p.d_gate = d_gate;
    p.d_up = d_up;
    p.ld_gate = ld_gate;
    p.ld_up = ld_up;
    p.ld_d = ld_d;
    p.ld_dgate = ld_dgate;
    p.ld_dup = ld_dup;
    p.rows = rows;
    p.cols = cols;
    p.bf16 = dtype == MUON_BF16;
    const double n = static_cast<double>(rows) * cols;
    return op_launch(kOpSwigluGrad, 11.0 * n, 5.0 * n * dtype_size(dtype), stream, [&] { return launch_swiglu(p, stream); });
}

int muon_int4_quantize_weight(const void* w, int dtype, int batch, long long rows, long long cols, int block, void* codes,
                              void* scale, cudaStream_t stream) {
    int rc = check_dtype(dtype, "w");
    if (rc != MUON_OK) return rc;
    if (batch < 0 || batch > kFp8MaxGroups) return fail(MUON_ERR_INVALID_ARG, "batch is %d (0 to %d)", batch, kFp8MaxGroups);
    if ((rc = check_dim(rows, "rows")) != MUON_OK || (rc = check_dim(cols, "cols")) != MUON_OK) return rc;
    if ((rc = check_block(block)) != MUON_OK) return rc;
    if (batch == 0) return MUON_OK;
    if ((rc = check_align(w, dtype_size(dtype), "w")) != MUON_OK) return rc;
    if ((rc = check_align(codes, 16, "codes")) != MUON_OK) return rc;
    if ((rc = check_align(scale, 2, "scale")) != MUON_OK) return rc;
    int sms = 0;
    if ((rc = op_device(&sms)) != MUON_OK) return rc;
    Int4QuantParams p = {};
    p.w = w;
    p.codes = static_cast<uint8_t*>(codes);
    p.scale = static_cast<__nv_bfloat16*>(scale);
    p.batch = batch;
    p.rows = rows;
    p.cols = cols;
    p.kblocks = up128(cols) / 128;
    p.block = block;
    p.bf16 = dtype == MUON_BF16;
    const double n = static_cast<double>(batch) * rows * cols;
    return op_launch(kOpInt4Quantize, 0.0, n * (dtype_size(dtype) + 0.5 + 2.0 / block), stream,
                     [&] { return launch_int4_quantize(p, stream); });
}

int muon_int4_linear(const void* x, int x_dtype, long long tokens, long long ld_x, const void* w_codes, const void* w_scale,
                     int block, int n, int k, int groups, const int* offsets, void* out, int out_dtype, long long ld_out,
                     cudaStream_t stream) {
    int rc = check_dtype(x_dtype, "x");
    if (rc != MUON_OK) return rc;
    if ((rc = check_dtype(out_dtype, "out")) != MUON_OK) return rc;
    if ((rc = check_groups(tokens, groups, offsets)) != MUON_OK) return rc;
    if ((rc = check_dim(n, "n")) != MUON_OK || (rc = check_dim(k, "k")) != MUON_OK) return rc;
    if ((rc = check_block(block)) != MUON_OK) return rc;
    if ((rc = check_align(w_codes, 16, "w_codes")) != MUON_OK) return rc;
    if ((rc = check_align(w_scale, 2, "w_scale")) != MUON_OK) return rc;
    if (tokens == 0) return MUON_OK;
    if ((rc = check_matrix(x, x_dtype, ld_x, k, "x")) != MUON_OK) return rc;
    if ((rc = check_matrix(out, out_dtype, ld_out, n, "out")) != MUON_OK) return rc;
    int sms = 0;
    if ((rc = op_device(&sms)) != MUON_OK) return rc;
    Int4Params p = {};
    p.x = x;
    p.w = static_cast<const uint8_t*>(w_codes);
    p.scale = static_cast<const __nv_bfloat16*>(w_scale);
    p.out = out;
    p.offsets = offsets;
    p.ld_x = ld_x;
    p.ldw = up128(k) / 2;
    p.ld_out = ld_out;
    p.tokens = static_cast<int>(tokens);
    p.n = n;
    p.k = k;
    p.kblocks = static_cast<int>(up128(k) / 128);
    p.groups = groups;
    p.block = block;
    p.w_batch = n * p.ldw;
    p.scale_batch = static_cast<long long>(p.kblocks) * (128 / block) * n;
    p.x_bf16 = x_dtype == MUON_BF16;
    p.out_f32 = out_dtype == MUON_F32;
    p.vec = reinterpret_cast<uintptr_t>(x) % 16 == 0 && ld_x * static_cast<long long>(dtype_size(x_dtype)) % 16 == 0;
    p.pairs = n % 2 == 0 && reinterpret_cast<uintptr_t>(w_scale) % 4 == 0;
    const double some = groups < tokens ? groups : static_cast<double>(tokens);
    const double bytes = some * n * k * (0.5 + 2.0 / block);
    return op_launch(kOpInt4Linear, 2.0 * tokens * n * k, bytes, stream, [&] { return launch_int4_linear(p, sms, stream); });
}

}  // extern "C"
