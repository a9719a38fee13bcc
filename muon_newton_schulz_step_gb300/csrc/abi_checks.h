// Checks of arguments that the entry points of the operators share.
#pragma once

#include <cstdarg>
#include <cstddef>
#include <cstdint>
#include <cstdio>

#include "internal.h"
#include "muon.h"

namespace muon {

inline int fail(int status, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return set_last_error(status, buf);
}

inline int check_dtype(int dtype, const char* what) {
    if (dtype != MUON_BF16 && dtype != MUON_F32) return fail(MUON_ERR_INVALID_ARG, "%s: unknown dtype %d", what, dtype);
    return MUON_OK;
}

inline size_t dtype_size(int dtype) { return dtype == MUON_F32 ? 4 : 2; }

inline int check_align(const void* p, size_t align, const char* what) {
    if (p == nullptr) return fail(MUON_ERR_INVALID_ARG, "%s is NULL", what);
    if (reinterpret_cast<uintptr_t>(p) % align != 0)
        return fail(MUON_ERR_INVALID_ARG, "%s is not %zu-byte aligned", what, align);
    return MUON_OK;
}

constexpr long long kMaxRows = 1ll << 30;

inline int check_groups(long long tokens, int groups, const int* offsets) {
    if (tokens < 0 || tokens > kMaxRows) return fail(MUON_ERR_INVALID_ARG, "rows is %lld (0 to 2^30)", tokens);
    if (groups < 1 || groups > kFp8MaxGroups)
        return fail(MUON_ERR_INVALID_ARG, "groups is %d (1 to %d)", groups, kFp8MaxGroups);
    if (groups > 1 && offsets == nullptr) return fail(MUON_ERR_INVALID_ARG, "offsets is NULL with %d groups", groups);
    if (offsets != nullptr && reinterpret_cast<uintptr_t>(offsets) % 4 != 0)
        return fail(MUON_ERR_INVALID_ARG, "offsets is not 4-byte aligned");
    return MUON_OK;
}

inline int check_dim(long long n, const char* what) {
    if (n < 1 || n > (1ll << 24)) return fail(MUON_ERR_INVALID_ARG, "%s is %lld (1 to 2^24)", what, n);
    return MUON_OK;
}

inline long long up128(long long n) { return (n + 127) / 128 * 128; }

inline int check_workspace(const void* ws, size_t have, size_t need) {
    if (need == 0) return MUON_OK;
    const int rc = check_align(ws, 16, "workspace");
    if (rc != MUON_OK) return rc;
    if (have < need) return fail(MUON_ERR_OOM, "workspace has %zu bytes; %zu are needed", have, need);
    return MUON_OK;
}

}  // namespace muon
