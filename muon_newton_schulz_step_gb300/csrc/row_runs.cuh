// Runs of E consecutive elements of a row, bf16 or fp32, as loaded and stored, for rows that
// start anywhere.  E is 16 bytes' worth where a kernel meets one type (a warp's vectors then lie
// side by side), and 8 where it meets both.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

namespace muon {

template <typename T, int E>
struct RowRun {
    static constexpr int kWords = static_cast<int>(sizeof(T)) * E / 4;
    uint32_t w[kWords];
};

// The elements of a matrix that may be read: [begin, end).
struct Extent {
    const char *begin, *end;
};

template <typename T>
__device__ __forceinline__ Extent extent_of(const void* p, long long rows, long long ld, long long cols) {
    const char* b = static_cast<const char*>(p);
    return {b, b + ((rows - 1) * ld + cols) * static_cast<long long>(sizeof(T))};
}

// ONCE: leave the first level alone.
template <bool ONCE>
__device__ __forceinline__ uint4 load_16(const char* p) {
    uint4 v;
    if (ONCE)
        asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "l"(p));
    else
        asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// 16 aligned bytes of which some lie outside of `in`: those read as zeros.
template <typename T>
__device__ __noinline__ uint4 load_edge(const char* p, Extent in) {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 16; i += static_cast<int>(sizeof(T))) {
        if (p + i < in.begin || p + i >= in.end) continue;
        if (sizeof(T) == 4) w[i / 4] = *reinterpret_cast<const uint32_t*>(p + i);
        else w[i / 4] |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(p + i)) << (8 * (i & 2));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The run that starts `off` bytes after the first of `w`.
template <typename T, int E>
__device__ __forceinline__ RowRun<T, E> shifted(uint32_t (&w)[RowRun<T, E>::kWords + 4], int off) {
    constexpr int kWords = RowRun<T, E>::kWords;
    RowRun<T, E> r;
    if (off & 8) {
#pragma unroll
        for (int i = 0; i < kWords + 2; ++i) w[i] = w[i + 2];
    }
    if (off & 4) {
#pragma unroll
        for (int i = 0; i < kWords + 1; ++i) w[i] = w[i + 1];
    }
#pragma unroll
    for (int i = 0; i < kWords; ++i)
        r.w[i] = sizeof(T) == 4 ? w[i] : __funnelshift_r(w[i], w[i + 1], 8 * (off & 2));
    return r;
}

// E elements from p on.  SHIFT: p is aligned to its elements alone; the 16-byte vectors
// around them are loaded and shifted (all lanes of a warp by the same amount).
template <typename T, int E, bool SHIFT, bool ONCE = false>
__device__ __forceinline__ RowRun<T, E> load_row(const T* p, Extent in) {
    constexpr int kWords = RowRun<T, E>::kWords;
    RowRun<T, E> r;
    const char* at = reinterpret_cast<const char*>(p);
    const int off = SHIFT ? static_cast<int>(reinterpret_cast<uintptr_t>(at) & 15) : 0;
    if (!SHIFT || off == 0) {
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i) {
            const uint4 v = load_16<ONCE>(at + 16 * i);
            r.w[4 * i] = v.x, r.w[4 * i + 1] = v.y, r.w[4 * i + 2] = v.z, r.w[4 * i + 3] = v.w;
        }
        return r;
    }
    uint32_t w[kWords + 4];
#pragma unroll
    for (int i = 0; i <= kWords / 4; ++i) {
        const char* q = at - off + 16 * i;
        const uint4 v = q >= in.begin && q + 16 <= in.end ? load_16<false>(q) : load_edge<T>(q, in);
        w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
    return shifted<T, E>(w, off);
}

// The same in two parts, for warps whose lanes take runs side by side: each lane loads the
// vectors at and below its run, and gets what its run has beyond them from the next lane.  The
// last lane's run stays unfinished: such a warp covers kShared runs.
constexpr int kShared = 31;

template <typename T, int E>
__device__ __forceinline__ RowRun<T, E> load_below(const T* p, Extent in) {
    RowRun<T, E> r;
    const char* at = reinterpret_cast<const char*>(p);
    at -= reinterpret_cast<uintptr_t>(at) & 15;
#pragma unroll
    for (int i = 0; i < RowRun<T, E>::kWords / 4; ++i) {
        const char* q = at + 16 * i;
        const uint4 v = q >= in.begin && q + 16 <= in.end ? load_16<true>(q) : load_edge<T>(q, in);
        r.w[4 * i] = v.x, r.w[4 * i + 1] = v.y, r.w[4 * i + 2] = v.z, r.w[4 * i + 3] = v.w;
    }
    return r;
}

// `off`: bytes of a run's start past its vector, the same in all lanes.
template <typename T, int E>
__device__ __forceinline__ RowRun<T, E> finished(const RowRun<T, E>& r, int off) {
    constexpr int kWords = RowRun<T, E>::kWords;
    if (off == 0) return r;
    uint32_t w[kWords + 4];
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = r.w[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[kWords + i] = __shfl_down_sync(0xffffffffu, r.w[i], 1);
    return shifted<T, E>(w, off);
}

// To 16 aligned bytes.
template <typename T, int E>
__device__ __forceinline__ void store_row(T* p, const RowRun<T, E>& r) {
#pragma unroll
    for (int i = 0; i < RowRun<T, E>::kWords / 4; ++i)
        reinterpret_cast<uint4*>(p)[i] = make_uint4(r.w[4 * i], r.w[4 * i + 1], r.w[4 * i + 2], r.w[4 * i + 3]);
}

template <typename T, int E>
__device__ __forceinline__ float element(const RowRun<T, E>& r, int i) {
    if (sizeof(T) == 4) return __uint_as_float(r.w[i]);
    return __uint_as_float((i & 1) ? r.w[i >> 1] & 0xffff0000u : r.w[i >> 1] << 16);
}

template <typename T, int E>
__device__ __forceinline__ RowRun<T, E> rounded(const float (&v)[E]) {
    RowRun<T, E> r;
#pragma unroll
    for (int i = 0; i < RowRun<T, E>::kWords; ++i) {
        if constexpr (sizeof(T) == 4) {
            r.w[i] = __float_as_uint(v[i]);
        } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            r.w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
    return r;
}

// A row of `cols` elements as the runs that lie on 16 bytes, with up to seven elements before and after them.
template <typename T, int E>
struct RowSpan {
    int head, runs, tail;
    __device__ __forceinline__ RowSpan(const T* row, long long cols) {
        const int off = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15) / static_cast<int>(sizeof(T));
        const int to = off == 0 ? 0 : 16 / static_cast<int>(sizeof(T)) - off;
        head = static_cast<int>(to < cols ? to : cols);
        runs = static_cast<int>(cols - head) / E;
        tail = static_cast<int>(cols - head) - E * runs;
    }
};

}  // namespace muon
