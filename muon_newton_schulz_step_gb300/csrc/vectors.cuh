// Runs of V consecutive elements of a row, bf16 or fp32, as fp32 in registers.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

namespace muon {

// As loaded and stored: words of up to 16 bytes, as wide as V elements are.
template <typename T, int V>
struct alignas(sizeof(T) * V >= 16 ? 16 : sizeof(T) * V) Run {
    T v[V];
};

// Loads leave the first level alone: what these kernels read, they read once.
template <typename T, int V>
__device__ __forceinline__ Run<T, V> load_run(const T* p) {
    constexpr int kBytes = sizeof(T) * V;
    Run<T, V> r;
    if constexpr (kBytes >= 16) {
        uint4* w = reinterpret_cast<uint4*>(&r);
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i)
            asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w)
                         : "l"(reinterpret_cast<const uint4*>(p) + i));
    } else {
        r = *reinterpret_cast<const Run<T, V>*>(p);
    }
    return r;
}

template <typename T, int V>
__device__ __forceinline__ void store_run(T* p, const Run<T, V>& r) {
    constexpr int kBytes = sizeof(T) * V;
    if constexpr (kBytes >= 16) {
        const uint4* w = reinterpret_cast<const uint4*>(&r);
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i) reinterpret_cast<uint4*>(p)[i] = w[i];
    } else {
        *reinterpret_cast<Run<T, V>*>(p) = r;
    }
}

__device__ __forceinline__ float as_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float as_float(float v) { return v; }
template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ float from_float<float>(float v) {
    return v;
}

// The widest run, of at most `most` elements, that every access of a call allows: `cols` in a
// row, row strides and addresses in elements of `size` bytes.
struct RunWidth {
    int v;
    RunWidth(long long cols, int most) : v(most) { fit(cols); }
    void fit(long long n) {
        while (v > 1 && n % v != 0) v >>= 1;
    }
    void array(const void* p, long long ld, int size) {
        fit(ld);
        while (v > 1 && reinterpret_cast<uintptr_t>(p) % (v * size >= 16 ? 16 : v * size) != 0) v >>= 1;
    }
};

}  // namespace muon
