// Global gradient norm over a list of tensors, and clipping by it.
//
//   norm = sqrt(sum over every element g of every tensor of g^2)
//   by   = min(1, max_norm / (norm + 1e-6)),   out = round(by * g)
//
// The step needs the norm of all gradients before any weight moves: the pages'
// recipe updates about 99.5 % of the parameters with Muon and the rest with
// AdamW ("Domyn is training a 1T-parameter MoE on Europe's Jupiter
// supercomputer, and published the recipe", table "The model and the machine"),
// and a global norm spans both.
//
// Bound by HBM: every gradient is read once for the norm (and read and written
// once more where clipping takes effect).  A tile is 32 KB of one tensor; a
// thread takes eight 16-byte vectors of it, all loaded before the first is
// used, so an SM keeps 8 x 16 bytes x its threads in flight.  A thread's 64 or
// 128 squares of a tile are summed in fp32 and added to a running double: the
// double costs one FP64 add per 64 elements and keeps the sum of billions of
// squares to a few units of 1e-9.  Where a thread's fp32 sum leaves
// [1e-30, 1e38] its squares over- or underflow, and that thread sums the same
// registers again in double, so the norm holds over the whole range of fp32.
//
// Each block writes one partial sum; the next launch adds them in a fixed
// order (no atomics: the same gradients give the same norm, bit for bit, on
// the same device).  In the clipping launch every block adds up the partials
// itself and walks the tiles from the last one back, so that what the norm
// pass read last is found in L2.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "internal.h"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = kNormTileBytes / 16 / kThreads;   // 16-byte vectors per thread and tile
constexpr float kClipEps = 1e-6f;

template <int N>
__device__ __forceinline__ int find_tensor(const NormParams<N>& p, int t) {
    int lo = 0, hi = p.h.ntensors - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.t[mid].tile0 <= t) lo = mid; else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ uint4 load_stream(const uint4* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

template <bool BF16>
__device__ __forceinline__ void add_squares(uint32_t w, float& s) {
    if (BF16) {
        const float lo = __uint_as_float(w << 16), hi = __uint_as_float(w & 0xffff0000u);
        s = fmaf(lo, lo, s);
        s = fmaf(hi, hi, s);
    } else {
        const float f = __uint_as_float(w);
        s = fmaf(f, f, s);
    }
}

template <bool BF16>
__device__ __noinline__ double exact_squares(const uint4* v, int n) {
    double s = 0.0;
    for (int i = 0; i < n; ++i) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        for (int j = 0; j < 4; ++j) {
            if (BF16) {
                const double lo = __uint_as_float(w[j] << 16), hi = __uint_as_float(w[j] & 0xffff0000u);
                s = fma(lo, lo, s);
                s = fma(hi, hi, s);
            } else {
                const double f = __uint_as_float(w[j]);
                s = fma(f, f, s);
            }
        }
    }
    return s;
}

// Sum of the squares of this thread's vectors.
template <bool BF16>
__device__ __forceinline__ double sum_vectors(const uint4 (&v)[kVecs]) {
    float a = 0.0f, b = 0.0f;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        add_squares<BF16>(v[i].x, a);
        add_squares<BF16>(v[i].y, b);
        add_squares<BF16>(v[i].z, a);
        add_squares<BF16>(v[i].w, b);
    }
    const float s = a + b;
    if (s >= 1e-30f && s <= 1e38f) return static_cast<double>(s);
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) any |= (v[i].x | v[i].y | v[i].z | v[i].w) & (BF16 ? 0x7fff7fffu : 0x7fffffffu);
    if (any == 0) return 0.0;
    uint4 copy[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) copy[i] = v[i];
    return exact_squares<BF16>(copy, kVecs);
}

template <bool BF16>
__device__ __forceinline__ float load_one(const void* g, long long e) {
    return BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(g)[e]) : static_cast<const float*>(g)[e];
}

template <bool BF16>
__device__ __forceinline__ double tile_squares(const NormTensor& T, int tile) {
    constexpr int kPer = BF16 ? 8 : 4;                              // elements per vector
    constexpr long long kTile = kNormTileBytes / (BF16 ? 2 : 4);
    const long long base = static_cast<long long>(tile) * kTile;
    if (base + kTile <= T.n && (reinterpret_cast<uintptr_t>(T.g) & 15u) == 0) {
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const char*>(T.g) +
                                                          static_cast<long long>(tile) * kNormTileBytes) + threadIdx.x;
        uint4 v[kVecs];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) v[i] = load_stream(src + i * kThreads);
        return sum_vectors<BF16>(v);
    }
    // the tensor's last tile, or a tensor that is not 16-byte aligned
    const long long end = base + kTile < T.n ? base + kTile : T.n;
    double d = 0.0;
    if ((reinterpret_cast<uintptr_t>(T.g) & 15u) == 0) {
        const long long vend = base + (end - base) / kPer * kPer;
        uint4 v[kVecs];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const long long e = base + static_cast<long long>(i * kThreads + threadIdx.x) * kPer;
            v[i] = make_uint4(0, 0, 0, 0);
            if (e < vend) v[i] = *reinterpret_cast<const uint4*>(static_cast<const char*>(T.g) + e * (BF16 ? 2 : 4));
        }
        d = sum_vectors<BF16>(v);
        const long long e = vend + threadIdx.x;
        if (e < end) {
            const double f = load_one<BF16>(T.g, e);
            d = fma(f, f, d);
        }
    } else {
        float s = 0.0f;
#pragma unroll 8
        for (long long e = base + threadIdx.x; e < end; e += kThreads) {
            const float f = load_one<BF16>(T.g, e);
            s = fmaf(f, f, s);
        }
        if (s >= 1e-30f && s <= 1e38f) return static_cast<double>(s);
        for (long long e = base + threadIdx.x; e < end; e += kThreads) {
            const double f = load_one<BF16>(T.g, e);
            d = fma(f, f, d);
        }
    }
    return d;
}

// Sum over the block, in a fixed order; the result in every thread.
__device__ __forceinline__ double block_sum(double d) {
    __shared__ double part[kThreads / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = d;
    __syncthreads();
    double s = 0.0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) s += part[w];
    return s;
}

__device__ __forceinline__ float total_norm(const NormHead& h) {
    double d = 0.0;
    for (int i = threadIdx.x; i < h.npartials; i += kThreads) d += h.partials[i];
    return static_cast<float>(sqrt(block_sum(d)));
}

template <int N>
__global__ void __launch_bounds__(kThreads) k_grad_norm(const __grid_constant__ NormParams<N> p) {
    asm volatile("griddepcontrol.launch_dependents;");
    double d = 0.0;
    for (int t = blockIdx.x; t < p.h.total_tiles; t += gridDim.x) {
        const NormTensor& T = p.t[find_tensor(p, t)];
        d += T.bf16 ? tile_squares<true>(T, t - T.tile0) : tile_squares<false>(T, t - T.tile0);
    }
    const double s = block_sum(d);
    if (threadIdx.x == 0) p.h.partials[blockIdx.x] = s;
}

__global__ void __launch_bounds__(kThreads) k_grad_norm_finish(const __grid_constant__ NormHead h) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const float norm = total_norm(h);
    if (threadIdx.x == 0) *h.norm = norm;
}

template <bool BF16>
__device__ __forceinline__ uint4 scale_vector(uint4 v, float by) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (BF16) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(__fmul_rn(__uint_as_float(w[j] << 16), by),
                                                           __fmul_rn(__uint_as_float(w[j] & 0xffff0000u), by));
            w[j] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
            w[j] = __float_as_uint(__fmul_rn(__uint_as_float(w[j]), by));
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool BF16>
__device__ __forceinline__ void scale_one(const NormTensor& T, long long e, float by) {
    const float f = __fmul_rn(load_one<BF16>(T.g, e), by);
    if (BF16) static_cast<__nv_bfloat16*>(T.out)[e] = __float2bfloat16_rn(f);
    else static_cast<float*>(T.out)[e] = f;
}

template <bool BF16>
__device__ __forceinline__ void tile_scale(const NormTensor& T, int tile, float by) {
    constexpr int kPer = BF16 ? 8 : 4;
    constexpr long long kTile = kNormTileBytes / (BF16 ? 2 : 4);
    const long long base = static_cast<long long>(tile) * kTile;
    const bool aligned = ((reinterpret_cast<uintptr_t>(T.g) | reinterpret_cast<uintptr_t>(T.out)) & 15u) == 0;
    if (base + kTile <= T.n && aligned) {
        const long long off = static_cast<long long>(tile) * kNormTileBytes;
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const char*>(T.g) + off) + threadIdx.x;
        uint4* dst = reinterpret_cast<uint4*>(static_cast<char*>(T.out) + off) + threadIdx.x;
        uint4 v[kVecs];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) v[i] = load_stream(src + i * kThreads);
#pragma unroll
        for (int i = 0; i < kVecs; ++i) __stcs(dst + i * kThreads, scale_vector<BF16>(v[i], by));   // not to push out what is still to be read
        return;
    }
    const long long end = base + kTile < T.n ? base + kTile : T.n;
    const long long vend = aligned ? base + (end - base) / kPer * kPer : base;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const long long e = base + static_cast<long long>(i * kThreads + threadIdx.x) * kPer;
        if (e < vend) {
            const long long off = e * (BF16 ? 2 : 4);
            *reinterpret_cast<uint4*>(static_cast<char*>(T.out) + off) =
                scale_vector<BF16>(*reinterpret_cast<const uint4*>(static_cast<const char*>(T.g) + off), by);
        }
    }
    for (long long e = vend + threadIdx.x; e < end; e += kThreads) scale_one<BF16>(T, e, by);
}

template <int N>
__global__ void __launch_bounds__(kThreads) k_grad_clip(const __grid_constant__ NormParams<N> p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const float norm = total_norm(p.h);
    if (p.h.norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *p.h.norm = norm;
    const float q = __fdiv_rn(p.h.max_norm, __fadd_rn(norm, kClipEps));
    const float by = q > 1.0f ? 1.0f : q;      // a NaN norm makes every gradient NaN, as the product says
    if (p.h.in_place && by == 1.0f) return;    // nothing to change
    for (int i = blockIdx.x; i < p.h.total_tiles; i += gridDim.x) {
        const int t = p.h.total_tiles - 1 - i;
        const NormTensor& T = p.t[find_tensor(p, t)];
        if (T.bf16) tile_scale<true>(T, t - T.tile0, by);
        else tile_scale<false>(T, t - T.tile0, by);
    }
}

// Launch that may start while the launch before it on the stream drains; its
// griddepcontrol.wait holds it until that launch's writes are visible.
template <class... A>
cudaError_t launch_after(void (*k)(A...), int grid, cudaStream_t s, const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, k, args...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

// One block per resident slot, no more than there are tiles or partial slots.
int norm_grid(int total_tiles, int sms) {
    const int cap = sms * 6 < kNormMaxBlocks ? sms * 6 : kNormMaxBlocks;
    return total_tiles < cap ? (total_tiles > 0 ? total_tiles : 1) : cap;
}

template <int N>
cudaError_t launch_grad_norm(const NormParams<N>& p, int grid, cudaStream_t s) {
    k_grad_norm<N><<<grid, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <int N>
cudaError_t launch_grad_clip(const NormParams<N>& p, int grid, bool first, cudaStream_t s) {
    if (first) return launch_after(k_grad_clip<N>, grid, s, p);
    k_grad_clip<N><<<grid, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_grad_norm_finish(const NormHead& h, cudaStream_t s) { return launch_after(k_grad_norm_finish, 1, s, h); }

template cudaError_t launch_grad_norm<kNormFewTensors>(const NormParams<kNormFewTensors>&, int, cudaStream_t);
template cudaError_t launch_grad_norm<kNormMaxTensors>(const NormParams<kNormMaxTensors>&, int, cudaStream_t);
template cudaError_t launch_grad_clip<kNormFewTensors>(const NormParams<kNormFewTensors>&, int, bool, cudaStream_t);
template cudaError_t launch_grad_clip<kNormMaxTensors>(const NormParams<kNormMaxTensors>&, int, bool, cudaStream_t);

}  // namespace muon
