// Tokens' rows on their way to the experts and, weighted, back.
//
//   dispatch   out[place[t, j]] = x[t]
//   combine    out[t] = sum over j of weights[t, j] y[place[t, j]]
//   backward   dy[place[t, j]] = weights[t, j] d[t],  dw[t, j] = <d[t], y[place[t, j]]>
//
// over entries whose place lies in [offsets[0], offsets[groups]); rows of the other
// places hold no expert's work: they are written as zeros and never read, whatever
// they hold.  All three walk the tokens and not the sorted rows: a token's row is then
// read (or written) once for all its entries, where a walk over the sorted rows
// would read it top_k times, from memory once the tokens outgrow L2.  The rows
// themselves are long (6144 bf16 are 12 KB), so their scattered places cost nothing.
// Sums are fp32 fused multiply-adds in the order of j, so that a call's result has
// one value whatever the order of the blocks.
//
// Bound by memory.  [8192 tokens x 8 x 6144 bf16; see the figures at each kernel]
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "vectors.cuh"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Lane j's place of a token's entry j; whether it holds a row of an expert is in `held`.
struct Entries {
    int place;
    unsigned held;
};

__device__ __forceinline__ Entries entries_of(const RowsParams& p, long long token) {
    const int lane = threadIdx.x & 31;
    Entries e;
    e.place = lane < p.top_k ? __ldg(p.place + token * p.top_k + lane) : -1;
    const int lo = max(0, __ldg(p.offsets)), hi = min(p.rows, __ldg(p.offsets + p.groups));
    e.held = __ballot_sync(0xffffffffu, e.place >= lo && e.place < hi);
    return e;
}

// A warp takes U x 32 runs of one token's row.
template <typename T, int V, int U>
__global__ void __launch_bounds__(kThreads) k_dispatch(const RowsParams p) {
    const int lane = threadIdx.x & 31;
    const long long item = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const long long token = item / p.parts;
    if (token >= p.tokens) return;
    const int run0 = static_cast<int>(item - token * p.parts) * (32 * U) + lane;
    const Entries e = entries_of(p, token);
    const T* x = static_cast<const T*>(p.x) + token * p.ld_x;
    Run<T, V> r[U] = {};
    if (e.held != 0u) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (run0 + 32 * u < p.runs) r[u] = load_run<T, V>(x + static_cast<long long>(run0 + 32 * u) * V);
    }
    for (int j = 0; j < p.top_k; ++j) {
        const int place = __shfl_sync(0xffffffffu, e.place, j);
        if (place < 0 || place >= p.rows) continue;
        const bool held = (e.held >> j) & 1u;
        T* out = static_cast<T*>(p.out) + place * p.ld_out;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (run0 + 32 * u >= p.runs) break;
            store_run<T, V>(out + static_cast<long long>(run0 + 32 * u) * V, held ? r[u] : Run<T, V>{});
        }
    }
}

template <typename T, typename O, int V, int U>
__global__ void __launch_bounds__(kThreads) k_combine(const RowsParams p) {
    constexpr int kAhead = 4;                          // entries whose rows are under way together
    const int lane = threadIdx.x & 31;
    const long long item = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const long long token = item / p.parts;
    if (token >= p.tokens) return;
    const int run0 = static_cast<int>(item - token * p.parts) * (32 * U) + lane;
    const Entries e = entries_of(p, token);
    const float weight = p.weights != nullptr && lane < p.top_k ? __ldg(p.weights + token * p.top_k + lane) : 1.0f;
    const T* y = static_cast<const T*>(p.x);
    float acc[U][V] = {};
    unsigned left = e.held;
    while (left != 0u) {
        Run<T, V> r[kAhead][U];
        float w[kAhead];
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
            const int j = left != 0u ? __ffs(left) - 1 : -1;
            left &= left - 1u;
            const long long place = __shfl_sync(0xffffffffu, e.place, max(j, 0));
            w[a] = __shfl_sync(0xffffffffu, weight, max(j, 0));
#pragma unroll
            for (int u = 0; u < U; ++u) {
                r[a][u] = Run<T, V>{};
                if (j >= 0 && run0 + 32 * u < p.runs)
                    r[a][u] = load_run<T, V>(y + place * p.ld_x + static_cast<long long>(run0 + 32 * u) * V);
            }
            if (j < 0) w[a] = 0.0f;                    // the rows past the last are zeros
        }
#pragma unroll
        for (int a = 0; a < kAhead; ++a)
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < V; ++i) acc[u][i] = fmaf(w[a], as_float(r[a][u].v[i]), acc[u][i]);
    }
    O* out = static_cast<O*>(p.out) + token * p.ld_out;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (run0 + 32 * u >= p.runs) break;
        Run<O, V> r;
#pragma unroll
        for (int i = 0; i < V; ++i) r.v[i] = from_float<O>(acc[u][i]);
        store_run<O, V>(out + static_cast<long long>(run0 + 32 * u) * V, r);
    }
}

// W warps take one token: each run of d is read once for up to kTogether entries,
// whose dot products stay in registers to the end of the row.
template <typename D, typename T, int V, int W>
__global__ void __launch_bounds__(kThreads) k_combine_backward(const RowsParams p) {
    constexpr int kTogether = 8;
    __shared__ float part[kWarps][kTogether];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int in = warp % W;                           // which of the token's warps
    const long long token = static_cast<long long>(blockIdx.x) * (kWarps / W) + warp / W;
    const bool here = token < p.tokens;
    const long long t = here ? token : p.tokens - 1;
    const Entries e = entries_of(p, t);
    const float weight = p.weights != nullptr && lane < p.top_k ? __ldg(p.weights + t * p.top_k + lane) : 1.0f;
    const D* d = static_cast<const D*>(p.d) + t * p.ld_d;
    const T* y = static_cast<const T*>(p.x);
    for (int j0 = 0; j0 < p.top_k; j0 += kTogether) {
        long long at[kTogether];
        float w[kTogether], dot[kTogether] = {};
        unsigned held = 0u, there = 0u;
#pragma unroll
        for (int a = 0; a < kTogether; ++a) {
            const int j = j0 + a;
            const int place = __shfl_sync(0xffffffffu, e.place, j & 31);
            w[a] = __shfl_sync(0xffffffffu, weight, j & 31);
            at[a] = place;
            if (here && j < p.top_k && place >= 0 && place < p.rows) there |= 1u << a;
            if (here && j < p.top_k && ((e.held >> j) & 1u)) held |= 1u << a;
        }
        for (int run = in * 32 + lane; run < p.runs; run += 32 * W) {
            const long long col = static_cast<long long>(run) * V;
            Run<D, V> dr = {};
            if (held != 0u) dr = load_run<D, V>(d + col);
            Run<T, V> r[kTogether];
            if (p.dw != nullptr) {
#pragma unroll
                for (int a = 0; a < kTogether; ++a)
                    if ((held >> a) & 1u) r[a] = load_run<T, V>(y + at[a] * p.ld_x + col);
            }
#pragma unroll
            for (int a = 0; a < kTogether; ++a) {
                if (p.out != nullptr && ((there >> a) & 1u)) {
                    Run<T, V> o = {};
                    if ((held >> a) & 1u) {
#pragma unroll
                        for (int i = 0; i < V; ++i) o.v[i] = from_float<T>(w[a] * as_float(dr.v[i]));
                    }
                    store_run<T, V>(static_cast<T*>(p.out) + at[a] * p.ld_out + col, o);
                }
                if (p.dw != nullptr && ((held >> a) & 1u)) {
#pragma unroll
                    for (int i = 0; i < V; ++i) dot[a] = fmaf(as_float(dr.v[i]), as_float(r[a].v[i]), dot[a]);
                }
            }
        }
        if (p.dw == nullptr) continue;
#pragma unroll
        for (int a = 0; a < kTogether; ++a) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) dot[a] += __shfl_xor_sync(0xffffffffu, dot[a], o);
        }
        if (W > 1) {
            __syncthreads();                           // the sums of the entries before have been read
            if (lane == 0) {
#pragma unroll
                for (int a = 0; a < kTogether; ++a) part[warp][a] = dot[a];
            }
            __syncthreads();
#pragma unroll
            for (int a = 0; a < kTogether; ++a) {
                dot[a] = 0.0f;
#pragma unroll
                for (int i = 0; i < W; ++i) dot[a] += part[warp / W * W + i][a];
            }
        }
        if (here && in == 0) {
#pragma unroll
            for (int a = 0; a < kTogether; ++a)
                if (lane == a && j0 + a < p.top_k) p.dw[t * p.top_k + j0 + a] = (held >> a) & 1u ? dot[a] : 0.0f;
        }
    }
}

template <int U>
unsigned warp_items(RowsParams& p) {
    p.parts = (p.runs + 32 * U - 1) / (32 * U);
    return static_cast<unsigned>((p.tokens * p.parts + kWarps - 1) / kWarps);
}

template <typename T, int V>
cudaError_t dispatch(RowsParams p, cudaStream_t s) {
    p.runs = static_cast<int>(p.cols / V);
    const unsigned grid = warp_items<4>(p);
    k_dispatch<T, V, 4><<<grid, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename T, typename O, int V>
cudaError_t combine(RowsParams p, cudaStream_t s) {
    p.runs = static_cast<int>(p.cols / V);
    const unsigned grid = warp_items<2>(p);
    k_combine<T, O, V, 2><<<grid, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename D, typename T, int V>
cudaError_t combine_backward(RowsParams p, cudaStream_t s) {
    p.runs = static_cast<int>(p.cols / V);
    const long long t = p.tokens;
    // as many warps as the row has runs of 32 for, so that none idles
    if (p.runs > 128) k_combine_backward<D, T, V, 8><<<static_cast<unsigned>(t), kThreads, 0, s>>>(p);
    else if (p.runs > 32) k_combine_backward<D, T, V, 4><<<static_cast<unsigned>((t + 1) / 2), kThreads, 0, s>>>(p);
    else k_combine_backward<D, T, V, 1><<<static_cast<unsigned>((t + 7) / 8), kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename F>
cudaError_t by_width(int v, F&& f) {
    switch (v) {
        case 8: return f(std::integral_constant<int, 8>());
        case 4: return f(std::integral_constant<int, 4>());
        case 2: return f(std::integral_constant<int, 2>());
        default: return f(std::integral_constant<int, 1>());
    }
}

}  // namespace

cudaError_t launch_dispatch(const RowsParams& p, cudaStream_t s) {
    const int size = p.x_bf16 ? 2 : 4;
    RunWidth w(p.cols);
    w.array(p.x, p.ld_x, size);
    w.array(p.out, p.ld_out, size);
    return by_width(w.v, [&](auto v) {
        return p.x_bf16 ? dispatch<__nv_bfloat16, v()>(p, s) : dispatch<float, v()>(p, s);
    });
}

cudaError_t launch_combine(const RowsParams& p, cudaStream_t s) {
    RunWidth w(p.cols);
    w.array(p.x, p.ld_x, p.x_bf16 ? 2 : 4);
    w.array(p.out, p.ld_out, p.out_bf16 ? 2 : 4);
    return by_width(w.v, [&](auto v) {
        if (p.x_bf16)
            return p.out_bf16 ? combine<__nv_bfloat16, __nv_bfloat16, v()>(p, s) : combine<__nv_bfloat16, float, v()>(p, s);
        return p.out_bf16 ? combine<float, __nv_bfloat16, v()>(p, s) : combine<float, float, v()>(p, s);
    });
}

cudaError_t launch_combine_backward(const RowsParams& p, cudaStream_t s) {
    RunWidth w(p.cols);
    w.array(p.d, p.ld_d, p.d_bf16 ? 2 : 4);
    if (p.dw != nullptr) w.array(p.x, p.ld_x, p.x_bf16 ? 2 : 4);
    if (p.out != nullptr) w.array(p.out, p.ld_out, p.x_bf16 ? 2 : 4);
    return by_width(w.v, [&](auto v) {
        if (p.d_bf16)
            return p.x_bf16 ? combine_backward<__nv_bfloat16, __nv_bfloat16, v()>(p, s)
                            : combine_backward<__nv_bfloat16, float, v()>(p, s);
        return p.x_bf16 ? combine_backward<float, __nv_bfloat16, v()>(p, s) : combine_backward<float, float, v()>(p, s);
    });
}

}  // namespace muon
