// The gated activation between an expert's projections, and its gradient:
//
//   s = 1 / (1 + exp(-gate)),  out = gate s up
//   d_gate = d up s (1 + gate (1 - s)),  d_up = d gate s
//
// Bound by memory: 3 and 5 elements move for each one of the result; the gradient of 65536 x
// 2048 in bf16 takes 191 us (1.34 GB, 7.0 TB/s), the forward 114 (0.81 GB, 7.1).  A thread takes
// U runs of up to 16 bytes, kThreads apart, all loaded before the first is used.
// Operands that lie row behind row are taken as one long row, so that odd widths
// cost no narrow loads; gate and up as the halves of one product have rows of their
// own, found by one multiplication (no division) from the run's number.
//
// Sums, quotients and products are fp32 in both types.  fp32 operands take the exponential in full and
// an exact division: out is off by 5 units of 2^-24 of its value (the exponential 2, the sum, the quotient
// and the product one each), what gate / (1 + exp(-gate)) * up in fp32 is.  bf16 takes the fast
// exponential (off by 2 + 1.173 |gate| units of 2^-23 by its documentation, 2^-16 at |gate| = 80) and
// the fast quotient (2 units): far below half a step of bf16, 2^-8.  The full ones cost fp32 nothing where rows
// load in 16 bytes (28042 x 916 45.4 and 74.9 us, as with the fast ones; 65536 x 2048 229 and 382), and 58 us
// for 54 where they go by single elements (28042 x 915, halves of one product; gradient 82 for 79).  Both
// types lose what lies below their exponents: fp32 gives 0 below gate = -88.7, where exp(-gate) is infinite,
// bf16 below -87.3, where the fast quotient is 0; there the result is below 2^-119 of up.  gate = -inf gives
// NaN, as its product -inf * 0 does.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "vectors.cuh"

namespace muon {
namespace {

constexpr int kThreads = 256;

// y / (1 + exp(-g))
template <typename T>
__device__ __forceinline__ float over(float y, float g) {
    if constexpr (sizeof(T) == 4) return __fdiv_rn(y, 1.0f + expf(-g));
    else return __fdividef(y, 1.0f + __expf(-g));
}

// Row and first column of run i: i / runs by the multiplier 2^64 / runs + 1, exact for i < 2^32.
struct Spot {
    long long row, col;
};

template <int V>
__device__ __forceinline__ Spot spot_of(const SwigluParams& p, unsigned i) {
    const unsigned row = p.runs == 1 ? i : static_cast<unsigned>(__umul64hi(p.by_runs, static_cast<unsigned long long>(i)));
    return {static_cast<long long>(row), static_cast<long long>(i - row * p.runs) * V};
}

template <typename T, int V>
__device__ __forceinline__ Run<T, V> forward(const Run<T, V>& g, const Run<T, V>& u) {
    Run<T, V> o;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float x = as_float(g.v[i]);
        o.v[i] = from_float<T>(over<T>(x, x) * as_float(u.v[i]));
    }
    return o;
}

template <typename T, int V>
__device__ __forceinline__ void backward(const Run<T, V>& g, const Run<T, V>& u, const Run<T, V>& d, Run<T, V>& dg,
                                         Run<T, V>& du) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float x = as_float(g.v[i]), y = as_float(d.v[i]), s = over<T>(1.0f, x);
        dg.v[i] = from_float<T>(y * as_float(u.v[i]) * (s * fmaf(x, 1.0f - s, 1.0f)));
        du.v[i] = from_float<T>(y * (x * s));
    }
}

template <typename T, int V, int U>
__global__ void __launch_bounds__(kThreads) k_swiglu(const SwigluParams p) {
    const T *gate = static_cast<const T*>(p.gate), *up = static_cast<const T*>(p.up);
    T* out = static_cast<T*>(p.out);
    const unsigned first = blockIdx.x * (kThreads * U) + threadIdx.x;
    Run<T, V> g[U], u[U];
    Spot at[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const unsigned i = first + k * kThreads;
        if (i >= p.total) break;
        at[k] = spot_of<V>(p, i);
        g[k] = load_run<T, V>(gate + at[k].row * p.ld_gate + at[k].col);
        u[k] = load_run<T, V>(up + at[k].row * p.ld_up + at[k].col);
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
        if (first + k * kThreads >= p.total) break;
        store_run<T, V>(out + at[k].row * p.ld_out + at[k].col, forward<T, V>(g[k], u[k]));
    }
    if (first < static_cast<unsigned>(p.rest)) {
        const long long i = p.cols + first;
        store_run<T, 1>(out + i, forward<T, 1>(load_run<T, 1>(gate + i), load_run<T, 1>(up + i)));
    }
}

template <typename T, int V, int U>
__global__ void __launch_bounds__(kThreads) k_swiglu_backward(const SwigluParams p) {
    const T *gate = static_cast<const T*>(p.gate), *up = static_cast<const T*>(p.up), *dy = static_cast<const T*>(p.d);
    T *d_gate = static_cast<T*>(p.d_gate), *d_up = static_cast<T*>(p.d_up);
    const unsigned first = blockIdx.x * (kThreads * U) + threadIdx.x;
    Run<T, V> g[U], u[U], d[U];
    Spot at[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const unsigned i = first + k * kThreads;
        if (i >= p.total) break;
        at[k] = spot_of<V>(p, i);
        g[k] = load_run<T, V>(gate + at[k].row * p.ld_gate + at[k].col);
        u[k] = load_run<T, V>(up + at[k].row * p.ld_up + at[k].col);
        d[k] = load_run<T, V>(dy + at[k].row * p.ld_d + at[k].col);
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
        if (first + k * kThreads >= p.total) break;
        Run<T, V> dg, du;
        backward<T, V>(g[k], u[k], d[k], dg, du);
        store_run<T, V>(d_gate + at[k].row * p.ld_dgate + at[k].col, dg);
        store_run<T, V>(d_up + at[k].row * p.ld_dup + at[k].col, du);
    }
    if (first < static_cast<unsigned>(p.rest)) {
        const long long i = p.cols + first;
        Run<T, 1> dg, du;
        backward<T, 1>(load_run<T, 1>(gate + i), load_run<T, 1>(up + i), load_run<T, 1>(dy + i), dg, du);
        store_run<T, 1>(d_gate + i, dg);
        store_run<T, 1>(d_up + i, du);
    }
}

// Launches of at most 2^31 runs: rows at a time where there are more.
template <int V, typename F>
cudaError_t in_parts(SwigluParams p, int size, int u, F&& launch) {
    const long long runs = p.cols >= V ? p.cols / V : 1;
    const long long most = (1ll << 31) / runs > 0 ? (1ll << 31) / runs : 1;
    auto move = [&](const void*& q, long long ld, long long rows) {
        if (q != nullptr) q = static_cast<const char*>(q) + rows * ld * size;
    };
    auto move_out = [&](void*& q, long long ld, long long rows) {
        if (q != nullptr) q = static_cast<char*>(q) + rows * ld * size;
    };
    p.runs = static_cast<unsigned>(runs);
    p.by_runs = ~0ull / static_cast<unsigned long long>(runs) + 1;
    for (long long left = p.rows; left > 0;) {
        const long long rows = left < most ? left : most;
        p.total = p.cols >= V ? static_cast<unsigned>(rows * runs) : 0u;    // 0: the rest alone
        const unsigned grid = (p.total + kThreads * u - 1) / (kThreads * u);
        const cudaError_t e = launch(p, grid > 0 ? grid : 1u);
        if (e != cudaSuccess) return e;
        left -= rows;
        move(p.gate, p.ld_gate, rows);
        move(p.up, p.ld_up, rows);
        move(p.d, p.ld_d, rows);
        move_out(p.out, p.ld_out, rows);
        move_out(p.d_gate, p.ld_dgate, rows);
        move_out(p.d_up, p.ld_dup, rows);
    }
    return cudaSuccess;
}

// Runs of a thread: one of 16 bytes, two narrower ones.  Forward of 65536 x 2048 in bf16: 114 us with
// one, 128 with two, 183 with four, whose registers leave few warps; of 65536 x 2046 as halves of one
// product (4-byte runs) 223, 151 and 177.
template <typename T, int V>
cudaError_t run(const SwigluParams& p, cudaStream_t s) {
    constexpr int kRuns = sizeof(T) * V >= 16 ? 1 : 2;
    return in_parts<V>(p, sizeof(T), kRuns, [&](const SwigluParams& q, unsigned grid) {
        if (q.d == nullptr) k_swiglu<T, V, kRuns><<<grid, kThreads, 0, s>>>(q);
        else k_swiglu_backward<T, V, kRuns><<<grid, kThreads, 0, s>>>(q);
        return cudaGetLastError();
    });
}

template <typename T>
cudaError_t by_width(const SwigluParams& p, int v, cudaStream_t s) {
    if constexpr (sizeof(T) == 2) {
        if (v == 8) return run<T, 8>(p, s);
    }
    return v == 4 ? run<T, 4>(p, s) : v == 2 ? run<T, 2>(p, s) : run<T, 1>(p, s);
}

}  // namespace

cudaError_t launch_swiglu(SwigluParams p, cudaStream_t s) {
    const int size = p.bf16 ? 2 : 4;
    struct Array {
        const void* p;
        long long ld;
    };
    const Array arrays[6] = {{p.gate, p.ld_gate}, {p.up, p.ld_up},         {p.d, p.ld_d},
                             {p.out, p.ld_out},   {p.d_gate, p.ld_dgate}, {p.d_up, p.ld_dup}};
    bool joined = true;
    for (const Array& a : arrays) joined = joined && (p.rows == 1 || a.p == nullptr || a.ld == p.cols);
    p.rest = 0;
    if (joined && p.cols * p.rows < (1ll << 31)) {       // one long row; what its last whole run leaves goes one by one
        p.cols *= p.rows;
        p.rows = 1;
        p.rest = static_cast<int>(p.cols % 8);
        p.cols -= p.rest;
    }
    // 16 bytes at most: a warp's vectors then lie side by side (fp32 in runs of 32 bytes: 4.4 TB/s backward)
    RunWidth w(p.cols > 0 ? p.cols : 8, 16 / size);
    for (const Array& a : arrays)
        if (a.p != nullptr) w.array(a.p, p.rows == 1 ? w.v : a.ld, size);
    return p.bf16 ? by_width<__nv_bfloat16>(p, w.v, s) : by_width<float>(p, w.v, s);
}

}  // namespace muon
