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
// Sums are fp32 fused multiply-adds in the order of j (a dot product's in the order of
// the columns of each thread, then of the lanes and warps), so that a call's result has one
// value whatever the order of the blocks.
//
// Bound by memory.  8192 tokens x 8 entries x 6144 in bf16, device time: dispatch 137 us (906
// MB, 6.6 TB/s), combine 133 us (6.8), backward 252 us (1.71 GB, 6.8); a plain copy runs
// at 6.8.  fp32 the same.  What it took is many loads under way and few registers: entries of
// an expert are gone through four at a time with no conditions inside (combine 151 -> 133 us,
// backward 730 -> 252: a loop over all entries with their conditions took 176 registers and
// left one block on an SM; a persistent form whose loads were renewed one by one as they were
// used, 568 us: more loads than a warp can wait for one by one).
//
// Rows are worked off in runs of elements that lie on 16 bytes of the row that is
// written; where the rows that are read lie otherwise (odd widths, views), their runs are
// put together from the 16-byte vectors around them (SHIFT), and the ends of a row go one
// by one.  4096 tokens x 8 x 6143 in bf16 against 6144: dispatch 81 us and 69, combine 94 and
// 65, backward 208 and 130.  (Element by element: 93, 133 and 484.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "row_runs.cuh"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(float v) { return v; }
template <typename T>
__device__ __forceinline__ T to_type(float v) {
    if constexpr (sizeof(T) == 4) return v;
    else return __float2bfloat16_rn(v);
}

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

// A warp takes U x 32 runs of one token's row.  4096 x 8 x 6144 and 6143 in bf16: 68.2 and 95 us with one,
// 68.6 and 81 with two, 70.0 and 82 with four.
template <typename T, int E, bool SHIFT, int U>
__global__ void __launch_bounds__(kThreads) k_dispatch(const RowsParams p) {
    const int lane = threadIdx.x & 31;
    const long long item = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const long long token = item / p.parts;
    if (token >= p.tokens) return;
    const int part = static_cast<int>(item - token * p.parts), first = part * (32 * U) + lane;
    const Entries e = entries_of(p, token);
    const T* x = static_cast<const T*>(p.x) + token * p.ld_x;
    const Extent in = extent_of<T>(p.x, p.tokens, p.ld_x, p.cols);
    RowRun<T, E> r[U] = {};
    if (!SHIFT && e.held != 0u) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (first + 32 * u < p.runs)
                r[u] = load_row<T, E, false>(x + static_cast<long long>(first + 32 * u) * E, in);
    }
    for (int j = 0; j < p.top_k; ++j) {
        const int place = __shfl_sync(0xffffffffu, e.place, j);
        if (place < 0 || place >= p.rows) continue;
        const bool held = (e.held >> j) & 1u;
        T* out = static_cast<T*>(p.out) + place * p.ld_out;
        if (!SHIFT) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (first + 32 * u >= p.runs) break;
                store_row<T, E>(out + static_cast<long long>(first + 32 * u) * E, held ? r[u] : RowRun<T, E>{});
            }
            continue;
        }
        const RowSpan<T, E> span(out, p.cols);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (held && first + 32 * u < span.runs)
                r[u] = load_row<T, E, true>(x + span.head + static_cast<long long>(first + 32 * u) * E, in);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (first + 32 * u >= span.runs) break;
            store_row<T, E>(out + span.head + static_cast<long long>(first + 32 * u) * E, held ? r[u] : RowRun<T, E>{});
        }
        if (part == 0) {                               // the ends of the row
            if (lane < span.head) out[lane] = held ? x[lane] : to_type<T>(0.0f);
            const long long at = p.cols - span.tail + lane;
            if (lane < span.tail) out[at] = held ? x[at] : to_type<T>(0.0f);
        }
    }
}

// N entries' rows are under way together, U runs of a lane from each: four entries of two runs, two
// of four for the layers that choose one or two experts (16384 x 2 x 6144 136 us with 4 x 2, 97), or two
// of two where they are put together (six blocks of 2 x 1: 121 us for 4096 x 8 x 6143, 95).
template <typename T, int E, bool SHIFT, int N, int U>
__device__ __forceinline__ void add_rows(const RowsParams& p, const Entries& e, float weight, unsigned& left, int first,
                                         int head, int runs, Extent in, float (&acc)[U][E]) {
    constexpr int kStep = SHIFT ? kShared : 32;
    RowRun<T, E> r[N][U] = {};
    float w[N];
    int off[N];
#pragma unroll
    for (int a = 0; a < N; ++a) {
        const int j = __ffs(left) - 1;
        left &= left - 1u;
        const long long place = __shfl_sync(0xffffffffu, e.place, j);
        w[a] = __shfl_sync(0xffffffffu, weight, j);
        const T* y = static_cast<const T*>(p.x) + place * p.ld_x + head;
        off[a] = static_cast<int>(reinterpret_cast<uintptr_t>(y) & 15);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const T* at = y + static_cast<long long>(first + kStep * u) * E;
            if (SHIFT) {                               // past the last run lies what that one has beyond its vector
                if (first + kStep * u <= runs) r[a][u] = load_below<T, E>(at, in);
            } else if (first + kStep * u < runs) {
                r[a][u] = load_row<T, E, false, true>(at, in);
            }
        }
    }
#pragma unroll
    for (int a = 0; a < N; ++a)
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const RowRun<T, E> v = SHIFT ? finished<T, E>(r[a][u], off[a]) : r[a][u];
#pragma unroll
            for (int i = 0; i < E; ++i) acc[u][i] = fmaf(w[a], element<T, E>(v, i), acc[u][i]);
        }
}

template <typename T, typename O, int E, bool SHIFT, int U>
__global__ void __launch_bounds__(kThreads, SHIFT ? 4 : 3) k_combine(const RowsParams p) {
    constexpr int kStep = SHIFT ? kShared : 32, kRows = SHIFT || U == 4 ? 2 : 4;
    const int lane = threadIdx.x & 31;
    const long long item = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const long long token = item / p.parts;
    if (token >= p.tokens) return;
    const int part = static_cast<int>(item - token * p.parts), first = part * (kStep * U) + lane;
    const Entries e = entries_of(p, token);
    const float weight = p.weights != nullptr && lane < p.top_k ? __ldg(p.weights + token * p.top_k + lane) : 1.0f;
    const T* y = static_cast<const T*>(p.x);
    const Extent in = extent_of<T>(p.x, p.rows, p.ld_x, p.cols);
    O* out = static_cast<O*>(p.out) + token * p.ld_out;
    const RowSpan<O, E> span(out, p.cols);
    const int head = SHIFT ? span.head : 0, runs = SHIFT ? span.runs : p.runs;
    float acc[U][E] = {};
    unsigned left = e.held;
    while (__popc(left) >= kRows) add_rows<T, E, SHIFT, kRows, U>(p, e, weight, left, first, head, runs, in, acc);
    if (kRows > 2 && __popc(left) >= 2) add_rows<T, E, SHIFT, 2, U>(p, e, weight, left, first, head, runs, in, acc);
    if (left != 0u) add_rows<T, E, SHIFT, 1, U>(p, e, weight, left, first, head, runs, in, acc);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (first + kStep * u >= runs || lane >= kStep) break;
        store_row<O, E>(out + head + static_cast<long long>(first + kStep * u) * E, rounded<O, E>(acc[u]));
    }
    if (SHIFT && part == 0) {                          // the ends of the row
        const long long at = lane < span.head ? lane : p.cols - span.tail + (lane - span.head);
        const bool mine = lane < span.head + span.tail;
        float sum = 0.0f;
        for (left = e.held; left != 0u; left &= left - 1u) {
            const int j = __ffs(left) - 1;
            const long long place = __shfl_sync(0xffffffffu, e.place, j);
            const float w = __shfl_sync(0xffffffffu, weight, j);
            if (mine) sum = fmaf(w, to_float(y[place * p.ld_x + at]), sum);
        }
        if (mine) out[at] = to_type<O>(sum);
    }
}

// A block takes one token, N of its entries at a time: d is read once for them, and their
// dot products stay in registers to the end of the row.  Three blocks per SM: with two 264 us,
// with four 267 (8192 x 8 x 6144), the registers of the loads under way against the warps.
template <typename D, typename T, int E, bool SHIFT, int N, int U>
__device__ __forceinline__ void backward_of(const RowsParams& p, long long token, const Entries& e, float weight,
                                            unsigned& left, float (*part)[kRowsMaxTopK]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const D* d = static_cast<const D*>(p.d) + token * p.ld_d;
    const Extent in_d = extent_of<D>(p.d, p.tokens, p.ld_d, p.cols), in_y = extent_of<T>(p.x, p.rows, p.ld_x, p.cols);
    const bool dots = p.dw != nullptr;
    const T* y[N];
    T* dy[N];
    float w[N], dot[N];
    int js[N];
#pragma unroll
    for (int a = 0; a < N; ++a) {
        js[a] = __ffs(left) - 1;
        left &= left - 1u;
        const long long place = __shfl_sync(0xffffffffu, e.place, js[a]);
        w[a] = __shfl_sync(0xffffffffu, weight, js[a]);
        y[a] = static_cast<const T*>(p.x) + place * p.ld_x;
        dy[a] = static_cast<T*>(p.out) + place * p.ld_out;
        dot[a] = 0.0f;
    }
    static_assert(!SHIFT || N == 1, "rows that lie differently go one at a time");
    // by the runs of y, so that the order of a sum does not depend on where dy lies; dy lies alike as a rule
    const RowSpan<T, E> span(dots ? y[0] : dy[0], p.cols);
    const bool alike = !SHIFT || reinterpret_cast<uintptr_t>(dy[0] + span.head) % 16 == 0;
    const int head = SHIFT ? span.head : 0, runs = SHIFT ? span.runs : p.runs;
    for (int at = threadIdx.x; at < runs; at += U * blockDim.x) {
        RowRun<D, E> g[U];
        RowRun<T, E> r[U][N];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = at + u * static_cast<int>(blockDim.x);
            if (i >= runs) break;
            const long long col = head + static_cast<long long>(i) * E;
            g[u] = load_row<D, E, SHIFT>(d + col, in_d);
            if (dots) {
#pragma unroll
                for (int a = 0; a < N; ++a) r[u][a] = load_row<T, E, SHIFT>(y[a] + col, in_y);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = at + u * static_cast<int>(blockDim.x);
            if (i >= runs) break;
            const long long col = head + static_cast<long long>(i) * E;
            float v[E];
#pragma unroll
            for (int k = 0; k < E; ++k) v[k] = element<D, E>(g[u], k);
#pragma unroll
            for (int a = 0; a < N; ++a) {
                if (dots) {
#pragma unroll
                    for (int k = 0; k < E; ++k) dot[a] = fmaf(v[k], element<T, E>(r[u][a], k), dot[a]);
                }
                if (p.out != nullptr) {
                    float o[E];
#pragma unroll
                    for (int k = 0; k < E; ++k) o[k] = w[a] * v[k];
                    if (alike) {
                        store_row<T, E>(dy[a] + col, rounded<T, E>(o));
                    } else {
#pragma unroll
                        for (int k = 0; k < E; ++k) dy[a][col + k] = to_type<T>(o[k]);
                    }
                }
            }
        }
    }
    if (SHIFT && threadIdx.x < span.head + span.tail) {    // the ends of the row
        const int i = threadIdx.x;
        const long long col = i < span.head ? i : p.cols - span.tail + (i - span.head);
        const float v = to_float(d[col]);
        if (dots) dot[0] = fmaf(v, to_float(y[0][col]), dot[0]);
        if (p.out != nullptr) dy[0][col] = to_type<T>(w[0] * v);
    }
    if (!dots) return;
#pragma unroll
    for (int a = 0; a < N; ++a) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot[a] += __shfl_xor_sync(0xffffffffu, dot[a], o);
        if (lane == 0) part[warp][js[a]] = dot[a];
    }
}

template <typename D, typename T, int E, bool SHIFT>
__global__ void __launch_bounds__(kThreads, 3) k_combine_backward(const RowsParams p) {
    constexpr int kU = SHIFT || sizeof(D) + sizeof(T) != 4 ? 1 : 2;   // runs of a lane under way
    __shared__ float part[kWarps][kRowsMaxTopK];
    const int lane = threadIdx.x & 31;
    const long long token = blockIdx.x;
    const Entries e = entries_of(p, token);
    const float weight = p.weights != nullptr && lane < p.top_k ? __ldg(p.weights + token * p.top_k + lane) : 1.0f;
    unsigned left = e.held;
    if (!SHIFT) {
        while (__popc(left) >= 4) backward_of<D, T, E, SHIFT, SHIFT ? 1 : 4, kU>(p, token, e, weight, left, part);
        if (__popc(left) >= 2) backward_of<D, T, E, SHIFT, SHIFT ? 1 : 2, kU>(p, token, e, weight, left, part);
    }
    while (left != 0u) backward_of<D, T, E, SHIFT, 1, kU == 2 ? 4 : 1>(p, token, e, weight, left, part);
    if (p.out != nullptr) {                            // rows of no expert
        const unsigned rest = __ballot_sync(0xffffffffu, e.place >= 0 && e.place < p.rows) & ~e.held;
        for (left = rest; left != 0u; left &= left - 1u) {
            const long long place = __shfl_sync(0xffffffffu, e.place, __ffs(left) - 1);
            T* dy = static_cast<T*>(p.out) + place * p.ld_out;
            const RowSpan<T, E> span(dy, p.cols);
            for (int i = threadIdx.x; i < span.runs; i += blockDim.x)
                store_row<T, E>(dy + span.head + static_cast<long long>(i) * E, RowRun<T, E>{});
            const int i = threadIdx.x;
            if (i < span.head + span.tail) dy[i < span.head ? i : p.cols - span.tail + (i - span.head)] = to_type<T>(0.0f);
        }
    }
    if (p.dw == nullptr) return;
    __syncthreads();
    if (threadIdx.x < p.top_k) {
        float sum = 0.0f;
        for (int i = 0; i < static_cast<int>(blockDim.x) / 32; ++i) sum += part[i][threadIdx.x];
        p.dw[token * p.top_k + threadIdx.x] = (e.held >> lane) & 1u ? sum : 0.0f;
    }
}

// STEP runs of a warp U times
template <int E, int U, int STEP = 32>
unsigned warp_items(RowsParams& p) {
    p.runs = static_cast<int>(p.cols / E);
    p.parts = (p.runs + STEP * U - 1) / (STEP * U);
    if (p.parts == 0) p.parts = 1;
    return static_cast<unsigned>((p.tokens * p.parts + kWarps - 1) / kWarps);
}

// 16 bytes of one type, 8 elements of two
template <typename A, typename B>
constexpr int run_of() {
    return sizeof(A) == 4 && sizeof(B) == 4 ? 4 : 8;
}

template <typename T, bool SHIFT>
cudaError_t dispatch(RowsParams p, cudaStream_t s) {
    constexpr int E = run_of<T, T>();
    const unsigned grid = warp_items<E, 2>(p);
    k_dispatch<T, E, SHIFT, 2><<<grid, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename T, typename O, bool SHIFT>
cudaError_t combine(RowsParams p, cudaStream_t s) {
    constexpr int E = run_of<T, O>(), kU = sizeof(T) * E > 16 ? 1 : 2;
    if constexpr (kU == 2 && !SHIFT) {
        if (p.top_k <= 2) {
            const unsigned grid = warp_items<E, 4>(p);
            k_combine<T, O, E, false, 4><<<grid, kThreads, 0, s>>>(p);
            return cudaGetLastError();
        }
    }
    const unsigned grid = warp_items<E, kU, SHIFT ? kShared : 32>(p);
    k_combine<T, O, E, SHIFT, kU><<<grid, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename D, typename T, bool SHIFT>
cudaError_t combine_backward(RowsParams p, cudaStream_t s) {
    constexpr int E = run_of<D, T>();
    p.runs = static_cast<int>(p.cols / E);
    // as many warps as the row has runs for
    const int warps = p.runs >= 256 ? 8 : p.runs >= 128 ? 4 : p.runs >= 64 ? 2 : 1;
    k_combine_backward<D, T, E, SHIFT><<<static_cast<unsigned>(p.tokens), 32 * warps, 0, s>>>(p);
    return cudaGetLastError();
}

bool on_16(const void* p, long long ld, bool bf16) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * (bf16 ? 2 : 4) % 16 == 0;
}

// Rows of whole runs
bool fills(const RowsParams& p, bool any_bf16) { return p.cols % (any_bf16 ? 8 : 4) == 0; }

template <typename F>
cudaError_t by_type(bool bf16, F&& f) {
    return bf16 ? f(__nv_bfloat16()) : f(float());
}

}  // namespace

cudaError_t launch_dispatch(const RowsParams& p, cudaStream_t s) {
    const bool whole = fills(p, p.x_bf16) && on_16(p.x, p.ld_x, p.x_bf16) && on_16(p.out, p.ld_out, p.x_bf16);
    return by_type(p.x_bf16, [&](auto t) {
        using T = decltype(t);
        return whole ? dispatch<T, false>(p, s) : dispatch<T, true>(p, s);
    });
}

cudaError_t launch_combine(const RowsParams& p, cudaStream_t s) {
    const bool whole = fills(p, p.x_bf16 || p.out_bf16) && on_16(p.x, p.ld_x, p.x_bf16) && on_16(p.out, p.ld_out, p.out_bf16);
    return by_type(p.x_bf16, [&](auto t) {
        return by_type(p.out_bf16, [&](auto o) {
            using T = decltype(t);
            using O = decltype(o);
            return whole ? combine<T, O, false>(p, s) : combine<T, O, true>(p, s);
        });
    });
}

cudaError_t launch_combine_backward(const RowsParams& p, cudaStream_t s) {
    const bool whole = fills(p, p.d_bf16 || p.x_bf16) && on_16(p.d, p.ld_d, p.d_bf16) &&
                       (p.dw == nullptr || on_16(p.x, p.ld_x, p.x_bf16)) && (p.out == nullptr || on_16(p.out, p.ld_out, p.x_bf16));
    return by_type(p.d_bf16, [&](auto d) {
        return by_type(p.x_bf16, [&](auto t) {
            using D = decltype(d);
            using T = decltype(t);
            return whole ? combine_backward<D, T, false>(p, s) : combine_backward<D, T, true>(p, s);
        });
    });
}

}  // namespace muon
