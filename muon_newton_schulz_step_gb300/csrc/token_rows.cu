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
// Rows are worked off in eights of elements that lie on 16 bytes of the row that is
// written; where the rows that are read lie otherwise (odd widths, views), their eights are
// put together from the 16-byte vectors around them (SHIFT), and the ends of a row go one
// by one.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "eights.cuh"
#include "internal.h"

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

// Whether eight i of a row ends in its middle (fp32 rows of 4 modulo 8).
__device__ __forceinline__ bool half_of(const RowsParams& p, int i) { return p.half != 0 && i == p.eights - 1; }

// A warp takes U x 32 eights of one token's row.
template <typename T, bool SHIFT, int U>
__global__ void __launch_bounds__(kThreads) k_dispatch(const RowsParams p) {
    const int lane = threadIdx.x & 31;
    const long long item = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const long long token = item / p.parts;
    if (token >= p.tokens) return;
    const int part = static_cast<int>(item - token * p.parts), first = part * (32 * U) + lane;
    const Entries e = entries_of(p, token);
    const T* x = static_cast<const T*>(p.x) + token * p.ld_x;
    const Extent in = extent_of<T>(p.x, p.tokens, p.ld_x, p.cols);
    Eight<T> r[U] = {};
    if (!SHIFT && e.held != 0u) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (first + 32 * u < p.eights)
                r[u] = load_eight<T, false>(x + static_cast<long long>(first + 32 * u) * 8, in, half_of(p, first + 32 * u));
    }
    for (int j = 0; j < p.top_k; ++j) {
        const int place = __shfl_sync(0xffffffffu, e.place, j);
        if (place < 0 || place >= p.rows) continue;
        const bool held = (e.held >> j) & 1u;
        T* out = static_cast<T*>(p.out) + place * p.ld_out;
        if (!SHIFT) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (first + 32 * u >= p.eights) break;
                store_eight<T>(out + static_cast<long long>(first + 32 * u) * 8, held ? r[u] : Eight<T>{},
                               half_of(p, first + 32 * u));
            }
            continue;
        }
        const RowSpan<T> span(out, p.cols);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (held && first + 32 * u < span.eights)
                r[u] = load_eight<T, true>(x + span.head + static_cast<long long>(first + 32 * u) * 8, in);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (first + 32 * u >= span.eights) break;
            store_eight<T>(out + span.head + static_cast<long long>(first + 32 * u) * 8, held ? r[u] : Eight<T>{});
        }
        if (part == 0) {                               // the ends of the row
            if (lane < span.head) out[lane] = held ? x[lane] : to_type<T>(0.0f);
            const long long at = p.cols - span.tail + lane;
            if (lane < span.tail) out[at] = held ? x[at] : to_type<T>(0.0f);
        }
    }
}

// N entries' rows are under way together, U eights of a lane from each.
template <typename T, bool SHIFT, int N, int U>
__device__ __forceinline__ void add_rows(const RowsParams& p, const Entries& e, float weight, unsigned& left, int first,
                                         int head, int eights, Extent in, float (&acc)[U][8]) {
    Eight<T> r[N][U];
    float w[N];
#pragma unroll
    for (int a = 0; a < N; ++a) {
        const int j = __ffs(left) - 1;
        left &= left - 1u;
        const long long place = __shfl_sync(0xffffffffu, e.place, j);
        w[a] = __shfl_sync(0xffffffffu, weight, j);
        const T* y = static_cast<const T*>(p.x) + place * p.ld_x + head;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (first + 32 * u < eights)
                r[a][u] = load_eight<T, SHIFT, !SHIFT>(y + static_cast<long long>(first + 32 * u) * 8, in,
                                                       !SHIFT && half_of(p, first + 32 * u));
    }
#pragma unroll
    for (int a = 0; a < N; ++a)
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[u][i] = fmaf(w[a], element<T>(r[a][u], i), acc[u][i]);
}

template <typename T, typename O, bool SHIFT, int U>
__global__ void __launch_bounds__(kThreads, SHIFT ? 5 : 3) k_combine(const RowsParams p) {
    const int lane = threadIdx.x & 31;
    const long long item = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const long long token = item / p.parts;
    if (token >= p.tokens) return;
    const int part = static_cast<int>(item - token * p.parts), first = part * (32 * U) + lane;
    const Entries e = entries_of(p, token);
    const float weight = p.weights != nullptr && lane < p.top_k ? __ldg(p.weights + token * p.top_k + lane) : 1.0f;
    const T* y = static_cast<const T*>(p.x);
    const Extent in = extent_of<T>(p.x, p.rows, p.ld_x, p.cols);
    O* out = static_cast<O*>(p.out) + token * p.ld_out;
    const RowSpan<O> span(out, p.cols);
    const int head = SHIFT ? span.head : 0, eights = SHIFT ? span.eights : p.eights;
    float acc[U][8] = {};
    unsigned left = e.held;
    while (__popc(left) >= 4) add_rows<T, SHIFT, 4, U>(p, e, weight, left, first, head, eights, in, acc);
    while (left != 0u) add_rows<T, SHIFT, 1, U>(p, e, weight, left, first, head, eights, in, acc);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (first + 32 * u >= eights) break;
        store_eight<O>(out + head + static_cast<long long>(first + 32 * u) * 8, rounded<O>(acc[u]),
                       !SHIFT && half_of(p, first + 32 * u));
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
// dot products stay in registers to the end of the row.
template <typename D, typename T, bool SHIFT, int N, int U>
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
    // by the eights of y, so that the order of a sum does not depend on where dy lies; dy lies alike as a rule
    const RowSpan<T> span(dots ? y[0] : dy[0], p.cols);
    const bool alike = !SHIFT || reinterpret_cast<uintptr_t>(dy[0] + span.head) % 16 == 0;
    const int head = SHIFT ? span.head : 0, eights = SHIFT ? span.eights : p.eights;
    for (int at = threadIdx.x; at < eights; at += U * blockDim.x) {
        Eight<D> g[U];
        Eight<T> r[U][N];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = at + u * static_cast<int>(blockDim.x);
            if (i >= eights) break;
            const long long col = head + static_cast<long long>(i) * 8;
            const bool half = !SHIFT && half_of(p, i);
            g[u] = load_eight<D, SHIFT>(d + col, in_d, half);
            if (dots) {
#pragma unroll
                for (int a = 0; a < N; ++a) r[u][a] = load_eight<T, SHIFT>(y[a] + col, in_y, half);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = at + u * static_cast<int>(blockDim.x);
            if (i >= eights) break;
            const long long col = head + static_cast<long long>(i) * 8;
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = element<D>(g[u], k);
#pragma unroll
            for (int a = 0; a < N; ++a) {
                if (dots) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) dot[a] = fmaf(v[k], element<T>(r[u][a], k), dot[a]);
                }
                if (p.out != nullptr) {
                    float o[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) o[k] = w[a] * v[k];
                    if (alike) {
                        store_eight<T>(dy[a] + col, rounded<T>(o), !SHIFT && half_of(p, i));
                    } else {
#pragma unroll
                        for (int k = 0; k < 8; ++k) dy[a][col + k] = to_type<T>(o[k]);
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

template <typename D, typename T, bool SHIFT>
__global__ void __launch_bounds__(kThreads, 3) k_combine_backward(const RowsParams p) {
    constexpr int kU = SHIFT || sizeof(D) + sizeof(T) != 4 ? 1 : 2;   // eights of a lane under way
    __shared__ float part[kWarps][kRowsMaxTopK];
    const int lane = threadIdx.x & 31;
    const long long token = blockIdx.x;
    const Entries e = entries_of(p, token);
    const float weight = p.weights != nullptr && lane < p.top_k ? __ldg(p.weights + token * p.top_k + lane) : 1.0f;
    unsigned left = e.held;
    if (!SHIFT) {
        while (__popc(left) >= 4) backward_of<D, T, SHIFT, SHIFT ? 1 : 4, kU>(p, token, e, weight, left, part);
    }
    while (left != 0u) backward_of<D, T, SHIFT, 1, kU>(p, token, e, weight, left, part);
    if (p.out != nullptr) {                            // rows of no expert
        const unsigned rest = __ballot_sync(0xffffffffu, e.place >= 0 && e.place < p.rows) & ~e.held;
        for (left = rest; left != 0u; left &= left - 1u) {
            const long long place = __shfl_sync(0xffffffffu, e.place, __ffs(left) - 1);
            T* dy = static_cast<T*>(p.out) + place * p.ld_out;
            const RowSpan<T> span(dy, p.cols);
            for (int i = threadIdx.x; i < span.eights; i += blockDim.x)
                store_eight<T>(dy + span.head + static_cast<long long>(i) * 8, Eight<T>{});
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

template <int U>
unsigned warp_items(RowsParams& p) {
    p.eights = static_cast<int>((p.cols + 4 * p.half) / 8);
    p.parts = (p.eights + 32 * U - 1) / (32 * U);
    if (p.parts == 0) p.parts = 1;
    return static_cast<unsigned>((p.tokens * p.parts + kWarps - 1) / kWarps);
}

template <typename T, bool SHIFT>
cudaError_t dispatch(RowsParams p, cudaStream_t s) {
    constexpr int kU = sizeof(T) == 2 ? 4 : 2;
    const unsigned grid = warp_items<kU>(p);
    k_dispatch<T, SHIFT, kU><<<grid, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename T, typename O, bool SHIFT>
cudaError_t combine(RowsParams p, cudaStream_t s) {
    constexpr int kU = sizeof(T) == 2 && !SHIFT ? 2 : 1;
    const unsigned grid = warp_items<kU>(p);
    k_combine<T, O, SHIFT, kU><<<grid, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename D, typename T, bool SHIFT>
cudaError_t combine_backward(RowsParams p, cudaStream_t s) {
    p.eights = static_cast<int>((p.cols + 4 * p.half) / 8);
    // as many warps as the row has eights for
    const int warps = p.eights >= 256 ? 8 : p.eights >= 128 ? 4 : p.eights >= 64 ? 2 : 1;
    k_combine_backward<D, T, SHIFT><<<static_cast<unsigned>(p.tokens), 32 * warps, 0, s>>>(p);
    return cudaGetLastError();
}

bool on_16(const void* p, long long ld, bool bf16) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * (bf16 ? 2 : 4) % 16 == 0;
}

// Rows that fill 16-byte vectors: eights, or in fp32 alone fours.
bool fills(const RowsParams& p, bool any_bf16) { return p.cols % (any_bf16 ? 8 : 4) == 0; }

template <typename F>
cudaError_t by_type(bool bf16, F&& f) {
    return bf16 ? f(__nv_bfloat16()) : f(float());
}

}  // namespace

cudaError_t launch_dispatch(const RowsParams& q, cudaStream_t s) {
    RowsParams p = q;
    const bool whole = fills(p, p.x_bf16) && on_16(p.x, p.ld_x, p.x_bf16) && on_16(p.out, p.ld_out, p.x_bf16);
    p.half = whole && p.cols % 8 != 0;
    return by_type(p.x_bf16, [&](auto t) {
        using T = decltype(t);
        return whole ? dispatch<T, false>(p, s) : dispatch<T, true>(p, s);
    });
}

cudaError_t launch_combine(const RowsParams& q, cudaStream_t s) {
    RowsParams p = q;
    const bool whole = fills(p, p.x_bf16 || p.out_bf16) && on_16(p.x, p.ld_x, p.x_bf16) && on_16(p.out, p.ld_out, p.out_bf16);
    p.half = whole && p.cols % 8 != 0;
    return by_type(p.x_bf16, [&](auto t) {
        return by_type(p.out_bf16, [&](auto o) {
            using T = decltype(t);
            using O = decltype(o);
            return whole ? combine<T, O, false>(p, s) : combine<T, O, true>(p, s);
        });
    });
}

cudaError_t launch_combine_backward(const RowsParams& q, cudaStream_t s) {
    RowsParams p = q;
    const bool whole = fills(p, p.d_bf16 || p.x_bf16) && on_16(p.d, p.ld_d, p.d_bf16) &&
                       (p.dw == nullptr || on_16(p.x, p.ld_x, p.x_bf16)) && (p.out == nullptr || on_16(p.out, p.ld_out, p.x_bf16));
    p.half = whole && p.cols % 8 != 0;
    return by_type(p.d_bf16, [&](auto d) {
        return by_type(p.x_bf16, [&](auto t) {
            using D = decltype(d);
            using T = decltype(t);
            return whole ? combine_backward<D, T, false>(p, s) : combine_backward<D, T, true>(p, s);
        });
    });
}

}  // namespace muon
