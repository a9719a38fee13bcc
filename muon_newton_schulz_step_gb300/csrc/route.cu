// Routing of tokens to experts, and its gradient.
//
// Per token, over `experts` logits x:
//   s_e   = softmax(x)_e or 1 / (1 + exp(-x_e))
//   c_e   = s_e + bias_e                        (the bias steers the choice only)
//   group score = the two largest c of the group added up (one group: no step)
//   the top_groups groups of largest score stay; of their experts the top_k
//   largest c are chosen, in descending order; equal values: lowest index first
//   w_k   = scale * s_k / sum of the chosen s   (renormalize)  or  scale * s_k
// Group-limited routing is the pages' ("Domyn is training a 1T-parameter MoE
// on Europe's Jupiter supercomputer, and published the recipe", section "What
// moved the number"); 384 experts, 8 chosen: its table "The model and the
// machine".
//
// A logit or a choice value of -inf masks the expert.  Where fewer than top_k
// experts are left (a padding token whose logits are all -inf has none), the
// remaining places get expert -1 and weight 0 and are not counted.  A NaN
// choice value orders below every number.
//
// Gradient of the logits from that of the weights (d_k):
//   renormalised: u_k = d_k - sum_j d_j w_j / scale,  ds_k = scale * u_k / S,
//   else          ds_k = scale * d_k;   S = sum of the chosen s
//   sigmoid: dx_k = ds_k s_k (1 - s_k), 0 elsewhere
//   softmax: dx_e = s_e (ds_e - sum_j ds_j s_j); renormalised the sum is zero
//            and dx_k = w_k u_k on the chosen, 0 elsewhere
// so only the softmax without renormalisation reads the whole row again.
//
// Forward: one warp per token.  A group owns `lanes` lanes, a lane `per_lane`
// consecutive experts of one group, in index order over the warp: so the lowest
// index among equal values is the lowest lane's, a group's two largest values
// meet in log2(lanes) exchanges for all groups at once, and everything stays
// in registers.  The top_k largest lane maxima bound the choice from below:
// whatever is chosen is at least the top_k-th of them.  The few experts at or
// above that bound (8 to about 12 of 384) are written to shared memory in index
// order, a lane takes one each and counts those before it: its place in the
// result.  Should more than 32 qualify (equal values, few lanes left), the
// largest is taken top_k times instead, which alone took 680 of about 1400
// instructions a token (73 us for 32768 tokens x 384 experts in fp32; now @@).
//
// Backward: one warp per token, lanes striped over the row in vectors of four.
// Scores of the chosen are recomputed from their logits; only the softmax without
// renormalisation reads the row.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cmath>

#include "groups.cuh"
#include "internal.h"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr uint32_t kAll = 0xffffffffu;

__device__ __forceinline__ float load_logit(const RouteParams& p, long long row, int e) {
    return p.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.logits)[row * p.ld + e])
                  : static_cast<const float*>(p.logits)[row * p.ld + e];
}

__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));   // NaN: not taken
    return r;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

// e^x to about 2 ulp: 2^k with k = x log2(e) rounded, times 1 + (what the rounding
// left) ln 2.  Arguments beyond +-200 give infinity and zero, NaN gives NaN.
__device__ __forceinline__ float exp_fast(float x) {
    const float c = fminf(fmaxf(x, -200.0f), 200.0f);
    const float k = c * 1.44269504f;
    float lo = fmaf(c, 1.44269504f, -k);
    lo = fmaf(c, 1.92596299e-8f, lo);                    // log2(e) - fp32(log2(e))
    float p;
    asm("ex2.approx.f32 %0, %1;" : "=f"(p) : "f"(k));
    p = p * fmaf(lo, 0.693147181f, 1.0f);
    return x == x ? p : x;
}

__device__ __forceinline__ float sigmoid_fast(float x) { return __fdividef(1.0f, 1.0f + exp_fast(-x)); }

// This lane's logits, -inf where it owns no expert.
template <int NV>
__device__ __forceinline__ void load_lane(const RouteParams& p, long long row, int e0, int n, float (&x)[NV]) {
    if (NV % 4 == 0 && p.vec) {
#pragma unroll
        for (int j = 0; j < NV / 4 * 4; j += 4) {
            float f[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            if (j < n) {
                if (p.bf16) {
                    const uint2 r = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.logits) +
                                                                    row * p.ld + e0 + j);
                    f[0] = __uint_as_float(r.x << 16);
                    f[1] = __uint_as_float(r.x & 0xffff0000u);
                    f[2] = __uint_as_float(r.y << 16);
                    f[3] = __uint_as_float(r.y & 0xffff0000u);
                } else {
                    const float4 r = *reinterpret_cast<const float4*>(static_cast<const float*>(p.logits) + row * p.ld +
                                                                      e0 + j);
                    f[0] = r.x; f[1] = r.y; f[2] = r.z; f[3] = r.w;
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) x[j + i] = f[i];
        }
    } else {
#pragma unroll
        for (int j = 0; j < NV; ++j) x[j] = j < n ? load_logit(p, row, e0 + j) : -INFINITY;
    }
}

template <int NV, bool SIGMOID>
__global__ void __launch_bounds__(kThreads) k_route(const __grid_constant__ RouteParams p) {
    extern __shared__ int hist[];
    __shared__ float2 pool[kWarps][32];                  // choice value, score
    __shared__ int pool_e[kWarps][32];
    __shared__ float2 order[kWarps][32];                 // score, expert
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int e = threadIdx.x; e < p.experts; e += kThreads) hist[e] = 0;
    __syncthreads();

    const int group = lane / p.lanes, in_group = lane % p.lanes;
    const int g0 = in_group * p.per_lane;               // first expert of this lane within its group
    const int e0 = group * p.group_size + g0;
    const int n = group < p.groups ? max(0, min(p.per_lane, p.group_size - g0)) : 0;
    float bias[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) bias[j] = p.bias != nullptr && j < n ? p.bias[e0 + j] : 0.0f;

    for (long long row = static_cast<long long>(blockIdx.x) * kWarps + warp; row < p.tokens;
         row += static_cast<long long>(gridDim.x) * kWarps) {
        float x[NV];
        load_lane<NV>(p, row, e0, n, x);
        // scores
        float top = 0.0f, scale = 1.0f;
        if (!SIGMOID) {
            float m = -INFINITY;
#pragma unroll
            for (int j = 0; j < NV; ++j) m = fmaxf(m, x[j]);
            top = warp_max(m);
        }
        float c[NV];                                     // choice values; -inf: masked
        float a = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const bool masked = x[j] == -INFINITY;
            x[j] = SIGMOID ? sigmoid_fast(x[j]) : exp_fast(x[j] - top);
            if (masked) x[j] = 0.0f;
            if (!SIGMOID) a += x[j];
            c[j] = masked ? -INFINITY : 0.0f;
        }
        if (!SIGMOID) scale = __fdiv_rn(1.0f, warp_sum(a));
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (!SIGMOID) x[j] *= scale;
            // a NaN orders below every number
            const float v = x[j] + bias[j];
            c[j] = c[j] < 0.0f ? c[j] : (v == v ? v : -FLT_MAX);
        }
        // group scores
        if (p.groups > 1) {
            float m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                m2 = fmaxf(m2, fminf(m1, c[j]));
                m1 = fmaxf(m1, c[j]);
            }
            for (int o = p.lanes >> 1; o > 0; o >>= 1) {
                const float o1 = __shfl_xor_sync(kAll, m1, o), o2 = __shfl_xor_sync(kAll, m2, o);
                m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
                m1 = fmaxf(m1, o1);
            }
            const float gv = m2 <= -FLT_MAX ? m1 : m1 + m2;   // one expert left (or one that is not NaN): its own
            int before = 0;
            for (int g = 0; g < p.groups; ++g) {
                const float v = __shfl_sync(kAll, gv, g * p.lanes);
                before += v > gv || (v == gv && g < group);
            }
            if (before >= p.top_groups) {
#pragma unroll
                for (int j = 0; j < NV; ++j) c[j] = -INFINITY;
            }
        }
        float best = -INFINITY;
#pragma unroll
        for (int j = 0; j < NV; ++j) best = fmaxf(best, c[j]);
        // the top_k-th largest lane maximum, by a bitonic sort of the maxima (descending)
        float v = best;
#pragma unroll
        for (int k = 2; k <= 32; k <<= 1) {
#pragma unroll
            for (int o = k >> 1; o > 0; o >>= 1) {
                const float w = __shfl_xor_sync(kAll, v, o);
                const bool larger = ((lane & o) == 0) == ((lane & k) == 0);
                v = larger ? fmaxf(v, w) : fminf(v, w);
            }
        }
        const float bound = __shfl_sync(kAll, v, p.top_k - 1);
        int cnt = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j) cnt += c[j] >= bound && c[j] > -INFINITY;
        const int upto = warp_inclusive_sum(cnt);
        const int total = __shfl_sync(kAll, upto, 31);
        int my_e = -1;
        float my_s = 0.0f;
        if (total <= 32) {
            int at = upto - cnt;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if (c[j] >= bound && c[j] > -INFINITY) {
                    pool[warp][at] = make_float2(c[j], x[j]);
                    pool_e[warp][at] = e0 + j;
                    ++at;
                }
            }
            __syncwarp();
            const float2 f = pool[warp][lane];
            const int e = pool_e[warp][lane];
            const float mine = lane < total ? f.x : -INFINITY;
            int place = 0;
            for (int i = 0; i < total; ++i) {
                const float o = __shfl_sync(kAll, mine, i);
                place += o > mine || (o == mine && i < lane);
            }
            __syncwarp();                                // the pool has been read
            if (lane < total && place < p.top_k) {
                order[warp][place] = make_float2(f.y, __int_as_float(e));
            }
            __syncwarp();
            if (lane < p.top_k && lane < total) {
                const float2 o = order[warp][lane];
                my_s = o.x;
                my_e = __float_as_int(o.y);
            }
        } else {
            for (int k = 0; k < p.top_k; ++k) {
                const float m = warp_max(best);
                if (m == -INFINITY) break;
                const int w = __ffs(__ballot_sync(kAll, best == m)) - 1;
                int e = -1;
                float s = 0.0f;
                if (lane == w) {
                    bool found = false;
                    best = -INFINITY;
#pragma unroll
                    for (int j = 0; j < NV; ++j) {
                        if (!found && c[j] == m) {
                            found = true;
                            e = e0 + j;
                            s = x[j];
                            c[j] = -INFINITY;
                        }
                        best = fmaxf(best, c[j]);
                    }
                }
                e = __shfl_sync(kAll, e, w);
                s = __shfl_sync(kAll, s, w);
                if (lane == k) {
                    my_e = e;
                    my_s = s;
                }
            }
        }
        const bool mine = lane < p.top_k;
        float w = my_s;
        if (p.renormalize) {
            if (!SIGMOID) {
                // renormalised softmax = softmax over the chosen logits, which holds
                // where every chosen score underflows, too
                const float v = my_e >= 0 ? load_logit(p, row, my_e) : -INFINITY;
                const float m = warp_max(v);
                if (my_e >= 0 && my_s == my_s) w = exp_fast(v - m);
            }
            const float t = warp_sum(w);
            w = t == 0.0f ? 0.0f : __fdiv_rn(w, t);
        }
        if (mine) {
            p.weights[row * p.top_k + lane] = w * p.scale;
            p.chosen[row * p.top_k + lane] = my_e;
            if (my_e >= 0) atomicAdd(&hist[my_e], 1);
        }
    }
    __syncthreads();
    if (gridDim.x == 1) {
        for (int e = threadIdx.x; e < p.experts; e += kThreads) p.counts[e] = hist[e];
    } else {
        for (int e = threadIdx.x; e < p.experts; e += kThreads)
            if (hist[e] != 0) atomicAdd(&p.counts[e], hist[e]);
    }
}

__device__ __forceinline__ void store_grad(const RouteParams& p, long long row, int e, float v) {
    if (p.bf16) static_cast<__nv_bfloat16*>(p.d_logits)[row * p.ld_d + e] = __float2bfloat16_rn(v);
    else static_cast<float*>(p.d_logits)[row * p.ld_d + e] = v;
}

// Four consecutive logits of a row (VEC: one load; else 32 apart, from lane).
template <bool BF16, bool VEC>
struct Row4 {
    static __device__ __forceinline__ int index(int i, int j, int lane) {
        return VEC ? 128 * i + 4 * lane + j : 128 * i + 32 * j + lane;
    }
    static __device__ __forceinline__ void load(const RouteParams& p, long long row, int i, int lane, float (&x)[4]) {
        if (VEC) {
            x[0] = x[1] = x[2] = x[3] = -INFINITY;
            if (index(i, 0, lane) < p.experts) {
                const long long at = row * p.ld + index(i, 0, lane);
                if (BF16) {
                    const uint2 r = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.logits) + at);
                    x[0] = __uint_as_float(r.x << 16);
                    x[1] = __uint_as_float(r.x & 0xffff0000u);
                    x[2] = __uint_as_float(r.y << 16);
                    x[3] = __uint_as_float(r.y & 0xffff0000u);
                } else {
                    const float4 r = *reinterpret_cast<const float4*>(static_cast<const float*>(p.logits) + at);
                    x[0] = r.x; x[1] = r.y; x[2] = r.z; x[3] = r.w;
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int e = index(i, j, lane);
                x[j] = e < p.experts ? load_logit(p, row, e) : -INFINITY;
            }
        }
    }
    static __device__ __forceinline__ void store(const RouteParams& p, long long row, int i, int lane, const float (&x)[4]) {
        if (VEC) {
            if (index(i, 0, lane) < p.experts) {
                const long long at = row * p.ld_d + index(i, 0, lane);
                if (BF16) {
                    const __nv_bfloat162 lo = __floats2bfloat162_rn(x[0], x[1]), hi = __floats2bfloat162_rn(x[2], x[3]);
                    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.d_logits) + at) =
                        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
                } else {
                    *reinterpret_cast<float4*>(static_cast<float*>(p.d_logits) + at) = make_float4(x[0], x[1], x[2], x[3]);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int e = index(i, j, lane);
                if (e < p.experts) store_grad(p, row, e, x[j]);
            }
        }
    }
};

// One warp per token.  Lane k holds the k-th chosen expert; the row's dense
// part is written first and the chosen entries over it.  N: 128-expert pieces
// of a row.  DENSE: softmax without renormalisation.
template <int N, bool BF16, bool VEC, bool DENSE>
__global__ void __launch_bounds__(kThreads) k_route_backward(const __grid_constant__ RouteParams p) {
    using R = Row4<BF16, VEC>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (long long row = static_cast<long long>(blockIdx.x) * kWarps + warp; row < p.tokens;
         row += static_cast<long long>(gridDim.x) * kWarps) {
        float s[N][4];
        if (DENSE) {
#pragma unroll
            for (int i = 0; i < N; ++i) R::load(p, row, i, lane, s[i]);
        }
        int e = -1;
        float d = 0.0f;
        if (lane < p.top_k) {
            e = p.chosen[row * p.top_k + lane];
            if (e >= p.experts) e = -1;
            if (e >= 0) d = p.d_weights[row * p.top_k + lane] * p.scale;
        }
        const float x = e >= 0 ? load_logit(p, row, e) : -INFINITY;
        float g = 0.0f;                                  // gradient of the chosen logit
        if (DENSE) {
            float m = -INFINITY;
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) m = fmaxf(m, s[i][j]);
            m = warp_max(m);
            float a = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i][j] = s[i][j] == -INFINITY ? 0.0f : exp_fast(s[i][j] - m);
                    a += s[i][j];
                }
            const float sum = warp_sum(a);
            const float inv = sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);
            const float c = e >= 0 ? exp_fast(x - m) * inv : 0.0f;
            const float dot = warp_sum(d * c);
            g = c * (d - dot);
            const float by = -dot * inv;
#pragma unroll
            for (int i = 0; i < N; ++i) {
#pragma unroll
                for (int j = 0; j < 4; ++j) s[i][j] *= by;
                R::store(p, row, i, lane, s[i]);
            }
        } else {
            const float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < N; ++i) R::store(p, row, i, lane, zero);
            float c = 0.0f, w = 1.0f;                    // score; derivative of its logarithm by the logit
            if (p.sigmoid) {
                if (e >= 0) {
                    c = sigmoid_fast(x);
                    w = 1.0f - c;
                }
            } else {
                const float m = warp_max(x);
                c = e >= 0 ? exp_fast(x - m) : 0.0f;
            }
            if (p.renormalize) {
                const float t = warp_sum(c);
                c = t == 0.0f ? 0.0f : __fdiv_rn(c, t);
                d -= warp_sum(d * c);
            }
            g = d * c * w;
        }
        __syncwarp();                                    // the dense part is written before the chosen entries
        if (e >= 0) store_grad(p, row, e, g);
    }
}

int route_grid(const RouteParams& p, int sms, int per_sm) {
    const long long need = (p.tokens + kWarps - 1) / kWarps;
    const long long cap = static_cast<long long>(sms) * per_sm;
    return static_cast<int>(need < cap ? (need > 0 ? need : 1) : cap);
}

template <int NV>
cudaError_t run_route(const RouteParams& p, int sms, cudaStream_t s) {
    const size_t smem = sizeof(int) * p.experts;
    const int grid = route_grid(p, sms, 4);
    if (grid > 1) {
        const cudaError_t e = cudaMemsetAsync(p.counts, 0, smem, s);
        if (e != cudaSuccess) return e;
    }
    if (p.sigmoid) k_route<NV, true><<<grid, kThreads, smem, s>>>(p);
    else k_route<NV, false><<<grid, kThreads, smem, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_route(const RouteParams& p, int sms, cudaStream_t s) {
    if (p.per_lane <= 1) return run_route<1>(p, sms, s);
    if (p.per_lane <= 2) return run_route<2>(p, sms, s);
    if (p.per_lane <= 4) return run_route<4>(p, sms, s);
    if (p.per_lane <= 8) return run_route<8>(p, sms, s);
    if (p.per_lane <= 12) return run_route<12>(p, sms, s);
    if (p.per_lane <= 16) return run_route<16>(p, sms, s);
    return run_route<32>(p, sms, s);
}

namespace {

template <int N, bool BF16>
cudaError_t run_backward(const RouteParams& p, int sms, cudaStream_t s) {
    const int grid = route_grid(p, sms, 8);
    const bool dense = !p.sigmoid && !p.renormalize;
    if (dense && p.vec) k_route_backward<N, BF16, true, true><<<grid, kThreads, 0, s>>>(p);
    else if (dense) k_route_backward<N, BF16, false, true><<<grid, kThreads, 0, s>>>(p);
    else if (p.vec) k_route_backward<N, BF16, true, false><<<grid, kThreads, 0, s>>>(p);
    else k_route_backward<N, BF16, false, false><<<grid, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <int N>
cudaError_t run_backward(const RouteParams& p, int sms, cudaStream_t s) {
    return p.bf16 ? run_backward<N, true>(p, sms, s) : run_backward<N, false>(p, sms, s);
}

}  // namespace

cudaError_t launch_route_backward(const RouteParams& p, int sms, cudaStream_t s) {
    if (p.experts <= 128) return run_backward<1>(p, sms, s);
    if (p.experts <= 256) return run_backward<2>(p, sms, s);
    if (p.experts <= 384) return run_backward<3>(p, sms, s);
    if (p.experts <= 512) return run_backward<4>(p, sms, s);
    return run_backward<8>(p, sms, s);
}

}  // namespace muon
