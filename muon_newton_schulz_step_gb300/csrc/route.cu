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
// in registers.  The top_k-th largest lane maximum bounds the choice from
// below.  The few experts at or
// above that bound (8 to about 12 of 384) are written to shared memory in index
// order, a lane takes one each and counts those before it: its place in the
// result.  Should more than 32 qualify (equal values, few lanes left), the
// largest is taken top_k times instead.  The choice works on scores from one ex2 and
// one rcp; the weights of the chosen are computed anew.  Bound by instructions:
// 32768 tokens x 384 experts in fp32, 4 of 8 groups: 73 us with the largest taken
// top_k times for every token (about 1400 instructions each), 45 with the bound and
// full-accuracy scores (1050), 34 now (780, four blocks per SM in one wave).
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

// For the choice: 2^x and 1 / x in one instruction each.  e^x by them is off by
// |x| 2^-24 on top of 2 ulp; the weights of what is chosen are computed anew.
__device__ __forceinline__ float exp2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

constexpr float kLog2e = 1.44269504f;

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

// Blocks per SM: the grid is that many, so that all are resident at once.
template <int NV>
constexpr int route_blocks() {
    return NV <= 4 ? 6 : NV <= 12 ? 4 : 2;
}

template <int NV, bool SIGMOID>
__global__ void __launch_bounds__(kThreads, route_blocks<NV>()) k_route(const __grid_constant__ RouteParams p) {
    extern __shared__ int hist[];
    __shared__ float2 pool[kWarps][32];                  // choice value, expert
    __shared__ int order[kWarps][32];                    // experts by place
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
    bool odd_bias = false;                               // of any lane: some bias is not finite
#pragma unroll
    for (int j = 0; j < NV; ++j) odd_bias |= !(fabsf(bias[j]) <= FLT_MAX);
    odd_bias = __any_sync(kAll, odd_bias);

    for (long long row = static_cast<long long>(blockIdx.x) * kWarps + warp; row < p.tokens;
         row += static_cast<long long>(gridDim.x) * kWarps) {
        float c[NV];                                     // logits, then choice values; -inf: masked
        load_lane<NV>(p, row, e0, n, c);
        float top = 0.0f, inv = 1.0f;                    // softmax: largest logit, 1 / sum
        float seen = 0.0f;                               // not finite: masked experts or NaN in this lane
        if (SIGMOID) {
#pragma unroll
            for (int j = 0; j < NV; ++j) seen += c[j];
        } else {
            float m = -INFINITY;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                m = fmaxf(m, c[j]);
                seen += c[j];
            }
            top = warp_max(m);
        }
        const bool plain = __all_sync(kAll, fabsf(seen) <= FLT_MAX) && top > -FLT_MAX;
        uint32_t masked = 0;                             // bit j: no expert, or masked
        if (!plain) {
#pragma unroll
            for (int j = 0; j < NV; ++j) masked |= (c[j] == -INFINITY ? 1u : 0u) << j;
        }
        if (SIGMOID) {
#pragma unroll
            for (int j = 0; j < NV; ++j) c[j] = rcp_approx(1.0f + exp2_approx(c[j] * -kLog2e));
        } else {
            float a = 0.0f;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                c[j] = exp2_approx((c[j] - top) * kLog2e);
                if (!plain && (masked >> j & 1u)) c[j] = 0.0f;
                a += c[j];
            }
            inv = __fdiv_rn(1.0f, warp_sum(a));
#pragma unroll
            for (int j = 0; j < NV; ++j) c[j] *= inv;
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) c[j] += bias[j];
        if (!plain || odd_bias) {
            // a NaN orders below every number
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const float v = c[j] == c[j] ? c[j] : -FLT_MAX;
                c[j] = masked >> j & 1u ? -INFINITY : v;
            }
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
        // a bound that at least top_k choice values reach: take the largest lane maximum
        // away top_k times (equal ones together: the bound is then lower)
        float bound = -INFINITY, v = best;
        for (int k = 0; k < p.top_k; ++k) {
            bound = warp_max(v);
            v = v == bound ? -INFINITY : v;
        }
        int cnt = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j) cnt += c[j] >= bound;
        const int upto = warp_inclusive_sum(cnt);
        const int total = __shfl_sync(kAll, upto, 31);
        int my_e = -1;
        if (bound > -INFINITY && total <= 32) {
            float2* at = &pool[warp][upto - cnt];
            if (cnt > 0) {
#pragma unroll
                for (int j = 0; j < NV; ++j)
                    if (c[j] >= bound) *at++ = make_float2(c[j], __int_as_float(e0 + j));
            }
            __syncwarp();
            const float2 f = pool[warp][lane];
            const float mine = lane < total ? f.x : -INFINITY;
            int place = 0;
            for (int i = 0; i < total; ++i) {
                const float o = __shfl_sync(kAll, mine, i);
                place += o > mine || (o == mine && i < lane);
            }
            if (lane < total && place < p.top_k) order[warp][place] = __float_as_int(f.y);
            __syncwarp();                                // and the pool has been read
            if (lane < p.top_k) my_e = order[warp][lane];
        } else {
            for (int k = 0; k < p.top_k; ++k) {
                const float m = warp_max(best);
                if (m == -INFINITY) break;
                const int w = __ffs(__ballot_sync(kAll, best == m)) - 1;
                int e = -1;
                if (lane == w) {
                    bool found = false;
                    best = -INFINITY;
#pragma unroll
                    for (int j = 0; j < NV; ++j) {
                        if (!found && c[j] == m) {
                            found = true;
                            e = e0 + j;
                            c[j] = -INFINITY;
                        }
                        best = fmaxf(best, c[j]);
                    }
                }
                e = __shfl_sync(kAll, e, w);
                if (lane == k) my_e = e;
            }
        }
        // the scores of the chosen, from their logits
        float w = 0.0f;
        const float logit = my_e >= 0 ? load_logit(p, row, my_e) : -INFINITY;
        if (SIGMOID) {
            if (my_e >= 0) w = sigmoid_fast(logit);
        } else {
            // renormalised softmax = softmax over the chosen logits, which holds where
            // every chosen score underflows, too (a NaN sum stays one)
            const float m = p.renormalize ? warp_max(logit) : top;
            if (my_e >= 0) w = exp_fast(logit - m) * (p.renormalize ? (inv == inv ? 1.0f : inv) : inv);
        }
        if (p.renormalize) {
            const float t = warp_sum(w);
            w = t == 0.0f ? 0.0f : __fdiv_rn(w, t);
        }
        if (lane < p.top_k) {
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
            const float m0 = m == -INFINITY ? 0.0f : m;   // every expert masked: all scores zero
            float a = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i][j] = exp2_approx((s[i][j] - m0) * kLog2e);
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
    const int grid = route_grid(p, sms, route_blocks<NV>());
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
