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
// One warp per token.  A group owns `lanes` lanes, a lane `per_lane`
// consecutive experts of one group, in index order over the warp: so the lowest
// index among equal values is the lowest lane's, a group's two largest values
// meet in log2(lanes) exchanges for all groups at once, and everything stays
// in registers.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

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

// Order-preserving image of a float in unsigned integers; 0: masked.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __float_as_uint(v);
    if (v != v) return 0x00800000u;                     // NaN: below every number
    if (v == -INFINITY) return 0u;
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    return v;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

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
        uint32_t key[NV];
        load_lane<NV>(p, row, e0, n, x);
        // scores
        float top = 0.0f, sum = 1.0f;
        if (!SIGMOID) {
            float m = -INFINITY;
            bool nan = false;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                m = fmaxf(m, x[j]);
                nan |= x[j] != x[j];
            }
            top = warp_max(m);
            float a = 0.0f;
#pragma unroll
            for (int j = 0; j < NV; ++j) a += x[j] == -INFINITY ? 0.0f : expf(x[j] - top);
            sum = warp_sum(nan ? NAN : a);
        }
        float c[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const float s = SIGMOID ? __fdiv_rn(1.0f, 1.0f + expf(-x[j])) : __fdiv_rn(expf(x[j] - top), sum);
            c[j] = x[j] == -INFINITY ? -INFINITY : s + bias[j];
            x[j] = s;
        }
        // group scores
        bool keep = true;
        if (p.groups > 1) {
            float m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const float v = c[j] == c[j] ? c[j] : -INFINITY;
                m2 = fmaxf(m2, fminf(m1, v));
                m1 = fmaxf(m1, v);
            }
            for (int o = p.lanes >> 1; o > 0; o >>= 1) {
                const float o1 = __shfl_xor_sync(kAll, m1, o), o2 = __shfl_xor_sync(kAll, m2, o);
                m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
                m1 = fmaxf(m1, o1);
            }
            const uint32_t gk = order_key(m2 == -INFINITY ? m1 : m1 + m2);
            int before = 0;
            for (int g = 0; g < p.groups; ++g) {
                const uint32_t k = __shfl_sync(kAll, gk, g * p.lanes);
                before += k > gk || (k == gk && g < group);
            }
            keep = before < p.top_groups;
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) key[j] = keep ? order_key(c[j]) : 0u;
        // the top_k largest, one after the other
        uint32_t best = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j) best = max(best, key[j]);
        int my_e = -1;
        float my_s = 0.0f;
        for (int k = 0; k < p.top_k; ++k) {
            const uint32_t m = __reduce_max_sync(kAll, best);
            int e = -1;
            float s = 0.0f;
            if (m != 0u) {
                const int w = __ffs(__ballot_sync(kAll, best == m)) - 1;
                if (lane == w) {
                    bool found = false;
                    best = 0;
#pragma unroll
                    for (int j = 0; j < NV; ++j) {
                        if (!found && key[j] == m) {
                            found = true;
                            e = e0 + j;
                            s = x[j];
                            key[j] = 0u;
                        }
                        best = max(best, key[j]);
                    }
                }
                e = __shfl_sync(kAll, e, w);
                s = __shfl_sync(kAll, s, w);
            }
            if (lane == k) {
                my_e = e;
                my_s = s;
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
                if (my_e >= 0 && my_s == my_s) w = expf(v - m);
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

// One warp per token.  Lane k holds the k-th chosen expert; the row's dense
// part is written first and the chosen entries over it.
__global__ void __launch_bounds__(kThreads) k_route_backward(const __grid_constant__ RouteParams p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool dense = !p.sigmoid && !p.renormalize;
    for (long long row = static_cast<long long>(blockIdx.x) * kWarps + warp; row < p.tokens;
         row += static_cast<long long>(gridDim.x) * kWarps) {
        int e = -1;
        float d = 0.0f;
        if (lane < p.top_k) {
            e = p.chosen[row * p.top_k + lane];
            if (e >= p.experts) e = -1;
            if (e >= 0) d = p.d_weights[row * p.top_k + lane] * p.scale;
        }
        const float x = e >= 0 ? load_logit(p, row, e) : -INFINITY;
        float g = 0.0f;                                  // gradient of the chosen logit
        if (dense) {
            float m = -INFINITY;
            for (int i = lane; i < p.experts; i += 32) m = fmaxf(m, load_logit(p, row, i));
            m = warp_max(m);
            float a = 0.0f;
            for (int i = lane; i < p.experts; i += 32) {
                const float v = load_logit(p, row, i);
                a += v == -INFINITY ? 0.0f : expf(v - m);
            }
            const float sum = warp_sum(a);
            const float s = e >= 0 ? __fdiv_rn(expf(x - m), sum) : 0.0f;
            const float dot = warp_sum(d * s);
            g = s * (d - dot);
            for (int i = lane; i < p.experts; i += 32) {
                const float v = load_logit(p, row, i);
                store_grad(p, row, i, v == -INFINITY ? 0.0f : -__fdiv_rn(expf(v - m), sum) * dot);
            }
        } else {
            for (int i = lane; i < p.experts; i += 32) store_grad(p, row, i, 0.0f);
            float s = 0.0f, w = 1.0f;                    // score; derivative of the score's logarithm by the logit
            if (p.sigmoid) {
                if (e >= 0) {
                    s = __fdiv_rn(1.0f, 1.0f + expf(-x));
                    w = 1.0f - s;
                }
            } else {
                const float m = warp_max(x);
                s = e >= 0 ? expf(x - m) : 0.0f;
            }
            if (p.renormalize) {
                const float t = warp_sum(s);
                s = t == 0.0f ? 0.0f : __fdiv_rn(s, t);
                d -= warp_sum(d * s);
            }
            g = d * s * w;
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

cudaError_t launch_route_backward(const RouteParams& p, int sms, cudaStream_t s) {
    k_route_backward<<<route_grid(p, sms, 8), kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace muon
