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
// Forward: a warp chooses for one token.  A group owns `lanes` lanes, a lane
// `per_lane` consecutive experts of one group, in index order over the warp: so a
// group's two largest values meet in log2(lanes) exchanges for all groups at once, and
// everything stays in registers.  The top_k-th largest lane maximum bounds the choice
// from below, and the few experts at or above that bound (8 to about 12 of 384) are
// noted in shared memory.  Should more than a pool of them qualify (equal values), or
// fewer lanes than top_k have an expert left, the largest is taken top_k times instead.
// Then a lane takes one each, makes its choice value again from its logit by the same
// operations, counts those before it (its place in the result), and computes its weight
// anew at full accuracy.  Two tokens go through that second half side by side, 16 lanes
// each, where top_k and the number of tokens allow it.  The choice works on scores from
// one ex2 and one rcp, and takes those below 2^-126 as zero, so as equal.  Bound by
// instructions:
// 32768 tokens x 384 experts in fp32, 4 of 8 groups: 73 us with the largest taken
// top_k times for every token (about 1400 instructions each), 45 with the bound and
// full-accuracy scores (1050), 34 with approximate ones (780), 28 with the second half
// for two tokens at once (issue slots 72 % busy), 25.4 with the counts zeroed beside
// it.  As it is now (609 a token; softmax 645), with biases: 27.9, softmax 24.4; 64 experts,
// softmax, one group 18.7.  (Approximate divisions would save half a microsecond, and leave
// the weights of a token 4e-9 above their sum on average.)
//
// Backward: one warp per token, lanes striped over the row in vectors of four.
// Scores of the chosen are recomputed from their logits; only the softmax without
// renormalisation reads the row.  Bound by the chain from a choice to its logits to
// the sums over them, so the next token's choice is loaded a token ahead: 32768 x 384
// without renormalisation, in L2, fp32 15.8 -> 13.4 us, bf16 12.1 -> 11.6; 32768 x 1000
// in fp32 43.3 -> 40.7 (6.4 TB/s).  On the chosen alone (32768 x 384, in L2): fp32 11.2 us,
// bf16 9.4.
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

// e^x to 6 * 2^-24 (ex2's 2^-22 and two roundings): 2^k with k = x log2(e) rounded,
// times 1 + (what the rounding left) ln 2.  Arguments beyond +-200 give infinity and zero, NaN gives NaN.
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

// e^(x - max): the difference first.  x log2(e) - (max log2(e) rounded), one operation
// less, is off by up to half a unit in the last place of max log2(e) in the exponent:
// 1e-5 of the scores at 200, and no number at all from 1e9 on.
__device__ __forceinline__ float exp_choice(float x, float max) { return exp2_approx((x - max) * kLog2e); }

// A choice value as the choice compares it: a NaN as -FLT_MAX, and every finite number
// above that.  -inf (masked by its bias) stays.
__device__ __forceinline__ float ordered(float c) {
    if (c != c) return -FLT_MAX;
    return c == -FLT_MAX ? -3.40282326e38f : c;
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

// Blocks per SM: the grid is that many, so that all are resident at once.
template <int NV>
constexpr int route_blocks() {
    return NV <= 4 ? 6 : NV <= 12 ? 4 : 2;
}

// W: lanes that finish one token, 16 (then a warp finishes two at once) or 32.
template <int NV, bool SIGMOID, int W>
__global__ void __launch_bounds__(kThreads, route_blocks<NV>()) k_route(const __grid_constant__ RouteParams p) {
    extern __shared__ int hist[];
    __shared__ int pool[kWarps][32];                     // experts at or above the bound
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t below = (1u << lane) - 1u;
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

    constexpr int kTokens = 32 / W;
    const int sub = lane & (W - 1), which = lane / W;
    const long long step = static_cast<long long>(gridDim.x) * kWarps * kTokens;
    for (long long row0 = (static_cast<long long>(blockIdx.x) * kWarps + warp) * kTokens; row0 < p.tokens; row0 += step) {
        // of this lane's token: candidates, and what their scores need
        int total = 0;
        float top = 0.0f, inv = 1.0f;
#pragma unroll 1
        for (int h = 0; h < kTokens; ++h) {
            const long long row = row0 + h;
            if (row >= p.tokens) break;
            float c[NV];                                     // logits, then choice values; -inf: masked
            load_lane<NV>(p, row, e0, n, c);
            float max_x = 0.0f, norm = 1.0f;                 // softmax: largest logit, 1 / sum
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
                m = warp_max(m);
                if (m > -INFINITY) max_x = m;                // every expert masked: all scores zero
            }
            const bool plain = __all_sync(kAll, fabsf(seen) <= FLT_MAX);
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
                for (int j = 0; j < NV; ++j) a += c[j] = exp_choice(c[j], max_x);
                norm = __frcp_rn(warp_sum(a));
            }
            if (which == h) {
                top = max_x;
                inv = norm;
            }
#pragma unroll
            for (int j = 0; j < NV; ++j) c[j] = SIGMOID ? __fadd_rn(c[j], bias[j]) : fmaf(c[j], norm, bias[j]);
            const bool odd = !plain || odd_bias;             // some may be masked or NaN
            if (odd) {
#pragma unroll
                for (int j = 0; j < NV; ++j) c[j] = masked >> j & 1u ? -INFINITY : ordered(c[j]);
            }
            // group scores
            float best = -INFINITY;
            bool kept = true;                                // this lane's group
            if (p.groups > 1) {
                float m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    m2 = fmaxf(m2, fminf(m1, c[j]));
                    m1 = fmaxf(m1, c[j]);
                }
                best = m1;
                for (int o = p.lanes >> 1; o > 0; o >>= 1) {
                    const float o1 = __shfl_xor_sync(kAll, m1, o), o2 = __shfl_xor_sync(kAll, m2, o);
                    m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
                    m1 = fmaxf(m1, o1);
                }
                // one expert left (or one that is not NaN): its own; a finite bias of
                // -FLT_MAX is a number like any other
                const float gv = m2 <= (odd ? -FLT_MAX : -INFINITY) ? m1 : m1 + m2;
                int before = 0;                              // groups ahead of this one: each lane compares some
                for (int g = 0; g < p.groups; g += p.lanes) {
                    const int other = g + in_group;
                    const float v = __shfl_sync(kAll, gv, other * p.lanes);
                    before += other < p.groups && (v > gv || (v == gv && other < group));
                }
                for (int o = p.lanes >> 1; o > 0; o >>= 1) before += __shfl_xor_sync(kAll, before, o);
                kept = before < p.top_groups;
                if (!kept) best = -INFINITY;
            } else {
#pragma unroll
                for (int j = 0; j < NV; ++j) best = fmaxf(best, c[j]);
            }
            // a bound that at least top_k choice values reach: take the largest lane maximum
            // away top_k times (equal ones together: the bound is then lower)
            float bound = -INFINITY, v = best;
            auto lower = [&] {
                bound = warp_max(v);
                v = v == bound ? -INFINITY : v;
            };
            int k = p.top_k;
            for (; k >= 4; k -= 4) {
                lower();
                lower();
                lower();
                lower();
            }
            for (; k > 0; --k) lower();
            // the experts that reach it, a round for each lane's first, second, ...
            uint32_t mine = 0;
#pragma unroll
            for (int j = 0; j < NV; ++j) mine |= (c[j] >= bound ? 1u : 0u) << j;
            if (!kept) mine = 0;
            int n_at = 0;                                    // candidates
            if (bound > -INFINITY) {
                for (uint32_t with = __ballot_sync(kAll, mine != 0); with != 0; with = __ballot_sync(kAll, mine != 0)) {
                    const int at = n_at + __popc(with & below);
                    if (mine != 0 && at < W) pool[warp][W * h + at] = e0 + __ffs(mine) - 1;
                    mine &= mine - 1;
                    n_at += __popc(with);
                }
            }
            if (n_at < p.top_k || n_at > W) {
                // few lanes have an expert left, or many values are equal: the largest, top_k times
                __syncwarp();
                n_at = 0;
                if (!kept) {
#pragma unroll
                    for (int j = 0; j < NV; ++j) c[j] = -INFINITY;
                }
                for (; n_at < p.top_k; ++n_at) {
                    const float m = warp_max(best);
                    if (m == -INFINITY) break;
                    const int w = __ffs(__ballot_sync(kAll, best == m)) - 1;
                    if (lane == w) {
                        bool found = false;
                        best = -INFINITY;
#pragma unroll
                        for (int j = 0; j < NV; ++j) {
                            if (!found && c[j] == m) {
                                found = true;
                                pool[warp][W * h + n_at] = e0 + j;
                                c[j] = -INFINITY;
                            }
                            best = fmaxf(best, c[j]);
                        }
                    }
                }
            }
            if (which == h) total = n_at;
        }
        // The candidates' order: a lane takes one, and counts those before it.  Their
        // choice values are made again, by the same operations, from their logits.
        __syncwarp();
        const long long row = row0 + which;
        int my_e = -1;
        float logit = -INFINITY, value = -INFINITY;
        if (sub < total) {
            my_e = pool[warp][lane];
            logit = load_logit(p, row, my_e);
            const float b = p.bias != nullptr ? p.bias[my_e] : 0.0f;
            if (SIGMOID) value = __fadd_rn(rcp_approx(1.0f + exp2_approx(logit * -kLog2e)), b);
            else value = fmaf(exp_choice(logit, top), inv, b);
            value = ordered(value);
        }
        __syncwarp();                                    // the pool has been read
        int most = total;
        if (W < 32) most = max(total, __shfl_xor_sync(kAll, total, W & 31));
        int place = 0;
        for (int i = 0; i < most; i += 4) {
#pragma unroll
            for (int u = 0; u < 4; ++u) place += __shfl_sync(kAll, value, i + u, W) > value;
        }
        // places that nobody has: some values are equal, and go by index
        const uint32_t taken = __reduce_or_sync(kAll, sub < total ? 1u << (W * which + place) : 0u);
        if (__popc(taken) != __popc(__ballot_sync(kAll, sub < total))) {
            for (int i = 0; i < most; ++i) {
                const float o = __shfl_sync(kAll, value, i, W);
                const int e = __shfl_sync(kAll, my_e, i, W);
                place += o == value && e < my_e;
            }
        }
        if (sub >= total) {
            place = sub;                                 // no expert: -1 in the places left over
        } else if (place >= p.top_k) {
            my_e = -1;
            logit = -INFINITY;
        }
        // the scores of the chosen, from their logits
        float w = 0.0f;
        if (SIGMOID) {
            if (my_e >= 0) w = sigmoid_fast(logit);
        } else {
            // renormalised softmax = softmax over the chosen logits, which holds where
            // every chosen score underflows, too (a NaN sum stays one)
            float m = top;
            if (p.renormalize) {
                m = logit;
#pragma unroll
                for (int o = W / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
            }
            if (my_e >= 0) w = exp_fast(logit - m) * (p.renormalize ? (inv == inv ? 1.0f : inv) : inv);
        }
        if (p.renormalize) {
            float sum = w;
#pragma unroll
            for (int o = W / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
            w = sum == 0.0f ? 0.0f : __fdiv_rn(w, sum);
        }
        if (row < p.tokens && place < p.top_k) {
            p.weights[row * p.top_k + place] = w * p.scale;
            p.chosen[row * p.top_k + place] = my_e;
            if (my_e >= 0) atomicAdd(&hist[my_e], 1);
        }
    }
    __syncthreads();
    if (gridDim.x == 1) {
        for (int e = threadIdx.x; e < p.experts; e += kThreads) p.counts[e] = hist[e];
    } else {
        asm volatile("griddepcontrol.wait;" ::: "memory");   // the counts are zero
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
    const long long step = static_cast<long long>(gridDim.x) * kWarps;
    // the next token's choice is on its way a token ahead: its logits wait for it
    int next_e = -1;
    float next_d = 0.0f;
    auto fetch = [&](long long row) {
        if (lane < p.top_k && row < p.tokens) {
            next_e = p.chosen[row * p.top_k + lane];
            next_d = p.d_weights[row * p.top_k + lane];
        }
    };
    long long row = static_cast<long long>(blockIdx.x) * kWarps + warp;
    fetch(row);
    for (; row < p.tokens; row += step) {
        float s[N][4];
        if (DENSE) {
#pragma unroll
            for (int i = 0; i < N; ++i) R::load(p, row, i, lane, s[i]);
        }
        const int e = next_e < p.experts ? next_e : -1;
        float d = e >= 0 ? next_d * p.scale : 0.0f;
        const float x = e >= 0 ? load_logit(p, row, e) : -INFINITY;
        fetch(row + step);
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
                    const float t = exp_fast(-x);
                    c = __fdividef(1.0f, 1.0f + t);
                    w = t <= FLT_MAX ? t * c : 1.0f;     // 1 - c would have no bits left near c = 1
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

__global__ void k_zero_counts(int* counts, int experts) {
    asm volatile("griddepcontrol.launch_dependents;");
    for (int e = threadIdx.x; e < experts; e += kThreads) counts[e] = 0;
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
    // two tokens at once only where every warp has several
    const bool two = p.top_k <= 16 && p.tokens > static_cast<long long>(grid) * kWarps;
    const auto kernel = two ? (p.sigmoid ? k_route<NV, true, 16> : k_route<NV, false, 16>)
                            : (p.sigmoid ? k_route<NV, true, 32> : k_route<NV, false, 32>);
    if (grid == 1) {
        kernel<<<grid, kThreads, smem, s>>>(p);
        return cudaGetLastError();
    }
    // The counts are added up over the blocks.  Their zeroing starts when what came before
    // has ended, and the routing beside it: only its last step waits.  With a memset in
    // front: 600 tokens x 384 experts 8.2 us against 5.0, 32768 tokens 28.4 against 25.0.
    k_zero_counts<<<1, kThreads, 0, s>>>(p.counts, p.experts);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kernel, p);
    return e != cudaSuccess ? e : cudaGetLastError();
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
