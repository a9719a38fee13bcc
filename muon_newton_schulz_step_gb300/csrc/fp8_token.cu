// The forward product for few tokens: y[t, n] = sum_k q(x)[t, k] W[n, k], with
// the rounding of x to E4M3 in the same launch.
//
// Serving makes this product for one token at a time: its time is the weight's
// bytes, read once, and the launch.  The tiled product would load 128 rows per CTA
// on a third of the SMs and needs the codes of x from a launch before it.  One token
// x 6144 x 6144: 13.8 us by tiles, 9.2 here (12.3 with the weight from memory, 3.1 TB/s;
// the launch and the rounding of x take about 4).  With experts the tiles fill the SMs
// and win (32 tokens over 16 experts of 2048 x 6144: 43 us against 56 here), so this
// kernel serves single weights.
//
// A block takes 16 rows of the weight, its eight warps take the reduction's
// blocks of 128 in turn.  A lane reads 16 consecutive bytes of a row at a time (the
// matrix fragments want 4 here and 4 there: the reduction index is permuted within
// 64, the same way for both operands), so a warp has several KB on their way, and
// the products of a block of 128 run on mma.sync: 16 rows x 8 tokens cost no more
// than one token.  (tcgen05 has nothing to add: the tensor core idles either way,
// and its operands would take a trip through shared memory.)  The block rounds x
// into shared memory itself, while its first weight bytes are under way.  Streaming
// the weight through shared memory by bulk copies was no faster from memory (12.2
// against 12.5 us) and slower from L2 (11.8 against 10.4).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fp8_codes.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = 8;
constexpr int kRows = 16;            // weight rows per block
constexpr int kTokens = 8;           // most tokens: one matrix fragment's
constexpr int kRound = 2;            // blocks of x that half a warp loads at a time
constexpr int kAhead = 3;            // blocks of 128 of the reduction that a warp loads at a time
constexpr int kMaxCodes = 100 * 1024;
constexpr int kSms = 152;

__device__ __forceinline__ uint4 load_stream(const uint8_t* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Weight codes of one block of 128 for a 16-row fragment: rows lane / 4 and + 8,
// bytes 16 (lane % 4) of either half.
struct WeightBlock {
    uint4 v[2][2];
    __device__ __forceinline__ void load(const uint8_t* lo, const uint8_t* hi, int kb) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            v[0][h] = load_stream(lo + kb * 128 + 64 * h);
            v[1][h] = load_stream(hi + kb * 128 + 64 * h);
        }
    }
};

// Eight consecutive elements of a token from column col on; zero past the last.
template <bool BF16>
__device__ __forceinline__ Raw load_eight(const Fp8TokenParams& p, long long row, int col) {
    Raw r;
    r.a = r.b = make_uint4(0, 0, 0, 0);
    if (p.vec && col + 8 <= p.k) {
        const char* s = static_cast<const char*>(p.x) + (row * p.ld_x + col) * (BF16 ? 2 : 4);
        r.a = *reinterpret_cast<const uint4*>(s);
        if (!BF16) r.b = *reinterpret_cast<const uint4*>(s + 16);
        return r;
    }
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        w[i] = 0;
        const long long at = row * p.ld_x + col + i;
        if (col + i < p.k)
            w[i] = BF16 ? static_cast<uint32_t>(static_cast<const uint16_t*>(p.x)[at]) : static_cast<const uint32_t*>(p.x)[at];
    }
    if (BF16) {
        r.a = make_uint4(w[0] | (w[1] << 16), w[2] | (w[3] << 16), w[4] | (w[5] << 16), w[6] | (w[7] << 16));
    } else {
        r.a = make_uint4(w[0], w[1], w[2], w[3]);
        r.b = make_uint4(w[4], w[5], w[6], w[7]);
    }
    return r;
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 3) k_fp8_token(const __grid_constant__ Fp8TokenParams p) {
    extern __shared__ uint4 smem[];                      // the tokens' codes, then their exponents
    __shared__ float part[kWarps][kTokens][kRows];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int blocks = static_cast<int>(p.ldk >> 7);
    // rows of codes 64 bytes apart modulo 128: two tokens' 16-byte reads meet no bank conflict
    const int pitch = static_cast<int>(p.ldk) + 64;
    uint8_t* const codes = reinterpret_cast<uint8_t*>(smem);
    int16_t* const exps = reinterpret_cast<int16_t*>(codes + p.tokens * pitch);

    const int n0 = blockIdx.x * kRows;
    const int r = lane >> 2, j = lane & 3;
    // rows past the last read the last one's codes; their results are not stored
    const uint8_t* lo = p.w + 16 * j + static_cast<long long>(min(n0 + r, p.n - 1)) * p.ldk;
    const uint8_t* hi = p.w + 16 * j + static_cast<long long>(min(n0 + r + 8, p.n - 1)) * p.ldk;
    const uint8_t* ws = p.w_scale + static_cast<long long>(n0 >> 7) * blocks;
    WeightBlock wb[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (warp + i * kWarps < blocks) wb[i].load(lo, hi, warp + i * kWarps);

    // half a warp rounds one block of 128, eight elements a lane, kRound blocks at a time
    {
        const int c = threadIdx.x & 15;
        constexpr int kStep = kThreads / 16;
        const uint32_t half = 0xffffu << (lane & 16);
        int t = 0, kb = threadIdx.x >> 4;
        auto settle = [&] {
            while (kb >= blocks) {
                kb -= blocks;
                ++t;
            }
        };
        settle();
        while (t < p.tokens) {
            Raw x[kRound];
            int at[kRound], kbs[kRound];
#pragma unroll
            for (int u = 0; u < kRound; ++u) {
                at[u] = t;
                kbs[u] = kb;
                if (t < p.tokens) x[u] = load_eight<BF16>(p, t, kb * 128 + 8 * c);
                kb += kStep;
                settle();
            }
#pragma unroll
            for (int u = 0; u < kRound; ++u) {
                if (at[u] >= p.tokens) break;
                uint32_t top = row_max<BF16>(x[u]);
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(half, top, o));
                if (top >= kInf) {                       // of the whole half warp
                    top = row_max<BF16>(replace_odd<BF16>(x[u], true));
#pragma unroll
                    for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(half, top, o));
                    x[u] = replace_odd<BF16>(x[u], false);
                }
                const int e = scale_exponent(top);
                *reinterpret_cast<uint2*>(codes + at[u] * pitch + kbs[u] * 128 + 8 * c) =
                    codes_of<BF16>(x[u], inverse_scale(e));
                if (c == 0) exps[at[u] * blocks + kbs[u]] = static_cast<int16_t>(e);
            }
        }
    }
    __syncthreads();

    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    // as B fragment a lane holds token r; as accumulator tokens 2 j and 2 j + 1
    const uint8_t* mine = codes + r * pitch + 16 * j;
    const bool have = r < p.tokens;
    const int16_t* e0p = exps + min(2 * j, p.tokens - 1) * blocks;
    const int16_t* e1p = exps + min(2 * j + 1, p.tokens - 1) * blocks;
    for (int kb0 = warp; kb0 < blocks; kb0 += kAhead * kWarps) {
        if (kb0 != warp) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (kb0 + i * kWarps < blocks) wb[i].load(lo, hi, kb0 + i * kWarps);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int kb = kb0 + i * kWarps;
            if (kb >= blocks) break;
            float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint4 b = make_uint4(0, 0, 0, 0);
                if (have) b = *reinterpret_cast<const uint4*>(mine + kb * 128 + 64 * h);
                const uint4 &u = wb[i].v[0][h], &v = wb[i].v[1][h];
                mma_e4m3(c, u.x, v.x, u.y, v.y, b.x, b.y);
                mma_e4m3(c, u.z, v.z, u.w, v.w, b.z, b.w);
            }
            // both scales as one exponent, in two factors that cannot leave fp32 on their own
            const int ew = static_cast<int>(ws[kb]) - 127;
            const int e0 = e0p[kb] + ew, e1 = e1p[kb] + ew;
            const float a0 = power_of_two(e0 >> 1), b0 = power_of_two(e0 - (e0 >> 1));
            const float a1 = power_of_two(e1 >> 1), b1 = power_of_two(e1 - (e1 >> 1));
            acc[0] = fmaf(c[0] * a0, b0, acc[0]);
            acc[1] = fmaf(c[1] * a1, b1, acc[1]);
            acc[2] = fmaf(c[2] * a0, b0, acc[2]);
            acc[3] = fmaf(c[3] * a1, b1, acc[3]);
        }
    }
    // accumulator: rows r, r + 8; tokens 2 j, 2 j + 1
    part[warp][2 * j][r] = acc[0];
    part[warp][2 * j + 1][r] = acc[1];
    part[warp][2 * j][r + 8] = acc[2];
    part[warp][2 * j + 1][r + 8] = acc[3];
    __syncthreads();
    if (threadIdx.x < kTokens * kRows) {
        const int t = threadIdx.x / kRows, n = threadIdx.x % kRows;
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) s += part[i][t][n];
        if (t < p.tokens && n0 + n < p.n) {
            const long long at = t * p.ld_out + n0 + n;
            if (p.out_f32) static_cast<float*>(p.out)[at] = s;
            else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(s);
        }
    }
}

size_t token_smem(int tokens, long long ldk) { return static_cast<size_t>(tokens) * (ldk + 64 + ldk / 128 * 2); }

template <bool BF16>
cudaError_t run(const Fp8TokenParams& p, cudaStream_t s) {
    const size_t smem = token_smem(p.tokens, p.ldk);
    const cudaError_t e =
        smem > 40 * 1024 ? cudaFuncSetAttribute(k_fp8_token<BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxCodes)
                         : cudaSuccess;
    if (e != cudaSuccess) return e;
    k_fp8_token<BF16><<<(p.n + kRows - 1) / kRows, kThreads, smem, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

// Whether this kernel serves a call: the tokens take one matrix fragment, their codes
// fit in shared memory, the blocks are resident at once (three per SM), and rounding x
// in every block costs no more than tiles and the launch that they need for it.  That
// costs 1.35 us per token and 6144 elements of k, and 2 us and n / 1280 us per 6144 the
// rest; tiles take 6 us more to begin with, 0.4 + n / 10300 less per 6144.  Measured, this
// kernel against tiles, the weight in L2: 3 tokens x 6144 x 6144 12.9 us, 13.8; 4 tokens
// 14.3; 4 x 2048 x 6144 9.7, 11.4; 8 tokens 14.9; 8 x 6144 x 2048 8.7, 9.7; 1 x 16384 x
// 6144 26.0, 24.2.  The SMs are this part's 152 and not asked for: the workspace's size
// depends on the rule, and follows from sizes alone.
bool fp8_token_serves(long long tokens, long long n, long long k) {
    const long long ldk = (k + 127) / 128 * 128;
    return tokens <= kTokens && token_smem(static_cast<int>(tokens), ldk) <= static_cast<size_t>(kMaxCodes) &&
           n <= kSms * 3 * kRows && k * (14000 * (tokens - 1) + 4000 + n) <= 310000000ll;
}

cudaError_t launch_fp8_token(const Fp8TokenParams& p, cudaStream_t s) {
    return p.bf16 ? run<true>(p, s) : run<false>(p, s);
}

}  // namespace muon
