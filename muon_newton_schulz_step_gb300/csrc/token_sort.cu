// The routed entries sorted by expert: a stable counting sort.
//
// An entry's bucket is its expert's number here plus one, or 0 where its expert
// is not held here.  place = (entries of smaller buckets) + (earlier entries of its
// own bucket); order is the inverse, offsets[e] the start of bucket e + 1.
//
// 12 bytes an entry are all that has to move (262144 entries: 0.5 us), so this is
// bound by latency: as few launches and as short chains as can be.  A block takes
// 2048 entries at a time, a warp 128 in a row, four times 32: lanes of one bucket
// find each other by votes, and the count of those before is their rank in the
// warp; a column sum over the warps' counts turns it into the rank in the block.
// Up to kSortAlone entries one block does it all; past that the first of two launches
// leaves each block's counts (at most kSortMaxBlocks, each of an equal run of entries),
// and every block of the second adds the table up for itself, which reads
// 128 x (experts + 1) counts from L2 and saves a launch and a chain of waits between
// blocks.  The second launch's set-up overlaps the first.  Device time: one token's 8 entries
// 2.7 us, 262144 entries of 96 experts 9.0, of 384 experts 13.5, 2 million of 96 70.  All sums are of whole
// numbers: results do not depend on the order of atomics.
#include <cuda_runtime.h>

#include "groups.cuh"
#include "internal.h"
#include "sort_split.h"

namespace muon {
namespace {

constexpr int kThreads = kSortThreads;
constexpr int kWarps = kThreads / 32;
constexpr int kRounds = kSortRounds;
constexpr int kChunk = kSortChunk;

__device__ __forceinline__ int bucket_of(const SortParams& p, int expert) {
    // as unsigned numbers: what lies below `first` wraps to the far end
    const unsigned e = static_cast<unsigned>(expert) - static_cast<unsigned>(p.first);
    return e < static_cast<unsigned>(p.experts) ? static_cast<int>(e) + 1 : 0;
}

// The lanes with this lane's bucket, bit by bit: a vote for the lanes that have an entry and up to
// eleven (1025 buckets), where match.any takes its time by the number of different buckets (4096 entries of 384
// experts: 9.4 us with it, 7.9).
__device__ __forceinline__ unsigned lanes_of(int bucket, int bits) {
    unsigned same = __ballot_sync(0xffffffffu, bucket >= 0);
    for (int i = 0; i < bits; ++i) {
        const bool on = (bucket >> i) & 1;
        const unsigned votes = __ballot_sync(0xffffffffu, on);
        same &= on ? votes : ~votes;
    }
    return same;
}

__device__ __forceinline__ void count_run(const SortParams& p, int lo, int hi, int* counts) {
    for (int i = lo + static_cast<int>(threadIdx.x); i < hi; i += kThreads) atomicAdd(counts + bucket_of(p, p.chosen[i]), 1);
}

__global__ void __launch_bounds__(kThreads) k_token_counts(const SortParams p) {
    extern __shared__ int counts[];
    const int buckets = p.experts + 1;
    for (int c = threadIdx.x; c < buckets; c += kThreads) counts[c] = 0;
    __syncthreads();
    asm volatile("griddepcontrol.launch_dependents;");
    const int lo = min(p.entries, static_cast<int>(blockIdx.x) * p.run), hi = min(p.entries, lo + p.run);
    count_run(p, lo, hi, counts);
    __syncthreads();
    for (int c = threadIdx.x; c < buckets; c += kThreads) p.table[blockIdx.x * buckets + c] = counts[c];
}

// Shared memory: next[buckets] (the next place of each), sums[buckets], then warps' counts of 16 bits.
template <bool ALONE>
__global__ void __launch_bounds__(kThreads) k_token_places(const SortParams p) {
    extern __shared__ int smem[];
    __shared__ int warp_sums[kWarps];
    const int buckets = p.experts + 1;
    int* const next = smem;
    int* const total = smem + buckets;
    uint16_t* const seen = reinterpret_cast<uint16_t*>(smem + 2 * buckets);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int lo = ALONE ? 0 : min(p.entries, static_cast<int>(blockIdx.x) * p.run);
    const int hi = ALONE ? p.entries : min(p.entries, lo + p.run);

    for (int c = threadIdx.x; c < buckets; c += kThreads) next[c] = total[c] = 0;
    __syncthreads();
    if (ALONE) {
        count_run(p, 0, p.entries, total);
    } else {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        // columns of the table to consecutive threads, its rows to as many parts as there is room for
        const int parts = sort_parts(p.blocks, buckets);
        const int part = buckets < kThreads ? static_cast<int>(threadIdx.x) / buckets : 0;
        if (part < parts) {
            for (int c = static_cast<int>(threadIdx.x) - part * buckets; c < buckets; c += kThreads) {
                // every block from a row of its own on: all at the same rows would queue for them
                int before = 0, all = 0;
                const int rows = sort_part_rows(p.blocks, parts, part), from = static_cast<int>(blockIdx.x) % rows;
#pragma unroll 16
                for (int i = 0; i < rows; ++i) {
                    const int b = part + (i + from < rows ? i + from : i + from - rows) * parts;
                    const int v = __ldcg(p.table + b * buckets + c);
                    all += v;
                    before += b < static_cast<int>(blockIdx.x) ? v : 0;
                }
                if (parts == 1) {
                    next[c] = before;
                    total[c] = all;
                } else {
                    atomicAdd(next + c, before);
                    atomicAdd(total + c, all);
                }
            }
        }
    }
    __syncthreads();
    // starts of the buckets: an exclusive sum over them, kThreads at a time
    int carry = 0;
    for (int c0 = 0; c0 < buckets; c0 += kThreads) {
        const int c = c0 + threadIdx.x;
        const int v = c < buckets ? total[c] : 0;
        int s = warp_inclusive_sum(v);
        if (lane == 31) warp_sums[warp] = s;
        __syncthreads();
        int base = carry, all = carry;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            base += w < warp ? warp_sums[w] : 0;
            all += warp_sums[w];
        }
        s += base;
        if (c < buckets) {
            next[c] += s - v;
            // bucket c ends where expert c starts; the last one's end is the number of entries
            if (ALONE || blockIdx.x == 0) p.offsets[c] = s;
        }
        carry = all;
        __syncthreads();
    }

    for (int at = lo; at < hi; at += kChunk) {
        for (int i = threadIdx.x; i < (kWarps * buckets + 1) / 2; i += kThreads) reinterpret_cast<int*>(seen)[i] = 0;
        int b[kRounds], rank[kRounds];
        const int first = at + warp * 32 * kRounds + lane;
#pragma unroll
        for (int r = 0; r < kRounds; ++r) b[r] = first + 32 * r < hi ? bucket_of(p, p.chosen[first + 32 * r]) : -1;
        __syncthreads();
        uint16_t* const mine = seen + warp * buckets;
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            if (first - lane + 32 * r >= hi) break;        // of the whole warp
            const unsigned same = lanes_of(b[r], p.bits);
            const int before = __popc(same & ((1u << lane) - 1u));
            const int had = b[r] >= 0 ? mine[b[r]] : 0;
            rank[r] = had + before;
            __syncwarp();
            if (before == 0 && b[r] >= 0) mine[b[r]] = static_cast<uint16_t>(had + __popc(same));
            __syncwarp();
        }
        __syncthreads();
        // each warp's count becomes the entries of the warps before it; the chunk's sum moves the next place on below
        for (int c = threadIdx.x; c < buckets; c += kThreads) {
            int sum = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const int v = seen[w * buckets + c];
                seen[w * buckets + c] = static_cast<uint16_t>(sum);
                sum += v;
            }
            total[c] = sum;
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            if (b[r] >= 0) {
                const int place = next[b[r]] + mine[b[r]] + rank[r];
                p.place[first + 32 * r] = place;
                p.order[place] = first + 32 * r;
            }
        }
        if (at + kChunk < hi) {
            __syncthreads();
            for (int c = threadIdx.x; c < buckets; c += kThreads) next[c] += total[c];
        }
    }
}

}  // namespace

int token_sort_blocks(long long entries) { return sort_blocks(entries); }

cudaError_t launch_token_sort(SortParams p, cudaStream_t s) {
    const int buckets = p.experts + 1;
    // 41 KB for 1024 experts
    const size_t smem = static_cast<size_t>(buckets) * 8 + (static_cast<size_t>(buckets) * kWarps * 2 + 3) / 4 * 4;
    p.blocks = token_sort_blocks(p.entries);
    p.bits = 0;
    while ((1 << p.bits) < buckets) ++p.bits;
    if (p.blocks == 0) {
        k_token_places<true><<<1, kThreads, smem, s>>>(p);
        return cudaGetLastError();
    }
    p.run = (p.entries + p.blocks - 1) / p.blocks;
    k_token_counts<<<p.blocks, kThreads, buckets * 4, s>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, k_token_places<false>, static_cast<const SortParams>(p));
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace muon
