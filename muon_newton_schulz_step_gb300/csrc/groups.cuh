// Rows sorted into groups (tokens by expert), from device offsets.
#pragma once

namespace muon {

// One warp walks the groups 32 at a time.  For lane l's group g0 + l: its first
// row and its rows, from offsets[g], offsets[g + 1] clamped to [0, rows] and to
// at least the largest end before it (`low`, carried from call to call), so
// that groups never overlap whatever the offsets hold.
struct GroupSpan {
    int lo, cnt;
};

__device__ __forceinline__ GroupSpan warp_group_spans(const int* offsets, int groups, int rows, int g0, int& low) {
    const int lane = threadIdx.x & 31;
    const int g = g0 + lane;
    int lo = 0, hi = rows;
    if (offsets != nullptr) {
        lo = g < groups ? offsets[g] : 0;
        hi = g < groups ? offsets[g + 1] : 0;
    } else if (g > 0) {
        hi = 0;                                          // no offsets: one group of every row
    }
    lo = lo < 0 ? 0 : (lo > rows ? rows : lo);
    hi = hi < 0 ? 0 : (hi > rows ? rows : hi);
    int top = hi > lo ? hi : lo;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, top, o);
        if (lane >= o) top = top > t ? top : t;
    }
    int prev = __shfl_up_sync(0xffffffffu, top, 1);
    if (lane == 0 || prev < low) prev = low;
    if (lo < prev) lo = prev;
    const int last = __shfl_sync(0xffffffffu, top, 31);
    low = low > last ? low : last;
    GroupSpan s;
    s.lo = lo;
    s.cnt = g < groups && hi > lo ? hi - lo : 0;
    return s;
}

__device__ __forceinline__ int warp_inclusive_sum(int v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += t;
    }
    return v;
}

}  // namespace muon
