// How the sort of routed entries (token_sort.cu) is split over blocks and threads: whole
// numbers only, for the host and the device, and for compilers without CUDA.
#pragma once

#ifdef __CUDACC__
#define MUON_BOTH __host__ __device__
#else
#define MUON_BOTH
#endif

namespace muon {

constexpr int kSortThreads = 512;
constexpr int kSortRounds = 4;                          // entries of a lane at a time
constexpr int kSortChunk = kSortThreads * kSortRounds;
constexpr int kSortMaxBlocks = 128;
constexpr int kSortAlone = 2 * kSortChunk;              // most entries for one block

// Blocks of the two launches; 0: one block does it all, without a table.
MUON_BOTH constexpr int sort_blocks(long long entries) {
    if (entries <= kSortAlone) return 0;
    const long long n = (entries + kSortChunk - 1) / kSortChunk;
    return static_cast<int>(n < kSortMaxBlocks ? n : kSortMaxBlocks);
}

// The parts that a block's threads make of the table's rows (a row of `buckets` counts for
// each of `blocks`), a thread to a column of each part: as many as there are threads
// for, and no more than rows, so that every part has one.
MUON_BOTH constexpr int sort_parts(int blocks, int buckets) {
    const int room = buckets < kSortThreads ? kSortThreads / buckets : 1;
    return room < blocks ? room : blocks;
}

// Rows of part `part`: part, part + parts, ..
MUON_BOTH constexpr int sort_part_rows(int blocks, int parts, int part) { return (blocks - part + parts - 1) / parts; }

}  // namespace muon

#undef MUON_BOTH
