/*
 * sort_layout.h -- how the order by expert shares its work out: the choices over
 * blocks, and the adding up of the blocks' counts over a block's threads.  Plain C++, so that a host
 * compiler can check the numbers.
 */
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define DLRM_SORT_LAYOUT __host__ __device__ constexpr
#else
#define DLRM_SORT_LAYOUT constexpr
#endif

namespace dlrm {

constexpr int kSortThreads = 512, kSortWarps = kSortThreads / 32;
constexpr int kSortChunk = 2048;        // choices of a block, while there are no more than kSortBlocks blocks
constexpr int kSortOne = 4096;          // so many choices are one block's
constexpr int kSortBlocks = 128;    // each of which reads all counts

struct SortShape {
    int blocks;
    int64_t chunk;
};

DLRM_SORT_LAYOUT SortShape sort_shape(int64_t n)
{
    if (n <= kSortOne) return {1, (n + kSortThreads - 1) / kSortThreads * kSortThreads};
    int64_t chunk = kSortChunk;
    if ((n + chunk - 1) / chunk > kSortBlocks)
        chunk = ((n + kSortBlocks - 1) / kSortBlocks + kSortThreads - 1) / kSortThreads * kSortThreads;
    return {(int)((n + chunk - 1) / chunk), chunk};
}

// The blocks' counts [blocks][bins] that a thread of block `block` adds up: those of one bin of every parts-th
// block from p on, `rows` of them (0: the thread has none), beginning with the from-th.
struct CountShare {
    int bin, p, parts, rows, from;
    DLRM_SORT_LAYOUT int block(int i) const { return p + (i + from < rows ? i + from : i + from - rows) * parts; }
};

DLRM_SORT_LAYOUT CountShare count_share(int thread, int bins, int blocks, int block)
{
    const int parts = kSortThreads / bins, p = thread / bins;
    if (p >= parts || p >= blocks) return {0, 0, 0, 0, 0};   // few bins have more parts than there are blocks
    const int rows = (blocks - p + parts - 1) / parts;
    return {thread % bins, p, parts, rows, block % rows};   // blocks do not all ask for the same row first
}

}  // namespace dlrm
