// row_units.cuh -- how kernels that pass over rows once share them out: a unit of threads takes part
// of a row, several runs of eight columns a lane.
#pragma once

#include "dense_ops.cuh"
#include "memo.h"

namespace dlrm {

// A lane's run of eight columns of a row, ES the element's size: on the 16-byte grid (VEC) 16-byte
// words, a warp's words one after another so that each access is of whole sectors (two words side by side
// in a lane cost fp32 every sector twice: norms of 16384 x 1024 80 us, 51 so); off it every 32nd column
// of 256, or pair of them.
template <bool VEC, int ES>
__device__ __forceinline__ int run_col(int first, int i)
{
    return first + (VEC ? ES == 2 ? i : i / 4 * 128 + i % 4 : ES == 2 ? i / 2 * 64 + i % 2 : i * 32);
}

// How units read rows: on the 16-byte grid, off it, or off it by a few lanes, every lanes-th column each.
enum { kOffGrid = 0, kOnGrid = 1, kFewLanes = 2 };

// A unit of `lanes` threads (a power of two; off the grid a warp) takes U runs a lane of one row at a
// time, whose loads are in flight together.
struct Unit {
    int lanes, l;                 // the unit's threads, and which of them this is
    int64_t units, unit;          // in the grid
    __device__ explicit Unit(int n) : lanes(n), l((int)threadIdx.x % n)
    {
        const int per = blockDim.x / n;
        units = (int64_t)gridDim.x * per;
        unit = (int64_t)blockIdx.x * per + threadIdx.x / n;
    }
    // the first column of the lane's run-th run of a row
    template <int LAY, int ES>
    __device__ __forceinline__ int first(int run) const
    {
        return run * lanes * 8 + l * (LAY == kOnGrid ? 16 / ES : LAY == kOffGrid && ES == 2 ? 2 : 1);
    }
};

// Runs a lane takes at once: as many as eight 16-byte words hold for K rows; off the grid one, whose
// single loads are as many (sums of two rows 40000 x 515 fp16: one run 41 us, four 62).
template <typename T, int LAY, int K>
constexpr int kRuns = LAY == kOnGrid && 16 / (K * (int)sizeof(T)) > 1 ? 16 / (K * (int)sizeof(T)) : 1;

// Whether two neighbouring 2-byte elements of a row are one 4-byte word.
__device__ __forceinline__ bool row_of_words(const void* row) { return ((uintptr_t)row & 3u) == 0; }

// The run's columns of a row; columns past its end read as 0 and are not stored.  On the grid a lane's second
// 16-byte word is `lanes` words behind its first.
template <typename T, int LAY>
__device__ __forceinline__ Raw8<T> load_cols(const T* row, int first, int H, int lanes)
{
    Raw8<T> r = {};
    if constexpr (LAY == kFewLanes) {
        T e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = first + i * lanes < H ? __ldg(row + first + i * lanes) : from_f32<T>(0.f);
        memcpy(&r, e, sizeof(e));
    } else if constexpr (LAY == kOnGrid) {
#pragma unroll
        for (int i = 0; i < (int)(sizeof(T) / 2); ++i)
            if (first + i * 4 * lanes < H) r.w[i] = ldg_nc_v4(row + first + i * 4 * lanes);
    } else if constexpr (sizeof(T) == 2) {
        uint32_t* const w = &r.w[0].x;
        const T* p = row + first;
        if (row_of_words(row)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (first + 64 * i + 1 < H) w[i] = __ldg(reinterpret_cast<const uint32_t*>(p) + 32 * i);
                else if (first + 64 * i < H) w[i] = __ldg(reinterpret_cast<const uint16_t*>(p) + 64 * i);
            }
        } else {
            uint16_t e[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                e[i] = run_col<false, 2>(first, i) < H ? __ldg((const uint16_t*)p + run_col<false, 2>(0, i)) : 0;
            memcpy(w, e, 16);
        }
    } else {
        float e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = first + 32 * i < H ? __ldg(row + first + 32 * i) : 0.f;
        memcpy(&r, e, 32);
    }
    return r;
}

template <typename T, int LAY>
__device__ __forceinline__ void store_raw(T* row, int first, int H, int lanes, const Raw8<T>& r)
{
    T* p = row + first;
    if constexpr (LAY == kFewLanes) {
        T e[8];
        memcpy(e, &r, sizeof(e));
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (first + i * lanes < H) p[i * lanes] = e[i];
    } else if constexpr (LAY == kOnGrid) {
#pragma unroll
        for (int i = 0; i < (int)(sizeof(T) / 2); ++i)
            if (first + i * 4 * lanes < H) *reinterpret_cast<uint4*>(p + i * 4 * lanes) = r.w[i];
    } else if constexpr (sizeof(T) == 2) {
        uint32_t w[4];
        memcpy(w, &r, 16);
        const bool words = row_of_words(row);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (words && first + 64 * i + 1 < H) {
                reinterpret_cast<uint32_t*>(p)[32 * i] = w[i];
            } else {
                if (first + 64 * i < H) reinterpret_cast<uint16_t*>(p)[64 * i] = (uint16_t)w[i];
                if (first + 64 * i + 1 < H) reinterpret_cast<uint16_t*>(p)[64 * i + 1] = (uint16_t)(w[i] >> 16);
            }
        }
    } else {
        float e[8];
        memcpy(e, &r, 32);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (first + 32 * i < H) p[32 * i] = e[i];
    }
}

template <typename T, int LAY>
__device__ __forceinline__ void store_cols(T* row, int first, int H, int lanes, const float (&f)[8])
{
    Raw8<T> r;
    if constexpr (sizeof(T) == 2) r.w[0] = pack8<T>(f);
    else memcpy(&r, f, 32);
    store_raw<T, LAY>(row, first, H, lanes, r);
}

// Walks (row, part of the row) pairs, a unit at a time, without a division after the first.  The runs of a row
// are shared out over its parts, `most` runs a lane at most: part * per + u for u < per.
struct Items {
    int64_t row, part, parts, drow, dpart;
    int per;
    __device__ Items(const Unit& u, int H, int most)
    {
        const int runs = (H - 1) / (u.lanes * 8) + 1, p = (runs - 1) / most + 1;
        parts = p;
        per = (runs - 1) / p + 1;
        row = u.unit / p;
        part = u.unit - row * p;
        drow = u.units / p;
        dpart = u.units - drow * p;
    }
    __device__ __forceinline__ int run(int u) const { return (int)part * per + u; }
    __device__ void next()
    {
        row += drow;
        part += dpart;
        if (part >= parts) {
            part -= parts;
            ++row;
        }
    }
};

// ---------------------------------------------------------------- host side
// How many blocks of 256 threads of a kernel without dynamic shared memory run at once.
inline int blocks_at_once(const void* kern)
{
    int dev = 0;
    cudaGetDevice(&dev);
    static KernelMemo memo;
    return memo.get({kern, dev, 0, 0}, [&] {
        int n = 0;
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, 256, 0) == cudaSuccess && n > 0) return n * num_sms();
        cudaGetLastError();
        return num_sms() * 8;
    });
}

// The blocks of a kernel whose threads stride over the work: as many as run at once, or without a kernel
// eight an SM.  (Five or six of eight run at once, the rest at the end: sums of 2 rows 65536 x 1024 bf16
// 61 us, 59 so; but rows written twice 63 and 66.)
inline unsigned grid_blocks(int64_t want, const void* kern)
{
    if (want <= num_sms()) return (unsigned)want;
    const int64_t most = kern ? blocks_at_once(kern) : num_sms() * 8;
    return (unsigned)(want < most ? want : most);
}

// The lanes of a unit, and the blocks of 256 threads for rows taken in parts of `runs` runs a lane.
// On the grid the most lanes of which four fifths have columns (160 fp32 columns of 5 rows: 8 lanes, not 32).
inline int unit_lanes(int H, int lay, int least = 1)
{
    if (lay == kOffGrid) return kWarp;
    const int64_t runs = ((int64_t)H + 7) / 8;
    int n = 1;
    while (n < kWarp && n < runs) n *= 2;
    while (lay == kOnGrid && n > 4 && 5 * runs < 4 * ((runs + n - 1) / n * n)) n /= 2;
    return n < least ? least : n;
}

// Rows off the grid of up to 128 columns are a few lanes' each.
inline int row_layout(bool vec, int H) { return vec ? kOnGrid : H <= 128 ? kFewLanes : kOffGrid; }

inline unsigned item_blocks(int64_t rows, int H, int lanes, int runs, const void* kern)
{
    const int64_t part = (int64_t)lanes * 8 * runs;
    return grid_blocks((rows * ((H + part - 1) / part) * lanes + 255) / 256, kern);
}

}  // namespace dlrm
