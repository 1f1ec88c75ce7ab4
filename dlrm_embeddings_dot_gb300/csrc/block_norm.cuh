// block_norm.cuh -- the norms after a block and before the next one, with the
// block's gate and residual scale:
//
//   u = norm(y) w_post + b_post;  r = residual + scale gate(g) u;  h = norm(r) w_pre + b_pre
//
// and its gradient.  Both are bound by memory: every matrix goes once, a row stays in
// registers between its sums.
//
// A row is taken by W warps, eight columns a lane, which holds its part of the vectors in
// registers.  The next rows are on their way meanwhile: a ring of rows in shared
// memory, each thread copying its own columns (cp.async), so that no thread waits for
// another's copies.  Sums of a row go by shuffles, then over its warps by shared memory.
// Short rows are a few lanes' each, and their loads go to registers.
//
//   forward    the statistics are taken in two passes over the registers (mean, then
//              squares about it)
//   backward   a lane also adds up its columns' sums over rows.  Blocks' sums go to `partial`
//              and block_norm_sum_kernel adds them in order
//
// Measured (us, share of the copy rate; 65536 x 1024 unless said): forward bf16 with a gate 106,
// 0.95; gradient fp16 with a gate 170, 0.94; 16384 x 1024 fp32 49 and 82, 0.98.  Pairs of fp32 values go
// through one instruction (fma.f32x2 and the like), and what depends on the row alone through the
// uniform datapath: the warp's number has to be read from one lane for that (gradient 236 us without).
//
// Nothing here depends on which columns a lane has.  On the 16-byte grid they are 16-byte words.
// Off it a warp copies the aligned 16-byte words that hold its 256 columns and a lane has every
// 32nd column, or pair of them, which shared memory gives without conflicts; the instructions for that
// bound it (40000 x 771 bf16, centred, a gate value a row: 121 and 186 us, 0.31 and 0.30).
#pragma once

#include "block_norm.h"
#include "row_units.cuh"

namespace dlrm {
namespace norms {
namespace {

// ------------------------------------------------------------- runs of a row
// How a row lies over lanes.  kGrid, kAny: 256 columns a warp, on the 16-byte grid and off it
// (row_units.cuh).  few<L>(grid), below 0: L lanes a row, several rows a warp; on the grid 16-byte words,
// off it every L-th column.
constexpr int kGrid = 1, kAny = 0, kFewGrid = -64;
constexpr int few(int lanes, bool grid) { return grid ? kFewGrid - lanes : -lanes; }
template <int LAY>
constexpr int kRowLanes = LAY < kFewGrid ? kFewGrid - LAY : LAY < 0 ? -LAY : kWarp;
template <int LAY>
constexpr bool kWords = LAY == kGrid || LAY < kFewGrid;   // 16-byte words

// A lane's first column of a row, and its i-th.
template <int LAY, int ES>
__device__ __forceinline__ int run_first(int warp, int lane)
{
    if constexpr (LAY < 0) return lane % kRowLanes<LAY> * (kWords<LAY> ? 16 / ES : 1);
    else return warp * 256 + lane * (LAY == kGrid ? 16 / ES : ES == 2 ? 2 : 1);
}

template <int LAY, int ES>
__device__ __forceinline__ int norm_col(int first, int i)
{
    constexpr int L = kRowLanes<LAY>;
    if constexpr (LAY < kFewGrid) return first + (ES == 2 ? i : i / 4 * 4 * L + i % 4);
    else if constexpr (LAY < 0) return first + i * L;
    else return run_col<LAY == kGrid, ES>(first, i);
}

// A tensor's row that a group of warps is at, stepped from one of its rows to the next.
template <typename T>
struct Cursor {
    const T *base, *row;
    int64_t inc;
    __device__ Cursor(const void* p, int64_t ld, int64_t row0, int64_t step)
        : base((const T*)p), row((const T*)p + row0 * ld), inc(step * ld)
    {
    }
    __device__ __forceinline__ const T* ahead(int rows) const { return row + rows * inc; }
    __device__ __forceinline__ T* out() const { return const_cast<T*>(row); }
    __device__ __forceinline__ void next() { row += inc; }
};

// A block's warps in groups of W, WARPS an SM at most: a row each, or several where a few lanes take one.
template <int W, int WARPS, int LAY>
struct Group {
    static constexpr int kGroups = norm_groups(W, WARPS), kWarps = kGroups * W, kThreads = kWarps * 32,
                         kPerSM = norm_per_sm(W, WARPS);
    static constexpr int kEach = kWarp / kRowLanes<LAY>, kRows = kGroups * kEach;
    // the places of a row's sums in shared memory, and an area's floats
    static constexpr int kPitch = W == 2 ? 2 : (W + 3) / 4 * 4, kArea = kGroups * 2 * kPitch;
};

// The rows to come: kAhead rows of NT tensors, three where the blocks that share an SM have the memory.
// Columns past the row's end are 0.
template <int STAGE, typename G>
constexpr int kRowsThatFit = (224 << 10) / G::kPerSM / STAGE;
template <int STAGE, typename G>
constexpr int kRowsAhead = kRowsThatFit<STAGE, G> < 3 ? kRowsThatFit<STAGE, G> : 3;

__device__ __forceinline__ void copy16(uint32_t to, const void* from, uint32_t bytes)   // the rest of the word becomes 0
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}

// On the grid: each thread copies and reads its own eight columns.
template <typename T, int LAY, int NT, typename G>
struct Ring {
    static constexpr int THREADS = G::kThreads;
    static constexpr int kWords = sizeof(T) / 2, kSlot = kWords * THREADS * 16, kStage = NT * kSlot;
    static constexpr int kAhead = kRowsAhead<kStage, G>;
    static_assert(kAhead >= 1, "a row fits");
    static constexpr size_t kBytes = (size_t)kAhead * kStage;
    uint8_t* mine;    // word 0 of slot 0 of stage 0
    uint32_t at;      // its shared address
    int N, first;

    __device__ Ring(uint8_t* smem, int n, int f, int) : mine(smem + threadIdx.x * 16), N(n), first(f)
    {
        at = (uint32_t)__cvta_generic_to_shared(mine);
        for (int i = 0; i < kAhead * NT * kWords; ++i)
            *reinterpret_cast<uint4*>(mine + i * THREADS * 16) = make_uint4(0, 0, 0, 0);
    }
    // Starts the copy of a tensor's row `rows` ahead to a slot.  inner: words that hold a part of the
    // row are in the matrix as a whole.
    __device__ __forceinline__ void fetch(int stage, int slot, const Cursor<T>& c, int rows, bool) const
    {
        const T* row = c.ahead(rows);
        const uint32_t to = at + stage * kStage + slot * kSlot;
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            if (first + i * 128 < N) copy16(to + i * THREADS * 16, row + first + i * 128, 16);
    }
    static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    // The oldest row's copies are complete.
    static __device__ __forceinline__ void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory"); }
    static __device__ __forceinline__ void done() {}
    __device__ __forceinline__ void read(int stage, int slot, const T*, float2 (&f)[4]) const
    {
        Raw8<T> r;
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            r.w[i] = *reinterpret_cast<const uint4*>(mine + stage * kStage + slot * kSlot + i * THREADS * 16);
        float v[8];
        widen8<T>(r, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = make_float2(v[2 * i], v[2 * i + 1]);
    }
};

// Off the grid: a warp's 256 columns lie in 16 ES + 1 aligned words at most, which its lanes copy.
// Near the matrix's ends the last word is cut there, and one that begins before the matrix is put
// together from its elements.
template <typename T, int NT, typename G>
struct Ring<T, kAny, NT, G> {
    static constexpr int THREADS = G::kThreads;
    static constexpr int kES = sizeof(T), kWords = 16 * kES + 1, kSlot = THREADS / kWarp * kWords * 16, kStage = NT * kSlot;
    static constexpr int kAhead = kRowsAhead<kStage, G>;
    static_assert(kAhead >= 1, "a row fits");
    static constexpr size_t kBytes = (size_t)kAhead * kStage;
    uint8_t* mine;    // the warp's word 0
    uint32_t at;
    int N, first, from, bytes;   // from: the warp's first column; bytes of its columns, 0 or less: none

    // f0: the row's warp's number times 256
    __device__ Ring(uint8_t* smem, int n, int f, int f0) : N(n), first(f), from(f0)
    {
        mine = smem + __shfl_sync(~0u, (int)threadIdx.x / kWarp, 0) * kWords * 16;
        at = (uint32_t)__cvta_generic_to_shared(mine);
        bytes = min(256, N - from) * kES;
    }
    __device__ __forceinline__ void fetch(int stage, int slot, const Cursor<T>& c, int rows, bool inner) const
    {
        const int lane = threadIdx.x % kWarp;
        const uint32_t to = at + stage * kStage + slot * kSlot + lane * 16;
        const uint8_t* p = reinterpret_cast<const uint8_t*>(c.ahead(rows) + from);
        const int off = (int)((uintptr_t)p & 15), end = off + bytes;
        const uint8_t* word = p - off + lane * 16;
        if (inner) {
#pragma unroll
            for (int i = 0; i < (kWords + kWarp - 1) / kWarp; ++i)
                if ((lane + kWarp * i) * 16 < end) copy16(to + kWarp * 16 * i, word + kWarp * 16 * i, 16);
        } else if (bytes > 0) {
            const bool cut = (uintptr_t)(p - off) < (uintptr_t)c.base;
            for (int w = lane; w * 16 < end; w += kWarp)
                if (w > 0 || !cut) copy16(to + (w - lane) * 16, p - off + w * 16, min(16, end - w * 16));
            if (cut && lane >= off / kES && lane < min(16, end) / kES)
                reinterpret_cast<T*>(mine + stage * kStage + slot * kSlot)[lane] =
                    __ldg(reinterpret_cast<const T*>(p) + lane - off / kES);
        }
    }
    static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    static __device__ __forceinline__ void wait()
    {
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
        __syncwarp();   // the other lanes' copies too
    }
    static __device__ __forceinline__ void done() { __syncwarp(); }   // all lanes have read the row
    __device__ __forceinline__ void read(int stage, int slot, const T* row, float2 (&f)[4]) const
    {
        const uint8_t* p = mine + stage * kStage + slot * kSlot + ((uintptr_t)(row + from) & 15) + (first - from) * kES;
        const T* e = reinterpret_cast<const T*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = make_float2(to_f32(e[norm_col<kAny, kES>(0, 2 * i)]), to_f32(e[norm_col<kAny, kES>(0, 2 * i + 1)]));
        if (bytes < 256 * kES) {   // what is left there from other rows
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[i].x = norm_col<kAny, kES>(first, 2 * i) < N ? f[i].x : 0.f;
                f[i].y = norm_col<kAny, kES>(first, 2 * i + 1) < N ? f[i].y : 0.f;
            }
        }
    }
};

// A few lanes a row: its columns straight to registers, all tensors' loads in flight together.
template <typename T, int LAY, int NT, typename G>
struct Few {
    static constexpr int kAhead = 1;
    static constexpr size_t kBytes = G::kThreads * 32;   // the backward adds up its blocks' sums there
    int N, first;
    Raw8<T> v[NT];
    __device__ Few(uint8_t*, int n, int f, int) : N(n), first(f) {}
    __device__ __forceinline__ void fetch(int, int slot, const Cursor<T>& c, int, bool here)
    {
        if constexpr (kWords<LAY>) {
#pragma unroll
            for (int i = 0; i < (int)(sizeof(T) / 2); ++i) {
                const int at = norm_col<LAY, sizeof(T)>(first, 4 * i);
                v[slot].w[i] = here && at < N ? ldg_nc_v4(c.row + at) : make_uint4(0, 0, 0, 0);
            }
        } else {
            T e[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int at = norm_col<LAY, sizeof(T)>(first, i);
                e[i] = here && at < N ? __ldg(c.row + at) : from_f32<T>(0.f);
            }
            memcpy(&v[slot], e, sizeof(e));
        }
    }
    static __device__ __forceinline__ void commit() {}
    static __device__ __forceinline__ void wait() {}
    static __device__ __forceinline__ void done() {}
    __device__ __forceinline__ void read(int, int slot, const T*, float2 (&f)[4]) const
    {
        float e[8];
        widen8<T>(v[slot], e);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = make_float2(e[2 * i], e[2 * i + 1]);
    }
};

template <typename T, int LAY, int NT, typename G>
using Rows = std::conditional_t<(LAY < 0), Few<T, LAY, NT, G>, Ring<T, LAY < 0 ? kGrid : LAY, NT, G>>;

// full: all columns are in the row; of a few lanes: there is a row.
template <typename T, int LAY>
__device__ __forceinline__ void store_run(T* row, int first, int N, bool full, const float2 (&v)[4])
{
    if constexpr (kWords<LAY>) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = v[i].x;
            f[2 * i + 1] = v[i].y;
        }
        if (LAY < 0 && !full) return;
        if constexpr (sizeof(T) == 2) {
            if (first < N) store8<T, true>(row + first, 8, f);
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int c = norm_col<LAY, 4>(first, 4 * i);
                if (c < N)
                    *reinterpret_cast<float4*>(row + c) = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
            }
        }
    } else if constexpr (LAY < 0) {
        if (full)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = norm_col<LAY, sizeof(T)>(first, 2 * i), d = norm_col<LAY, sizeof(T)>(first, 2 * i + 1);
                if (c < N) row[c] = from_f32<T>(v[i].x);
                if (d < N) row[d] = from_f32<T>(v[i].y);
            }
    } else if constexpr (sizeof(T) == 2) {
        T* const p = row + first;
        if (full && row_of_words(row)) {
            float f[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = v[i].x;
                f[2 * i + 1] = v[i].y;
            }
            const uint4 w = pack8<T>(f);
            uint32_t* const q = reinterpret_cast<uint32_t*>(p);
            q[0] = w.x;
            q[32] = w.y;
            q[64] = w.z;
            q[96] = w.w;
        } else if (full) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p[64 * i] = from_f32<T>(v[i].x);
                p[64 * i + 1] = from_f32<T>(v[i].y);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (first + 64 * i < N) p[64 * i] = from_f32<T>(v[i].x);
                if (first + 64 * i + 1 < N) p[64 * i + 1] = from_f32<T>(v[i].y);
            }
        }
    } else {
        T* const p = row + first;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (full || first + 64 * i < N) p[64 * i] = v[i].x;
            if (full || first + 64 * i + 32 < N) p[64 * i + 32] = v[i].y;
        }
    }
}

// The run's part of a vector: `fill` everywhere where there is none, 0 past the row's end; and of an fp32 output.
template <int LAY, int ES>
__device__ __forceinline__ void load_vector(const float* p, int first, int N, float fill, float2 (&f)[4])
{
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int c = norm_col<LAY, ES>(first, i);
        v[i] = c >= N ? 0.f : p ? __ldg(p + c) : fill;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = make_float2(v[2 * i], v[2 * i + 1]);
}

template <int LAY, int ES>
__device__ __forceinline__ void store_vector(float* p, int first, int N, const float2 (&v)[4])
{
    if constexpr (kWords<LAY>) {   // N is a multiple of eight
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (norm_col<LAY, ES>(first, 4 * i) < N)
                *reinterpret_cast<float4*>(p + norm_col<LAY, ES>(first, 4 * i)) =
                    make_float4(v[2 * i].x, v[2 * i].y, v[2 * i + 1].x, v[2 * i + 1].y);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = norm_col<LAY, ES>(first, 2 * i), d = norm_col<LAY, ES>(first, 2 * i + 1);
            if (c < N) p[c] = v[i].x;
            if (d < N) p[d] = v[i].y;
        }
    }
}

// Sums of V (1 or 2) values over the W warps of a row, the same in all of them.  red: two areas
// that take turns, so that one barrier a sum is enough.
template <typename G, int W, int LANES, int V>
__device__ __forceinline__ void row_sum(float (&v)[V], float* red, int& turn, int warp)
{
    const int lane = threadIdx.x % kWarp;
    if constexpr (LANES < kWarp) {
#pragma unroll
        for (int m = LANES / 2; m; m /= 2)
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] += __shfl_xor_sync(~0u, v[i], m);
        return;
    }
    float s = v[0];
    if constexpr (V == 2) {   // each half of the warp goes on with one of the two
        const bool up = lane & 16;
        s = (up ? v[1] : v[0]) + __shfl_xor_sync(~0u, up ? v[0] : v[1], 16);
    } else {
        s += __shfl_xor_sync(~0u, s, 16);
    }
#pragma unroll
    for (int m = 8; m; m /= 2) s += __shfl_xor_sync(~0u, s, m);
    if constexpr (W == 1) {
        if constexpr (V == 2) {
            const float o = __shfl_xor_sync(~0u, s, 16);
            v[0] = lane & 16 ? o : s;
            v[1] = lane & 16 ? s : o;
        } else {
            v[0] = s;
        }
    } else {
        constexpr int P = G::kPitch;
        float* area = red + turn * G::kArea;   // [row][2 values][warp]: rows' sums of one and two values may meet
        turn ^= 1;
        if (V == 2 ? lane % 16 == 0 : lane == 0) area[(warp / W * 2 + lane / 16) * P + warp % W] = s;
        if constexpr (G::kGroups == 1) __syncthreads();
        else asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / W), "r"(W * 32) : "memory");
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float* p = area + (warp / W * 2 + i) * P;
            if constexpr (W == 2) {
                const float2 q = *reinterpret_cast<const float2*>(p);
                v[i] = q.x + q.y;
            } else {
                v[i] = 0.f;
#pragma unroll
                for (int w = 0; w < W / 4 * 4; w += 4) {
                    const float4 q = *reinterpret_cast<const float4*>(p + w);
                    v[i] += (q.x + q.y) + (q.z + q.w);
                }
#pragma unroll
                for (int w = W / 4 * 4; w < W; ++w) v[i] += p[w];
            }
        }
    }
}

// (s, s) and sums of pairs
__device__ __forceinline__ float2 both(float s) { return make_float2(s, s); }
__device__ __forceinline__ float add_up(const float2 (&v)[4])
{
    const float2 a = __fadd2_rn(__fadd2_rn(v[0], v[1]), __fadd2_rn(v[2], v[3]));
    return a.x + a.y;
}

// gate(g), and gate'(g): with s the sigmoid, SIGMOID s and s (1 - s), SILU s g and s (1 + g (1 - s)).
template <typename T>
__device__ __forceinline__ float gate_f(float g, int act)
{
    if (act == DLRM_GATE_NONE) return g;
    return sigmoid<T>(g) * (act == DLRM_GATE_SIGMOID ? 1.f : g);
}

template <typename T>
__device__ __forceinline__ void gate_both(float& g, int act, float& slope)
{
    slope = 1.f;
    if (act == DLRM_GATE_NONE) return;
    float rest;
    const float s = sigmoid<T>(g, rest), m = act == DLRM_GATE_SIGMOID ? 1.f : g;
    g = s * m;
    slope = s * fmaf(m, rest, act == DLRM_GATE_SIGMOID ? 0.f : 1.f);
}

// ------------------------------------------------------------------- forward
template <int W, int LAY>
using FwdGroup = Group<W, fwd_warps(W, LAY == kAny), LAY>;

// (mean, 1 / sqrt(mean square + eps)) of a row; f becomes what is left without the mean, 0 past the end
template <typename G, int LAY, int ES, int W>
__device__ __forceinline__ float2 centre(float2 (&f)[4], int first, bool full, const NormFwd& a, float* red, int& turn,
                                         int warp)
{
    float s[1], mean = 0.f;
    if (a.layer) {
        s[0] = add_up(f);
        row_sum<G, W, kRowLanes<LAY>>(s, red, turn, warp);
        mean = s[0] * a.inv_n;
        if (full && LAY >= 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = __fadd2_rn(f[i], both(-mean));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[i].x = norm_col<LAY, ES>(first, 2 * i) < a.N ? f[i].x - mean : 0.f;
                f[i].y = norm_col<LAY, ES>(first, 2 * i + 1) < a.N ? f[i].y - mean : 0.f;
            }
        }
    }
    float2 q = __fmul2_rn(f[0], f[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) q = __ffma2_rn(f[i], f[i], q);
    s[0] = q.x + q.y;
    row_sum<G, W, kRowLanes<LAY>>(s, red, turn, warp);
    return make_float2(mean, 1.f / sqrtf(fmaf(s[0], a.inv_n, a.eps)));
}

template <typename T, int LAY, int W>
__global__ void __launch_bounds__(FwdGroup<W, LAY>::kThreads, FwdGroup<W, LAY>::kPerSM)
block_norm_fwd_kernel(const __grid_constant__ NormFwd a)
{
    using G = FwdGroup<W, LAY>;
    using R = Rows<T, LAY, 3, G>;
    constexpr int kAhead = R::kAhead;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float red[W > 1 ? 2 * G::kArea : 1];
    // the same in all lanes, so that what depends on the row alone takes the uniform datapath
    const int warp = __shfl_sync(~0u, (int)threadIdx.x / kWarp, 0), lane = threadIdx.x % kWarp, N = a.N;
    const bool whole = warp % W * 256 + 256 <= N;   // all columns of the warp are in the row
    const int sub = lane / kRowLanes<LAY>;          // the lane's row of the group's
    const int first = run_first<LAY, sizeof(T)>(warp % W, lane);
    int turn = 0;
    R ring(smem, N, first, warp % W * 256);
    pdl_wait();
    const int64_t step = (int64_t)gridDim.x * G::kRows;
    const int64_t row0 = (int64_t)blockIdx.x * G::kRows + warp / W * G::kEach + sub;
    Cursor<T> cy(a.y, a.ldy, row0, step), cg(a.gate, a.ldg, row0, step), cres(a.res, a.ldres, row0, step),
        cr(a.r, a.ldr, row0, step), ch(a.h, a.ldh, row0, step);
    auto fetch = [&](int stage, int64_t row, int rows) {
        const int64_t at = row + rows * step;
        if (at - sub < a.M) {
            const bool inner = LAY < 0 ? at < a.M : at >= a.margin && at < a.M - a.margin;
            if (a.y) ring.fetch(stage, 0, cy, rows, inner);
            if (a.gate_cols > 1) ring.fetch(stage, 1, cg, rows, inner);
            if (a.res) ring.fetch(stage, 2, cres, rows, inner);
        }
        R::commit();
    };
#pragma unroll
    for (int k = 0; k < kAhead - 1; ++k) fetch(k, row0, k);
    float2 aw[4], ab[4], wp[4], bp[4];   // scale w_post, scale b_post, w_pre, b_pre
    load_vector<LAY, sizeof(T)>(a.scale, first, N, 1.f, wp);
    load_vector<LAY, sizeof(T)>(a.w_post, first, N, 1.f, aw);
    load_vector<LAY, sizeof(T)>(a.b_post, first, N, 0.f, ab);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        aw[i] = __fmul2_rn(aw[i], wp[i]);
        ab[i] = __fmul2_rn(ab[i], wp[i]);
    }
    load_vector<LAY, sizeof(T)>(a.w_pre, first, N, 1.f, wp);
    load_vector<LAY, sizeof(T)>(a.b_pre, first, N, 0.f, bp);
    int stage = 0;
    for (int64_t row = row0; row - sub < a.M; row += step) {   // the lanes of a warp together
        const bool here = LAY >= 0 || row < a.M, full = LAY < 0 ? here : whole;
        fetch(stage == 0 ? kAhead - 1 : stage - 1, row, kAhead - 1);
        R::wait();
        float4 st = make_float4(0.f, 0.f, 0.f, 0.f);
        float2 r[4];
        if (a.res) ring.read(stage, 2, cres.row, r);
        else
#pragma unroll
            for (int i = 0; i < 4; ++i) r[i] = both(0.f);
        if (a.y) {
            float2 f[4], g[4];
            ring.read(stage, 0, cy.row, f);
            if (a.gate_cols > 1) {
                ring.read(stage, 1, cg.row, g);
                if (a.gate_act != DLRM_GATE_NONE)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        g[i].x = gate_f<T>(g[i].x, a.gate_act);
                        g[i].y = gate_f<T>(g[i].y, a.gate_act);
                    }
            } else {
                const float g1 = a.gate_cols == 1 ? gate_f<T>(here ? to_f32(__ldg(cg.row)) : 0.f, a.gate_act) : 1.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) g[i] = both(g1);
            }
            const float2 s = centre<G, LAY, sizeof(T), W>(f, first, full, a, red, turn, warp);
            st.x = s.x;
            st.y = s.y;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 u = __ffma2_rn(__fmul2_rn(f[i], both(s.y)), aw[i], ab[i]);   // scale u
                r[i] = __ffma2_rn(u, g[i], r[i]);
            }
            store_run<T, LAY>(cr.out(), first, N, full, r);
        }
        if (a.h) {
            const float2 s = centre<G, LAY, sizeof(T), W>(r, first, full, a, red, turn, warp);
            st.z = s.x;
            st.w = s.y;
#pragma unroll
            for (int i = 0; i < 4; ++i) r[i] = __ffma2_rn(__fmul2_rn(r[i], both(s.y)), wp[i], bp[i]);
            store_run<T, LAY>(ch.out(), first, N, full, r);
        }
        if (a.stats && here && warp % W == 0 && lane % kRowLanes<LAY> == 0) a.stats[row] = st;
        R::done();
        cy.next();
        cg.next();
        cres.next();
        cr.next();
        ch.next();
        stage = stage == kAhead - 1 ? 0 : stage + 1;
    }
}

// fn(the layout and the warps of a row as constants)
template <typename Fn>
dlrm_status with_rows(int N, bool vec, Fn&& fn)
{
    using std::integral_constant;
    constexpr integral_constant<int, 1> one;
    switch (norm_lanes(N)) {
    case 4: return vec ? fn(integral_constant<int, few(4, true)>(), one) : fn(integral_constant<int, few(4, false)>(), one);
    case 8: return vec ? fn(integral_constant<int, few(8, true)>(), one) : fn(integral_constant<int, few(8, false)>(), one);
    case 16: return vec ? fn(integral_constant<int, few(16, true)>(), one) : fn(integral_constant<int, few(16, false)>(), one);
    default: break;
    }
    auto wide = [&](auto lay) {
        switch (norm_warps(N)) {
        case 1: return fn(lay, one);
        case 2: return fn(lay, integral_constant<int, 2>());
        case 3: return fn(lay, integral_constant<int, 3>());
        case 4: return fn(lay, integral_constant<int, 4>());
        case 5: return fn(lay, integral_constant<int, 5>());
        case 6: return fn(lay, integral_constant<int, 6>());
        case 7: return fn(lay, integral_constant<int, 7>());
        case 8: return fn(lay, integral_constant<int, 8>());
        case 10: return fn(lay, integral_constant<int, 10>());
        case 12: return fn(lay, integral_constant<int, 12>());
        case 16: return fn(lay, integral_constant<int, 16>());
        case 20: return fn(lay, integral_constant<int, 20>());
        case 24: return fn(lay, integral_constant<int, 24>());
        default: return fn(lay, integral_constant<int, 32>());
        }
    };
    return vec ? wide(integral_constant<int, kGrid>()) : wide(integral_constant<int, kAny>());
}

template <typename K, typename A>
dlrm_status launch_norm(const char* what, K kern, const A& a, int warps, int threads, size_t smem, cudaStream_t st)
{
    const cudaError_t e =   // the first 48 KB need no leave
        smem > 46 << 10 ? cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) : cudaSuccess;
    if (e != cudaSuccess) return fail(DLRM_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
    return check_launch_pdl(launch_pdl(kern, dim3(norm_blocks(a.M, a.N, warps)), dim3(threads), smem, st, a), what);
}

template <typename T>
dlrm_status launch_fwd(const NormFwd& a, bool vec, cudaStream_t st)
{
    return with_rows(a.N, vec, [&](auto l, auto w) {
        constexpr int LAY = decltype(l)::value, W = decltype(w)::value;
        using G = FwdGroup<W, LAY>;
        return launch_norm("block_norm_fwd_kernel", block_norm_fwd_kernel<T, LAY, W>, a, fwd_warps(W, LAY == kAny), G::kThreads,
                           Rows<T, LAY, 3, G>::kBytes, st);
    });
}

// ------------------------------------------------------------------ backward
template <int W, int LAY, bool POST, bool PRE>
using BwdGroup = Group<W, bwd_warps(POST, PRE, LAY == kGrid), LAY>;

template <typename T, int LAY, int W, bool POST, bool PRE>
__global__ void __launch_bounds__(BwdGroup<W, LAY, POST, PRE>::kThreads, BwdGroup<W, LAY, POST, PRE>::kPerSM)
block_norm_bwd_kernel(const __grid_constant__ NormBwd a)
{
    using G = BwdGroup<W, LAY, POST, PRE>;
    constexpr int kGr = 0, kGh = 1, kR = 2, kY = PRE ? 3 : 1, kGate = kY + 1;   // slots
    using Rg = Rows<T, LAY, POST && PRE ? 5 : 3, G>;
    constexpr int kAhead = Rg::kAhead;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float red[W > 1 ? 2 * G::kArea : 1];
    // the same in all lanes, so that what depends on the row alone takes the uniform datapath
    const int warp = __shfl_sync(~0u, (int)threadIdx.x / kWarp, 0), lane = threadIdx.x % kWarp, N = a.N;
    const bool whole = warp % W * 256 + 256 <= N;   // all columns of the warp are in the row
    const int sub = lane / kRowLanes<LAY>;          // the lane's row of the group's
    const int first = run_first<LAY, sizeof(T)>(warp % W, lane);
    int turn = 0;
    Rg ring(smem, N, first, warp % W * 256);
    pdl_wait();
    const int64_t step = (int64_t)gridDim.x * G::kRows, row0 = (int64_t)blockIdx.x * G::kRows + warp / W * G::kEach + sub;
    Cursor<T> cgr(a.gr, a.ldgr, row0, step), cgh(a.gh, a.ldgh, row0, step), cr(a.r, a.ldr, row0, step),
        cy(a.y, a.ldy, row0, step), cg(a.gate, a.ldg, row0, step), cgy(a.gy, a.ldgy, row0, step), cgg(a.gg, a.ldgg, row0, step),
        cgres(a.gres, a.ldgres, row0, step);
    auto fetch = [&](int stage, int64_t row, int rows) {
        const int64_t at = row + rows * step;
        if (at - sub < a.M) {
            const bool inner = LAY < 0 ? at < a.M : at >= a.margin && at < a.M - a.margin;
            if (a.gr) ring.fetch(stage, kGr, cgr, rows, inner);
            if (PRE) {
                ring.fetch(stage, kGh, cgh, rows, inner);
                ring.fetch(stage, kR, cr, rows, inner);
            }
            if (POST) {
                ring.fetch(stage, kY, cy, rows, inner);
                if (a.gate_cols > 1) ring.fetch(stage, kGate, cg, rows, inner);
            }
        }
        Rg::commit();
    };
#pragma unroll
    for (int k = 0; k < kAhead - 1; ++k) fetch(k, row0, k);
    float2 aw[4], ab[4], wp[4];   // scale w_post, scale b_post, w_pre; 0 past the row's end
    load_vector<LAY, sizeof(T)>(a.scale, first, N, 1.f, wp);
    load_vector<LAY, sizeof(T)>(a.w_post, first, N, 1.f, aw);
    load_vector<LAY, sizeof(T)>(a.b_post, first, N, 0.f, ab);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        aw[i] = __fmul2_rn(aw[i], wp[i]);
        ab[i] = __fmul2_rn(ab[i], wp[i]);
    }
    load_vector<LAY, sizeof(T)>(a.w_pre, first, N, 1.f, wp);
    float2 sum[4][4] = {};
    // what a row has one of is loaded a row ahead
    float4 st_next = row0 < a.M ? __ldg(a.stats + row0) : make_float4(0, 0, 0, 0);
    float g_next = a.gate_cols == 1 && row0 < a.M ? to_f32(__ldg(cg.row)) : 1.f;
    int stage = 0;
    for (int64_t row = row0; row - sub < a.M; row += step) {   // the lanes of a warp together
        const bool here = LAY >= 0 || row < a.M, full = LAY < 0 ? here : whole;
        fetch(stage == 0 ? kAhead - 1 : stage - 1, row, kAhead - 1);
        const float4 st = st_next;
        float g1 = g_next, slope1 = 1.f;
        st_next = make_float4(0, 0, 0, 0);
        g_next = 1.f;   // lanes without a next row: not this row's gate, which may be infinite
        if (row + step < a.M) {
            st_next = __ldg(a.stats + row + step);
            if (a.gate_cols == 1) g_next = to_f32(__ldg(cg.ahead(1)));
        }
        Rg::wait();
        float2 dr[4];
        if (a.gr) ring.read(stage, kGr, cgr.row, dr);
        else
#pragma unroll
            for (int i = 0; i < 4; ++i) dr[i] = both(0.f);
        if (PRE) {
            float2 d[4], x[4], p, q;
            ring.read(stage, kGh, cgh.row, d);
            ring.read(stage, kR, cr.row, x);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = __fmul2_rn(__fadd2_rn(x[i], both(-st.z)), both(st.w));
                sum[2][i] = __ffma2_rn(d[i], x[i], sum[2][i]);
                sum[3][i] = __fadd2_rn(sum[3][i], d[i]);
                d[i] = __fmul2_rn(d[i], wp[i]);
                p = i ? __ffma2_rn(d[i], x[i], p) : __fmul2_rn(d[i], x[i]);
                q = i ? __fadd2_rn(d[i], q) : d[i];
            }
            float c0, c1 = 0.f;
            if (a.layer) {
                float c[2] = {p.x + p.y, q.x + q.y};
                row_sum<G, W, kRowLanes<LAY>>(c, red, turn, warp);
                c0 = c[0] * -a.inv_n;
                c1 = c[1] * -a.inv_n;
            } else {
                float c[1] = {p.x + p.y};
                row_sum<G, W, kRowLanes<LAY>>(c, red, turn, warp);
                c0 = c[0] * -a.inv_n;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                dr[i] = __ffma2_rn(__ffma2_rn(x[i], both(c0), __fadd2_rn(d[i], both(c1))), both(st.w), dr[i]);
        }
        if (a.gres) store_run<T, LAY>(cgres.out(), first, N, full, dr);
        if (POST) {
            float2 x[4], g[4], k[4], p, q, t = both(0.f);
            ring.read(stage, kY, cy.row, x);
            if (a.gate_cols > 1) {
                ring.read(stage, kGate, cg.row, g);
                if (a.gate_act != DLRM_GATE_NONE)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        gate_both<T>(g[i].x, a.gate_act, k[i].x);
                        gate_both<T>(g[i].y, a.gate_act, k[i].y);
                    }
                else
#pragma unroll
                    for (int i = 0; i < 4; ++i) k[i] = both(1.f);
            } else {
                if (a.gate_cols == 1) gate_both<T>(g1, a.gate_act, slope1);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    g[i] = both(g1);
                    k[i] = both(1.f);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = __fmul2_rn(__fadd2_rn(x[i], both(-st.x)), both(st.y));
                const float2 su = __ffma2_rn(x[i], aw[i], ab[i]);   // scale u
                t = __ffma2_rn(dr[i], su, t);
                k[i] = __fmul2_rn(__fmul2_rn(dr[i], su), k[i]);
                dr[i] = __fmul2_rn(dr[i], g[i]);
                sum[0][i] = __ffma2_rn(dr[i], x[i], sum[0][i]);
                sum[1][i] = __fadd2_rn(sum[1][i], dr[i]);
                dr[i] = __fmul2_rn(dr[i], aw[i]);
                p = i ? __ffma2_rn(dr[i], x[i], p) : __fmul2_rn(dr[i], x[i]);
                q = i ? __fadd2_rn(dr[i], q) : dr[i];
            }
            if (a.gg && a.gate_cols > 1) store_run<T, LAY>(cgg.out(), first, N, full, k);
            float c0, c1 = 0.f;
            if (a.layer) {
                float c[2] = {p.x + p.y, q.x + q.y};
                row_sum<G, W, kRowLanes<LAY>>(c, red, turn, warp);
                c0 = c[0] * -a.inv_n;
                c1 = c[1] * -a.inv_n;
            } else {
                float c[1] = {p.x + p.y};
                row_sum<G, W, kRowLanes<LAY>>(c, red, turn, warp);
                c0 = c[0] * -a.inv_n;
            }
            if (a.gg && a.gate_cols == 1) {
                float c[1] = {t.x + t.y};
                row_sum<G, W, kRowLanes<LAY>>(c, red, turn, warp);
                if (here && warp % W == 0 && lane % kRowLanes<LAY> == 0) *cgg.out() = from_f32<T>(c[0] * slope1);
            }
            if (a.gy) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    dr[i] = __fmul2_rn(__ffma2_rn(x[i], both(c0), __fadd2_rn(dr[i], both(c1))), both(st.y));
                store_run<T, LAY>(cgy.out(), first, N, full, dr);
            }
        }
        Rg::done();
        cgr.next();
        cgh.next();
        cr.next();
        cy.next();
        cg.next();
        cgy.next();
        cgg.next();
        cgres.next();
        stage = stage == kAhead - 1 ? 0 : stage + 1;
    }
    if (!a.partial) return;
    // the rows' sums of a block: its groups one after another, by way of the ring's memory
    float2* const tile = reinterpret_cast<float2*>(smem);
    asm volatile("cp.async.wait_all;" ::: "memory");
    constexpr int kGroups = G::kGroups, kThreads = G::kThreads;
    static_assert(Rg::kBytes >= kThreads * 32, "a tile fits");
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        if (s < 2 ? !POST : !PRE) continue;
#pragma unroll
        for (int m = kRowLanes<LAY>; m < kWarp; m *= 2)   // a warp's rows
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sum[s][i].x += __shfl_xor_sync(~0u, sum[s][i].x, m);
                sum[s][i].y += __shfl_xor_sync(~0u, sum[s][i].y, m);
            }
        if constexpr (kGroups > 1) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 4; ++i) tile[i * kThreads + threadIdx.x] = sum[s][i];
            __syncthreads();
            if (warp < W) {
#pragma unroll
                for (int g = 1; g < kGroups; ++g)
#pragma unroll
                    for (int i = 0; i < 4; ++i) sum[s][i] = __fadd2_rn(sum[s][i], tile[i * kThreads + g * W * 32 + threadIdx.x]);
            }
        }
        if (warp < W && lane < kRowLanes<LAY>)
            store_vector<LAY, sizeof(T)>(a.partial + ((int64_t)blockIdx.x * 4 + s) * a.Np, first, N, sum[s]);
    }
}

template <typename T, bool POST, bool PRE>
dlrm_status launch_bwd(const NormBwd& a, bool vec, cudaStream_t st)
{
    return with_rows(a.N, vec, [&](auto l, auto w) {
        constexpr int LAY = decltype(l)::value, W = decltype(w)::value, kWarps = bwd_warps(POST, PRE, LAY == kGrid);
        using G = BwdGroup<W, LAY, POST, PRE>;
        return launch_norm("block_norm_bwd_kernel", block_norm_bwd_kernel<T, LAY, W, POST, PRE>, a, kWarps, G::kThreads,
                           Rows<T, LAY, POST && PRE ? 5 : 3, G>::kBytes, st);
    });
}

}  // namespace

template <typename T>
dlrm_status forward(const NormFwd& a, bool vec, cudaStream_t st)
{
    return launch_fwd<T>(a, vec, st);
}

template <typename T>
dlrm_status backward(const NormBwd& a, bool vec, cudaStream_t st)
{
    return !a.y ? launch_bwd<T, false, true>(a, vec, st) : a.gh ? launch_bwd<T, true, true>(a, vec, st)
                                                               : launch_bwd<T, true, false>(a, vec, st);
}

}  // namespace norms
}  // namespace dlrm
