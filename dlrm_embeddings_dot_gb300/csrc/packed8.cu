// packed8.cu -- matrices to 8 bits and back: 8-bit floats with a power of two for
// every 32 columns, so that scaling is exact and the only rounding is the one to four bits.
// Bound by memory, several 16-byte words a lane in flight.  Four lanes have a block of 32 columns,
// eight of fp32, a word each.
#include "packed8.cuh"
#include "dlrm_block.h"
#include "row_units.cuh"

namespace dlrm {
namespace {

constexpr int kThreads8 = 256;

constexpr int kWords8 = 4;

template <typename T>
constexpr int kRuns8 = kRuns<T, kOnGrid, 2>;

// Walks the words of rows, `groups` of them a row, kWords8 at a time: each(k, row, word) for those
// there are, in a loop over k that the compiler unrolls.
struct Words {
    int64_t i, end, stride, row, g, groups, drow, dg;
    __device__ Words(int64_t rows, int64_t n) : groups(n)
    {
        end = groups * rows;
        stride = (int64_t)gridDim.x * kThreads8;
        i = (int64_t)blockIdx.x * kThreads8 + threadIdx.x;
        row = i / groups;
        g = i - row * groups;
        drow = stride / groups;
        dg = stride - drow * groups;
    }
    __device__ __forceinline__ bool more() const { return i < end; }
    __device__ __forceinline__ void next()
    {
        i += stride;
        row += drow;
        g += dg;
        if (g >= groups) {
            g -= groups;
            ++row;
        }
    }
};

// The exponent byte for the largest size 1.m 2^(E - 127): that is at most 448 2^(e - 127) from
// e = E - 8 on, or E - 7 where 1.m > 1.75.
__device__ __forceinline__ int exponent8(uint32_t top)
{
    return max(0, (int)(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u));
}

__device__ __forceinline__ float scale_up(int e) { return __uint_as_float((uint32_t)(254 - e) << 23); }   // 2^(127 - e)

__device__ __forceinline__ uint16_t round8(float lo, float hi)
{
    uint16_t h;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(hi), "f"(lo));
    return h;
}

// The largest size in a block, which LANES neighbouring lanes have a 16-byte word each of, as fp32's bits.
template <typename T, int LANES>
__device__ __forceinline__ uint32_t block_size8(const uint4& v)
{
    const uint32_t those = (LANES == 32 ? ~0u : (1u << LANES % 32) - 1) << (threadIdx.x % kWarp / LANES * LANES);
    if constexpr (sizeof(T) == 2) {   // sizes of numbers order as their bits do: two at a time
        uint32_t top = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
#pragma unroll
        for (int m = 1; m < LANES; m *= 2) top = __vmaxu2(top, __shfl_xor_sync(those, top, m));
        const uint16_t h = (uint16_t)max(top & 0xffffu, top >> 16);
        T t;
        memcpy(&t, &h, 2);
        return __float_as_uint(to_f32(t));
    } else {
        uint32_t top = max(max(v.x & 0x7fffffffu, v.y & 0x7fffffffu), max(v.z & 0x7fffffffu, v.w & 0x7fffffffu));
#pragma unroll
        for (int m = 1; m < LANES; m *= 2) top = max(top, __shfl_xor_sync(those, top, m));
        return top;
    }
}

// A word with its infinities and NaN as zeros, and which they were.
template <typename T>
__device__ __forceinline__ uint32_t drop_wild(uint4& v)
{
    constexpr int V = 16 / sizeof(T);
    T e[V];
    memcpy(e, &v, 16);
    uint32_t gone = 0;
#pragma unroll
    for (int i = 0; i < V; ++i)
        if ((__float_as_uint(to_f32(e[i])) & 0x7fffffffu) >= 0x7f800000u) {
            e[i] = from_f32<T>(0.f);
            gone |= 1u << i;
        }
    memcpy(&v, e, 16);
    return gone;
}

// The exponent of a block, and the lane's word of it in its scale as bytes.  Infinities and NaN become NaN
// and do not count for the block.
template <typename T>
__device__ __forceinline__ int block8(uint4 v, uint32_t (&w)[4 / sizeof(T)])
{
    constexpr int V = 16 / sizeof(T), kLanes = kBlock8 / V;
    uint32_t top = block_size8<T, kLanes>(v), gone = 0;
    if (top >= 0x7f800000u) {   // the same in all of the block's lanes
        gone = drop_wild<T>(v);
        top = block_size8<T, kLanes>(v);
    }
    const int e = exponent8(top);
    const float up = scale_up(e);
    float f[8];
    if constexpr (sizeof(T) == 2) {
        unpack8<T>(v, f);
    } else {
        const float4 g = u4_as_f4(v);
        f[0] = g.x; f[1] = g.y; f[2] = g.z; f[3] = g.w;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] *= up;
    if (gone)
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (gone >> i & 1) f[i] = __uint_as_float(0x7fc00000u);
#pragma unroll
    for (int i = 0; i < V / 4; ++i)
        w[i] = round8(f[4 * i], f[4 * i + 1]) | (uint32_t)round8(f[4 * i + 2], f[4 * i + 3]) << 16;
    return e;
}

// blocks: exponent bytes of a row.  Rows go by units of lanes (row_units.cuh): as one sequence of words,
// as in unpack8_kernel, the places of four words cost registers (65536 x 1024 bf16 46 us, so 40).
template <typename T>
__global__ void __launch_bounds__(kThreads8)
pack8_kernel(const T* __restrict__ x, int64_t ldx, int M, int N, int lanes, uint8_t* __restrict__ q, int64_t ldq,
             uint8_t* __restrict__ exps, int blocks)
{
    constexpr int U = kRuns8<T>, V = 16 / sizeof(T);
    pdl_wait();
    const Unit unit(lanes);
    for (Items it(unit, N, U); it.row < M; it.next()) {
        Raw8<T> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (u < it.per)
                v[u] = load_cols<T, kOnGrid>(x + it.row * ldx, unit.first<kOnGrid, sizeof(T)>(it.run(u)), N, lanes);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (u >= it.per) break;
            const int c = unit.first<kOnGrid, sizeof(T)>(it.run(u));
#pragma unroll
            for (int h = 0; h < 8 / V; ++h) {   // the run's 16-byte words
                uint32_t w[V / 4];
                const int e = block8<T>(v[u].w[h], w), at = c + h * 4 * lanes;
                if (at < N) {
                    uint8_t* p = q + it.row * ldq + at;
                    if constexpr (V == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
                    else *reinterpret_cast<uint32_t*>(p) = w[0];
                    if (at % kBlock8 == 0) exps[it.row * blocks + at / kBlock8] = (uint8_t)e;
                }
            }
        }
    }
}

// The same of eight neighbours a lane, four lanes a block.
template <typename T>
__device__ __forceinline__ int run8(Raw8<T> v, uint32_t (&w)[2])
{
    if constexpr (sizeof(T) == 2) {
        return block8<T>(v.w[0], w);
    } else {
        uint32_t gone = 0, top = max(block_size8<T, 4>(v.w[0]), block_size8<T, 4>(v.w[1]));
        if (top >= 0x7f800000u) {
            gone = drop_wild<T>(v.w[0]) | drop_wild<T>(v.w[1]) << 4;
            top = max(block_size8<T, 4>(v.w[0]), block_size8<T, 4>(v.w[1]));
        }
        const int e = exponent8(top);
        const float up = scale_up(e);
        float f[8];
        widen8<T>(v, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = gone >> i & 1 ? __uint_as_float(0x7fc00000u) : f[i] * up;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            w[i] = round8(f[4 * i], f[4 * i + 1]) | (uint32_t)round8(f[4 * i + 2], f[4 * i + 3]) << 16;
        return e;
    }
}

// Off the grid: the runs of all rows are one sequence, four a block; a run is read as the 16-byte words
// that it lies in and leaves in the widest pieces that its address allows.  (Every 32nd column a lane
// instead: 60000 x 515 bf16 62 us, where single loads of neighbours took 35.)
template <typename T>
__global__ void __launch_bounds__(kThreads8)
pack8_any_kernel(const T* __restrict__ x, int64_t ldx, int M, int N, uint8_t* __restrict__ q, int64_t ldq,
                 uint8_t* __restrict__ exps, int blocks)
{
    pdl_wait();
    const T* const end = x + (M - 1) * ldx + N;
    for (Words w8(M, (int64_t)blocks * 4); w8.more(); w8.next()) {   // a quad's lanes leave together
        const int64_t row = w8.row, c = w8.g * 8;
        const int n = (int)min((int64_t)8, N - c);    // 0 or less: past the row's end
        Raw8<T> v = {};
        if (n > 0) {
            v = load8_shifted<T>(x + row * ldx + c, n, x, end);
            if (n < 8) {
                T e[8];
                memcpy(e, &v, sizeof(e));
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i >= n) e[i] = from_f32<T>(0.f);
                memcpy(&v, e, sizeof(e));
            }
        }
        uint32_t w[2];
        const int e = run8<T>(v, w);
        uint8_t* p = q + row * ldq + c;
        const uint32_t off = (uint32_t)(uintptr_t)p & 7u;
        if (n == 8 && off == 0) {
            *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        } else if (n == 8 && off == 4) {
            reinterpret_cast<uint32_t*>(p)[0] = w[0];
            reinterpret_cast<uint32_t*>(p)[1] = w[1];
        } else if (n == 8 && off % 2 == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)(w[i / 2] >> 16 * (i % 2));
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n) p[i] = (uint8_t)(w[i / 4] >> 8 * (i % 4));
        }
        if (w8.g % 4 == 0) exps[row * blocks + w8.g / 4] = (uint8_t)e;
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads8)
unpack8_kernel(const __grid_constant__ Packed8 m, int M, int N, T* __restrict__ y, int64_t ldy)
{
    constexpr int V = 16 / sizeof(T);
    pdl_wait();
    Words w(M, N / V);
    while (w.more()) {
        uint2 v[kWords8];
        uint32_t e[kWords8];
        T* to[kWords8];
        int live = 0;
#pragma unroll
        for (int k = 0; k < kWords8; ++k)
            if (w.more()) {
                const int col = (int)w.g * V;
                const uint8_t* p = m.q + w.row * m.ld + col;
                if constexpr (V == 8) v[k] = __ldg(reinterpret_cast<const uint2*>(p));
                else v[k] = make_uint2(__ldg(reinterpret_cast<const uint32_t*>(p)), 0);
                e[k] = __ldg(m.exps + w.row * m.blocks + col / kBlock8);
                to[k] = y + w.row * ldy + col;
                live = k + 1;
                w.next();
            }
#pragma unroll
        for (int k = 0; k < kWords8; ++k) {
            if (k >= live) break;
            float f[8];
            widen_run8<T>({v[k], e[k]}, f);
            if constexpr (V == 8) store8<T, true>(to[k], 8, f);
            else *reinterpret_cast<float4*>(to[k]) = make_float4(f[0], f[1], f[2], f[3]);
        }
    }
}

// Off the grid: rows by warps (row_units.cuh), every 32nd column a lane or pair of them; FEW: by a few lanes
// (to 8 bits and back, us, a warp a row / so: 56414 x 44 bf16 25 / 16, 65536 x 7 fp16 25 / 10).
template <typename T, bool FEW>
__global__ void __launch_bounds__(kThreads8)
unpack8_any_kernel(const __grid_constant__ Packed8 m, int M, int N, int lanes, T* __restrict__ y, int64_t ldy)
{
    pdl_wait();
    const Unit unit(FEW ? lanes : kWarp);
    if constexpr (FEW) {
        for (int64_t row = unit.unit; row < M; row += unit.units) {
            const uint8_t *q = m.q + row * m.ld, *e = m.exps + row * m.blocks;
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int c = min(unit.l + i * lanes, N - 1);
                f[i] = value8<T>(__ldg(q + c), __ldg(e + c / kBlock8));
            }
            store_cols<T, kFewLanes>(y + row * ldy, unit.l, N, lanes, f);
        }
        return;
    }
    const int lane = threadIdx.x % kWarp;
    for (Items it(unit, N, 1); it.row < M; it.next()) {
        const int c = unit.first<kOffGrid, sizeof(T)>((int)it.part);
        const uint8_t* row = m.q + it.row * m.ld;
        const bool words = sizeof(T) == 2 && ((uintptr_t)row & 1u) == 0;
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int x = run_col<false, sizeof(T)>(c, 2 * i), z = run_col<false, sizeof(T)>(c, 2 * i + 1);
            uint32_t h = 0;
            if (words && z < N) {
                h = __ldg(reinterpret_cast<const uint16_t*>(row + x));
            } else {
                if (x < N) h = __ldg(row + x);
                if (z < N) h |= (uint32_t)__ldg(row + z) << 8;
            }
            w[i / 2] |= h << 16 * (i % 2);
        }
        const int64_t b = it.part * 8 + lane;   // lane i has the part's i-th block's exponent
        const float own = scale8(lane < 8 && b < m.blocks ? __ldg(m.exps + it.row * m.blocks + b) : 0);
        float f[8];
        if constexpr (sizeof(T) == 2) {
            float scale[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) scale[i] = __shfl_sync(~0u, own, 2 * i + lane / 16);
            widen_codes8<T>(make_uint2(w[0], w[1]), scale, f);
        } else {   // a scale each: the values without it, then it
            const float one[4] = {1.f, 1.f, 1.f, 1.f};
            widen_codes8<T>(make_uint2(w[0], w[1]), one, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                f[i] *= __shfl_sync(~0u, own, i);
                if (fabsf(f[i]) > kMost8<T>) f[i] = copysignf(kMost8<T>, f[i]);
            }
        }
        store_cols<T, kOffGrid>(y + it.row * ldy, c, N, kWarp, f);
    }
}

dlrm_status check_sizes8(const char* fn, dlrm_dtype dtype, int M, int N)
{
    if (!dense_dtype_ok(dtype)) return fail(DLRM_ERR_INVALID_ARG, "%s: bad dtype", fn);
    if (M < 0 || N < 1) return fail(DLRM_ERR_INVALID_ARG, "%s: need M >= 0 and N >= 1", fn);
    if (M > kMaxSize || N > kMaxSize) return fail(DLRM_ERR_UNSUPPORTED, "%s: sizes up to %d", fn, kMaxSize);
    return DLRM_OK;
}

// Blocks for lanes that take `each` words at a time.
unsigned word_blocks(int64_t words, int each, const void* kern)
{
    return grid_blocks((words + kThreads8 * each - 1) / (kThreads8 * each), kern);
}

}  // namespace
}  // namespace dlrm

using namespace dlrm;

extern "C" dlrm_status dlrm_pack8(const void* d_x, int64_t ldx, dlrm_dtype dtype, int M, int N, uint8_t* d_q, int64_t ldq,
                                  uint8_t* d_exps, void* stream)
{
    DLRM_API_RANGE("dlrm_pack8");
    clear_error();
    const char* fn = "dlrm_pack8";
    dlrm_status s = check_sizes8(fn, dtype, M, N);
    if (s != DLRM_OK || M == 0) return s;
    const int es = dense_dtype_size(dtype);
    if ((s = check_matrix(fn, "d_x", d_x, ldx, M, N, es)) != DLRM_OK) return s;
    if ((s = check_packed(fn, "d_q", d_q, ldq, d_exps, M, N)) != DLRM_OK) return s;
    const bool vec = N % 8 == 0 && rows_aligned16(d_x, ldx, M, es) && rows_aligned8(d_q, ldq, M);
    return with_type(dtype, [&](auto t) {
        using T = decltype(t);
        const int lanes = unit_lanes(N, kOnGrid, sizeof(T) == 2 ? 4 : 8), blocks = blocks8(N);   // a block's lanes at least
        if (vec) {
            auto kern = pack8_kernel<T>;
            const unsigned grid = item_blocks(M, N, lanes, kRuns8<T>, (const void*)kern);
            return check_launch_pdl(launch_pdl(kern, dim3(grid), dim3(kThreads8), 0, as_stream(stream), (const T*)d_x, ldx, M, N,
                                               lanes, d_q, ldq, d_exps, blocks),
                                    "pack8_kernel");
        }
        auto kern = pack8_any_kernel<T>;
        const unsigned grid = word_blocks((int64_t)M * blocks * 4, 1, (const void*)kern);
        return check_launch_pdl(launch_pdl(kern, dim3(grid), dim3(kThreads8), 0, as_stream(stream), (const T*)d_x, ldx, M, N, d_q,
                                           ldq, d_exps, blocks),
                                "pack8_any_kernel");
    });
}

extern "C" dlrm_status dlrm_unpack8(const uint8_t* d_q, int64_t ldq, const uint8_t* d_exps, dlrm_dtype dtype, int M, int N,
                                    void* d_y, int64_t ldy, void* stream)
{
    DLRM_API_RANGE("dlrm_unpack8");
    clear_error();
    const char* fn = "dlrm_unpack8";
    dlrm_status s = check_sizes8(fn, dtype, M, N);
    if (s != DLRM_OK || M == 0) return s;
    const int es = dense_dtype_size(dtype);
    if ((s = check_packed(fn, "d_q", d_q, ldq, d_exps, M, N)) != DLRM_OK) return s;
    if ((s = check_matrix(fn, "d_y", d_y, ldy, M, N, es)) != DLRM_OK) return s;
    const bool vec = N % 8 == 0 && rows_aligned16(d_y, ldy, M, es) && rows_aligned8(d_q, ldq, M);
    const Packed8 m = packed8(d_q, ldq, d_exps, M, N);
    return with_type(dtype, [&](auto t) {
        using T = decltype(t);
        if (vec) {
            auto kern = unpack8_kernel<T>;
            const unsigned blocks = word_blocks((int64_t)M * N * (int)sizeof(T) / 16, kWords8, (const void*)kern);
            return check_launch_pdl(launch_pdl(kern, dim3(blocks), dim3(kThreads8), 0, as_stream(stream), m, M, N, (T*)d_y, ldy),
                                    "unpack8_kernel");
        }
        const int lay = row_layout(false, N), lanes = unit_lanes(N, lay);
        auto kern = lay == kFewLanes ? unpack8_any_kernel<T, true> : unpack8_any_kernel<T, false>;
        return check_launch_pdl(launch_pdl(kern, dim3(item_blocks(M, N, lanes, 1, (const void*)kern)), dim3(kThreads8), 0,
                                           as_stream(stream), m, M, N, lanes, (T*)d_y, ldy),
                                "unpack8_any_kernel");
    });
}
