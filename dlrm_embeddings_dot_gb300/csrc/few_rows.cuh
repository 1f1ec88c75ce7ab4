// few_rows.cuh -- products of weight rows with a few tokens (at most 64),
// where the weights are the traffic: every weight goes from HBM straight into
// the registers of one warp as a matrix fragment.
//
// A warp multiplies WT tiles of 16 weight rows with NT tiles of 8 tokens over a
// range of K (mma.sync m16n8k16: at these shapes the tensor pipe idles, and
// unlike tcgen05 it takes both operands from registers, so nothing passes
// through shared memory).  The order of K inside a step is free as long as both
// operands use the same one: lane (g, t) = (lane / 4, lane % 4) takes the
// 16 consecutive bytes at 16 t of rows g and g + 8 and of token g, so every
// load is 16 bytes wide and four lanes cover 64 contiguous bytes of a row.
//   2-byte types: 8 values, the fragments of two k16 steps (32 of K)
//   fp32: 4 values, each split into three bf16 parts (8 + 8 + 8 bits); six
//   products of the parts, the smallest first, give the fp32 product (16 of K)
#pragma once

#include "dense_ops.cuh"

namespace dlrm {
namespace few {

constexpr int kRows = 16;         // weight rows of a tile
constexpr int kMaxTokens = 64;
constexpr int kPitch = 20;        // floats between tokens of a partial tile in shared memory: the fragment
                                  // stores of a warp (tokens 2t, rows g) then hit 32 different banks

template <typename T>
constexpr int kLane = 16 / (int)sizeof(T);   // values of K a lane loads at once
template <typename T>
constexpr int kStep = 4 * kLane<T>;          // values of K a warp covers at once

template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    if constexpr (std::is_same_v<T, __half>)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The lane's 16 bytes of a row: values [0, n) of the kLane at p, zeros behind.
template <typename T, bool VEC>
__device__ __forceinline__ uint4 load_part(const T* p, int n)
{
    if (VEC && n >= kLane<T>) return ldg_nc_l1_v4(p);
    T e[kLane<T>];
#pragma unroll
    for (int i = 0; i < kLane<T>; ++i) e[i] = i < n ? __ldg(p + i) : from_f32<T>(0.f);
    uint4 v;
    memcpy(&v, e, 16);
    return v;
}

// All kLane values.  KEEP: allocate in L1 (tokens, read by every warp); weights
// pass through once.
template <typename T, bool VEC, bool KEEP>
__device__ __forceinline__ uint4 load_lane(const T* p)
{
    if constexpr (!VEC) return load_part<T, false>(p, kLane<T>);
    else return KEEP ? ldg_nc_l1_v4(p) : ldg_nc_v4(p);
}

// Three bf16 parts of each of four floats (split1), two values to a word.
struct Parts {
    uint32_t hi[2], mid[2], lo[2];
};

__device__ __forceinline__ Parts split4(uint4 v)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    Parts p;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t h0, h1, m0, m1;
        float l0, l1;
        split1(__uint_as_float(w[2 * i]), h0, m0, l0);
        split1(__uint_as_float(w[2 * i + 1]), h1, m1, l1);
        p.hi[i] = __byte_perm(h0, h1, 0x7632);
        p.mid[i] = __byte_perm(m0, m1, 0x7632);
        const __nv_bfloat162 l = __floats2bfloat162_rn(l0, l1);
        memcpy(&p.lo[i], &l, 4);
    }
    return p;
}

// acc += the 16 rows (lane's bytes a of row g, b of row g + 8) times 8 tokens (x of token g).
template <typename T>
__device__ __forceinline__ void mac(float (&acc)[4], uint4 a, uint4 b, uint4 x)
{
    if constexpr (std::is_same_v<T, float>) {
        const Parts p = split4(a), q = split4(b), y = split4(x);
        mma16816<bf16>(acc, p.hi[0], q.hi[0], p.hi[1], q.hi[1], y.lo[0], y.lo[1]);
        mma16816<bf16>(acc, p.lo[0], q.lo[0], p.lo[1], q.lo[1], y.hi[0], y.hi[1]);
        mma16816<bf16>(acc, p.mid[0], q.mid[0], p.mid[1], q.mid[1], y.mid[0], y.mid[1]);
        mma16816<bf16>(acc, p.hi[0], q.hi[0], p.hi[1], q.hi[1], y.mid[0], y.mid[1]);
        mma16816<bf16>(acc, p.mid[0], q.mid[0], p.mid[1], q.mid[1], y.hi[0], y.hi[1]);
        mma16816<bf16>(acc, p.hi[0], q.hi[0], p.hi[1], q.hi[1], y.hi[0], y.hi[1]);
    } else {
        mma16816<T>(acc, a.x, b.x, a.y, b.y, x.x, x.y);
        mma16816<T>(acc, a.z, b.z, a.w, b.w, x.z, x.w);
    }
}

// acc[i][j] += tile i of 16 weight rows times tile j of 8 tokens over [k0, k1) of K
// (k0 a multiple of kStep).  w[i][0] / w[i][1]: rows g and g + 8 of tile i;
// x[j]: token g of tile j.  Every pointer is a readable row: where a tile has no
// such row or token any other does, as rows and tokens meet only in results
// that the caller then leaves alone.  XP: terms each token is the sum of, term i
// at x[j] + i * xplane.
template <typename T, int WT, int NT, bool VEC, int XP = 1>
__device__ __forceinline__ void rows_mac(float (&acc)[WT][NT][4], const T* (&w)[WT][2], const T* (&x)[NT], int k0, int k1,
                                         int64_t xplane = 0)
{
    // steps whose weight loads are issued together: what the registers beside the accumulators hold
    constexpr int U = (NT == 8 ? 2 : 4) / WT;
    constexpr int kBlock = U * kStep<T>;
    const int t = (threadIdx.x % kWarp) % 4;
    if (k0 >= k1) return;
#pragma unroll
    for (int i = 0; i < WT; ++i) {
        w[i][0] += k0 + t * kLane<T>;
        w[i][1] += k0 + t * kLane<T>;
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) x[j] += k0 + t * kLane<T>;
    int left = k1 - k0;
    auto load = [&](uint4 (&a)[U][WT][2], int at) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < WT; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) a[u][i][h] = load_lane<T, VEC, false>(w[i][h] + at + u * kStep<T>);
    };
    auto multiply = [&](const uint4 (&a)[U][WT][2], int at) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int q = 0; q < XP; ++q) {
                    const uint4 b = load_lane<T, VEC, true>(x[j] + q * xplane + at + u * kStep<T>);
#pragma unroll
                    for (int i = 0; i < WT; ++i) mac<T>(acc[i][j], a[u][i][0], a[u][i][1], b);
                }
    };
    auto advance = [&](int by) {
#pragma unroll
        for (int i = 0; i < WT; ++i) {
            w[i][0] += by;
            w[i][1] += by;
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) x[j] += by;
        left -= by;
    };
    if constexpr (NT <= 2 && VEC) {   // the next block's weights are on their way while one is multiplied
        uint4 a[U][WT][2], b[U][WT][2];
        if (left >= kBlock) load(a, 0);
#pragma unroll 1
        while (left >= 2 * kBlock) {
            load(b, kBlock);
            multiply(a, 0);
            if (left >= 3 * kBlock) load(a, 2 * kBlock);
            multiply(b, kBlock);
            advance(2 * kBlock);
        }
        if (left >= kBlock) {
            multiply(a, 0);
            advance(kBlock);
        }
    } else {
#pragma unroll 1
        while (left >= kBlock) {
            uint4 a[U][WT][2];
            load(a, 0);
            multiply(a, 0);
            advance(kBlock);
        }
    }
#pragma unroll 1
    while (left > 0) {   // the last steps, one at a time; past K both sides are zero
        const int n = left - t * kLane<T>;
        uint4 a[WT][2];
#pragma unroll
        for (int i = 0; i < WT; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) a[i][h] = load_part<T, VEC>(w[i][h], n);
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int q = 0; q < XP; ++q) {
                const uint4 b = load_part<T, VEC>(x[j] + q * xplane, n);
#pragma unroll
                for (int i = 0; i < WT; ++i) mac<T>(acc[i][j], a[i][0], a[i][1], b);
            }
        advance(kStep<T>);
    }
}

// The warp's partial tile to shared memory: part[token * kPitch + row].
template <int NT>
__device__ __forceinline__ void put_partial(float* part, const float (&acc)[NT][4])
{
    const int lane = threadIdx.x % kWarp, g = lane / 4, t = lane % 4;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        float* p = part + (j * 8 + 2 * t) * kPitch + g;
        p[0] = acc[j][0];
        p[kPitch] = acc[j][1];
        p[8] = acc[j][2];
        p[kPitch + 8] = acc[j][3];
    }
}

// Calls fn(std::integral_constant<int, NT>) with the least NT of 1, 2, 4, 8 that covers n tokens.
template <typename Fn>
__device__ __forceinline__ void with_token_tiles(int n, Fn&& fn)
{
    if (n <= 8) fn(std::integral_constant<int, 1>{});
    else if (n <= 16) fn(std::integral_constant<int, 2>{});
    else if (n <= 32) fn(std::integral_constant<int, 4>{});
    else fn(std::integral_constant<int, 8>{});
}

// ------------------------------------------------------- thread-block cluster
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of the same shared variable in block `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_map(const void* p, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(r)
                 : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ float cluster_ld(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void cluster_st(uint32_t addr, float v)
{
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

}  // namespace few
}  // namespace dlrm
