// few_rows.cuh -- products of weight rows with a few tokens (at most 64),
// where the weights are the traffic: every weight goes from HBM straight into
// the registers of one warp as a matrix fragment.
//
// A warp multiplies WT tiles of 16 weight rows with tokens over a range of K.
// The order of K inside a step is free as long as both sides use the same one:
// lane (g, t) = (lane / 4, lane % 4) takes the 32 consecutive bytes at 32 t of
// rows g and g + 8 and of its token, so a load is up to 32 bytes wide and four
// lanes cover 128 contiguous bytes of a row (with 16-byte loads L1's tag stage
// alone held the weights to half of HBM's rate).
//   2-byte types: 16 values, the fragments of four mma.sync m16n8k16 (64 of K)
//     against NT tiles of 8 tokens.  At these shapes the tensor pipe idles, and
//     unlike tcgen05 it takes both operands from registers
//   fp32, up to 8 tokens: 8 values (32 of K), multiplied and added in fp32;
//     the four lanes of a row add up their shares at the end
//   fp32, more tokens: the same values as three bf16 parts each (8 + 8 + 8
//     bits), whose six products, the smallest first, give the fp32 product.  The
//     tensor cores cut what they add to an accumulator instead of rounding it, so
//     16 of K are summed from zero and added in fp32: in one accumulator through
//     all of K the error was 3 to 7 times an fp32 product's (32 x 4096 x 4096:
//     3.7e-6 against 1.2e-6, 32768 x 256 to 16: 1.9e-6 against 2.9e-7)
#pragma once

#include "dense_ops.cuh"

namespace dlrm {
namespace few {

constexpr int kRows = 16;         // weight rows of a tile
constexpr int kMaxTokens = 64;
constexpr int kPitch = 20;         // floats between tokens of a partial tile in shared memory: the fragment
                                   // stores of a warp (tokens 2t, rows g) then hit 32 different banks

template <typename T>
constexpr int kLane = 32 / (int)sizeof(T);   // values of K a lane loads at once
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

struct Chunk {
    uint4 v[2];
};

// The lane's 32 bytes of a row: values [0, n) of the kLane at p, zeros behind.
template <typename T>
__device__ __forceinline__ Chunk load_part(const T* p, int n)
{
    T e[kLane<T>];
#pragma unroll
    for (int i = 0; i < kLane<T>; ++i) e[i] = i < n ? __ldg(p + i) : from_f32<T>(0.f);
    Chunk c;
    memcpy(&c, e, 32);
    return c;
}

// All kLane values; VEC: 2 on the 32-byte grid, 1 on the 16-byte grid, 0 off it.
// KEEP: allocate in L1 (tokens, read by every warp); weights pass through once.
template <typename T, int VEC, bool KEEP>
__device__ __forceinline__ Chunk load_lane(const T* p)
{
    Chunk c;
    if constexpr (VEC == 2 && !KEEP) {
        asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(c.v[0].x), "=r"(c.v[0].y), "=r"(c.v[0].z), "=r"(c.v[0].w), "=r"(c.v[1].x), "=r"(c.v[1].y),
                       "=r"(c.v[1].z), "=r"(c.v[1].w)
                     : "l"(p));
    } else if constexpr (VEC == 2) {
        asm volatile("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(c.v[0].x), "=r"(c.v[0].y), "=r"(c.v[0].z), "=r"(c.v[0].w), "=r"(c.v[1].x), "=r"(c.v[1].y),
                       "=r"(c.v[1].z), "=r"(c.v[1].w)
                     : "l"(p));
    } else if constexpr (VEC == 1) {
        const uint4* q = reinterpret_cast<const uint4*>(p);
        c.v[0] = KEEP ? ldg_nc_l1_v4(q) : ldg_nc_v4(q);
        c.v[1] = KEEP ? ldg_nc_l1_v4(q + 1) : ldg_nc_v4(q + 1);
    } else {
        c = load_part<T>(p, kLane<T>);
    }
    return c;
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

// acc += the 16 rows (lane's bytes a of row g, b of row g + 8) times 8 tokens (x of token g), 16 bytes each.
template <typename T>
__device__ __forceinline__ void mac16(float (&acc)[4], uint4 a, uint4 b, uint4 x)
{
    if constexpr (std::is_same_v<T, float>) {
        const Parts p = split4(a), q = split4(b), y = split4(x);
        float d[4] = {};
        mma16816<bf16>(d, p.hi[0], q.hi[0], p.hi[1], q.hi[1], y.lo[0], y.lo[1]);
        mma16816<bf16>(d, p.lo[0], q.lo[0], p.lo[1], q.lo[1], y.hi[0], y.hi[1]);
        mma16816<bf16>(d, p.mid[0], q.mid[0], p.mid[1], q.mid[1], y.mid[0], y.mid[1]);
        mma16816<bf16>(d, p.hi[0], q.hi[0], p.hi[1], q.hi[1], y.mid[0], y.mid[1]);
        mma16816<bf16>(d, p.mid[0], q.mid[0], p.mid[1], q.mid[1], y.hi[0], y.hi[1]);
        mma16816<bf16>(d, p.hi[0], q.hi[0], p.hi[1], q.hi[1], y.hi[0], y.hi[1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] += d[i];
    } else {
        mma16816<T>(acc, a.x, b.x, a.y, b.y, x.x, x.y);
        mma16816<T>(acc, a.z, b.z, a.w, b.w, x.z, x.w);
    }
}

template <typename T>
__device__ __forceinline__ void mac(float (&acc)[4], const Chunk& a, const Chunk& b, const Chunk& x)
{
#pragma unroll
    for (int h = 0; h < 2; ++h) mac16<T>(acc, a.v[h], b.v[h], x.v[h]);
}

// s += the eight products of two chunks of floats
__device__ __forceinline__ void dot8(float& s, const Chunk& a, const Chunk& x)
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float4 u = u4_as_f4(a.v[h]), v = u4_as_f4(x.v[h]);
        s = fmaf(u.x, v.x, s);
        s = fmaf(u.y, v.y, s);
        s = fmaf(u.z, v.z, s);
        s = fmaf(u.w, v.w, s);
    }
}

// Visits [k0, k1) of K (k0 a multiple of kStep) for WT tiles of 16 weight rows and
// NX tokens of this lane: mul(i, j, a, b, x) gets the lane's chunks of rows g and
// g + 8 of tile i and of its token j.  w[i][0] / w[i][1]: rows g and g + 8 of tile
// i.  Every pointer is a readable row: where a tile has no such row or token any
// other does, as rows and tokens meet only in results that the caller then leaves
// alone.  XP: terms each token is the sum of, term q at x[j] + q * xplane.  fix(j, k, x)
// may change a chunk of token j, whose first value is k values behind k0, before use.
template <typename T, int WT, int NX, int VEC, int XP, int U, bool AHEAD, typename Mul, typename Fix>
__device__ __forceinline__ void visit_k(const T* (&w)[WT][2], const T* (&x)[NX], int k0, int k1, int64_t xplane, Mul&& mul,
                                        Fix&& fix)
{
    constexpr int kBlock = U * kStep<T>;   // K whose weight loads are issued together
    const int t = (threadIdx.x % kWarp) % 4;
    if (k0 >= k1) return;
#pragma unroll
    for (int i = 0; i < WT; ++i) {
        w[i][0] += k0 + t * kLane<T>;
        w[i][1] += k0 + t * kLane<T>;
    }
#pragma unroll
    for (int j = 0; j < NX; ++j) x[j] += k0 + t * kLane<T>;
    int left = k1 - k0;
    auto load = [&](Chunk (&a)[U][WT][2], int at) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < WT; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) a[u][i][h] = load_lane<T, VEC, false>(w[i][h] + at + u * kStep<T>);
    };
    auto multiply = [&](const Chunk (&a)[U][WT][2], int at) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < NX; ++j)
#pragma unroll
                for (int q = 0; q < XP; ++q) {
                    Chunk b = load_lane<T, VEC, true>(x[j] + q * xplane + at + u * kStep<T>);
                    fix(j, k1 - k0 - left + at + u * kStep<T> + t * kLane<T>, b);
#pragma unroll
                    for (int i = 0; i < WT; ++i) mul(i, j, a[u][i][0], a[u][i][1], b);
                }
    };
    auto advance = [&](int by) {
#pragma unroll
        for (int i = 0; i < WT; ++i) {
            w[i][0] += by;
            w[i][1] += by;
        }
#pragma unroll
        for (int j = 0; j < NX; ++j) x[j] += by;
        left -= by;
    };
    if constexpr (AHEAD && VEC > 0) {   // the next block's weights are on their way while one is multiplied
        Chunk a[U][WT][2], b[U][WT][2];
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
            Chunk a[U][WT][2];
            load(a, 0);
            multiply(a, 0);
            advance(kBlock);
        }
    }
#pragma unroll 1
    while (left > 0) {   // the last steps, one at a time; past K both sides are zero
        const int n = left - t * kLane<T>;
        Chunk a[WT][2];
        if (VEC > 0 && left >= kStep<T>) {
#pragma unroll
            for (int i = 0; i < WT; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) a[i][h] = load_lane<T, VEC, false>(w[i][h]);
#pragma unroll
            for (int j = 0; j < NX; ++j)
#pragma unroll
                for (int q = 0; q < XP; ++q) {
                    Chunk b = load_lane<T, VEC, true>(x[j] + q * xplane);
                    fix(j, k1 - k0 - left + t * kLane<T>, b);
#pragma unroll
                    for (int i = 0; i < WT; ++i) mul(i, j, a[i][0], a[i][1], b);
                }
        } else {
#pragma unroll
            for (int i = 0; i < WT; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) a[i][h] = load_part<T>(w[i][h], n);
#pragma unroll
            for (int j = 0; j < NX; ++j)
#pragma unroll
                for (int q = 0; q < XP; ++q) {
                    Chunk b = load_part<T>(x[j] + q * xplane, n);
                    fix(j, k1 - k0 - left + t * kLane<T>, b);
#pragma unroll
                    for (int i = 0; i < WT; ++i) mul(i, j, a[i][0], a[i][1], b);
                }
        }
        advance(kStep<T>);
    }
}

// out(i, token, row, value) for every sum of the warp's WT tiles of 16 weight rows
// (pointers as for visit_k) with tokens [0, n), n <= 8 NT, over [k0, k1) of K.
// token(j) gives the row of token j (j < n).  fix as for visit_k, j counting the lane's
// tokens 8 j + g (2-byte types).
struct Unchanged {
    __device__ __forceinline__ void operator()(int, int, Chunk&) const {}
};
template <typename T, int WT, int NT, int VEC, int XP = 1, typename Token, typename Out, typename Fix = Unchanged>
__device__ __forceinline__ void rows_times_tokens(const T* (&w)[WT][2], Token&& token, int n, int k0, int k1,
                                                  int64_t xplane, Out&& out, Fix&& fix = Fix())
{
    const int lane = threadIdx.x % kWarp, g = lane / 4, t = lane % 4;
    if constexpr (std::is_same_v<T, float> && NT == 1) {
        // every lane has all the tokens, for its share of K
        auto with = [&](auto nn) {
            constexpr int NX = decltype(nn)::value;
            const T* x[NX];
#pragma unroll
            for (int j = 0; j < NX; ++j) x[j] = token(min(j, n - 1));
            float acc[WT][NX][2] = {};
            visit_k<T, WT, NX, VEC, XP, 2 / WT, (NX <= 2)>(w, x, k0, k1, xplane,
                                                            [&](int i, int j, const Chunk& a, const Chunk& b, const Chunk& c) {
                                                                dot8(acc[i][j][0], a, c);
                                                                dot8(acc[i][j][1], b, c);
                                                            }, Unchanged());
#pragma unroll
            for (int i = 0; i < WT; ++i)
#pragma unroll
                for (int j = 0; j < NX; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float v = acc[i][j][h];
                        v += __shfl_xor_sync(~0u, v, 1);
                        v += __shfl_xor_sync(~0u, v, 2);
                        if (t == 0 && j < n) out(i, j, g + 8 * h, v);
                    }
        };
        if (n == 1) with(std::integral_constant<int, 1>{});
        else if (n == 2) with(std::integral_constant<int, 2>{});
        else if (n <= 4) with(std::integral_constant<int, 4>{});
        else with(std::integral_constant<int, 8>{});
    } else {
        const T* x[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) x[j] = token(min(j * 8 + g, n - 1));
        float acc[WT][NT][4] = {};
        constexpr int U = WT == 1 && NT < 8 ? 2 : 1;
        visit_k<T, WT, NT, VEC, XP, U, (NT == 1)>(w, x, k0, k1, xplane,
                                                  [&](int i, int j, const Chunk& a, const Chunk& b, const Chunk& c) {
                                                      mac<T>(acc[i][j], a, b, c);
                                                  }, fix);
#pragma unroll
        for (int i = 0; i < WT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int tok = j * 8 + 2 * t + (c & 1);
                    if (tok < n) out(i, tok, g + 8 * (c >> 1), acc[i][j][c]);
                }
    }
}

// 2, 1 or 0: whether rows of `width` elements lie on the 32-byte grid, on the 16-byte grid, or off both.
inline int row_grid(const void* p, int64_t ld, int rows, int es)
{
    if ((reinterpret_cast<uintptr_t>(p) & 31u) == 0 && (rows <= 1 || ld * es % 32 == 0)) return 2;
    return rows_aligned16(p, ld, rows, es) ? 1 : 0;
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
