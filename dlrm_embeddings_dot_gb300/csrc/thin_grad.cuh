// thin_grad.cuh -- the gradient of a dense layer of up to 16 outputs (the logit
// layer of a click model):
//
//   dZ = a'(z) drop(dY);  dX = dZ W;  dW = dZ^T x;  db = sum dZ
//
// One pass: x is read once and dX written once, both products beside it; the
// tcgen05 tiles' 64 columns would be mostly padding.  A block owns some columns of
// x and a chunk of its rows.  dZ of 256 rows goes to shared memory; then the warps walk
// rows, the columns' part of W and of dW in registers.  Chunks' sums are added in order by
// thin_sum_kernel.
//
//   2-byte types: mma.sync m16n8k16.  A warp takes 16 rows x 64 columns at a time, a
//   lane eight columns of four rows; the order of the columns within the fragments is
//   chosen so that its loads and stores are whole 16-byte words.
//   fp32: 2 N multiply-adds an element on the ordinary pipes, so nothing is split.
//
// HBM bounds few outputs, the instructions of a row many: 65536 x 1024, us, for 1, 8 and 16
// outputs: fp16 63, 65, 74 (two passes over x at the measured copy rate: 40), fp32 99, 114,
// 172 (79).  One launch and the sum of the chunks is all that a small batch pays (300 x 64: 6.4).
#pragma once

#include "dense_epilogue.cuh"
#include "few_rows.cuh"

namespace dlrm {
namespace thin {

constexpr int kMaxOutputs = 16;
constexpr int kTile = 256;   // rows of dZ in shared memory, one a thread

struct Grad {
    const void *dy, *pre, *x, *w;
    int64_t ldg, ldp, ldx, ldw;
    int M, N, K, act;
    Drop drop;
    float scale, bias_scale;   // of the products' and of the bias gradient's sums
    int cg, rows;       // threads along the columns; rows of a chunk
    void *dx, *dw;      // each may be NULL
    int64_t lddx, lddw;
    float* db;          // may be NULL
    float* partial;     // [chunks][N * K + N], NULL for one chunk
};

// dZ of the rows t0 .. t0 + rows - 1 (256 at most, one a thread), eight outputs at a time:
// store(group, values).  Where bias is summed, lane n of a warp adds the warp's rows of output n to b.
template <typename T, typename Store>
__device__ __forceinline__ void tile_of_dz(const Grad& a, const DropKey& key, int t0, int rows, float& b, Store store)
{
    const int tid = threadIdx.x, row = t0 + tid;
    const bool bias = a.db && blockIdx.x == 0;
#pragma unroll 1
    for (int g = 0; g * 8 < a.N; ++g) {
        const int n = a.N - g * 8;
        float f[8] = {};
        if (tid < rows) {
            widen8<T>(load8<T, false>((const T*)a.dy + row * a.ldg + g * 8, n), f);
            if (a.act != DLRM_ACT_NONE) {
                float z[8];
                widen8<T>(load8<T, false>((const T*)a.pre + row * a.ldp + g * 8, n), z);
                slope8<T>(f, z, a.act);
            }
            if (a.drop.thr) drop8(f, a.drop, key, (uint32_t)row, (uint32_t)g);
        }
        store(g, f);
        if (!bias) continue;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float s = f[i];
#pragma unroll
            for (int m = 16; m; m /= 2) s += __shfl_xor_sync(~0u, s, m);
            if (tid % 32 == g * 8 + i) b += s;
        }
    }
}

// The sums of one chunk, where they go.
template <typename T>
struct Sums {
    const Grad& a;
    int64_t NK;
    float* partial;
    __device__ explicit Sums(const Grad& g) : a(g), NK((int64_t)g.N * g.K)
    {
        partial = g.partial ? g.partial + blockIdx.y * (NK + g.N) : nullptr;
    }
    __device__ void weight(int n, int64_t k, float s)
    {
        s *= a.scale;
        if (partial) partial[(int64_t)n * a.K + k] = s;
        else ((T*)a.dw)[n * a.lddw + k] = from_f32<T>(s);
    }
    // lane n's sum b of output n, over the block's eight warps
    __device__ void bias(float b, float* red)
    {
        const int tid = threadIdx.x, lane = tid % 32;
        __syncthreads();
        if (lane < kMaxOutputs) red[tid / 32 * kMaxOutputs + lane] = b;
        __syncthreads();
        if (tid >= a.N) return;
        float s = red[tid];
#pragma unroll
        for (int y = 1; y < 8; ++y) s += red[y * kMaxOutputs + tid];
        s *= a.bias_scale;
        if (partial) partial[NK + tid] = s;
        else a.db[tid] = s;
    }
};

// ------------------------------------------------------------ 2-byte types
constexpr int kPitch = 24;   // elements between rows of dZ: ldmatrix's eight rows fall on different banks

template <bool TRANS>
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr)
{
    if constexpr (TRANS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(T lo, T hi)
{
    uint16_t a, b;
    memcpy(&a, &lo, 2);
    memcpy(&b, &hi, 2);
    return (uint32_t)b << 16 | a;
}

// VEC: rows of x and dX are on the 16-byte grid and K is a multiple of eight.  Lane 4 g + q, step j
// of a warp's eight products of each kind: for dW column g of a product is column 8 g + j of x; for
// dX column 2 q + b of a product is 16 q + 2 j + b (j * 8 + 2 q + b where rows go by shared memory).
// Measured, us, products / multiply-adds as in fp32: 65536 x 256 fp16 22 / 22 for 1 output, 24 / 39
// for 8, 30 / 70 for 16.
// TERMS: dZ as one value of the type, or as the sum of two (GELU and SILU, whose slopes it does not
// hold): the products of the second are added first.
template <typename T, bool VEC, int TERMS>
__global__ void __launch_bounds__(256, 2) thin_grad_mma_kernel(const __grid_constant__ Grad a)
{
    pdl_wait();
    __shared__ __align__(16) T dzs[TERMS][kTile * kPitch];
    using Stage = T[8][16][72];                              // a warp's 16 x 64 of dX where rows are off the 16-byte grid
    constexpr size_t kRed = 8 * 8 * 64 * 4;
    __shared__ __align__(16) uint8_t pool[!VEC && sizeof(Stage) > kRed ? sizeof(Stage) : kRed];
    float* const red = reinterpret_cast<float*>(pool);       // the block's sums, once all rows are through
    Stage& stage = *reinterpret_cast<Stage*>(pool);
    const int tid = threadIdx.x, lane = tid % 32, g = lane / 4, q = lane % 4;
    const int cw = tid / 32 % a.cg, rw = tid / 32 / a.cg, step = 8 / a.cg;   // a.cg warps side by side
    const int64_t c0 = ((int64_t)blockIdx.x * a.cg + cw) * 64;
    const int64_t left = a.K - c0;                                           // columns from c0 on
    const DropKey key = drop_key(a.drop);
    const T zero = from_f32<T>(0.f);

    uint32_t wf[8][2];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int col = VEC ? g / 2 * 16 + 2 * j + g % 2 : j * 8 + g;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            T v[2];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int n = 2 * q + 8 * h + b;
                v[b] = a.dx && n < a.N && col < left ? __ldg((const T*)a.w + n * a.ldw + c0 + col) : zero;
            }
            wf[j][h] = pack2(v[0], v[1]);
        }
    }
    float acc[8][4], bsum = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
    uint4* mine[TERMS];
#pragma unroll
    for (int u = 0; u < TERMS; ++u) {
        mine[u] = reinterpret_cast<uint4*>(dzs[u] + tid * kPitch);
        mine[u][0] = mine[u][1] = make_uint4(0, 0, 0, 0);   // outputs past N stay zero
    }

    const T* const xend = (const T*)a.x + (a.M - 1) * a.ldx + a.K;
    // rows s + 2 q, + 1, + 8, + 9 of a tile; element j of a row is step j's
    auto fetch = [&](int t0, int rows, int s, uint4 (&v)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = s + 2 * q + i % 2 + i / 2 * 8;
            const T* p = (const T*)a.x + (t0 + r) * a.ldx + c0;
            v[i] = make_uint4(0, 0, 0, 0);
            if (r < rows && g * 8 < left) {
                if constexpr (VEC) v[i] = ldg_nc_v4(reinterpret_cast<const uint4*>(p) + g);
                else v[i] = load8_shifted<T>(p + g * 8, (int)min((int64_t)8, left - g * 8), (const T*)a.x, xend).w[0];
            }
        }
    };

    const int r0 = blockIdx.y * a.rows, r1 = min(a.M, r0 + a.rows);
    for (int t0 = r0; t0 < r1; t0 += kTile) {
        const int rows = min(kTile, r1 - t0);
        uint4 xn[4];
        if (a.dw) fetch(t0, rows, rw * 16, xn);
        __syncthreads();
        tile_of_dz<T>(a, key, t0, rows, bsum, [&](int h, const float (&f)[8]) {
            if constexpr (TERMS == 2) {
                float hi[8], lo[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) split2<T>(f[i], hi[i], lo[i]);
                mine[0][h] = pack8<T>(hi);
                mine[1][h] = pack8<T>(lo);
            } else {
                mine[0][h] = pack8<T>(f);
            }
        });
        __syncthreads();
        if (left <= 0) continue;
        for (int s = rw * 16; s < rows; s += step * 16) {
            uint4 xv[4];
            if (a.dw) {
#pragma unroll
                for (int i = 0; i < 4; ++i) xv[i] = xn[i];
                fetch(t0, rows, s + step * 16, xn);
            }
            const uint32_t at = (uint32_t)__cvta_generic_to_shared(dzs[0]) + (s * kPitch) * 2;
            constexpr uint32_t kTerm = kTile * kPitch * 2;
            if (a.dx) {
                uint32_t d[TERMS][4];
#pragma unroll
                for (int u = 0; u < TERMS; ++u) ldmatrix4<false>(d[u], at + u * kTerm + (lane % 16 * kPitch + lane / 16 * 8) * 2);
                uint32_t out[2][8];
                if constexpr (!VEC) __syncwarp();   // the last rows have left the stage
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float o[4] = {};
#pragma unroll
                    for (int u = TERMS - 1; u >= 0; --u)
                        few::mma16816<T>(o, d[u][0], d[u][1], d[u][2], d[u][3], wf[j][0], wf[j][1]);
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        out[h][j] = pack2(from_f32<T>(o[2 * h] * a.scale), from_f32<T>(o[2 * h + 1] * a.scale));
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = s + g + 8 * h;
                    T* p = (T*)a.dx + (t0 + r) * a.lddx + c0;
                    if constexpr (VEC) {
                        uint4* v = reinterpret_cast<uint4*>(p + q * 16);
                        if (r < rows && q * 16 < left) v[0] = make_uint4(out[h][0], out[h][1], out[h][2], out[h][3]);
                        if (r < rows && q * 16 + 8 < left) v[1] = make_uint4(out[h][4], out[h][5], out[h][6], out[h][7]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            *reinterpret_cast<uint32_t*>(&stage[tid / 32][g + 8 * h][j * 8 + 2 * q]) = out[h][j];
                    }
                }
                if constexpr (!VEC) {
                    // four rows at a time from shared memory, eight lanes a row: its whole 16-byte words, then the
                    // elements before and behind them
                    __syncwarp();
                    const int lim = (int)min((int64_t)64, left), k = lane % 8;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = i * 4 + lane / 8;
                        if (s + r >= rows) break;
                        const T* from = stage[tid / 32][r];
                        T* p = (T*)a.dx + (t0 + s + r) * a.lddx + c0;
                        const int off = (int)((uintptr_t)p >> 1 & 7), head = off ? 8 - off : 0, e = head + 8 * k;
                        if (e + 8 <= lim) {
                            const uint32_t* w = reinterpret_cast<const uint32_t*>(from) + e / 2;
                            const uint32_t u[5] = {w[0], w[1], w[2], w[3], w[4]};
                            const int sh = (e & 1) * 16;
                            *reinterpret_cast<uint4*>(p + e) =
                                make_uint4(__funnelshift_r(u[0], u[1], sh), __funnelshift_r(u[1], u[2], sh),
                                           __funnelshift_r(u[2], u[3], sh), __funnelshift_r(u[3], u[4], sh));
                        }
                        const int tail = lim > head ? head + (lim - head) / 8 * 8 + k : lim;
                        if (k < min(head, lim)) p[k] = from[k];
                        if (tail < lim) p[tail] = from[tail];
                    }
                }
            }
            if (a.dw) {
                uint32_t d[TERMS][4];
#pragma unroll
                for (int u = 0; u < TERMS; ++u)
                    ldmatrix4<true>(d[u], at + u * kTerm + ((lane % 8 + lane / 16 * 8) * kPitch + lane / 8 % 2 * 8) * 2);
                const uint32_t* x0 = &xv[0].x;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t pick = j % 2 ? 0x7632 : 0x5410;
                    const uint32_t b0 = __byte_perm(x0[j / 2], x0[4 + j / 2], pick);
                    const uint32_t b1 = __byte_perm(x0[8 + j / 2], x0[12 + j / 2], pick);
#pragma unroll
                    for (int u = TERMS - 1; u >= 0; --u)
                        few::mma16816<T>(acc[j], d[u][0], d[u][1], d[u][2], d[u][3], b0, b1);
                }
            }
        }
    }

    Sums<T> sums(a);
    if (a.dw) {
        // outputs 0..7, then 8..15: a row warp's sums side by side, added by one thread each
        const int width = a.cg * 64;
        const int64_t b0 = (int64_t)blockIdx.x * width;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (h * 8 >= a.N) break;
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int b = 0; b < 2; ++b)
                    red[(rw * 8 + g) * width + cw * 64 + 8 * (2 * q + b) + j] = acc[j][2 * h + b];
            __syncthreads();
            for (int i = tid; i < 8 * width; i += 256) {
                const int n = h * 8 + i / width;
                const int64_t k = b0 + i % width;
                if (n >= a.N || k >= a.K) continue;
                float s = red[i];
                for (int y = 1; y < step; ++y) s += red[y * 8 * width + i];
                sums.weight(n, k, s);
            }
        }
    }
    if (a.db && blockIdx.x == 0) sums.bias(bsum, red);
}

// -------------------------------------------------------------------- fp32
// C consecutive floats, the address on their 8- or 16-byte grid.
template <int C>
__device__ __forceinline__ void load_run(const float* p, float (&v)[C])
{
    if constexpr (C == 2) {
        const float2 u = __ldg(reinterpret_cast<const float2*>(p));
        v[0] = u.x;
        v[1] = u.y;
    } else {
#pragma unroll
        for (int i = 0; i < C; i += 4) {
            const float4 u = u4_as_f4(ldg_nc_v4(reinterpret_cast<const uint4*>(p + i)));
            v[i] = u.x;
            v[i + 1] = u.y;
            v[i + 2] = u.z;
            v[i + 3] = u.w;
        }
    }
}

template <int C>
__device__ __forceinline__ void store_run(float* p, const float (&v)[C])
{
    if constexpr (C == 2) {
        *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
    } else {
#pragma unroll
        for (int i = 0; i < C; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    }
}

// NT: outputs rounded up; a thread's C columns fall as NT grows, so that W's and dW's
// values are 32 each at most.  VEC: rows of x, W and dX are on the 16-byte grid and K is
// a multiple of C; a thread's columns lie cg apart without it, which keeps a warp's
// accesses on consecutive elements.
template <int NT, int C, bool VEC>
__global__ void __launch_bounds__(256, 2) thin_grad_f32_kernel(const __grid_constant__ Grad a)
{
    pdl_wait();
    constexpr int kAhead = NT == 1 ? 4 : 16 / C;             // rows whose loads are in flight together
    constexpr int kOut = NT < 8 ? NT : 8;                      // outputs whose sums meet at once
    __shared__ __align__(16) float dzs[kTile][NT];
    __shared__ float red[kOut * 256 * C];
    const int tid = threadIdx.x, tx = tid % a.cg, ty = tid / a.cg, step = 256 / a.cg;
    const int64_t c0 = (int64_t)blockIdx.x * a.cg * C;
    const DropKey key = drop_key(a.drop);
    auto at = [&](int c, int x) { return VEC ? x * C + c : c * a.cg + x; };   // thread x's columns within the block
    auto in = [&](int c) { return c0 + at(c, tx) < a.K; };
    auto load = [&](const float* row, float (&v)[C]) {
        if constexpr (VEC) {
            if (in(0)) load_run<C>(row + c0 + at(0, tx), v);
        } else {
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (in(c)) v[c] = __ldg(row + c0 + at(c, tx));
        }
    };

    float wv[NT][C], acc[NT][C], bsum = 0.f;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int c = 0; c < C; ++c) wv[n][c] = acc[n][c] = 0.f;
        if (a.dx && n < a.N) load((const float*)a.w + n * a.ldw, wv[n]);
    }

    const int r0 = blockIdx.y * a.rows, r1 = min(a.M, r0 + a.rows);
    for (int t0 = r0; t0 < r1; t0 += kTile) {
        const int rows = min(kTile, r1 - t0);
        __syncthreads();
        tile_of_dz<float>(a, key, t0, rows, bsum, [&](int h, const float (&f)[8]) {
#pragma unroll
            for (int i = 0; i < (NT < 8 ? NT : 8); ++i) dzs[tid][h * 8 + i] = f[i];
        });
        __syncthreads();
        for (int r = ty; r < rows; r += step * kAhead) {
            float xv[kAhead][C] = {};
            if (a.dw)
#pragma unroll
                for (int k = 0; k < kAhead; ++k)
                    if (r + k * step < rows) load((const float*)a.x + (t0 + r + k * step) * a.ldx, xv[k]);
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int rr = r + k * step;
                if (rr >= rows) break;
                float d[NT];
                if constexpr (NT % 4 == 0) {
#pragma unroll
                    for (int n = 0; n < NT; n += 4) {
                        const float4 v = *reinterpret_cast<const float4*>(&dzs[rr][n]);
                        d[n] = v.x;
                        d[n + 1] = v.y;
                        d[n + 2] = v.z;
                        d[n + 3] = v.w;
                    }
                } else {
#pragma unroll
                    for (int n = 0; n < NT; ++n) d[n] = dzs[rr][n];
                }
                if (a.dw)
#pragma unroll
                    for (int c = 0; c < C; ++c)
#pragma unroll
                        for (int n = 0; n < NT; ++n) acc[n][c] = fmaf(d[n], xv[k][c], acc[n][c]);
                if (!a.dx) continue;
                float* out = (float*)a.dx + (t0 + rr) * a.lddx + c0;
                float o[C];
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    o[c] = d[0] * wv[0][c];
#pragma unroll
                    for (int n = 1; n < NT; ++n) o[c] = fmaf(d[n], wv[n][c], o[c]);
                }
                if constexpr (VEC) {
                    if (in(0)) store_run<C>(out + at(0, tx), o);
                } else {
#pragma unroll
                    for (int c = 0; c < C; ++c)
                        if (in(c)) out[at(c, tx)] = o[c];
                }
            }
        }
    }

    Sums<float> sums(a);
    if (a.dw) {
        const int width = a.cg * C;
#pragma unroll
        for (int h = 0; h < NT / kOut; ++h) {
            if (h * kOut >= a.N) break;
            __syncthreads();
#pragma unroll
            for (int n = 0; n < kOut; ++n)
#pragma unroll
                for (int c = 0; c < C; ++c) red[((ty * kOut + n) * C + c) * a.cg + tx] = acc[h * kOut + n][c];
            __syncthreads();
            for (int i = tid; i < kOut * width; i += 256) {
                const int n = h * kOut + i / width, u = i % width;
                const int64_t k = c0 + at(u / a.cg, u % a.cg);
                if (n >= a.N || k >= a.K) continue;
                float s = red[i];
                for (int y = 1; y < step; ++y) s += red[y * kOut * width + i];
                sums.weight(n, k, s);
            }
        }
    }
    if (a.db && blockIdx.x == 0) sums.bias(bsum, red);
}

// dW and db from the chunks' sums: of columns [first, end) of the N * K + N, 1024 / Y a block, Y
// threads a sum.
template <typename T, int Y>
__global__ void __launch_bounds__(1024)
thin_sum_kernel(const float* __restrict__ partial, int chunks, int N, int K, int64_t first, int64_t end,
                T* __restrict__ dw, int64_t lddw, float* __restrict__ db)
{
    pdl_wait();
    constexpr int X = 1024 / Y;
    __shared__ float red[Y][X + 1];
    const int tx = threadIdx.x % X, ty = threadIdx.x / X;
    const int64_t NK = (int64_t)N * K, i = first + (int64_t)blockIdx.x * X + tx;
    float s = 0.f;
    if (i < end)
#pragma unroll 8
        for (int r = ty; r < chunks; r += Y) s += partial[r * (NK + N) + i];
    red[ty][tx] = s;
    __syncthreads();
    if (ty || i >= end) return;
#pragma unroll
    for (int y = 1; y < Y; ++y) s += red[y][tx];
    if (i >= NK) db[i - NK] = s;
    else dw[i / K * lddw + i % K] = from_f32<T>(s);
}

// The split: units of columns (a thread's, or a warp's 64), side by side in a block; chunks of rows
// for two blocks an SM, of four rows a thread or more.  A function of the sizes and the type alone.
struct Shape {
    int cg, blocks_x, chunks, rows;
};

inline int columns(int N) { return N <= 4 ? 8 : N <= 8 ? 4 : 2; }   // a thread's, fp32

inline Shape shape(dlrm_dtype dt, int M, int N, int K)
{
    const bool f32 = dt == DLRM_F32;
    const int unit = f32 ? columns(N) : 64, most_cg = f32 ? 64 : 8;
    const int units = (int)(((int64_t)K + unit - 1) / unit);
    Shape s = {most_cg, 0, 1, M};
    // as wide as leaves no more than an eighth of the columns idle, fp32 not under a warp's 256 bytes
    while (s.cg > (f32 ? 8 : 1) && ((int64_t)units + s.cg - 1) / s.cg * s.cg * 8 > (int64_t)units * 9) s.cg /= 2;
    s.blocks_x = (units + s.cg - 1) / s.cg;
    const int least = f32 ? 4 * 256 / s.cg : 16 * 8 / s.cg;   // rows
    int64_t chunks = (int64_t)num_sms() * 2 / s.blocks_x, most = ((int64_t)M + least - 1) / least;
    if (chunks > most) chunks = most;
    if (chunks < 1) chunks = 1;
    s.rows = (int)((M + chunks - 1) / chunks);
    if (s.rows < M) s.rows = (s.rows + 15) / 16 * 16;
    s.chunks = (int)(((int64_t)M + s.rows - 1) / s.rows);
    return s;
}

inline size_t workspace_bytes(dlrm_dtype dt, int M, int N, int K)
{
    const Shape s = shape(dt, M, N, K);
    return s.chunks > 1 ? dlrm_ws_align((size_t)s.chunks * ((size_t)N * K + N) * 4) : 0;
}

// a.cg, a.rows and a.partial are set here.
template <typename T>
dlrm_status run(dlrm_dtype dt, Grad a, float* ws, cudaStream_t st)
{
    const Shape s = shape(dt, a.M, a.N, a.K);
    a.cg = s.cg;
    a.rows = s.rows;
    a.partial = s.chunks > 1 ? ws : nullptr;
    const dim3 grid(a.dx || a.dw ? s.blocks_x : 1, s.chunks);
    const int es = sizeof(T);
    const bool vec = (!a.dw || rows_aligned16(a.x, a.ldx, a.M, es)) && (!a.dx || rows_aligned16(a.dx, a.lddx, a.M, es));
    dlrm_status r;
    if constexpr (std::is_same_v<T, float>) {
        const bool v = vec && a.K % columns(a.N) == 0 && (!a.dx || rows_aligned16(a.w, a.ldw, a.N, es));
        auto go = [&](auto n) {
            constexpr int NT = decltype(n)::value, C = NT <= 4 ? 8 : NT <= 8 ? 4 : 2;
            auto kern = v ? thin_grad_f32_kernel<NT, C, true> : thin_grad_f32_kernel<NT, C, false>;
            return check_launch_pdl(launch_pdl(kern, grid, dim3(256), 0, st, a), "thin_grad_f32_kernel");
        };
        r = a.N == 1   ? go(std::integral_constant<int, 1>{})
            : a.N <= 4 ? go(std::integral_constant<int, 4>{})
            : a.N <= 8 ? go(std::integral_constant<int, 8>{})
                       : go(std::integral_constant<int, 16>{});
    } else {
        const bool v = vec && a.K % 8 == 0, two = a.act == DLRM_ACT_GELU || a.act == DLRM_ACT_SILU;
        auto kern = two ? (v ? thin_grad_mma_kernel<T, true, 2> : thin_grad_mma_kernel<T, false, 2>)
                        : (v ? thin_grad_mma_kernel<T, true, 1> : thin_grad_mma_kernel<T, false, 1>);
        r = check_launch_pdl(launch_pdl(kern, grid, dim3(256), 0, st, a), "thin_grad_mma_kernel");
    }
    if (r != DLRM_OK || s.chunks == 1 || !(a.dw || a.db)) return r;
    const int64_t NK = (int64_t)a.N * a.K, first = a.dw ? 0 : NK, end = a.db ? NK + a.N : NK;
    auto sum = [&](auto y) {
        constexpr int Y = decltype(y)::value;
        return check_launch_pdl(launch_pdl(thin_sum_kernel<T, Y>, dim3((unsigned)((end - first + 1024 / Y - 1) / (1024 / Y))),
                                           dim3(1024), 0, st, (const float*)a.partial, s.chunks, a.N, a.K, first, end,
                                           (T*)a.dw, a.lddw, a.db),
                                "thin_sum_kernel");
    };
    return s.chunks <= 8 ? sum(std::integral_constant<int, 4>{}) : sum(std::integral_constant<int, 32>{});
}

}  // namespace thin
}  // namespace dlrm
