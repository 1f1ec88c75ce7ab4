// block_norm.cu -- the norms after a block and before the next one, with the
// block's gate and residual scale:
//
//   u = norm(y) w_post + b_post;  r = residual + scale gate(g) u;  h = norm(r) w_pre + b_pre
//
// and its gradient.  Both are bound by memory: every matrix goes once, a row stays in
// registers between its sums.
//
//   forward    a row by W warps of C runs of eight columns a lane; the statistics are
//              taken in two passes over the registers (mean, then squares about it)
//   backward   a row by W warps of one run a lane, which then holds the vectors' part
//              and the sums over rows of its columns in registers, and the next row's
//              loads are in flight while a row is computed.  Blocks' sums go to `partial`
//              and block_norm_sum_kernel adds them in order
//
// Nothing here depends on which column a lane has, so rows off the 16-byte grid give a
// lane every 32nd column instead of eight in a row: whole sectors a load, whatever the base.
#include "dense_ops.cuh"
#include "dlrm_block.h"

namespace dlrm {
namespace {

// ------------------------------------------------------------- runs of a row
// A lane's run c of a row: columns first .. first + 7, or first, first + 32, ..
template <bool VEC>
__device__ __forceinline__ int run_first(int chunk, int lane)
{
    return chunk * 256 + (VEC ? lane * 8 : lane);
}

template <bool VEC>
__device__ __forceinline__ bool run_has(int first, int i, int N)
{
    return VEC ? first < N : first + 32 * i < N;
}

// The run's columns of a row, 0 past its end.
template <typename T, bool VEC>
__device__ __forceinline__ Raw8<T> load_run(const T* row, int first, int N)
{
    Raw8<T> r;
    if constexpr (VEC) {
        if (first < N) return load8<T, true>(row + first, 8);
#pragma unroll
        for (int i = 0; i < (int)(sizeof(T) / 2); ++i) r.w[i] = make_uint4(0, 0, 0, 0);
    } else {
        T e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = first + 32 * i < N ? __ldg(row + first + 32 * i) : from_f32<T>(0.f);
        memcpy(&r, e, sizeof(r));
    }
    return r;
}

template <typename T, bool VEC>
__device__ __forceinline__ void store_run(T* row, int first, int N, const float (&f)[8])
{
    if constexpr (VEC) {
        if (first < N) store8<T, true>(row + first, 8, f);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (first + 32 * i < N) row[first + 32 * i] = from_f32<T>(f[i]);
    }
}

// The run's part of a vector, `fill` everywhere where there is none.
template <bool VEC>
__device__ __forceinline__ void load_vector(const float* p, int first, int N, float fill, float (&f)[8])
{
    if (!p) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = fill;
    } else if constexpr (VEC) {
        float4 a = make_float4(0, 0, 0, 0), b = a;
        if (first < N) {
            a = __ldg(reinterpret_cast<const float4*>(p + first));
            b = __ldg(reinterpret_cast<const float4*>(p + first) + 1);
        }
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = first + 32 * i < N ? __ldg(p + first + 32 * i) : 0.f;
    }
}

// Sums of V values over the W warps of a row, the same in all of them.  red: two areas that
// take turns, so that one barrier a sum is enough.
template <int W, int V>
__device__ __forceinline__ void row_sum(float (&v)[V], float* red, int& turn, int warp)
{
#pragma unroll
    for (int m = 16; m; m /= 2)
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] += __shfl_xor_sync(~0u, v[i], m);
    if constexpr (W > 1) {
        constexpr int kWarps = W > 8 ? W : 8;
        float* area = red + turn * kWarps * 4;
        turn ^= 1;
        if (threadIdx.x % kWarp == 0)
#pragma unroll
            for (int i = 0; i < V; ++i) area[warp * 4 + i] = v[i];
        if constexpr (W >= 8) __syncthreads();
        else asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / W), "r"(W * 32) : "memory");
        const float* row = area + warp / W * W * 4;
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = row[i];
#pragma unroll
        for (int w = 1; w < W; ++w)
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] += row[w * 4 + i];
    }
}

template <typename T>
__device__ __forceinline__ float gate_f(float g, int act)
{
    if (act == DLRM_GATE_NONE) return g;
    const float s = sigmoid<T>(g);
    return act == DLRM_GATE_SIGMOID ? s : g * s;
}

// gate(g) and gate'(g)
template <typename T>
__device__ __forceinline__ void gate_both(float g, int act, float& v, float& slope)
{
    v = g;
    slope = 1.f;
    if (act == DLRM_GATE_NONE) return;
    const float s = sigmoid<T>(g);
    v = act == DLRM_GATE_SIGMOID ? s : g * s;
    slope = act == DLRM_GATE_SIGMOID ? s * (1.f - s) : s * fmaf(g, 1.f - s, 1.f);
}

// ------------------------------------------------------------------- forward
struct NormFwd {
    const void *y, *gate, *res;
    int64_t ldy, ldg, ldres;
    int gate_cols;                   // 0: no gate
    const float *w_post, *b_post, *scale, *w_pre, *b_pre;
    int M, N, layer, gate_act;
    float eps, inv_n;
    void *r, *h;
    int64_t ldr, ldh;
    float4* stats;
};

// (mean, 1 / sqrt(mean square + eps)) of a row
template <bool VEC, int C, int W>
__device__ __forceinline__ float2 row_stats(const float (&f)[C][8], const int (&first)[C], const NormFwd& a, float* red,
                                            int& turn, int warp)
{
    float mean = 0.f, s[1] = {0.f};
    if (a.layer) {
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) s[0] += f[c][i];
        row_sum<W>(s, red, turn, warp);
        mean = s[0] * a.inv_n;
        s[0] = 0.f;
    }
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float d = run_has<VEC>(first[c], i, a.N) ? f[c][i] - mean : 0.f;
            s[0] = fmaf(d, d, s[0]);
        }
    row_sum<W>(s, red, turn, warp);
    return make_float2(mean, 1.f / sqrtf(fmaf(s[0], a.inv_n, a.eps)));
}

template <typename T, bool VEC, int C, int W>
__global__ void __launch_bounds__(W > 8 ? W * 32 : 256)
block_norm_fwd_kernel(const __grid_constant__ NormFwd a)
{
    constexpr int kWarps = W > 8 ? W : 8, G = kWarps / W;   // G rows of a block at a time
    __shared__ float red[W > 1 ? 2 * kWarps * 4 : 1];
    pdl_wait();
    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
    int turn = 0, first[C];
#pragma unroll
    for (int c = 0; c < C; ++c) first[c] = run_first<VEC>(warp % W + W * c, lane);
    for (int64_t row = (int64_t)blockIdx.x * G + warp / W; row < a.M; row += (int64_t)gridDim.x * G) {
        Raw8<T> ry[C], rg[C], rr[C];
        float g1 = 1.f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (a.y) ry[c] = load_run<T, VEC>((const T*)a.y + row * a.ldy, first[c], a.N);
            if (a.gate_cols > 1) rg[c] = load_run<T, VEC>((const T*)a.gate + row * a.ldg, first[c], a.N);
            if (a.res) rr[c] = load_run<T, VEC>((const T*)a.res + row * a.ldres, first[c], a.N);
        }
        if (a.gate_cols == 1) g1 = gate_f<T>(to_f32(__ldg((const T*)a.gate + row * a.ldg)), a.gate_act);
        float r[C][8];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (a.res) widen8<T>(rr[c], r[c]);
            else
#pragma unroll
                for (int i = 0; i < 8; ++i) r[c][i] = 0.f;
        }
        float4 st = make_float4(0.f, 0.f, 0.f, 0.f);
        if (a.y) {
            float f[C][8];
#pragma unroll
            for (int c = 0; c < C; ++c) widen8<T>(ry[c], f[c]);
            const float2 s = row_stats<VEC, C, W>(f, first, a, red, turn, warp);
            st.x = s.x;
            st.y = s.y;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float w[8], b[8], sc[8], g[8];
                load_vector<VEC>(a.w_post, first[c], a.N, 1.f, w);
                load_vector<VEC>(a.b_post, first[c], a.N, 0.f, b);
                load_vector<VEC>(a.scale, first[c], a.N, 1.f, sc);
                if (a.gate_cols > 1) widen8<T>(rg[c], g);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float u = fmaf((f[c][i] - s.x) * s.y, w[i], b[i]);
                    u *= a.gate_cols > 1 ? gate_f<T>(g[i], a.gate_act) : g1;
                    r[c][i] = fmaf(sc[i], u, r[c][i]);
                }
                store_run<T, VEC>((T*)a.r + row * a.ldr, first[c], a.N, r[c]);
            }
        }
        if (a.h) {
            if (a.y)   // columns past the row's end hold what the vectors' fill made of them
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (!run_has<VEC>(first[c], i, a.N)) r[c][i] = 0.f;
            const float2 s = row_stats<VEC, C, W>(r, first, a, red, turn, warp);
            st.z = s.x;
            st.w = s.y;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float w[8], b[8], o[8];
                load_vector<VEC>(a.w_pre, first[c], a.N, 1.f, w);
                load_vector<VEC>(a.b_pre, first[c], a.N, 0.f, b);
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = fmaf((r[c][i] - s.x) * s.y, w[i], b[i]);
                store_run<T, VEC>((T*)a.h + row * a.ldh, first[c], a.N, o);
            }
        }
        if (a.stats && warp % W == 0 && lane == 0) a.stats[row] = st;
    }
}

template <typename T, bool VEC>
dlrm_status launch_fwd(const NormFwd& a, cudaStream_t st)
{
    auto go = [&](auto c, auto w) {
        constexpr int C = decltype(c)::value, W = decltype(w)::value, kWarps = W > 8 ? W : 8;
        const int64_t want = ((int64_t)a.M + kWarps / W - 1) / (kWarps / W), most = (int64_t)num_sms() * 8;
        return check_launch_pdl(launch_pdl(block_norm_fwd_kernel<T, VEC, C, W>, dim3((unsigned)(want < most ? want : most)),
                                           dim3(kWarps * 32), 0, st, a),
                                "block_norm_fwd_kernel");
    };
    using std::integral_constant;
    constexpr int L = sizeof(T) == 4 ? 2 : 4;   // runs a lane: what three tensors' words leave registers for
    constexpr integral_constant<int, 1> one;
    constexpr integral_constant<int, 2> two;
    constexpr integral_constant<int, L> most;
    if (a.N <= 256) return go(one, one);
    if (a.N <= 512) return go(two, one);
    if (a.N <= 1024) return go(most, integral_constant<int, 4 / L>());
    if (a.N <= 2048) return go(most, integral_constant<int, 8 / L>());
    if (a.N <= 4096) return go(most, integral_constant<int, 16 / L>());
    return go(most, integral_constant<int, 32 / L>());
}

// ------------------------------------------------------------------ backward
struct NormBwd {
    const void *gr, *gh, *y, *gate, *r;
    int64_t ldgr, ldgh, ldy, ldg, ldr;
    int gate_cols;
    const float4* stats;
    const float *w_post, *b_post, *scale, *w_pre;
    int M, N, layer, gate_act;
    float inv_n;
    void *gy, *gg, *gres;
    int64_t ldgy, ldgg, ldgres;
    float* partial;   // [gridDim.x][4][Np]: sums of dr gate norm(y), dr gate, grad_h norm(r), grad_h; or NULL
    int64_t Np;
};

template <typename T>
struct BwdRow {
    Raw8<T> gr, gh, y, gate, r;
    float4 st;
    float g1;
};

template <typename T, bool VEC, bool POST, bool PRE>
__device__ __forceinline__ void load_bwd(BwdRow<T>& q, const NormBwd& a, int64_t row, int first)
{
    if (PRE) {
        q.gh = load_run<T, VEC>((const T*)a.gh + row * a.ldgh, first, a.N);
        q.r = load_run<T, VEC>((const T*)a.r + row * a.ldr, first, a.N);
    }
    if (a.gr) q.gr = load_run<T, VEC>((const T*)a.gr + row * a.ldgr, first, a.N);
    if (POST) {
        q.y = load_run<T, VEC>((const T*)a.y + row * a.ldy, first, a.N);
        if (a.gate_cols > 1) q.gate = load_run<T, VEC>((const T*)a.gate + row * a.ldg, first, a.N);
        q.g1 = a.gate_cols == 1 ? to_f32(__ldg((const T*)a.gate + row * a.ldg)) : 1.f;
    }
    q.st = __ldg(a.stats + row);
}

template <typename T, bool VEC, int W, bool POST, bool PRE>
__global__ void __launch_bounds__(W > 8 ? W * 32 : 256, W > 8 ? 1 : 2)
block_norm_bwd_kernel(const __grid_constant__ NormBwd a)
{
    constexpr int kWarps = W > 8 ? W : 8, G = kWarps / W;
    __shared__ float red[W > 1 ? 2 * kWarps * 4 : 1];
    __shared__ float tile[G > 1 ? 8 * 256 : 1];
    pdl_wait();
    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
    const int first = run_first<VEC>(warp % W, lane), N = a.N;
    int turn = 0;
    // scale w_post, scale b_post, w_pre; 0 past the row's end
    float aw[8], ab[8], wp[8];
    {
        float sc[8];
        load_vector<VEC>(a.w_post, first, N, 1.f, aw);
        load_vector<VEC>(a.b_post, first, N, 0.f, ab);
        load_vector<VEC>(a.scale, first, N, 1.f, sc);
        load_vector<VEC>(a.w_pre, first, N, 1.f, wp);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool in = run_has<VEC>(first, i, N);
            aw[i] = in ? aw[i] * sc[i] : 0.f;
            ab[i] = in ? ab[i] * sc[i] : 0.f;
            wp[i] = in ? wp[i] : 0.f;
        }
    }
    float sum[4][8] = {};
    const int64_t step = (int64_t)gridDim.x * G;
    int64_t row = (int64_t)blockIdx.x * G + warp / W;
    BwdRow<T> q;
    if (row < a.M) load_bwd<T, VEC, POST, PRE>(q, a, row, first);
    for (; row < a.M; row += step) {
        BwdRow<T> next;
        if (row + step < a.M) load_bwd<T, VEC, POST, PRE>(next, a, row + step, first);
        float dr[8];
        if (a.gr) widen8<T>(q.gr, dr);
        else
#pragma unroll
            for (int i = 0; i < 8; ++i) dr[i] = 0.f;
        if (PRE) {
            float d[8], x[8], c[2] = {0.f, 0.f};
            widen8<T>(q.gh, d);
            widen8<T>(q.r, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[i] = (x[i] - q.st.z) * q.st.w;
                sum[2][i] = fmaf(d[i], x[i], sum[2][i]);
                sum[3][i] += d[i];
                d[i] *= wp[i];
                c[0] = fmaf(d[i], x[i], c[0]);
                c[1] += d[i];
            }
            row_sum<W>(c, red, turn, warp);
            c[0] *= a.inv_n;
            c[1] = a.layer ? c[1] * a.inv_n : 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) dr[i] = fmaf(d[i] - c[1] - x[i] * c[0], q.st.w, dr[i]);
        }
        if (a.gres) store_run<T, VEC>((T*)a.gres + row * a.ldgres, first, N, dr);
        if (POST) {
            float x[8], c[3] = {0.f, 0.f, 0.f}, dg[8], g1 = q.g1, slope1 = 1.f;
            widen8<T>(q.y, x);
            if (a.gate_cols > 1) widen8<T>(q.gate, dg);
            else if (a.gate_cols == 1) gate_both<T>(q.g1, a.gate_act, g1, slope1);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[i] = (x[i] - q.st.x) * q.st.y;
                float g = g1, slope = 1.f;
                if (a.gate_cols > 1) gate_both<T>(dg[i], a.gate_act, g, slope);
                const float du = dr[i] * g, su = fmaf(x[i], aw[i], ab[i]);   // su: scale u
                dg[i] = dr[i] * su * slope;
                c[2] = fmaf(dr[i], su, c[2]);
                sum[0][i] = fmaf(du, x[i], sum[0][i]);
                sum[1][i] += du;
                dr[i] = du * aw[i];
                c[0] = fmaf(dr[i], x[i], c[0]);
                c[1] += dr[i];
            }
            row_sum<W>(c, red, turn, warp);
            if (a.gg) {
                if (a.gate_cols > 1) store_run<T, VEC>((T*)a.gg + row * a.ldgg, first, N, dg);
                else if (warp % W == 0 && lane == 0) ((T*)a.gg)[row * a.ldgg] = from_f32<T>(c[2] * slope1);
            }
            if (a.gy) {
                c[0] *= a.inv_n;
                c[1] = a.layer ? c[1] * a.inv_n : 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) dr[i] = (dr[i] - c[1] - x[i] * c[0]) * q.st.y;
                store_run<T, VEC>((T*)a.gy + row * a.ldgy, first, N, dr);
            }
        }
        q = next;
    }
    if (!a.partial) return;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        if (s < 2 ? !POST : !PRE) continue;
        if constexpr (G > 1) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 8; ++i) tile[i * 256 + threadIdx.x] = sum[s][i];
            __syncthreads();
            if (warp < W) {
#pragma unroll
                for (int g = 1; g < G; ++g)
#pragma unroll
                    for (int i = 0; i < 8; ++i) sum[s][i] += tile[i * 256 + g * W * 32 + threadIdx.x];
            }
        }
        if (warp < W) store_run<float, VEC>(a.partial + ((int64_t)blockIdx.x * 4 + s) * a.Np, first, N, sum[s]);
    }
}

struct NormSum {
    const float* partial;
    int64_t Np;
    int blocks, N;
    const float *w_post, *b_post, *scale;
    float *gw_post, *gb_post, *gscale, *gw_pre, *gb_pre;
};

// The vectors' gradients: 32 columns a block, 32 threads a column; blockIdx.y 0 the side of the
// norm after the block, 1 that of the norm before the next.
__global__ void __launch_bounds__(1024) block_norm_sum_kernel(const __grid_constant__ NormSum a)
{
    pdl_wait();
    __shared__ float red[2][32][33];
    const int tx = threadIdx.x % 32, ty = threadIdx.x / 32, n = blockIdx.x * 32 + tx;
    const bool pre = blockIdx.y == 1;
    if (pre ? !a.gw_pre && !a.gb_pre : !a.gw_post && !a.gb_post && !a.gscale) return;
    float s = 0.f, t = 0.f;
    if (n < a.N) {
        const float* p = a.partial + (pre ? 2 * a.Np : 0) + n;
#pragma unroll 4
        for (int b = ty; b < a.blocks; b += 32) {
            s += p[(int64_t)b * 4 * a.Np];
            t += p[(int64_t)b * 4 * a.Np + a.Np];
        }
    }
    red[0][ty][tx] = s;
    red[1][ty][tx] = t;
    __syncthreads();
    if (ty || n >= a.N) return;
#pragma unroll
    for (int y = 1; y < 32; ++y) {
        s += red[0][y][tx];
        t += red[1][y][tx];
    }
    if (pre) {
        if (a.gw_pre) a.gw_pre[n] = s;
        if (a.gb_pre) a.gb_pre[n] = t;
    } else {
        const float scale = a.scale ? a.scale[n] : 1.f;
        if (a.gw_post) a.gw_post[n] = scale * s;
        if (a.gb_post) a.gb_post[n] = scale * t;
        if (a.gscale) a.gscale[n] = fmaf(a.w_post ? a.w_post[n] : 1.f, s, (a.b_post ? a.b_post[n] : 0.f) * t);
    }
}

// Warps of a row, a power of two, and the blocks of the backward.
int bwd_warps(int N)
{
    int w = 1;
    while (w * 256 < N) w *= 2;
    return w;
}

int bwd_blocks(int M, int N)
{
    const int w = bwd_warps(N), rows = w > 8 ? 1 : 8 / w;
    const int64_t want = ((int64_t)M + rows - 1) / rows, most = (int64_t)num_sms() * (w > 8 ? 1 : 2);
    return (int)(want < most ? want : most);
}

template <typename T, bool VEC, bool POST, bool PRE>
dlrm_status launch_bwd(const NormBwd& a, cudaStream_t st)
{
    auto go = [&](auto w) {
        constexpr int W = decltype(w)::value;
        return check_launch_pdl(launch_pdl(block_norm_bwd_kernel<T, VEC, W, POST, PRE>, dim3(bwd_blocks(a.M, a.N)),
                                           dim3(W > 8 ? W * 32 : 256), 0, st, a),
                                "block_norm_bwd_kernel");
    };
    using std::integral_constant;
    switch (bwd_warps(a.N)) {
    case 1: return go(integral_constant<int, 1>());
    case 2: return go(integral_constant<int, 2>());
    case 4: return go(integral_constant<int, 4>());
    case 8: return go(integral_constant<int, 8>());
    case 16: return go(integral_constant<int, 16>());
    default: return go(integral_constant<int, 32>());
    }
}

// ------------------------------------------------------------------- checks
dlrm_status check_norm(const char* fn, dlrm_dtype dtype, int M, int N, int norm, int gate_act)
{
    if (!dense_dtype_ok(dtype)) return fail(DLRM_ERR_INVALID_ARG, "%s: bad dtype", fn);
    if (M < 0 || N < 1) return fail(DLRM_ERR_INVALID_ARG, "%s: need M >= 0 and N >= 1", fn);
    if (M > kMaxSize || N > DLRM_BLOCK_MAX_WIDTH)
        return fail(DLRM_ERR_UNSUPPORTED, "%s: up to %d rows of %d columns", fn, kMaxSize, DLRM_BLOCK_MAX_WIDTH);
    if (norm != DLRM_NORM_RMS && norm != DLRM_NORM_LAYER) return fail(DLRM_ERR_INVALID_ARG, "%s: bad norm", fn);
    if (gate_act < DLRM_GATE_NONE || gate_act > DLRM_GATE_SILU) return fail(DLRM_ERR_INVALID_ARG, "%s: bad gate", fn);
    return DLRM_OK;
}

// Checks fp32 vectors of N elements, each of which may be NULL; *vec: whether all start on 16-byte boundaries.
dlrm_status check_vectors(const char* fn, std::initializer_list<const void*> v, bool* vec)
{
    for (const void* p : v) {
        if (reinterpret_cast<uintptr_t>(p) & 3u)
            return fail(DLRM_ERR_INVALID_ARG, "%s: a vector is not aligned to its element size", fn);
        *vec = *vec && aligned16(p);
    }
    return DLRM_OK;
}

dlrm_status check_gate(const char* fn, const void* gate, int64_t ldg, int gate_cols, int M, int N, int es)
{
    if (gate_cols != 1 && gate_cols != N) return fail(DLRM_ERR_INVALID_ARG, "%s: gate_cols is neither 1 nor N", fn);
    return check_matrix(fn, "d_gate", gate, ldg, M, gate_cols, es);
}

}  // namespace
}  // namespace dlrm

using namespace dlrm;

extern "C" dlrm_status dlrm_block_norm_fwd(const void* d_y, int64_t ldy, const void* d_gate, int64_t ldg, int gate_cols,
                                           const void* d_residual, int64_t ldres, const float* d_w_post,
                                           const float* d_b_post, const float* d_scale, const float* d_w_pre,
                                           const float* d_b_pre, dlrm_dtype dtype, int M, int N, dlrm_norm norm,
                                           dlrm_gate gate_act, double eps, void* d_r, int64_t ldr, void* d_h,
                                           int64_t ldh, float* d_stats, void* stream)
{
    DLRM_API_RANGE("dlrm_block_norm_fwd");
    clear_error();
    const char* fn = "dlrm_block_norm_fwd";
    dlrm_status s = check_norm(fn, dtype, M, N, norm, gate_act);
    if (s != DLRM_OK) return s;
    if (!(eps >= 0.0 && eps <= 3.0e38)) return fail(DLRM_ERR_INVALID_ARG, "%s: eps must be finite and not negative", fn);
    if (M == 0) return DLRM_OK;
    const int es = dense_dtype_size(dtype);
    if (!d_y && (d_r || d_gate || d_w_post || d_b_post || d_scale))
        return fail(DLRM_ERR_INVALID_ARG, "%s: d_r, d_gate, d_w_post, d_b_post and d_scale need d_y", fn);
    if (!d_h && (d_w_pre || d_b_pre)) return fail(DLRM_ERR_INVALID_ARG, "%s: d_w_pre and d_b_pre need d_h", fn);
    if (!d_y && !d_h) return fail(DLRM_ERR_INVALID_ARG, "%s: neither d_y nor d_h", fn);
    bool vec = N % 8 == 0;
    if ((s = check_vectors(fn, {d_w_post, d_b_post, d_scale, d_w_pre, d_b_pre}, &vec)) != DLRM_OK) return s;
    if (d_y && (s = check_matrix(fn, "d_y", d_y, ldy, M, N, es)) != DLRM_OK) return s;
    if (d_gate && (s = check_gate(fn, d_gate, ldg, gate_cols, M, N, es)) != DLRM_OK) return s;
    if ((d_residual || !d_y) && (s = check_matrix(fn, "d_residual", d_residual, ldres, M, N, es)) != DLRM_OK) return s;
    if (d_y && (s = check_matrix(fn, "d_r", d_r, ldr, M, N, es)) != DLRM_OK) return s;
    if (d_h && (s = check_matrix(fn, "d_h", d_h, ldh, M, N, es)) != DLRM_OK) return s;
    if (!aligned16(d_stats)) return fail(DLRM_ERR_INVALID_ARG, "%s: d_stats must be 16-byte aligned", fn);
    const bool wide_gate = d_gate && N > 1 && gate_cols == N;
    vec = vec && (!d_y || (rows_aligned16(d_y, ldy, M, es) && rows_aligned16(d_r, ldr, M, es))) &&
          (!wide_gate || rows_aligned16(d_gate, ldg, M, es)) && (!d_residual || rows_aligned16(d_residual, ldres, M, es)) &&
          (!d_h || rows_aligned16(d_h, ldh, M, es));
    const NormFwd a = {d_y, d_gate, d_residual, ldy, ldg, ldres, !d_gate ? 0 : wide_gate ? N : 1, d_w_post, d_b_post,
                       d_scale, d_w_pre, d_b_pre, M, N, norm == DLRM_NORM_LAYER, (int)gate_act, (float)eps,
                       (float)(1.0 / N), d_r, d_h, ldr, ldh, (float4*)d_stats};
    return with_type(dtype, [&](auto t) {
        using T = decltype(t);
        return vec ? launch_fwd<T, true>(a, as_stream(stream)) : launch_fwd<T, false>(a, as_stream(stream));
    });
}

extern "C" size_t dlrm_block_norm_bwd_workspace_size(int M, int N)
{
    if (M < 1 || N < 1 || M > kMaxSize || N > DLRM_BLOCK_MAX_WIDTH) return 0;
    return dlrm_ws_align((size_t)bwd_blocks(M, N) * 4 * ((N + 7) / 8 * 8) * 4);
}

extern "C" dlrm_status dlrm_block_norm_bwd(
    const void* d_grad_r, int64_t ldgr, const void* d_grad_h, int64_t ldgh, const void* d_y, int64_t ldy,
    const void* d_gate, int64_t ldg, int gate_cols, const void* d_r, int64_t ldr, const float* d_stats,
    const float* d_w_post, const float* d_b_post, const float* d_scale, const float* d_w_pre, dlrm_dtype dtype, int M, int N,
    dlrm_norm norm, dlrm_gate gate_act, void* d_grad_y, int64_t ldgy, void* d_grad_gate, int64_t ldgg,
    void* d_grad_residual, int64_t ldgres, float* d_grad_w_post, float* d_grad_b_post, float* d_grad_scale,
    float* d_grad_w_pre, float* d_grad_b_pre, void* d_workspace, size_t workspace_bytes, void* stream)
{
    DLRM_API_RANGE("dlrm_block_norm_bwd");
    clear_error();
    const char* fn = "dlrm_block_norm_bwd";
    dlrm_status s = check_norm(fn, dtype, M, N, norm, gate_act);
    if (s != DLRM_OK) return s;
    const int es = dense_dtype_size(dtype);
    bool vec = N % 8 == 0, grads_vec = true;
    float* const grads[5] = {d_grad_w_post, d_grad_b_post, d_grad_scale, d_grad_w_pre, d_grad_b_pre};
    if ((s = check_vectors(fn, {d_w_post, d_b_post, d_scale, d_w_pre}, &vec)) != DLRM_OK) return s;
    if ((s = check_vectors(fn, {grads[0], grads[1], grads[2], grads[3], grads[4]}, &grads_vec)) != DLRM_OK) return s;
    const cudaStream_t st = as_stream(stream);
    if (M == 0) {
        for (float* g : grads)   // no rows: the sums over them are zero
            if (g) {
                const cudaError_t ce = cudaMemsetAsync(g, 0, (size_t)N * 4, st);
                if (ce != cudaSuccess) return fail(DLRM_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(ce));
            }
        return DLRM_OK;
    }
    if (!d_grad_h && (!d_grad_r || !d_y))
        return fail(DLRM_ERR_INVALID_ARG, "%s: need d_grad_h, or d_grad_r and d_y", fn);
    if (!d_y && (d_gate || d_w_post || d_b_post || d_scale || d_grad_y || d_grad_gate || d_grad_w_post || d_grad_b_post ||
                 d_grad_scale))
        return fail(DLRM_ERR_INVALID_ARG, "%s: the block's side needs d_y", fn);
    if (!d_grad_h && (d_r || d_w_pre || d_grad_w_pre || d_grad_b_pre))
        return fail(DLRM_ERR_INVALID_ARG, "%s: d_r, d_w_pre, d_grad_w_pre and d_grad_b_pre need d_grad_h", fn);
    if (d_grad_gate && !d_gate) return fail(DLRM_ERR_INVALID_ARG, "%s: d_grad_gate needs d_gate", fn);
    if (d_grad_r && (s = check_matrix(fn, "d_grad_r", d_grad_r, ldgr, M, N, es)) != DLRM_OK) return s;
    if (d_grad_h && (s = check_matrix(fn, "d_grad_h", d_grad_h, ldgh, M, N, es)) != DLRM_OK) return s;
    if (d_grad_h && (s = check_matrix(fn, "d_r", d_r, ldr, M, N, es)) != DLRM_OK) return s;
    if (d_y && (s = check_matrix(fn, "d_y", d_y, ldy, M, N, es)) != DLRM_OK) return s;
    if (d_gate && (s = check_gate(fn, d_gate, ldg, gate_cols, M, N, es)) != DLRM_OK) return s;
    if (!d_stats || !aligned16(d_stats))
        return fail(DLRM_ERR_INVALID_ARG, "%s: d_stats is NULL or not 16-byte aligned", fn);
    if (d_grad_y && (s = check_matrix(fn, "d_grad_y", d_grad_y, ldgy, M, N, es)) != DLRM_OK) return s;
    if (d_grad_gate && (s = check_matrix(fn, "d_grad_gate", d_grad_gate, ldgg, M, gate_cols, es)) != DLRM_OK) return s;
    if (d_grad_residual && (s = check_matrix(fn, "d_grad_residual", d_grad_residual, ldgres, M, N, es)) != DLRM_OK) return s;
    bool sums = false;
    for (float* g : grads) sums = sums || g;
    if (sums) {
        const size_t need = dlrm_block_norm_bwd_workspace_size(M, N);
        if (!d_workspace || workspace_bytes < need)
            return fail(DLRM_ERR_WORKSPACE, "%s: workspace %zu bytes < %zu", fn, d_workspace ? workspace_bytes : 0, need);
        if (reinterpret_cast<uintptr_t>(d_workspace) & 255u)
            return fail(DLRM_ERR_INVALID_ARG, "%s: the workspace must be 256-byte aligned", fn);
    }
    const bool wide_gate = d_gate && N > 1 && gate_cols == N;
    vec = vec && (!d_grad_r || rows_aligned16(d_grad_r, ldgr, M, es)) &&
          (!d_grad_h || (rows_aligned16(d_grad_h, ldgh, M, es) && rows_aligned16(d_r, ldr, M, es))) &&
          (!d_y || rows_aligned16(d_y, ldy, M, es)) && (!wide_gate || rows_aligned16(d_gate, ldg, M, es)) &&
          (!d_grad_y || rows_aligned16(d_grad_y, ldgy, M, es)) &&
          (!wide_gate || !d_grad_gate || rows_aligned16(d_grad_gate, ldgg, M, es)) &&
          (!d_grad_residual || rows_aligned16(d_grad_residual, ldgres, M, es));
    const int64_t Np = (N + 7) / 8 * 8;
    const NormBwd a = {d_grad_r, d_grad_h, d_y, d_gate, d_r, ldgr, ldgh, ldy, ldg, ldr, !d_gate ? 0 : wide_gate ? N : 1,
                       (const float4*)d_stats, d_w_post, d_b_post, d_scale, d_w_pre, M, N, norm == DLRM_NORM_LAYER,
                       (int)gate_act, (float)(1.0 / N), d_grad_y, d_grad_gate, d_grad_residual, ldgy, ldgg, ldgres,
                       sums ? (float*)d_workspace : nullptr, Np};
    s = with_type(dtype, [&](auto t) {
        using T = decltype(t);
        auto go = [&](auto v) {
            constexpr bool VEC = decltype(v)::value;
            return !d_y ? launch_bwd<T, VEC, false, true>(a, st) : d_grad_h ? launch_bwd<T, VEC, true, true>(a, st)
                                                                           : launch_bwd<T, VEC, true, false>(a, st);
        };
        return vec ? go(std::true_type()) : go(std::false_type());
    });
    if (s != DLRM_OK || !sums) return s;
    const NormSum q = {a.partial, Np, bwd_blocks(M, N), N, d_w_post, d_b_post, d_scale,
                       d_grad_w_post, d_grad_b_post, d_grad_scale, d_grad_w_pre, d_grad_b_pre};
    return check_launch_pdl(launch_pdl(block_norm_sum_kernel, dim3((N + 31) / 32, 2), dim3(1024), 0, st, q),
                            "block_norm_sum_kernel");
}
