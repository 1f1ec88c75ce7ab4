// linear.cu -- the dense layer and its gradient: argument checks, workspaces
// and the launches.
//
//   forward   z = x W^T + b;  y = residual + drop(a(z))
//   backward  dZ = a'(z) drop(dY);  dX = dZ W;  dW = dZ^T x;  db = sum dZ
#include "dense_ops.cuh"

namespace dlrm {
namespace {

// What follows a product: bias, activation, dropout and residual, with the
// pre-activation kept where it is asked for.
struct Epilogue {
    const float* bias;
    const void* res;
    int64_t ldr;
    void* pre;
    int64_t ldp;
    int act;
    Drop drop;
};

constexpr int kTile = 64, kStepK = 16;

// C[m][n] = sum_k A[m * sam + k * sak] * B[n * sbn + k * sbk], then the epilogue.
template <typename T>
__global__ void __launch_bounds__(256)
product_kernel(const T* __restrict__ A, int64_t sam, int64_t sak, const T* __restrict__ B, int64_t sbn, int64_t sbk,
               int M, int N, int K, Epilogue e, T* __restrict__ C, int64_t ldc)
{
    pdl_wait();
    __shared__ float as[kStepK][kTile + 1], bs[kStepK][kTile + 1];
    const int n_tiles = (N + kTile - 1) / kTile;
    const int m0 = blockIdx.x / n_tiles * kTile, n0 = blockIdx.x % n_tiles * kTile;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float acc[4][4] = {};
    for (int k0 = 0; k0 < K; k0 += kStepK) {
        for (int i = threadIdx.x; i < kTile * kStepK; i += 256) {
            const int k = sak == 1 ? i % kStepK : i / kTile, r = sak == 1 ? i / kStepK : i % kTile;
            as[k][r] = m0 + r < M && k0 + k < K ? to_f32(A[(m0 + r) * sam + (k0 + k) * sak]) : 0.f;
        }
        for (int i = threadIdx.x; i < kTile * kStepK; i += 256) {
            const int k = sbk == 1 ? i % kStepK : i / kTile, r = sbk == 1 ? i / kStepK : i % kTile;
            bs[k][r] = n0 + r < N && k0 + k < K ? to_f32(B[(n0 + r) * sbn + (k0 + k) * sbk]) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kStepK; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(as[k][ty * 4 + i], bs[k][tx * 4 + j], acc[i][j]);
        __syncthreads();
    }
    const DropKey key = drop_key(e.drop);
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
            if (m >= M || n >= N) continue;
            const float z = acc[i][j] + (e.bias ? e.bias[n] : 0.f);
            if (e.pre) ((T*)e.pre)[m * e.ldp + n] = from_f32<T>(z);
            float f[8] = {};
            f[n & 7] = act_f(z, e.act);
            if (e.drop.thr) drop8(f, e.drop, key, (uint32_t)m, (uint32_t)n >> 3);
            const float y = f[n & 7] + (e.res ? to_f32(((const T*)e.res)[m * e.ldr + n]) : 0.f);
            C[m * ldc + n] = from_f32<T>(y);
        }
}

// dZ = a'(pre) drop(dY) for a chunk of rows, and that chunk's column sums.
template <typename T>
__global__ void __launch_bounds__(256)
grad_z_kernel(const T* __restrict__ dy, int64_t ldg, const T* __restrict__ pre, int64_t ldp, int act, Drop drop, int M,
              int N, int rows, T* __restrict__ dz, float* __restrict__ partial)
{
    pdl_wait();
    const DropKey key = drop_key(drop);
    const int g = blockIdx.x * 256 + threadIdx.x, col = g * 8, n = N - col;
    if (n <= 0) return;
    float sum[8] = {};
    const int r0 = blockIdx.y * rows, r1 = min(M, r0 + rows);
    for (int r = r0; r < r1; ++r) {
        float f[8], z[8];
        widen8<T>(load8<T, false>(dy + r * ldg + col, n), f);
        if (drop.thr) drop8(f, drop, key, (uint32_t)r, (uint32_t)g);
        if (act != DLRM_ACT_NONE) {
            widen8<T>(load8<T, false>(pre + r * ldp + col, n), z);
            for (int j = 0; j < 8; ++j) f[j] *= act_slope(z[j], act);
        }
        for (int j = 0; j < 8; ++j) sum[j] += f[j];
        store8<T, false>(dz + (int64_t)r * N + col, n, f);
    }
    if (partial)
        for (int j = 0; j < 8; ++j)
            if (j < n) partial[(int64_t)blockIdx.y * N + col + j] = sum[j];
}

__global__ void sum_rows_kernel(const float* __restrict__ partial, int rows, int N, float* __restrict__ out)
{
    pdl_wait();
    const int n = blockIdx.x * blockDim.x + threadIdx.x;
    if (n >= N) return;
    float s = 0.f;
    for (int r = 0; r < rows; ++r) s += partial[(int64_t)r * N + n];
    out[n] = s;
}

template <typename T>
dlrm_status launch_product(const T* A, int64_t sam, int64_t sak, const T* B, int64_t sbn, int64_t sbk, int M, int N,
                           int K, const Epilogue& e, T* C, int64_t ldc, cudaStream_t st)
{
    const int64_t tiles = (int64_t)((M + kTile - 1) / kTile) * ((N + kTile - 1) / kTile);
    if (tiles > INT32_MAX) return fail(DLRM_ERR_UNSUPPORTED, "dense layer: %lld output tiles", (long long)tiles);
    return check_launch_pdl(launch_pdl(product_kernel<T>, dim3((unsigned)tiles), dim3(256), 0, st, A, sam, sak, B, sbn,
                                       sbk, M, N, K, e, C, ldc),
                            "product_kernel");
}

constexpr int kChunkRows = 64;

dlrm_status check_sizes(const char* fn, dlrm_dtype dtype, int M, int N, int K, dlrm_act act)
{
    if (!dense_dtype_ok(dtype)) return fail(DLRM_ERR_INVALID_ARG, "%s: bad dtype", fn);
    if (M < 0 || N < 1 || K < 1) return fail(DLRM_ERR_INVALID_ARG, "%s: need M >= 0, N >= 1 and K >= 1", fn);
    if (act < DLRM_ACT_NONE || act > DLRM_ACT_SILU) return fail(DLRM_ERR_INVALID_ARG, "%s: bad activation", fn);
    return DLRM_OK;
}

dlrm_status check_workspace(const char* fn, const void* ws, size_t bytes, size_t need)
{
    if (need == 0) return DLRM_OK;
    if (bytes < need || !ws) return fail(DLRM_ERR_WORKSPACE, "%s: workspace %zu bytes < %zu", fn, ws ? bytes : 0, need);
    if (reinterpret_cast<uintptr_t>(ws) & 255u)
        return fail(DLRM_ERR_INVALID_ARG, "%s: the workspace must be 256-byte aligned", fn);
    return DLRM_OK;
}

}  // namespace
}  // namespace dlrm

using namespace dlrm;

extern "C" size_t dlrm_linear_fwd_workspace_size(const void* d_x, int64_t ldx, const void* d_w, int64_t ldw,
                                                 dlrm_dtype dtype, int M, int N, int K)
{
    return 0;
}

extern "C" dlrm_status dlrm_linear_fwd(const void* d_x, int64_t ldx, const void* d_w, int64_t ldw, const float* d_bias,
                                       const void* d_residual, int64_t ldr, dlrm_dtype dtype, int M, int N, int K,
                                       dlrm_act act, double p, const uint64_t* d_rng, void* d_y, int64_t ldy,
                                       void* d_pre, int64_t ldp, void* d_workspace, size_t workspace_bytes,
                                       uint32_t* d_status, void* stream)
{
    DLRM_API_RANGE("dlrm_linear_fwd");
    clear_error();
    const char* fn = "dlrm_linear_fwd";
    dlrm_status s = check_sizes(fn, dtype, M, N, K, act);
    if (s != DLRM_OK) return s;
    Epilogue e = {d_bias, d_residual, ldr, d_pre, ldp, act, {}};
    if ((s = make_drop(fn, p, d_rng, &e.drop)) != DLRM_OK) return s;
    if (M == 0) return DLRM_OK;
    const int es = dense_dtype_size(dtype);
    if ((s = check_matrix(fn, "d_x", d_x, ldx, M, K, es)) != DLRM_OK) return s;
    if ((s = check_matrix(fn, "d_w", d_w, ldw, N, K, es)) != DLRM_OK) return s;
    if (d_bias && (s = check_matrix(fn, "d_bias", d_bias, N, 1, N, 4)) != DLRM_OK) return s;
    if (d_residual && (s = check_matrix(fn, "d_residual", d_residual, ldr, M, N, es)) != DLRM_OK) return s;
    if (d_pre && (s = check_matrix(fn, "d_pre", d_pre, ldp, M, N, es)) != DLRM_OK) return s;
    if ((s = check_matrix(fn, "d_y", d_y, ldy, M, N, es)) != DLRM_OK) return s;
    s = check_workspace(fn, d_workspace, workspace_bytes,
                        dlrm_linear_fwd_workspace_size(d_x, ldx, d_w, ldw, dtype, M, N, K));
    if (s != DLRM_OK) return s;
    return with_type(dtype, [&](auto t) {
        using T = decltype(t);
        return launch_product<T>((const T*)d_x, ldx, 1, (const T*)d_w, ldw, 1, M, N, K, e, (T*)d_y, ldy,
                                 as_stream(stream));
    });
}

extern "C" size_t dlrm_linear_bwd_workspace_size(const void* d_grad_y, int64_t ldg, const void* d_x, int64_t ldx,
                                                 const void* d_w, int64_t ldw, dlrm_dtype dtype, int M, int N, int K,
                                                 dlrm_act act, double p)
{
    if (check_sizes("", dtype, M, N, K, act) != DLRM_OK || M == 0) return 0;
    return dlrm_ws_align((size_t)M * N * dense_dtype_size(dtype)) +
           dlrm_ws_align((size_t)((M + kChunkRows - 1) / kChunkRows) * N * 4);
}

extern "C" dlrm_status dlrm_linear_bwd(const void* d_grad_y, int64_t ldg, const void* d_x, int64_t ldx,
                                       const void* d_w, int64_t ldw, const void* d_pre, int64_t ldp, dlrm_dtype dtype,
                                       int M, int N, int K, dlrm_act act, double p, const uint64_t* d_rng,
                                       void* d_grad_x, int64_t lddx, void* d_grad_w, int64_t lddw, float* d_grad_bias,
                                       void* d_workspace, size_t workspace_bytes, uint32_t* d_status, void* stream)
{
    DLRM_API_RANGE("dlrm_linear_bwd");
    clear_error();
    const char* fn = "dlrm_linear_bwd";
    dlrm_status s = check_sizes(fn, dtype, M, N, K, act);
    if (s != DLRM_OK) return s;
    Drop drop;
    if ((s = make_drop(fn, p, d_rng, &drop)) != DLRM_OK) return s;
    const int es = dense_dtype_size(dtype);
    if (d_grad_w && (s = check_matrix(fn, "d_grad_w", d_grad_w, lddw, N, K, es)) != DLRM_OK) return s;
    if (d_grad_bias && (s = check_matrix(fn, "d_grad_bias", d_grad_bias, N, 1, N, 4)) != DLRM_OK) return s;
    cudaStream_t st = as_stream(stream);
    if (M == 0) {
        // no rows: the gradients that sum over them are zero
        cudaError_t ce = cudaSuccess;
        if (d_grad_w)
            ce = cudaMemset2DAsync(d_grad_w, (size_t)(N > 1 ? lddw : K) * es, 0, (size_t)K * es, (size_t)N, st);
        if (ce == cudaSuccess && d_grad_bias) ce = cudaMemsetAsync(d_grad_bias, 0, (size_t)N * 4, st);
        return ce == cudaSuccess ? DLRM_OK : fail(DLRM_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(ce));
    }
    if ((s = check_matrix(fn, "d_grad_y", d_grad_y, ldg, M, N, es)) != DLRM_OK) return s;
    if (act != DLRM_ACT_NONE && (s = check_matrix(fn, "d_pre", d_pre, ldp, M, N, es)) != DLRM_OK) return s;
    if (d_grad_w && (s = check_matrix(fn, "d_x", d_x, ldx, M, K, es)) != DLRM_OK) return s;
    if (d_grad_x && (s = check_matrix(fn, "d_w", d_w, ldw, N, K, es)) != DLRM_OK) return s;
    if (d_grad_x && (s = check_matrix(fn, "d_grad_x", d_grad_x, lddx, M, K, es)) != DLRM_OK) return s;
    s = check_workspace(fn, d_workspace, workspace_bytes,
                        dlrm_linear_bwd_workspace_size(d_grad_y, ldg, d_x, ldx, d_w, ldw, dtype, M, N, K, act, p));
    if (s != DLRM_OK) return s;
    const int chunks = (M + kChunkRows - 1) / kChunkRows;
    return with_type(dtype, [&](auto t) -> dlrm_status {
        using T = decltype(t);
        T* dz = (T*)d_workspace;
        float* partial = (float*)((uint8_t*)d_workspace + dlrm_ws_align((size_t)M * N * sizeof(T)));
        dlrm_status r = check_launch_pdl(
            launch_pdl(grad_z_kernel<T>, dim3(((N + 7) / 8 + 255) / 256, chunks), dim3(256), 0, st, (const T*)d_grad_y,
                       ldg, (const T*)d_pre, ldp, (int)act, drop, M, N, kChunkRows, dz, d_grad_bias ? partial : nullptr),
            "grad_z_kernel");
        if (r == DLRM_OK && d_grad_bias)
            r = check_launch_pdl(launch_pdl(sum_rows_kernel, dim3((N + 255) / 256), dim3(256), 0, st, partial, chunks, N,
                                            d_grad_bias),
                                 "sum_rows_kernel");
        const Epilogue none = {};
        if (r == DLRM_OK && d_grad_x)
            r = launch_product<T>(dz, N, 1, (const T*)d_w, 1, ldw, M, K, N, none, (T*)d_grad_x, lddx, st);
        if (r == DLRM_OK && d_grad_w)
            r = launch_product<T>(dz, 1, N, (const T*)d_x, 1, ldx, N, K, M, none, (T*)d_grad_w, lddw, st);
        return r;
    });
}
