// block_norm.cu -- the norms after a block and before the next one, with the block's gate and residual
// scale: argument checks, and the sums of the vectors' gradients.  The kernels are block_norm.cuh's.
#include "block_norm.h"

#include <algorithm>

namespace dlrm {
namespace {

using norms::norm_blocks;
using norms::NormBwd;
using norms::NormFwd;

struct NormSum {
    const float* partial;
    int64_t Np;
    int blocks, N;
    const float *w_post, *b_post, *scale;
    float *gw_post, *gb_post, *gscale, *gw_pre, *gb_pre;
};

// The vectors' gradients: COLS columns a block, 1024 / COLS threads a column; blockIdx.y 0 the side of the
// norm after the block, 1 that of the norm before the next.  Eight columns are a sector of each block's
// sums; 32 are four, where there are columns for as many blocks (us, 8 / 32: 771 columns 4.7 / 5.2, 8192 18 / 7).
template <int COLS>
__global__ void __launch_bounds__(1024) block_norm_sum_kernel(const __grid_constant__ NormSum a)
{
    constexpr int kRows = 1024 / COLS, kEach = kWarp / COLS;   // threads a column; of them in a warp
    pdl_wait();
    __shared__ float red[2][kRows / kEach][COLS];
    const int tx = threadIdx.x % COLS, ty = threadIdx.x / COLS, n = blockIdx.x * COLS + tx;
    const bool pre = blockIdx.y == 1;
    if (pre ? !a.gw_pre && !a.gb_pre : !a.gw_post && !a.gb_post && !a.gscale) return;
    float s = 0.f, t = 0.f;
    if (n < a.N) {
        const float* p = a.partial + (pre ? 2 * a.Np : 0) + n;
#pragma unroll 4
        for (int b = ty; b < a.blocks; b += kRows) {
            s += p[(int64_t)b * 4 * a.Np];
            t += p[(int64_t)b * 4 * a.Np + a.Np];
        }
    }
#pragma unroll
    for (int m = 16; m >= COLS; m /= 2) {   // a warp's rows
        s += __shfl_xor_sync(~0u, s, m);
        t += __shfl_xor_sync(~0u, t, m);
    }
    if (ty % kEach == 0) {
        red[0][ty / kEach][tx] = s;
        red[1][ty / kEach][tx] = t;
    }
    __syncthreads();
    if (ty || n >= a.N) return;
#pragma unroll
    for (int y = 1; y < kRows / kEach; ++y) {
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

// Checks fp32 vectors of N elements, each of which may be NULL; *vec (may be NULL): whether all start on 16-byte boundaries.
dlrm_status check_vectors(const char* fn, std::initializer_list<const void*> v, bool* vec)
{
    for (const void* p : v) {
        if (reinterpret_cast<uintptr_t>(p) & 3u)
            return fail(DLRM_ERR_INVALID_ARG, "%s: a vector is not aligned to its element size", fn);
        if (vec) *vec = *vec && aligned16(p);
    }
    return DLRM_OK;
}

// The rows at the ends of matrices of N columns or more whose neighbours' bytes may be fewer than 16.
int end_rows(int N, int es) { return 16 / (N * es) + 1; }

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
                       d_scale, d_w_pre, d_b_pre, M, N, end_rows(N, es), norm == DLRM_NORM_LAYER, (int)gate_act, (float)eps,
                       (float)(1.0 / N), d_r, d_h, ldr, ldh, (float4*)d_stats};
    return with_type(dtype, [&](auto t) {
        using T = decltype(t);
        return norms::forward<T>(a, vec, as_stream(stream));
    });
}

extern "C" size_t dlrm_block_norm_bwd_workspace_size(int M, int N)
{
    if (M < 1 || N < 1 || M > kMaxSize || N > DLRM_BLOCK_MAX_WIDTH) return 0;
    int most = norm_blocks(M, N, norms::bwd_warps(true, true, true));
    if (norms::on_grid(N % 8 == 0, N))   // the rows may be: whichever norms are asked for, on the grid or off it
        for (const bool post : {false, true})
            most = std::max(most, norm_blocks(M, N, norms::bwd_warps(post, !post, true)));
    return dlrm_ws_align((size_t)most * 4 * ((N + 7) / 8 * 8) * 4);
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
    bool vec = N % 8 == 0;
    float* const grads[5] = {d_grad_w_post, d_grad_b_post, d_grad_scale, d_grad_w_pre, d_grad_b_pre};
    if ((s = check_vectors(fn, {d_w_post, d_b_post, d_scale, d_w_pre}, &vec)) != DLRM_OK) return s;
    if ((s = check_vectors(fn, {grads[0], grads[1], grads[2], grads[3], grads[4]}, nullptr)) != DLRM_OK) return s;
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
                       (const float4*)d_stats, d_w_post, d_b_post, d_scale, d_w_pre, M, N, end_rows(N, es),
                       norm == DLRM_NORM_LAYER,
                       (int)gate_act, (float)(1.0 / N), d_grad_y, d_grad_gate, d_grad_residual, ldgy, ldgg, ldgres,
                       sums ? (float*)d_workspace : nullptr, Np};
    s = with_type(dtype, [&](auto t) {
        using T = decltype(t);
        return norms::backward<T>(a, vec, st);
    });
    if (s != DLRM_OK || !sums) return s;
    const int blocks = norm_blocks(M, N, norms::bwd_warps(d_y, d_grad_h, norms::on_grid(vec, N)));
    const NormSum q = {a.partial, Np, blocks, N, d_w_post, d_b_post, d_scale,
                       d_grad_w_post, d_grad_b_post, d_grad_scale, d_grad_w_pre, d_grad_b_pre};
    const int cols = N > 1024 ? 32 : 8;
    return check_launch_pdl(launch_pdl(cols == 32 ? block_norm_sum_kernel<32> : block_norm_sum_kernel<8>,
                                       dim3((N + cols - 1) / cols, 2), dim3(1024), 0, st, q),
                            "block_norm_sum_kernel");
}
