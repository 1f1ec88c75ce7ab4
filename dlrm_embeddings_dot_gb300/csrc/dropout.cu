// dropout.cu -- dropout from the counter-based generator of dense_ops.cuh, with
// an optional residual: y = residual + drop(x).  The backward is the same map
// of the gradient.
//
// Bound by memory: x (and the residual) read once, y written once.  A thread
// takes one run of eight columns (one Philox call) at a time; the runs of all
// rows are one sequence that the grid strides over, the row and the run within
// it stepped without a division.
#include "dense_ops.cuh"

namespace dlrm {
namespace {

constexpr int kDropThreads = 256;
constexpr int kAhead = 2;

template <typename T, bool VEC>
__global__ void __launch_bounds__(kDropThreads)
dropout_kernel(const T* __restrict__ x, int64_t ldx, const T* __restrict__ res, int64_t ldr, int M, int N, Drop drop,
               T* __restrict__ y, int64_t ldy)
{
    pdl_wait();
    const DropKey key = drop_key(drop);
    const int64_t groups = (N - 1) / 8 + 1, runs = groups * M;   // N + 7 may pass 2^31
    const int64_t stride = (int64_t)gridDim.x * kDropThreads;
    int64_t i = (int64_t)blockIdx.x * kDropThreads + threadIdx.x;
    int64_t row = i / groups, g = i - row * groups;
    const int64_t drow = stride / groups, dg = stride - drow * groups;
    // two runs a turn, so that twice the loads are in flight
    auto next = [&] {
        i += stride;
        row += drow;
        g += dg;
        if (g >= groups) {
            g -= groups;
            ++row;
        }
    };
    while (i < runs) {
        Raw8<T> rx[kAhead], rr[kAhead];
        int64_t at[kAhead], gs[kAhead];
        int live = 0;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (i < runs) {
                const int col = (int)g * 8;
                at[k] = row;
                gs[k] = g;
                rx[k] = load8<T, VEC>(x + row * ldx + col, N - col);
                if (res) rr[k] = load8<T, VEC>(res + row * ldr + col, N - col);
                live = k + 1;
                next();
            }
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (k >= live) break;
            const int col = (int)gs[k] * 8;
            float f[8];
            widen8<T>(rx[k], f);
            if (drop.thr) drop8(f, drop, key, (uint32_t)at[k], (uint32_t)gs[k]);
            if (res) {
                float r[8];
                widen8<T>(rr[k], r);
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] += r[j];
            }
            store8<T, VEC>(y + at[k] * ldy + col, N - col, f);
        }
    }
}

dlrm_status run_dropout(const char* fn, const void* x, int64_t ldx, const void* res, int64_t ldr, dlrm_dtype dtype,
                        int M, int N, double p, const uint64_t* rng, void* y, int64_t ldy, void* stream)
{
    clear_error();
    if (!dense_dtype_ok(dtype)) return fail(DLRM_ERR_INVALID_ARG, "%s: bad dtype", fn);
    if (M < 0 || N < 1) return fail(DLRM_ERR_INVALID_ARG, "%s: need M >= 0 and N >= 1", fn);
    Drop drop;
    dlrm_status s = make_drop(fn, p, rng, &drop);
    if (s != DLRM_OK) return s;
    if (M == 0) return DLRM_OK;
    const int es = dense_dtype_size(dtype);
    if ((s = check_matrix(fn, "the input", x, ldx, M, N, es)) != DLRM_OK) return s;
    if (res && (s = check_matrix(fn, "d_residual", res, ldr, M, N, es)) != DLRM_OK) return s;
    if ((s = check_matrix(fn, "the output", y, ldy, M, N, es)) != DLRM_OK) return s;
    const bool vec = N % 8 == 0 && rows_aligned16(x, ldx, M, es) && rows_aligned16(y, ldy, M, es) &&
                     (!res || rows_aligned16(res, ldr, M, es));
    const int64_t runs = (int64_t)((N - 1) / 8 + 1) * M;
    const int64_t want = (runs + kDropThreads - 1) / kDropThreads, most = (int64_t)num_sms() * 8;
    const int blocks = (int)(want < most ? want : most);
    return with_type(dtype, [&](auto t) {
        using T = decltype(t);
        auto kern = vec ? dropout_kernel<T, true> : dropout_kernel<T, false>;
        return check_launch_pdl(launch_pdl(kern, blocks, kDropThreads, 0, as_stream(stream), (const T*)x, ldx,
                                           (const T*)res, ldr, M, N, drop, (T*)y, ldy),
                                "dropout_kernel");
    });
}

}  // namespace
}  // namespace dlrm

using namespace dlrm;

extern "C" dlrm_status dlrm_dropout_fwd(const void* d_x, int64_t ldx, const void* d_residual, int64_t ldr,
                                        dlrm_dtype dtype, int M, int N, double p, const uint64_t* d_rng, void* d_y,
                                        int64_t ldy, void* stream)
{
    DLRM_API_RANGE("dlrm_dropout_fwd");
    return run_dropout("dlrm_dropout_fwd", d_x, ldx, d_residual, ldr, dtype, M, N, p, d_rng, d_y, ldy, stream);
}

extern "C" dlrm_status dlrm_dropout_bwd(const void* d_grad_y, int64_t ldg, dlrm_dtype dtype, int M, int N, double p,
                                        const uint64_t* d_rng, void* d_grad_x, int64_t lddx, void* stream)
{
    DLRM_API_RANGE("dlrm_dropout_bwd");
    return run_dropout("dlrm_dropout_bwd", d_grad_y, ldg, nullptr, 0, dtype, M, N, p, d_rng, d_grad_x, lddx, stream);
}
