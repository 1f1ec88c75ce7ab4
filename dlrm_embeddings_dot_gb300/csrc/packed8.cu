// packed8.cu -- matrices to 8 bits and back: 8-bit floats with a power of two for
// every 32 columns, so that scaling is exact and the only rounding is the one to four bits.
// Bound by memory.  A lane has eight columns, four lanes a block of 32, whose largest
// size they find by two shuffles.
#include "packed8.cuh"
#include "dlrm_block.h"

namespace dlrm {
namespace {

constexpr int kThreads8 = 256;

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads8)
pack8_kernel(const T* __restrict__ x, int64_t ldx, int M, int N, uint8_t* __restrict__ q, int64_t ldq,
             uint8_t* __restrict__ exps)
{
    pdl_wait();
    const int64_t groups = ((int64_t)N + kBlock8 - 1) / kBlock8 * 4, runs = groups * M;   // four a block, some past the row's end
    const int64_t stride = (int64_t)gridDim.x * kThreads8;
    const uint32_t quad = 0xfu << (threadIdx.x % kWarp & ~3);
    int64_t i = (int64_t)blockIdx.x * kThreads8 + threadIdx.x;
    int64_t row = i / groups, g = i - row * groups;
    const int64_t drow = stride / groups, dg = stride - drow * groups;
    while (i < runs) {   // a quad's lanes leave together: runs and stride are multiples of four
        const int64_t col = g * 8;
        const int n = (int)min((int64_t)8, N - col);   // 0 or less: past the row's end
        float f[8] = {};
        if (n > 0) widen8<T>(load8<T, VEC>(x + row * ldx + col, n), f);
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t b = __float_as_uint(f[j]) & 0x7fffffffu;
            if (b >= 0x7f800000u) f[j] = __uint_as_float(0x7fc00000u);
            else top = max(top, b);
        }
        top = max(top, __shfl_xor_sync(quad, top, 1));
        top = max(top, __shfl_xor_sync(quad, top, 2));
        // top = 1.m 2^(E - 127) is at most 448 2^(e - 127) from e = E - 8 on, or E - 7 where 1.m > 1.75
        const int e = max(0, (int)(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u));
        const float up = __uint_as_float((uint32_t)(254 - e) << 23);   // 2^(127 - e)
        if (n > 0) {
            uint16_t h[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h[j]) : "f"(f[2 * j + 1] * up), "f"(f[2 * j] * up));
            uint8_t* p = q + row * ldq + col;
            if constexpr (VEC) {
                uint2 v;
                memcpy(&v, h, 8);
                *reinterpret_cast<uint2*>(p) = v;
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j < n) p[j] = (uint8_t)(h[j / 2] >> 8 * (j % 2));
            }
        }
        if (g % 4 == 0) exps[row * (groups / 4) + g / 4] = (uint8_t)e;
        i += stride;
        row += drow;
        g += dg;
        if (g >= groups) {
            g -= groups;
            ++row;
        }
    }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads8)
unpack8_kernel(const __grid_constant__ Packed8 m, int M, int N, T* __restrict__ y, int64_t ldy)
{
    pdl_wait();
    const int64_t groups = (N - 1) / 8 + 1, runs = groups * M;
    const int64_t stride = (int64_t)gridDim.x * kThreads8;
    int64_t i = (int64_t)blockIdx.x * kThreads8 + threadIdx.x;
    int64_t row = i / groups, g = i - row * groups;
    const int64_t drow = stride / groups, dg = stride - drow * groups;
    while (i < runs) {
        const int col = (int)g * 8, n = N - col;
        float f[8];
        widen_run8<T>(load_run8<VEC>(m, row, col, n), f);
        store8<T, VEC>(y + row * ldy + col, n, f);
        i += stride;
        row += drow;
        g += dg;
        if (g >= groups) {
            g -= groups;
            ++row;
        }
    }
}

dlrm_status check_sizes8(const char* fn, dlrm_dtype dtype, int M, int N)
{
    if (!dense_dtype_ok(dtype)) return fail(DLRM_ERR_INVALID_ARG, "%s: bad dtype", fn);
    if (M < 0 || N < 1) return fail(DLRM_ERR_INVALID_ARG, "%s: need M >= 0 and N >= 1", fn);
    if (M > kMaxSize || N > kMaxSize) return fail(DLRM_ERR_UNSUPPORTED, "%s: sizes up to %d", fn, kMaxSize);
    return DLRM_OK;
}

inline unsigned blocks_for(int64_t runs)
{
    const int64_t want = (runs + kThreads8 - 1) / kThreads8, most = (int64_t)num_sms() * 8;
    return (unsigned)(want < most ? want : most);
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
        auto kern = vec ? pack8_kernel<T, true> : pack8_kernel<T, false>;
        return check_launch_pdl(launch_pdl(kern, dim3(blocks_for((int64_t)M * blocks8(N) * 4)), dim3(kThreads8), 0,
                                           as_stream(stream), (const T*)d_x, ldx, M, N, d_q, ldq, d_exps),
                                "pack8_kernel");
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
    const Packed8 m = {d_q, ldq, d_exps, blocks8(N)};
    return with_type(dtype, [&](auto t) {
        using T = decltype(t);
        auto kern = vec ? unpack8_kernel<T, true> : unpack8_kernel<T, false>;
        return check_launch_pdl(launch_pdl(kern, dim3(blocks_for((int64_t)M * ((N - 1) / 8 + 1))), dim3(kThreads8), 0,
                                           as_stream(stream), m, M, N, (T*)d_y, ldy),
                                "unpack8_kernel");
    });
}
