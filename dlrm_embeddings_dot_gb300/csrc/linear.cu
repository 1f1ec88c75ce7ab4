// linear.cu -- the dense layer and its gradient: argument checks, workspaces,
// and the kernels around the products.
//
//   forward   z = x W^T + b;  y = residual + drop(a(z))
//   backward  dZ = a'(z) drop(dY);  dX = dZ W;  dW = dZ^T x;  db = sum dZ
//
// Few rows (few_rows): the forward streams the weights into matrix fragments
// (linear_few_kernel).  Few outputs (few_columns): it streams the rows of x so
// (linear_thin_kernel, and thin_grad.cuh backward).  The other products run on tcgen05 (gemm_tc.cuh), which
// wants 2-byte operands with rows on the 16-byte grid.  pack_kernel lays out
// again what is not like that: misaligned rows, and fp32 as three bf16 planes.
#include "dlrm_block.h"
#include "few_rows.cuh"
#include "gemm_tc.cuh"
#include "packed8.cuh"
#include "row_units.cuh"
#include "thin_grad.cuh"

namespace dlrm {
namespace {

using gemm::Operand;
using gemm::padded;
using gemm::Shape;

// Whether the forward streams the weights (linear_few_kernel) instead of running on
// tcgen05 tiles.  Measured, us, streamed / tiles.  bf16: 1024 x 480 2.6 / 6.0 at 16 rows, 4.0 /
// 6.0 at 64; 4096 x 1024 5.2 / 8.2 at 48 rows; 1024 x 4096 8.9 / 8.9 at 48; 4096 x 4096 10.3 / 14.3 at 32
// rows but 13.0 / 13.1 at 40 and 15 / 13 at 48: there a block's 16 weight rows come with more
// token bytes from L2 than weight bytes.  fp32: 1024 x 480 3.5 / 10.3 at 16 rows, 8.1 / 10.7 at
// 64; 4096 x 1024 13.1 / 19.0 at 32 rows but 20.4 / 19.6 at 48; 2048 x 4096 24.5 / 31.1 and 39.5 /
// 32.0; 4096 x 4096 42 / 54 and 72 / 55.
// So weights of 16 MB and more are streamed for up to 32 rows only.
inline bool few_rows(int M, int N, int K, int es)
{
    return M <= 32 || (M <= few::kMaxTokens && (int64_t)N * K * es < 1 << 24);
}

// Whether the forward streams the rows of x (linear_thin_kernel).  Measured, us,
// streamed / tiles (whose 64 columns are mostly waste): 65536 x 256 fp16 5.6 / 16.8 for 1
// output, 8.4 / 9.9 for 16 (fp32 14 / 71, 40 / 59); 300 x 64 1.8 / 6.1; but 1711 x 1285
// 20.8 / 10.0 (fp32 35.1 / 17.6 for 16): a warp walks K alone, and there too few warps do.
inline bool few_columns(int M, int N, int K) { return N <= 16 && (K <= 512 || M >= 1 << 14); }

// Whether the backward is the one pass of thin_grad.cuh.  Measured, us, one pass / dZ and
// two tiled products, 1 and 16 outputs: 65536 x 256 fp16 22 / 42 and 30 / 38, fp32 30 / 142
// and 53 / 124; 40942 x 1049 fp16 109 / 137 and 125 / 133, fp32 75 / 265 and 156 / 235;
// 65536 x 1024 fp16 63 / 82 and 74 / 75; 1711 x 1285 fp16 12 / 28 and 19 / 24; 300 x 64
// 6.4 / 13 and 9.2 / 13.  Its fragments hold 16 outputs.
inline bool few_outputs(int N) { return N <= thin::kMaxOutputs; }

constexpr int kOneChunk = 1024;   // rows that grad_z_kernel takes as one chunk

// ------------------------------------------------------------------ packing
// Stores eight columns as a 2-byte operand; fp32 as three planes, `two`: as two.
template <typename T>
__device__ __forceinline__ void store_operand8(void* dst, int64_t at, int64_t plane, const float (&f)[8], bool two = false)
{
    if constexpr (std::is_same_v<T, float>) {
        uint32_t hi[8], mid[8];
        float lo[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) split1(f[i], hi[i], mid[i], lo[i]);
        uint4 h, m;
        uint32_t *hw = &h.x, *mw = &m.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            hw[i] = __byte_perm(hi[2 * i], hi[2 * i + 1], 0x7632);
            mw[i] = __byte_perm(mid[2 * i], mid[2 * i + 1], 0x7632);
        }
        bf16* p = (bf16*)dst + at;
        *reinterpret_cast<uint4*>(p) = h;
        *reinterpret_cast<uint4*>(p + plane) = m;
        *reinterpret_cast<uint4*>(p + 2 * plane) = pack8<bf16>(lo);
    } else if (two) {
        float hi[8], lo[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) split2<T>(f[i], hi[i], lo[i]);
        *reinterpret_cast<uint4*>((T*)dst + at) = pack8<T>(hi);
        *reinterpret_cast<uint4*>((T*)dst + at + plane) = pack8<T>(lo);
    } else {
        *reinterpret_cast<uint4*>((T*)dst + at) = pack8<T>(f);
    }
}

struct PackJob {
    const void* src;
    int64_t ld;
    int rows, cols, vec;
    void* dst;          // [planes][rows][padded(cols)]
};

// Up to two matrices laid out as operands, runs of eight columns a thread.
template <typename T>
__global__ void __launch_bounds__(256) pack_kernel(PackJob j0, PackJob j1, Overlap overlap)
{
    pdl_begin(overlap);
    const int64_t n0 = (int64_t)j0.rows * ((j0.cols + 7) / 8), n1 = (int64_t)j1.rows * ((j1.cols + 7) / 8);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n0 + n1; i += (int64_t)gridDim.x * 256) {
        const PackJob& j = i < n0 ? j0 : j1;
        const int64_t k = i < n0 ? i : i - n0;
        const int groups = (j.cols + 7) / 8;
        const int64_t row = k / groups;
        const int col = (int)(k - row * groups) * 8, n = j.cols - col;
        const T* p = (const T*)j.src + row * j.ld + col;
        float f[8];
        if (j.vec && n >= 8) widen8<T>(load8<T, true>(p, 8), f);
        else widen8<T>(load8<T, false>(p, n), f);
        store_operand8<T>(j.dst, k * 8, j.rows * (int64_t)groups * 8, f);
    }
}

template <typename T>
dlrm_status launch_pack(const PackJob& a, const PackJob& b, cudaStream_t st, Overlap overlap = {})
{
    const int64_t runs = (int64_t)a.rows * ((a.cols + 7) / 8) + (int64_t)b.rows * ((b.cols + 7) / 8);
    if (runs == 0) return DLRM_OK;
    const int64_t want = (runs + 255) / 256, most = (int64_t)num_sms() * 8;
    return check_launch_pdl(launch_pdl(pack_kernel<T>, dim3((unsigned)(want < most ? want : most)), dim3(256), 0, st, a, b,
                                       overlap),
                            "pack_kernel");
}

struct Unpack8Job {
    Packed8 src;
    int rows, cols, vec;
    void* dst;          // [rows][padded(cols)], T; for fp32 bf16, which holds every value of 8 bits from exponent 3 on
    int blocks;
};

// The input in 8 bits read back as an operand, and beside it the weights' copy as in pack_kernel: blocks from
// j0.blocks on.
template <typename T>
__global__ void __launch_bounds__(256) unpack_kernel(const __grid_constant__ Unpack8Job j0, const __grid_constant__ PackJob j1,
                                                     Overlap overlap)
{
    using X = std::conditional_t<std::is_same_v<T, float>, bf16, T>;
    pdl_begin(overlap);
    if ((int)blockIdx.x < j0.blocks) {
        const int64_t groups = (j0.cols + 7) / 8, n = groups * j0.rows, stride = (int64_t)j0.blocks * 256;
        const int64_t drow = stride / groups, dg = stride - drow * groups;
        int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, row = i / groups, g = i - row * groups;
        while (i < n) {   // kUnpack runs at a time, whose loads are in flight together
            constexpr int kUnpack = 4;
            Run8 r[kUnpack];
            X* to[kUnpack];
            int live = 0;
#pragma unroll
            for (int k = 0; k < kUnpack; ++k)
                if (i < n) {
                    const int col = (int)g * 8, left = j0.cols - col;
                    r[k] = j0.vec && left >= 8 ? load_run8<true>(j0.src, row, col, 8) : load_run8<false>(j0.src, row, col, left);
                    to[k] = (X*)j0.dst + i * 8;
                    live = k + 1;
                    i += stride;
                    row += drow;
                    g += dg;
                    if (g >= groups) {
                        g -= groups;
                        ++row;
                    }
                }
#pragma unroll
            for (int k = 0; k < kUnpack; ++k) {
                if (k >= live) break;
                float f[8];
                widen_run8<T>(r[k], f);
                *reinterpret_cast<uint4*>(to[k]) = pack8<X>(f);
            }
        }
        return;
    }
    const int64_t n1 = (int64_t)j1.rows * ((j1.cols + 7) / 8), stride = (int64_t)(gridDim.x - j0.blocks) * 256;
    for (int64_t k = (int64_t)(blockIdx.x - j0.blocks) * 256 + threadIdx.x; k < n1; k += stride) {
        const int groups = (j1.cols + 7) / 8;
        const int64_t row = k / groups;
        const int col = (int)(k - row * groups) * 8, n = j1.cols - col;
        const T* p = (const T*)j1.src + row * j1.ld + col;
        float f[8];
        if (j1.vec && n >= 8) widen8<T>(load8<T, true>(p, 8), f);
        else widen8<T>(load8<T, false>(p, n), f);
        store_operand8<T>(j1.dst, k * 8, j1.rows * (int64_t)groups * 8, f);
    }
}

template <typename T>
dlrm_status launch_unpack(Unpack8Job a, const PackJob& b, cudaStream_t st, Overlap overlap)
{
    // (two blocks an SM, so that dZ's run beside them: 65536 x 1024 x 1024 fp16 333 us in all, eight 313)
    const int64_t most = blocks_at_once((const void*)unpack_kernel<T>);
    auto blocks = [&](int64_t runs, int each) {
        const int64_t want = (runs + each - 1) / each;
        return (int)(want < most ? want : most);
    };
    a.blocks = blocks((int64_t)a.rows * ((a.cols + 7) / 8), 1024);
    const int more = blocks((int64_t)b.rows * ((b.cols + 7) / 8), 256);
    if (a.blocks + more == 0) return DLRM_OK;
    return check_launch_pdl(launch_pdl(unpack_kernel<T>, dim3(a.blocks + more), dim3(256), 0, st, a, b, overlap), "unpack_kernel");
}

// A matrix argument as an operand: itself, or its copy at ws of `planes` planes.
Operand operand(const void* p, int64_t ld, int rows, int cols, void* ws, int planes, bool mn)
{
    if (!ws) return {p, ld, 0, 1, mn};
    return {ws, padded(cols), rows * padded(cols), planes, mn};
}

int planes_of(dlrm_dtype dt) { return dt == DLRM_F32 ? 3 : 1; }

// Planes of dZ, held without the dropout's scale (that goes to the products' sums): a'
// of NONE and RELU is 0 or 1, so it is dY's own values and one plane of the type
// holds it.  The other slopes need the digits behind: rounded to one plane the
// gradients' error against 64 bits was 1.4 times that of their own last rounding
// (256 x 512 x 1024 bf16: 2.3e-3, two planes 1.7e-3), and fp16 lost what dY / (1 - p)
// takes past 65504.
int z_planes(dlrm_dtype dt, dlrm_act act)
{
    return dt == DLRM_F32 ? 3 : act == DLRM_ACT_GELU || act == DLRM_ACT_SILU ? 2 : 1;
}

bool needs_pack(const void* p, int64_t ld, int rows, dlrm_dtype dt)
{
    return dt == DLRM_F32 || !rows_aligned16(p, ld, rows, 2);
}

size_t operand_bytes(int rows, int cols, int planes) { return dlrm_ws_align((size_t)planes * rows * padded(cols) * 2); }

// --------------------------------------------------------------- few rows
// The forward of up to 64 rows: a cluster owns 16 output columns (weight rows),
// its warps share out K, and their partial tiles are added in a fixed order.
template <typename T, int NT, int VEC>
__global__ void __launch_bounds__(256, 2)
linear_few_kernel(const T* __restrict__ x, int64_t ldx, const T* __restrict__ w, int64_t ldw, int M, int N, int K,
                  const __grid_constant__ Epilogue e)
{
    using namespace few;
    pdl_wait();
    constexpr int kWarps = 8;
    __shared__ __align__(16) float red[kWarps * NT * 8 * kPitch];
    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp, g = lane / 4;
    const int S = (int)cluster_size(), rank = (int)cluster_rank();
    const int row0 = (int)(blockIdx.x / S) * kRows;
    const int steps = (K + kStep<T> - 1) / kStep<T>, parts = S * kWarps, part = rank * kWarps + warp;
    const int per = (steps + parts - 1) / parts * kStep<T>;
    {
        const T* wp[1][2];
#pragma unroll
        for (int b = 0; b < 2; ++b) wp[0][b] = w + min(row0 + g + 8 * b, N - 1) * ldw;
        float* mine = red + warp * NT * 8 * kPitch;
        rows_times_tokens<T, 1, NT, VEC>(
            wp, [&](int t) { return x + t * ldx; }, M, part * per, min(K, (part + 1) * per), 0,
            [&](int, int t, int r, float v) { mine[t * kPitch + r] = v; });
    }
    __syncthreads();
    constexpr int kMine = (NT * 8 * kRows + 255) / 256;
    float sum[kMine];
#pragma unroll
    for (int m = 0; m < kMine; ++m) {
        const int i = threadIdx.x + m * 256;
        sum[m] = 0.f;
        if (i < M * kRows)
#pragma unroll
            for (int q = 0; q < kWarps; ++q) sum[m] += red[(q * NT * 8 + i / kRows) * kPitch + i % kRows];
    }
    __syncthreads();
    float* tot = red;    // [token][kRows], over the partial tiles
#pragma unroll
    for (int m = 0; m < kMine; ++m)
        if (threadIdx.x + m * 256 < NT * 8 * kRows) tot[threadIdx.x + m * 256] = sum[m];
    if (S > 1) cluster_sync();
    else __syncthreads();
    const DropKey key = drop_key(e.drop);
    for (int i = threadIdx.x * S + rank; i < M * (kRows / 8); i += 256 * S) {
        const int t = i / 2, col = row0 + i % 2 * 8, n = N - col;
        if (n <= 0) continue;
        float f[8] = {}, b[8];
        for (int q = 0; q < S; ++q) {
            const uint32_t at = cluster_map(tot + t * kRows + i % 2 * 8, q);
#pragma unroll
            for (int c = 0; c < 8; ++c) f[c] += cluster_ld(at + 4 * c);
        }
        bias8(e.bias, col, N, b);
        finish8_any<T>(e, key, t, col, n, f, b);
    }
    if (S > 1) cluster_sync();   // no block leaves while another reads its sums
}

template <typename T>
dlrm_status launch_few(const void* x, int64_t ldx, const void* w, int64_t ldw, int M, int N, int K, const Epilogue& e,
                       cudaStream_t st)
{
    const int row_tiles = (N + few::kRows - 1) / few::kRows, steps = (K + few::kStep<T> - 1) / few::kStep<T>;
    // a cluster splits K further while blocks are few and every warp keeps two steps
    int S = 1;
    while (S < 8 && row_tiles * S < num_sms() && steps >= S * 8 * 4) S *= 2;
    const int gx = few::row_grid(x, ldx, M, sizeof(T)), gw = few::row_grid(w, ldw, N, sizeof(T)), grid = gx < gw ? gx : gw;
    auto go = [&](auto n) {
        constexpr int NT = decltype(n)::value;
        auto kern = grid == 2 ? linear_few_kernel<T, NT, 2> : grid == 1 ? linear_few_kernel<T, NT, 1> : linear_few_kernel<T, NT, 0>;
        return check_launch_pdl(launch_cluster(kern, dim3((unsigned)row_tiles * S), dim3(256), 0, st, S,
                                                    (const T*)x, ldx, (const T*)w, ldw, M, N, K, e),
                                "linear_few_kernel");
    };
    if (M <= 8) return go(std::integral_constant<int, 1>{});
    if (M <= 16) return go(std::integral_constant<int, 2>{});
    if (M <= 32) return go(std::integral_constant<int, 4>{});
    return go(std::integral_constant<int, 8>{});
}

// ------------------------------------------------------------- few columns
// The forward of up to 16 outputs (the logit layer): the rows of x are the stream
// and the weights' rows the tokens.  A warp takes 16 rows of x at a time, the whole
// of K, and 32 lanes finish its 16 x 16 outputs.
template <typename T, int NT, int VEC>
__global__ void __launch_bounds__(256, 2)
linear_thin_kernel(const T* __restrict__ x, int64_t ldx, const T* __restrict__ w, int64_t ldw, int M, int N, int K,
                   const __grid_constant__ Epilogue e)
{
    using namespace few;
    pdl_wait();
    __shared__ float tile[8][kRows][kPitch];
    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp, g = lane / 4;
    const int tiles = (M + kRows - 1) / kRows;
    const DropKey key = drop_key(e.drop);
    for (int i = blockIdx.x * 8 + warp; i < tiles; i += gridDim.x * 8) {
        const int m0 = i * kRows;
        const T* rows[1][2];
#pragma unroll
        for (int b = 0; b < 2; ++b) rows[0][b] = x + min(m0 + g + 8 * b, M - 1) * ldx;
        rows_times_tokens<T, 1, NT, VEC>(rows, [&](int n) { return w + n * ldw; }, N, 0, K, 0,
                                         [&](int, int n, int r, float v) { tile[warp][r][n] = v; });
        __syncwarp();
        const int row = m0 + lane / 2, col = lane % 2 * 8, n = N - col;
        if (row < M && n > 0) {
            float f[8], b[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) f[c] = c < n ? tile[warp][lane / 2][col + c] : 0.f;
            bias8(e.bias, col, N, b);
            finish8_any<T>(e, key, row, col, n, f, b);
        }
        __syncwarp();
    }
}

template <typename T>
dlrm_status launch_thin(const void* x, int64_t ldx, const void* w, int64_t ldw, int M, int N, int K, const Epilogue& e,
                        cudaStream_t st)
{
    const int64_t want = (M + few::kRows * 8 - 1) / (few::kRows * 8), most = (int64_t)num_sms() * 2;
    const int gx = few::row_grid(x, ldx, M, sizeof(T)), gw = few::row_grid(w, ldw, N, sizeof(T)), grid = gx < gw ? gx : gw;
    auto go = [&](auto n) {
        constexpr int NT = decltype(n)::value;
        auto kern = grid == 2 ? linear_thin_kernel<T, NT, 2> : grid == 1 ? linear_thin_kernel<T, NT, 1> : linear_thin_kernel<T, NT, 0>;
        return check_launch_pdl(launch_pdl(kern, dim3((unsigned)(want < most ? want : most)), dim3(256), 0, st, (const T*)x,
                                           ldx, (const T*)w, ldw, M, N, K, e),
                                "linear_thin_kernel");
    };
    return N <= 8 ? go(std::integral_constant<int, 1>{}) : go(std::integral_constant<int, 2>{});
}

// ------------------------------------------------------- gradient of z and b
// dZ = a'(pre) drop(dY) as an operand of the products (dz, may be NULL; two: of two
// planes; pre of type T, or in 8 bits), and column sums of it times scale (partial [gridDim.y][N], may be NULL).  A block covers
// cg * 8 columns and `rows` rows: a thread owns eight columns of every
// (256 / cg)-th row and adds them up in registers, then the block adds its
// threads' sums in shared memory.
template <typename T>
struct PreMatrix {
    const T* p;
    int64_t ld;
    static constexpr bool kShifted = false;
    using Run = Raw8<T>;
    __device__ Run load(int r, int col, int n, bool v, int) const
    {
        const T* q = p + r * ld + col;
        return v ? load8<T, true>(q, 8) : load8<T, false>(q, n);
    }
    static __device__ void slope(float (&f)[8], const Run& r, int act)   // f times a'(the run)
    {
        float z[8];
        widen8<T>(r, z);
        slope8<T>(f, z, act);
    }
};

template <typename T>
struct PreMatrix8 {
    Packed8 m;
    static constexpr bool kShifted = true;    // rows off the grid are read as the words they lie in
    using Run = Run8;
    // RELU asks for the sign alone, which the bytes have without their exponent
    __device__ Run load(int r, int col, int n, bool v, int act) const
    {
        const bool scaled = act != DLRM_ACT_RELU;
        return v ? load_run8<true>(m, r, col, 8, scaled) : load_run8<false>(m, r, col, n, scaled);
    }
    static __device__ void slope(float (&f)[8], const Run& r, int act)
    {
        if (act == DLRM_ACT_RELU) {
            const uint32_t w[2] = {r.q.x, r.q.y};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t b = w[i / 4] >> 8 * (i % 4) & 0xffu;
                if (b - 1u >= 0x7fu && b != 0xffu) f[i] = 0.f;    // 0 or the sign bit, but for a NaN
            }
            return;
        }
        float z[8];
        widen_run8<T>(r, z);
        slope8<T>(f, z, act);
    }
};

template <typename T, typename Pre>
__global__ void __launch_bounds__(256, 3)
grad_z_kernel(const T* __restrict__ dy, int64_t ldg, const Pre pre, int act, int vec,
              Drop drop, float scale, int M, int N, int cg, int rows, int two, void* __restrict__ dz,
              float* __restrict__ partial, Overlap overlap)
{
    pdl_begin(overlap);
    __shared__ float red[256][8 + 1];
    const DropKey key = drop_key(drop);
    const int tx = threadIdx.x % cg, ty = threadIdx.x / cg, step = 256 / cg;
    const int g = blockIdx.x * cg + tx, col = g * 8, n = N - col;
    const int64_t Np = padded(N);
    float sum[8] = {};
    if (n > 0) {
        constexpr int kAhead = 4 / sizeof(T);   // rows whose loads are in flight together
        const int r0 = blockIdx.y * rows + ty, r1 = min(M, (int)(blockIdx.y + 1) * rows);
        const bool v = vec && n >= 8;
        for (int r = r0; r < r1; r += step * kAhead) {
            Raw8<T> a[kAhead];
            typename Pre::Run b[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int rr = r + k * step;
                if (rr < r1) {
                    const T* gp = dy + rr * ldg + col;
                    if (v) {
                        a[k] = load8<T, true>(gp, 8);
                    } else if (Pre::kShifted && n >= 8) {
                        a[k] = load8_shifted<T>(gp, 8, dy, dy + (M - 1) * ldg + N);
                    } else {
                        a[k] = load8<T, false>(gp, n);
                    }
                    if (act != DLRM_ACT_NONE) b[k] = pre.load(rr, col, n, v, act);
                }
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int rr = r + k * step;
                if (rr >= r1) break;
                float f[8];
                widen8<T>(a[k], f);
                if (act != DLRM_ACT_NONE) Pre::slope(f, b[k], act);
                if (drop.thr) drop8(f, drop, key, (uint32_t)rr, (uint32_t)g);
#pragma unroll
                for (int i = 0; i < 8; ++i) sum[i] += f[i];
                if (dz) store_operand8<T>(dz, rr * Np + col, M * Np, f, two);
            }
        }
    }
    if (!partial) return pdl_end(overlap);
#pragma unroll
    for (int i = 0; i < 8; ++i) red[threadIdx.x][i] = sum[i];
    __syncthreads();
    for (int i = threadIdx.x; i < cg * 8; i += 256) {
        float s = 0.f;
        for (int y = 0; y < step; ++y) s += red[y * cg + i / 8][i % 8];
        const int c = blockIdx.x * cg * 8 + i;
        if (c < N) partial[(int64_t)blockIdx.y * N + c] = s * scale;
    }
    pdl_end(overlap);
}

struct GradZ {
    int cg, blocks_x, chunks, rows;
};

// Few rows: one chunk of narrow blocks, whose sums are the bias gradient itself.
// Otherwise chunks of rows for eight blocks an SM, and sum_rows_kernel behind.
GradZ grad_z_shape(int M, int N)
{
    const int groups = (N + 7) / 8;
    GradZ s = {1, 0, 1, M};
    if (M <= kOneChunk) {
        while (s.cg < 32 && s.cg < groups && 256 / (2 * s.cg) * 4 >= M) s.cg *= 2;   // four rows a thread
        s.blocks_x = (groups + s.cg - 1) / s.cg;
        return s;
    }
    while (s.cg < 32 && s.cg < groups) s.cg *= 2;
    s.blocks_x = (groups + s.cg - 1) / s.cg;
    const int step = 256 / s.cg;
    int64_t chunks = (int64_t)num_sms() * 8 / s.blocks_x, most = ((int64_t)M + 4 * step - 1) / (4 * step);
    if (chunks > most) chunks = most;
    if (chunks < 1) chunks = 1;
    s.rows = (int)((M + chunks - 1) / chunks);
    s.chunks = (M + s.rows - 1) / s.rows;
    return s;
}

// out[n] = the sum of partial's rows: 32 columns a block, 32 threads a column.
__global__ void __launch_bounds__(1024)
sum_rows_kernel(const float* __restrict__ partial, int rows, int N, float* __restrict__ out, Overlap overlap)
{
    pdl_begin(overlap);
    __shared__ float red[32][33];
    const int tx = threadIdx.x % 32, ty = threadIdx.x / 32, n = blockIdx.x * 32 + tx;
    float s = 0.f;
    if (n < N)
#pragma unroll 8
        for (int r = ty; r < rows; r += 32) s += partial[(int64_t)r * N + n];
    red[ty][tx] = s;
    __syncthreads();
    if (ty == 0 && n < N) {
#pragma unroll
        for (int y = 1; y < 32; ++y) s += red[y][tx];
        out[n] = s;
    }
    pdl_end(overlap);
}

// ------------------------------------------------------------------- checks
dlrm_status check_sizes(const char* fn, dlrm_dtype dtype, int M, int N, int K, dlrm_act act)
{
    if (!dense_dtype_ok(dtype)) return fail(DLRM_ERR_INVALID_ARG, "%s: bad dtype", fn);
    if (M < 0 || N < 1 || K < 1) return fail(DLRM_ERR_INVALID_ARG, "%s: need M >= 0, N >= 1 and K >= 1", fn);
    if (M > kMaxSize || N > kMaxSize || K > kMaxSize)
        return fail(DLRM_ERR_UNSUPPORTED, "%s: sizes up to %d", fn, kMaxSize);
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

bool sizes_ok(dlrm_dtype dtype, int M, int N, int K)
{
    return dense_dtype_ok(dtype) && M >= 1 && N >= 1 && K >= 1 && M <= kMaxSize && N <= kMaxSize && K <= kMaxSize;
}

// The products as shapes: output rows, output columns, summed index.
Shape fwd_shape(dlrm_dtype dt, int M, int N, int K)
{
    return {M, N, K, dt == DLRM_F32 ? gemm::kMaxPairs : 1, gemm::column_cycles(N, dense_dtype_size(dt), true)};
}

Shape grad_shape(dlrm_dtype dt, dlrm_act act, int M, int N, int K)
{
    return {M, N, K, dt == DLRM_F32 ? gemm::kMaxPairs : z_planes(dt, act),
            gemm::column_cycles(N, dense_dtype_size(dt), false)};
}

// dW's shape where the input comes in 8 bits: one plane holds it, whatever the type.
Shape grad_shape8(dlrm_dtype dt, dlrm_act act, int M, int N, int K)
{
    return {M, N, K, z_planes(dt, act), gemm::column_cycles(N, dense_dtype_size(dt), false)};
}

// The workspaces' pieces, one after another.
struct FwdLayout {
    size_t x, w, partial, total;   // x, w: bytes of the operands' copies (0: used as they are)
};

FwdLayout fwd_layout(const void* x, int64_t ldx, const void* w, int64_t ldw, dlrm_dtype dt, int M, int N, int K)
{
    FwdLayout l = {};
    if (few_rows(M, N, K, dense_dtype_size(dt)) || few_columns(M, N, K)) return l;
    l.x = needs_pack(x, ldx, M, dt) ? operand_bytes(M, K, planes_of(dt)) : 0;
    l.w = needs_pack(w, ldw, N, dt) ? operand_bytes(N, K, planes_of(dt)) : 0;
    l.partial = gemm::partial_bytes(fwd_shape(dt, M, N, K));
    l.total = l.x + l.w + l.partial;
    return l;
}

struct BwdLayout {
    size_t dz, x, w, sums, partial_x, partial_w, total;
};

// The layer's input and pre-activation, of the call's type or in 8 bits (bits8).
struct Kept {
    bool bits8;
    const void *x, *pre;
    int64_t ldx, ldp;
    Packed8 x8, pre8;
};

BwdLayout bwd_layout(const void* dy, int64_t ldg, const Kept& in, const void* w, int64_t ldw, dlrm_dtype dt, int M, int N,
                     int K, dlrm_act act, double p)
{
    BwdLayout l = {};
    if (few_outputs(N)) {
        l.total = l.sums = thin::workspace_bytes(dt, M, N, K);
        return l;
    }
    l.dz = act != DLRM_ACT_NONE || p > 0 || needs_pack(dy, ldg, M, dt) ? operand_bytes(M, N, z_planes(dt, act)) : 0;
    l.x = in.bits8 ? operand_bytes(M, K, 1) : needs_pack(in.x, in.ldx, M, dt) ? operand_bytes(M, K, planes_of(dt)) : 0;
    l.w = needs_pack(w, ldw, N, dt) ? operand_bytes(N, K, planes_of(dt)) : 0;
    const GradZ g = grad_z_shape(M, N);
    l.sums = g.chunks > 1 ? dlrm_ws_align((size_t)g.chunks * N * 4) : 0;
    l.partial_x = gemm::partial_bytes(grad_shape(dt, act, M, K, N));
    l.partial_w = gemm::partial_bytes(in.bits8 ? grad_shape8(dt, act, N, K, M) : grad_shape(dt, act, N, K, M));
    l.total = l.dz + l.x + l.w + l.sums + l.partial_x + l.partial_w;
    return l;
}

// dlrm_linear_bwd, and dlrm_linear_bwd8: the same with the kept tensors in 8 bits.
dlrm_status run_bwd(const char* fn, const void* d_grad_y, int64_t ldg, const Kept& in, const void* d_w, int64_t ldw,
                    dlrm_dtype dtype, int M, int N, int K, dlrm_act act, double p, const uint64_t* d_rng, void* d_grad_x,
                    int64_t lddx, void* d_grad_w, int64_t lddw, float* d_grad_bias, void* d_workspace,
                    size_t workspace_bytes, uint32_t* d_status, void* stream)
{
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
    if (in.bits8) {
        if (act != DLRM_ACT_NONE && (s = check_packed(fn, "d_pre_q", in.pre8.q, in.pre8.ld, in.pre8.exps, M, N)) != DLRM_OK)
            return s;
        if (d_grad_w && (s = check_packed(fn, "d_x_q", in.x8.q, in.x8.ld, in.x8.exps, M, K)) != DLRM_OK) return s;
    } else {
        if (act != DLRM_ACT_NONE && (s = check_matrix(fn, "d_pre", in.pre, in.ldp, M, N, es)) != DLRM_OK) return s;
        if (d_grad_w && (s = check_matrix(fn, "d_x", in.x, in.ldx, M, K, es)) != DLRM_OK) return s;
    }
    if (d_grad_x && (s = check_matrix(fn, "d_w", d_w, ldw, N, K, es)) != DLRM_OK) return s;
    if (d_grad_x && (s = check_matrix(fn, "d_grad_x", d_grad_x, lddx, M, K, es)) != DLRM_OK) return s;
    const BwdLayout l = bwd_layout(d_grad_y, ldg, in, d_w, ldw, dtype, M, N, K, act, p);
    if ((s = check_workspace(fn, d_workspace, workspace_bytes, l.total)) != DLRM_OK) return s;
    // 2-byte types: dZ without the dropout's scale, the sums times it (fp32's planes hold the scaled values)
    const float scale = dtype == DLRM_F32 ? 1.f : drop.scale;
    if (dtype != DLRM_F32) drop.scale = 1.f;
    const int zp = z_planes(dtype, act), planes = planes_of(dtype);
    return with_type(dtype, [&](auto t) -> dlrm_status {
        using T = decltype(t);
        const float z_scale = zp == 2 ? scale / kFit<T> : scale;
        if (few_outputs(N)) {
            if (!d_grad_x && !d_grad_w && !d_grad_bias) return DLRM_OK;
            thin::Grad a = {d_grad_y, in.pre, in.x, d_w, ldg, in.ldp, in.ldx, ldw, M, N, K, (int)act, drop, z_scale, scale};
            a.x8 = in.x8;
            a.pre8 = in.pre8;
            a.dx = d_grad_x;
            a.dw = d_grad_w;
            a.lddx = lddx;
            a.lddw = lddw;
            a.db = d_grad_bias;
            float* const sums = (float*)d_workspace;
            return in.bits8 ? thin::run8(dtype, a, sums, st) : thin::run<T, false>(dtype, a, sums, st);
        }
        const bool bf = dtype != DLRM_F16;
        uint8_t* ws = (uint8_t*)d_workspace;
        void *dz = l.dz ? ws : nullptr, *xs = l.x ? ws + l.dz : nullptr, *wsp = l.w ? ws + l.dz + l.x : nullptr;
        float* sums = (float*)(ws + l.dz + l.x + l.w);
        float* px = (float*)(ws + l.dz + l.x + l.w + l.sums);
        float* pw = (float*)(ws + l.dz + l.x + l.w + l.sums + l.partial_x);
        // the copies and dZ run together, then dX, dW and the sum of the bias gradient
        const bool products = d_grad_x || d_grad_w;
        const GradZ g = grad_z_shape(M, N);
        const bool make_z = (dz && products) || d_grad_bias, sum = d_grad_bias && g.chunks > 1;
        PackJob jx = {}, jw = {};
        Unpack8Job j8 = {};
        if (in.bits8 && d_grad_w) j8 = {in.x8, M, K, rows_aligned8(in.x8.q, in.x8.ld, M), xs};
        else if (xs && d_grad_w) jx = {in.x, in.ldx, M, K, rows_aligned16(in.x, in.ldx, M, es), xs};
        if (wsp && d_grad_x) jw = {d_w, ldw, N, K, rows_aligned16(d_w, ldw, N, es), wsp};
        const bool packs = jx.src || jw.src || j8.dst;
        dlrm_status r = in.bits8 ? launch_unpack<T>(j8, jw, st, {0, make_z}) : launch_pack<T>(jx, jw, st, {0, make_z});
        if (r == DLRM_OK && make_z) {
            auto go = [&](auto pre, bool pre_vec) {
                const int vec = rows_aligned16(d_grad_y, ldg, M, es) && (act == DLRM_ACT_NONE || pre_vec);
                return check_launch_pdl(launch_pdl(grad_z_kernel<T, decltype(pre)>, dim3(g.blocks_x, g.chunks), dim3(256), 0,
                                                   st, (const T*)d_grad_y, ldg, pre, (int)act, vec, drop, scale, M, N, g.cg,
                                                   g.rows, (int)(zp == 2), products ? dz : nullptr,
                                                   d_grad_bias ? (sum ? sums : d_grad_bias) : nullptr, Overlap{packs, 0}),
                                        "grad_z_kernel");
            };
            r = in.bits8 ? go(PreMatrix8<T>{in.pre8}, rows_aligned8(in.pre8.q, in.pre8.ld, M))
                         : go(PreMatrix<T>{(const T*)in.pre, in.ldp}, rows_aligned16(in.pre, in.ldp, M, es));
        }
        Epilogue ex = {}, ew = {};
        ex.scale = ew.scale = z_scale;
        const Shape sx = grad_shape(dtype, act, M, K, N),
                    sw = in.bits8 ? grad_shape8(dtype, act, N, K, M) : grad_shape(dtype, act, N, K, M);
        if (r == DLRM_OK && d_grad_x) {
            ex.out = d_grad_x;
            ex.ldo = lddx;
            ex.vec = epilogue_vec(ex, M, es);
            r = gemm::run<T>(fn, sx, operand(d_grad_y, ldg, M, N, dz, zp, false), operand(d_w, ldw, N, K, wsp, planes, true),
                             bf, ex, px, d_status, st, {0, d_grad_w || sum});
        }
        if (r == DLRM_OK && d_grad_w) {
            ew.out = d_grad_w;
            ew.ldo = lddw;
            ew.vec = epilogue_vec(ew, N, es);
            r = gemm::run<T>(fn, sw, operand(d_grad_y, ldg, M, N, dz, zp, true), operand(in.x, in.ldx, M, K, xs, in.bits8 ? 1 : planes, true),
                             bf, ew, pw, d_status, st, {d_grad_x != nullptr, sum});
        }
        if (r == DLRM_OK && sum)
            r = check_launch_pdl(launch_pdl(sum_rows_kernel, dim3((N + 31) / 32), dim3(1024), 0, st, (const float*)sums,
                                            g.chunks, N, d_grad_bias, Overlap{products, 0}),
                                 "sum_rows_kernel");
        if (r == DLRM_OK && d_grad_x) r = gemm::finish<T>(sx, ex, px, st);
        if (r == DLRM_OK && d_grad_w) r = gemm::finish<T>(sw, ew, pw, st);
        return r;
    });
}

}  // namespace
}  // namespace dlrm

using namespace dlrm;

extern "C" size_t dlrm_linear_fwd_workspace_size(const void* d_x, int64_t ldx, const void* d_w, int64_t ldw,
                                                 dlrm_dtype dtype, int M, int N, int K)
{
    return sizes_ok(dtype, M, N, K) ? fwd_layout(d_x, ldx, d_w, ldw, dtype, M, N, K).total : 0;
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
    Epilogue e = {d_bias, d_residual, ldr, d_pre, ldp, d_y, ldy, act, 0, {}};
    if ((s = make_drop(fn, p, d_rng, &e.drop)) != DLRM_OK) return s;
    if (M == 0) return DLRM_OK;
    const int es = dense_dtype_size(dtype);
    if ((s = check_matrix(fn, "d_x", d_x, ldx, M, K, es)) != DLRM_OK) return s;
    if ((s = check_matrix(fn, "d_w", d_w, ldw, N, K, es)) != DLRM_OK) return s;
    if (d_bias && (s = check_matrix(fn, "d_bias", d_bias, N, 1, N, 4)) != DLRM_OK) return s;
    if (d_residual && (s = check_matrix(fn, "d_residual", d_residual, ldr, M, N, es)) != DLRM_OK) return s;
    if (d_pre && (s = check_matrix(fn, "d_pre", d_pre, ldp, M, N, es)) != DLRM_OK) return s;
    if ((s = check_matrix(fn, "d_y", d_y, ldy, M, N, es)) != DLRM_OK) return s;
    const FwdLayout l = fwd_layout(d_x, ldx, d_w, ldw, dtype, M, N, K);
    if ((s = check_workspace(fn, d_workspace, workspace_bytes, l.total)) != DLRM_OK) return s;
    e.vec = epilogue_vec(e, M, es);
    const cudaStream_t st = as_stream(stream);
    return with_type(dtype, [&](auto t) -> dlrm_status {
        using T = decltype(t);
        if (few_rows(M, N, K, es)) return launch_few<T>(d_x, ldx, d_w, ldw, M, N, K, e, st);
        if (few_columns(M, N, K)) return launch_thin<T>(d_x, ldx, d_w, ldw, M, N, K, e, st);
        uint8_t* ws = (uint8_t*)d_workspace;
        void *xs = l.x ? ws : nullptr, *wsp = l.w ? ws + l.x : nullptr;
        float* partial = (float*)(ws + l.x + l.w);
        PackJob jx = {}, jw = {};
        if (xs) jx = {d_x, ldx, M, K, rows_aligned16(d_x, ldx, M, es), xs};
        if (wsp) jw = {d_w, ldw, N, K, rows_aligned16(d_w, ldw, N, es), wsp};
        const dlrm_status r = launch_pack<T>(jx, jw, st);
        if (r != DLRM_OK) return r;
        const Shape z = fwd_shape(dtype, M, N, K);
        const int planes = planes_of(dtype);
        const dlrm_status q = gemm::run<T>(fn, z, operand(d_x, ldx, M, K, xs, planes, false),
                                           operand(d_w, ldw, N, K, wsp, planes, false), dtype != DLRM_F16, e, partial, d_status, st);
        return q == DLRM_OK ? gemm::finish<T>(z, e, partial, st) : q;
    });
}

extern "C" size_t dlrm_linear_bwd_workspace_size(const void* d_grad_y, int64_t ldg, const void* d_x, int64_t ldx,
                                                 const void* d_w, int64_t ldw, dlrm_dtype dtype, int M, int N, int K,
                                                 dlrm_act act, double p)
{
    if (!sizes_ok(dtype, M, N, K)) return 0;
    Kept in = {};
    in.x = d_x;
    in.ldx = ldx;
    return bwd_layout(d_grad_y, ldg, in, d_w, ldw, dtype, M, N, K, act, p).total;
}

extern "C" dlrm_status dlrm_linear_bwd(const void* d_grad_y, int64_t ldg, const void* d_x, int64_t ldx,
                                       const void* d_w, int64_t ldw, const void* d_pre, int64_t ldp, dlrm_dtype dtype,
                                       int M, int N, int K, dlrm_act act, double p, const uint64_t* d_rng,
                                       void* d_grad_x, int64_t lddx, void* d_grad_w, int64_t lddw, float* d_grad_bias,
                                       void* d_workspace, size_t workspace_bytes, uint32_t* d_status, void* stream)
{
    DLRM_API_RANGE("dlrm_linear_bwd");
    clear_error();
    Kept in = {};
    in.x = d_x;
    in.ldx = ldx;
    in.pre = d_pre;
    in.ldp = ldp;
    return run_bwd("dlrm_linear_bwd", d_grad_y, ldg, in, d_w, ldw, dtype, M, N, K, act, p, d_rng, d_grad_x, lddx, d_grad_w,
                   lddw, d_grad_bias, d_workspace, workspace_bytes, d_status, stream);
}

extern "C" size_t dlrm_linear_bwd8_workspace_size(const void* d_grad_y, int64_t ldg, const void* d_w, int64_t ldw,
                                                  dlrm_dtype dtype, int M, int N, int K, dlrm_act act, double p)
{
    if (!sizes_ok(dtype, M, N, K)) return 0;
    Kept in = {};
    in.bits8 = true;
    return bwd_layout(d_grad_y, ldg, in, d_w, ldw, dtype, M, N, K, act, p).total;
}

extern "C" dlrm_status dlrm_linear_bwd8(const void* d_grad_y, int64_t ldg, const uint8_t* d_x_q, int64_t ldx,
                                        const uint8_t* d_x_exps, const void* d_w, int64_t ldw, const uint8_t* d_pre_q,
                                        int64_t ldp, const uint8_t* d_pre_exps, dlrm_dtype dtype, int M, int N, int K,
                                        dlrm_act act, double p, const uint64_t* d_rng, void* d_grad_x, int64_t lddx,
                                        void* d_grad_w, int64_t lddw, float* d_grad_bias, void* d_workspace,
                                        size_t workspace_bytes, uint32_t* d_status, void* stream)
{
    DLRM_API_RANGE("dlrm_linear_bwd8");
    clear_error();
    Kept in = {};
    in.bits8 = true;
    in.x8 = packed8(d_x_q, ldx, d_x_exps, M, K);
    in.pre8 = packed8(d_pre_q, ldp, d_pre_exps, M, N);
    return run_bwd("dlrm_linear_bwd8", d_grad_y, ldg, in, d_w, ldw, dtype, M, N, K, act, p, d_rng, d_grad_x, lddx, d_grad_w,
                   lddw, d_grad_bias, d_workspace, workspace_bytes, d_status, stream);
}
