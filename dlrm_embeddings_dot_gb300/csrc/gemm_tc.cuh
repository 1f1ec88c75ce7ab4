// gemm_tc.cuh -- the dense layer's products on the tcgen05 tensor cores:
// out[M][N] = A B^T with a fused epilogue, A and B each either K-major (K
// contiguous: x and W of the forward, dZ of dX) or MN-major (the output's row
// or column index contiguous: W of dX, dZ and x of dW).
//
// A persistent block per SM walks 128 x BN output tiles (BN = 256, 128 or 64):
//   warp 0      TMA producer: per 64 of K a 128 x 64 tile of A and a BN x 64
//               tile of B, 128-byte swizzle, into an NS-stage ring
//   warp 1      TMEM allocation and MMA issue (M = 128, N = BN, K = 16 steps)
//   warps 2..9  epilogue: TMEM lane quarter q = warp % 4, alternate 32-column
//               slices.  A slice goes through 4 KB of shared memory, so that a
//               lane then holds eight consecutive columns of a row: one Philox
//               call, 16-byte loads and stores, and 64 contiguous bytes of a
//               row for every four lanes
// Two TMEM accumulators let the products of the next tile run under the
// epilogue of this one.
//
// fp32 operands come as three bf16 planes (see split planes in linear.cu); the
// K loop then runs over six plane pairs, the smallest products first.  Few
// output tiles: K is split over blocks, each writing its fp32 partial tile, and
// finish_kernel adds them in order and applies the epilogue.
#pragma once

#include "dense_epilogue.cuh"
#include "tcgen05.cuh"

namespace dlrm {
namespace gemm {

using namespace tc;

constexpr int kBM = 128;            // output rows of a tile
constexpr int kKB = 64;             // K elements of a stage (128-byte rows)
constexpr int kEpiWarps = 8;
constexpr int kThreads = (2 + kEpiWarps) * 32;
constexpr int kMaxStages = 8;
constexpr int kSmemLimit = 232448;  // 227 KB opt-in per block
constexpr int kScratch = kEpiWarps * 32 * 128;
constexpr int kMaxPairs = 6;

struct Args {
    int M, N;
    int kb, last_steps;             // 64-wide blocks of K, and 16-wide steps of the last one
    int pairs;                      // plane pairs: 1, or 6 for fp32
    int splits;                     // parts of K; above 1 the tiles go to `partial`
    int tiles_m, tiles_n, BN, NS;
    uint32_t idesc, tmem_cols;
    float* partial;                 // [splits][M][Np]
    int64_t Np;
    Epilogue e;
    uint32_t* status;
    long long wait_cycles;
};

// Plane pair p of the fp32 products, (A plane << 2) | B plane: hi = 0, mid = 1, lo = 2.
__device__ __forceinline__ int plane_pair(int pairs, int p)
{
    constexpr uint32_t order = 0x2u | 0x8u << 4 | 0x5u << 8 | 0x1u << 12 | 0x4u << 16 | 0x0u << 20;
    return pairs == 1 ? 0 : (int)(order >> (4 * p)) & 15;
}

inline size_t smem_bytes(int BN, int ns)
{
    return 1024 + (size_t)ns * (kBM * 128 + BN * 128) + kScratch + (size_t)(2 * ns + 4) * 8 + 16;
}

// The warp's 32 x 32 slice of the accumulator at taddr to rows of eight columns
// a lane, then fn(pass, row within the slice, f).
template <typename Fn>
__device__ __forceinline__ void transpose_slice(uint32_t taddr, uint8_t* scratch, Fn&& fn)
{
    const int lane = threadIdx.x % kWarp;
    uint32_t v[32];
    tmem_ld_x32(taddr, v);
    tmem_wait_ld(v);
    __syncwarp();   // the previous slice has been read
#pragma unroll
    for (int c = 0; c < 8; ++c)
        *reinterpret_cast<uint4*>(scratch + lane * 128 + ((c ^ (lane & 7)) << 4)) =
            make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
    __syncwarp();
#pragma unroll
    for (int pass = 0; pass < 4; ++pass) {
        const int r = pass * 8 + lane / 4, c = 2 * (lane % 4);
        const float4 lo = *reinterpret_cast<const float4*>(scratch + r * 128 + ((c ^ (r & 7)) << 4));
        const float4 hi = *reinterpret_cast<const float4*>(scratch + r * 128 + (((c + 1) ^ (r & 7)) << 4));
        float f[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        fn(pass, r, f);
    }
}

template <typename T, bool A_MN, bool B_MN>
__global__ void __launch_bounds__(kThreads, 1)
gemm_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
            const __grid_constant__ Args a)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int BN = a.BN, NS = a.NS;
    constexpr int a_bytes = kBM * 128;
    const int stage_bytes = a_bytes + BN * 128;
    uint8_t* scratch = smem + (size_t)NS * stage_bytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(scratch + kScratch);
    uint64_t* empty = full + NS;
    uint64_t* tfull = empty + NS;
    uint64_t* tempty = tfull + 2;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(tempty + 2);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
    const int per_split = a.tiles_m * a.tiles_n, tiles = per_split * a.splits;

    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], kEpiWarps);
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_holder)),
                     "r"(a.tmem_cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;
    pdl_wait();

    if (warp == 0) {
        if (lane == 0) {
            // ---------------------------------------------------- TMA producer
            int q = 0;
            bool ok = true;
            for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
                const int split = t / per_split, tt = t - split * per_split;
                const int m0 = tt / a.tiles_n * kBM, n0 = tt % a.tiles_n * BN;
                const int b0 = (int)((int64_t)a.kb * split / a.splits), b1 = (int)((int64_t)a.kb * (split + 1) / a.splits);
                for (int p = 0; ok && p < a.pairs; ++p) {
                    const int pp = plane_pair(a.pairs, p), pa = pp >> 2, pb = pp & 3;
                    for (int kb = b0; kb < b1; ++kb, ++q) {
                        const int stage = q % NS;
                        if (!mbar_wait(&empty[stage], ((uint32_t)(q / NS) & 1u) ^ 1u, abort_flag, a.wait_cycles)) {
                            ok = false;
                            break;
                        }
                        uint8_t* sa = smem + (size_t)stage * stage_bytes;
                        mbar_expect_tx(&full[stage], (uint32_t)stage_bytes);
                        if constexpr (A_MN) {
#pragma unroll
                            for (int i = 0; i < kBM / 64; ++i)
                                tma_load_3d(sa + i * 8192, &map_a, m0 + i * 64, kb * kKB, pa, &full[stage]);
                        } else {
                            tma_load_3d(sa, &map_a, kb * kKB, m0, pa, &full[stage]);
                        }
                        if constexpr (B_MN) {
                            for (int i = 0; i < BN / 64; ++i)
                                tma_load_3d(sa + a_bytes + i * 8192, &map_b, n0 + i * 64, kb * kKB, pb, &full[stage]);
                        } else {
                            tma_load_3d(sa + a_bytes, &map_b, kb * kKB, n0, pb, &full[stage]);
                        }
                    }
                }
            }
            if (*abort_flag)   // the copies already issued must land before the block exits
                for (int j = (q > NS ? q - NS : 0); j < q; ++j) mbar_drain(&full[j % NS], (uint32_t)(j / NS) & 1u);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // ---------------------------------------------------- MMA issuer
            int q = 0, it = 0;
            bool ok = true;
            for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x, ++it) {
                const int split = t / per_split;
                const int b0 = (int)((int64_t)a.kb * split / a.splits), b1 = (int)((int64_t)a.kb * (split + 1) / a.splits);
                const int buf = it & 1;
                if (!mbar_wait(&tempty[buf], ((uint32_t)(it >> 1) & 1u) ^ 1u, abort_flag, a.wait_cycles)) break;
                tc_fence_after();
                const uint32_t d = tmem_base + (uint32_t)(buf * BN);
                uint32_t accumulate = 0;
                for (int p = 0; ok && p < a.pairs; ++p) {
                    for (int kb = b0; kb < b1; ++kb, ++q) {
                        const int stage = q % NS;
                        if (!mbar_wait(&full[stage], (uint32_t)(q / NS) & 1u, abort_flag, a.wait_cycles)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t sa = smem_u32(smem + (size_t)stage * stage_bytes), sb = sa + a_bytes;
                        const int steps = kb == a.kb - 1 ? a.last_steps : kKB / 16;
                        for (int kk = 0; kk < steps; ++kk) {
                            const uint64_t ad = A_MN ? sw128_desc_mn(sa + kk * 2048, 8192, 1024) : sw128_desc(sa + kk * 32);
                            const uint64_t bd = B_MN ? sw128_desc_mn(sb + kk * 2048, 8192, 1024) : sw128_desc(sb + kk * 32);
                            tc_mma_f16(d, ad, bd, a.idesc, accumulate);
                            accumulate = 1;
                        }
                        tc_commit(&empty[stage]);
                    }
                }
                if (ok) tc_commit(&tfull[buf]);
            }
            if (*abort_flag) {   // MMAs already issued must finish before TMEM is freed
                tc_commit(&tfull[it & 1]);
                mbar_drain(&tfull[it & 1], (uint32_t)(it >> 1) & 1u);
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue
        const int quarter = warp & 3, half = (warp - 2) / 4;
        uint8_t* mine = scratch + (warp - 2) * (32 * 128);
        const DropKey key = drop_key(a.e.drop);
        int it = 0;
        for (int t = blockIdx.x; t < tiles; t += gridDim.x, ++it) {
            const int buf = it & 1;
            if (!mbar_wait(&tfull[buf], (uint32_t)(it >> 1) & 1u, abort_flag, a.wait_cycles)) break;
            __syncwarp();
            tc_fence_after();
            const int split = t / per_split, tt = t - split * per_split;
            const int row0 = tt / a.tiles_n * kBM + 32 * quarter, n0 = tt % a.tiles_n * BN;
            const uint32_t taddr = tmem_base + ((uint32_t)(32 * quarter) << 16) + (uint32_t)(buf * BN);
            for (int c0 = 32 * half; c0 < BN; c0 += 64) {
                if (n0 + c0 >= a.N) break;
                const int col = n0 + c0 + 8 * (lane % 4), n = a.N - col;
                if (a.splits > 1) {
                    transpose_slice(taddr + c0, mine, [&](int, int r, float (&f)[8]) {
                        const int row = row0 + r;
                        if (row < a.M && n > 0) {
                            float4* p = reinterpret_cast<float4*>(a.partial + ((int64_t)split * a.M + row) * a.Np + col);
                            p[0] = make_float4(f[0], f[1], f[2], f[3]);
                            p[1] = make_float4(f[4], f[5], f[6], f[7]);
                        }
                    });
                } else {
                    float b[8];
                    bias8(a.e.bias, col, a.N, b);
                    if (a.e.vec && n0 + c0 + 32 <= a.N) {
                        Raw8<T> res[4];
                        if (a.e.res) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int row = row0 + i * 8 + lane / 4;
                                if (row < a.M) res[i] = load8<T, true>((const T*)a.e.res + row * a.e.ldr + col, 8);
                            }
                        }
                        transpose_slice(taddr + c0, mine, [&](int pass, int r, float (&f)[8]) {
                            if (row0 + r < a.M) finish8<T, true>(a.e, key, row0 + r, col, 8, f, b, res[pass]);
                        });
                    } else {   // a ragged slice, or rows off the 16-byte grid
                        transpose_slice(taddr + c0, mine, [&](int, int r, float (&f)[8]) {
                            if (row0 + r < a.M && n > 0) finish8_any<T>(a.e, key, row0 + r, col, n, f, b);
                        });
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[buf]);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(a.tmem_cols)
                     : "memory");
    }
    if (threadIdx.x == 0 && *abort_flag) set_status(a.status, DLRM_STATUS_TIMEOUT);
}

// The partial tiles of a split product added in order, then the epilogue.
template <typename T>
__global__ void __launch_bounds__(256)
finish_kernel(const float* __restrict__ partial, int splits, int64_t Np, int M, int N, const __grid_constant__ Epilogue e)
{
    pdl_wait();
    const DropKey key = drop_key(e.drop);
    const int64_t groups = Np / 8, runs = groups * M, plane = (int64_t)M * Np;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < runs; i += (int64_t)gridDim.x * 256) {
        const int row = (int)(i / groups), col = (int)(i - row * groups) * 8, n = N - col;
        float f[8] = {};
        for (int s = 0; s < splits; ++s) {
            const float4* p = reinterpret_cast<const float4*>(partial + s * plane + i * 8);
            const float4 lo = __ldcs(p), hi = __ldcs(p + 1);
            f[0] += lo.x; f[1] += lo.y; f[2] += lo.z; f[3] += lo.w;
            f[4] += hi.x; f[5] += hi.y; f[6] += hi.z; f[7] += hi.w;
        }
        float b[8];
        bias8(e.bias, col, N, b);
        finish8_any<T>(e, key, row, col, n, f, b);
    }
}

// ---------------------------------------------------------------- host side
// One operand: `outer` rows (K-major: of the output index, ld apart, K
// contiguous; MN-major: of K, ld apart, the output index contiguous).
struct Operand {
    const void* p;
    int64_t ld, plane;   // elements between rows, and between planes
    int planes;
    bool mn;
};

struct Shape {
    int M, N, K, pairs;
};

struct Plan {
    int BN, splits;
};

// How a product is cut: the plan with the least estimated time.  The unit is
// one 16-wide MMA step of a 128 x 64 tile.
inline Plan plan(const Shape& s)
{
    const int sms = num_sms();
    const int64_t kb = (s.K + kKB - 1) / kKB;
    Plan best = {256, 1};
    double least = 0;
    for (int BN = 256; BN >= 64; BN /= 2) {
        if (BN > 64 && BN / 2 >= s.N) continue;
        const int64_t tiles = (int64_t)((s.M + kBM - 1) / kBM) * ((s.N + BN - 1) / BN);
        for (int S = 1; S <= 32 && S <= kb; ++S) {
            if (S > 1 && tiles * S > 4 * (int64_t)sms) break;
            const int64_t waves = (tiles * S + sms - 1) / sms;
            const int64_t blocks = (kb + S - 1) / S * s.pairs;
            // a stage's products (a narrow tile is bound by its operands' arrival), a tile's epilogue, the finish pass
            double cost = (double)waves * blocks * (BN == 256 ? 16.0 : BN == 128 ? 9.0 : 6.0) + waves * BN * 0.25 + 40;
            if (S > 1) cost += 80 + (double)s.M * s.N * S / sms / 1200.0;
            if (least == 0 || cost < least) {
                least = cost;
                best = {BN, S};
            }
        }
    }
    return best;
}

__host__ __device__ inline int64_t padded(int64_t n) { return (n + 7) / 8 * 8; }

inline size_t partial_bytes(const Shape& s)
{
    const Plan p = plan(s);
    return p.splits > 1 ? dlrm_ws_align((size_t)p.splits * s.M * padded(s.N) * 4) : 0;
}

inline dlrm_status make_map(const char* fn, CUtensorMap* m, const Operand& o, bool bf, int64_t index, int64_t K, int tile)
{
    EncodeTiledFn enc = encode_fn();
    if (!enc) return fail(DLRM_ERR_CUDA, "%s: cuTensorMapEncodeTiled unavailable", fn);
    const int64_t inner = o.mn ? index : K, outer = o.mn ? K : index;
    // a single row's distance is never used, but has to be a legal one
    const int64_t ld = outer > 1 ? o.ld : padded(inner);
    const cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)outer, (cuuint64_t)o.planes};
    const cuuint64_t str[2] = {(cuuint64_t)ld * 2, (cuuint64_t)(o.planes > 1 ? o.plane : ld) * 2};
    const cuuint32_t box[3] = {(cuuint32_t)kKB, (cuuint32_t)(o.mn ? kKB : tile), 1}, ones[3] = {1, 1, 1};
    const CUresult r = enc(m, bf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                           const_cast<void*>(o.p), dims, str, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(DLRM_ERR_CUDA, "%s: tensor map (%d)", fn, (int)r);
    return DLRM_OK;
}

// out = A B^T and the epilogue; T the type of the epilogue's tensors, bf
// whether the operands are bf16 (fp16 otherwise).  partial: partial_bytes(s).
template <typename T, bool A_MN, bool B_MN>
dlrm_status run(const char* fn, const Shape& s, const Operand& A, const Operand& B, bool bf, const Epilogue& e,
                float* partial, uint32_t* status, cudaStream_t st)
{
    const Plan p = plan(s);
    CUtensorMap ma, mb;
    dlrm_status r = make_map(fn, &ma, A, bf, s.M, s.K, kBM);
    if (r == DLRM_OK) r = make_map(fn, &mb, B, bf, s.N, s.K, p.BN);
    if (r != DLRM_OK) return r;
    Args a = {};
    a.M = s.M;
    a.N = s.N;
    a.kb = (s.K + kKB - 1) / kKB;
    a.last_steps = (s.K - (a.kb - 1) * kKB + 15) / 16;
    a.pairs = s.pairs;
    a.splits = p.splits;
    a.BN = p.BN;
    const int64_t tm = (s.M + kBM - 1) / kBM, tn = (s.N + p.BN - 1) / p.BN;
    if (tm * tn > INT32_MAX / 64) return fail(DLRM_ERR_UNSUPPORTED, "%s: %lld output tiles", fn, (long long)(tm * tn));
    a.tiles_m = (int)tm;
    a.tiles_n = (int)tn;
    a.NS = kMaxStages;
    while (smem_bytes(p.BN, a.NS) > (size_t)kSmemLimit) --a.NS;
    a.idesc = idesc_f16(kBM, p.BN) | (bf ? 1u << 7 | 1u << 10 : 0u) | (A_MN ? 1u << 15 : 0u) | (B_MN ? 1u << 16 : 0u);
    a.tmem_cols = 2 * p.BN;
    a.partial = partial;
    a.Np = padded(s.N);
    a.e = e;
    a.status = status;
    a.wait_cycles = wait_limit_cycles();
    const int64_t tiles = tm * tn * p.splits;
    const int grid = (int)(tiles < num_sms() ? tiles : num_sms());
    const size_t smem = smem_bytes(p.BN, a.NS);
    auto kern = gemm_kernel<T, A_MN, B_MN>;
    cudaError_t ce = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (ce != cudaSuccess) return fail(DLRM_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(ce));
    r = check_launch_pdl(launch_pdl(kern, dim3(grid), dim3(kThreads), smem, st, ma, mb, a), "gemm_kernel");
    if (r != DLRM_OK || p.splits == 1) return r;
    const int64_t runs = a.Np / 8 * s.M, want = (runs + 255) / 256, most = (int64_t)num_sms() * 8;
    return check_launch_pdl(launch_pdl(finish_kernel<T>, dim3((unsigned)(want < most ? want : most)), dim3(256), 0, st,
                                       (const float*)partial, p.splits, a.Np, s.M, s.N, e),
                            "finish_kernel");
}

}  // namespace gemm
}  // namespace dlrm
