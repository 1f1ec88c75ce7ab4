// gemm_tc.cuh -- the dense layer's products on the tcgen05 tensor cores:
// out[M][N] = A B^T with a fused epilogue, A and B each either K-major (K
// contiguous: x and W of the forward, dZ of dX) or MN-major (the output's row
// or column index contiguous: W of dX, dZ and x of dW).
//
// A persistent block per SM, or pair of blocks (PAIR), walks output tiles of 128
// (256) x BN rows and columns, BN = 256, 128 or 64:
//   warp 0      TMA producer: per 64 of K a 128 x 64 tile of A and a BN x 64
//               tile of B, 128-byte swizzle, into an NS-stage ring; in a pair
//               each block loads its own 128 rows of A and half of B's rows
//   warp 1      TMEM allocation and MMA issue (M = 128 or 256, N = BN, K = 16
//               steps; the pair's leader issues for both blocks, whose tensor
//               cores read both halves of B)
//   warps 2..17 epilogue: TMEM lane quarter q = warp % 4, every fourth 32-column
//               slice; a lane has 32 columns of a row, i.e. four runs of the
//               generator.  Results leave as boxes of 32 rows and columns by
//               TMA stores from swizzled shared memory, and the residual comes
//               in the same way.  A slice is a chain of latencies (TMEM,
//               barriers, fence, store), which is why there are many warps
// Two TMEM accumulators let the products of the next tile run under the
// epilogue of this one.
//
// fp32 operands come as three bf16 planes (see split planes in linear.cu); the
// K loop then runs over six plane pairs, the smallest products first.  The tensor
// cores cut what they add to an accumulator instead of rounding it, which shrinks a
// sum by 8e-10 of itself for each of K: past kChain blocks of K (LONG) the products of
// the first planes go to the accumulators in segments, which the epilogue warps add up
// in registers while the next one runs (16384 x 1024 outputs, error against 64 bits,
// one accumulator / segments: K = 1024 9.7e-7 / 3.5e-7, 152 / 155 us; K = 4096 4.3e-6 / 4.0e-7;
// the library's fp32 5.7e-7 and 1.2e-6).  A gradient
// that its 2-byte type does not hold comes as two planes of A.  Few
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
constexpr int kEpiWarps = 16;
constexpr int kThreads = (2 + kEpiWarps) * 32;
constexpr int kSlice = 32;          // columns of an epilogue slice
constexpr int kSliceStep = kEpiWarps / 4 * kSlice;
constexpr int kMaxStages = 8;
constexpr int kMaxPairs = 6;         // products of two operands of three planes each
constexpr int kChain = 6;           // 64-wide blocks of K that fp32's first planes add up in one accumulator
constexpr int kSmemLimit = 232448;  // 227 KB opt-in per block

struct Args {
    int M, N;
    int kb, last_steps;             // 64-wide blocks of K, and 16-wide steps of the last one
    int pairs;                      // plane pairs: 1, 2 (A has two planes), or 6 for fp32
    int splits;                     // parts of K; above 1 the tiles go to `partial`
    int tiles_m, tiles_n, BN, NS;
    int a_mn, b_mn;                 // operand layouts
    int bias_vec;                   // the bias starts on a 16-byte boundary
    int warp_bytes;                 // an epilogue warp's shared memory
    uint32_t idesc, tmem_cols;
    float* partial;                 // [splits][M][Np]
    int64_t Np;
    Epilogue e;
    uint32_t* status;
    long long wait_cycles;
    Overlap overlap;
};

// Plane pair p, (A plane << 2) | B plane, the small products first.  fp32: planes hi = 0,
// mid = 1, lo = 2 of both; two pairs: planes hi = 0, lo = 1 of A.
__device__ __forceinline__ int plane_pair(int pairs, int p)
{
    constexpr uint32_t order = 0x2u | 0x8u << 4 | 0x5u << 8 | 0x1u << 12 | 0x4u << 16 | 0x0u << 20;
    return pairs == kMaxPairs ? (int)(order >> (4 * p)) & 15 : p + 1 < pairs ? 0x4 : 0;
}

// A slice of 32 rows as a TMA box: rows of 64 bytes with the 64-byte swizzle
// (2-byte types) or of 128 bytes with the 128-byte one (fp32).  An epilogue warp
// holds one box of each tensor.
template <typename T>
constexpr int kBoxBytes = 32 * kSlice * (int)sizeof(T);

inline size_t smem_bytes(int b_rows, int ns, int warp_bytes)
{
    return 1024 + (size_t)ns * (kBM * 128 + b_rows * 128) + (size_t)kEpiWarps * warp_bytes +
           (size_t)(2 * ns + 4 + kEpiWarps) * 8 + 16;
}

// 16-byte chunk c of the lane's row of a box.
template <typename T>
__device__ __forceinline__ uint4* box_at(uint8_t* box, int c)
{
    const int lane = threadIdx.x % kWarp;
    const int at = sizeof(T) == 2 ? lane * 64 + ((c ^ (lane >> 1 & 3)) << 4) : lane * 128 + (((c ^ lane) & 7) << 4);
    return reinterpret_cast<uint4*>(box + at);
}

// f += the lane's row of a box
template <typename T>
__device__ __forceinline__ void add_box_row(uint8_t* box, float (&f)[kSlice])
{
#pragma unroll
    for (int q = 0; q < kSlice / 8; ++q) {
        Raw8<T> r;
#pragma unroll
        for (int i = 0; i < (int)(sizeof(T) / 2); ++i) r.w[i] = *box_at<T>(box, q * (int)(sizeof(T) / 2) + i);
        float g[8];
        widen8<T>(r, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[8 * q + i] += g[i];
    }
}

template <typename T>
__device__ __forceinline__ void write_box_row(uint8_t* box, const float (&f)[kSlice])
{
#pragma unroll
    for (int c = 0; c < kSlice * (int)sizeof(T) / 16; ++c) {
        if constexpr (std::is_same_v<T, float>)
            *box_at<T>(box, c) = f4_as_u4(make_float4(f[4 * c], f[4 * c + 1], f[4 * c + 2], f[4 * c + 3]));
        else
            *box_at<T>(box, c) = pack8<T>(reinterpret_cast<const float(&)[8]>(f[8 * c]));
    }
}

// K blocks [b0, b1) of part `split`.
struct Range {
    int b0, b1;
};
__device__ __forceinline__ Range k_range(const Args& a, int split)
{
    if (a.splits == 1) return {0, a.kb};   // a 64-bit division takes as long as a K block's products
    return {(int)((int64_t)a.kb * split / a.splits), (int)((int64_t)a.kb * (split + 1) / a.splits)};
}

// Segments of a range of K, and their length in blocks (the last may be shorter).
struct Segments {
    int n, len;
};
template <bool LONG>
__device__ __forceinline__ Segments segments(const Range& r)
{
    const int blocks = r.b1 - r.b0;
    if (!LONG || blocks <= kChain) return {1, blocks};
    const int n = (blocks + kChain - 1) / kChain, len = (blocks + n - 1) / n;
    return {(blocks + len - 1) / len, len};
}

// sum += the warp's 32 x 32 slice of the accumulator at taddr
__device__ __forceinline__ void add_slice(uint32_t taddr, float (&sum)[kSlice])
{
#pragma unroll
    for (int h = 0; h < kSlice; h += 16) {
        uint32_t v[16];
        tmem_ld_x16(taddr + h, v);
        tmem_wait_ld(v);
#pragma unroll
        for (int i = 0; i < 16; ++i) sum[h + i] += __uint_as_float(v[i]);
    }
}

// The slice at taddr = sum
__device__ __forceinline__ void put_slice(uint32_t taddr, const float (&sum)[kSlice])
{
#pragma unroll
    for (int h = 0; h < kSlice; h += 16) {
        uint32_t v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(sum[h + i]);
        tmem_st_x16(taddr + h, v);
    }
}

// The warp's 32 x 32 slice of the accumulator at taddr into its scratch, a row
// as eight swizzled 16-byte chunks; loaded() once TMEM has been read.
template <typename Loaded>
__device__ __forceinline__ void stage_slice(uint32_t taddr, uint8_t* scratch, Loaded&& loaded)
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
    loaded();
    __syncwarp();
}

// Columns 8 (lane % 4) and on of rows lane / 4, lane / 4 + 8, ... of the staged slice.
__device__ __forceinline__ void take_rows(const uint8_t* scratch, float (&f)[4][8])
{
    const int lane = threadIdx.x % kWarp, c = 2 * (lane % 4);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const int r = p * 8 + lane / 4;
        const float4 lo = *reinterpret_cast<const float4*>(scratch + r * 128 + ((c ^ (r & 7)) << 4));
        const float4 hi = *reinterpret_cast<const float4*>(scratch + r * 128 + (((c + 1) ^ (r & 7)) << 4));
        f[p][0] = lo.x, f[p][1] = lo.y, f[p][2] = lo.z, f[p][3] = lo.w;
        f[p][4] = hi.x, f[p][5] = hi.y, f[p][6] = hi.z, f[p][7] = hi.w;
    }
}

// The epilogue of rows that do not start and end on the 16-byte grid: a lane takes
// one column of each row, so that a warp's loads and stores are contiguous
// whatever the alignment, eight rows a turn, each step over all of them.
template <typename T, typename Loaded>
__device__ __forceinline__ void ragged_slice(const Epilogue& e, const DropKey& key, uint32_t taddr, uint8_t* scratch,
                                             int row0, int M, int c0, int N, Loaded&& loaded)
{
    constexpr int kTurn = 8;
    const int lane = threadIdx.x % kWarp, col = c0 + lane, rows = min(32, M - row0);
    const bool in = col < N;
    const float bias = e.bias && in ? __ldg(e.bias + col) : 0.f;
    const T* rp = (const T*)e.res + (int64_t)row0 * e.ldr + col;
    float res[kTurn], ahead[kTurn];   // the residual of this turn and of the next
    auto fetch = [&](int r0) {
#pragma unroll
        for (int i = 0; i < kTurn; ++i) ahead[i] = in && r0 + i < rows ? to_f32(__ldg(rp + (r0 + i) * e.ldr)) : 0.f;
    };
    if (e.res) fetch(0);
    uint32_t keep = 0;   // byte p: row 8 p + lane / 4, columns 8 (lane % 4) and on
    if (e.drop.thr)
#pragma unroll
        for (int p = 0; p < 4; ++p)
            keep |= keep8(e.drop, key, (uint32_t)(row0 + 8 * p + lane / 4), (uint32_t)c0 / 8 + lane % 4) << 8 * p;
    stage_slice(taddr, scratch, loaded);
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += kTurn) {
        float f[kTurn];
#pragma unroll
        for (int i = 0; i < kTurn; ++i) {
            const int r = r0 + i;
            const float v = *reinterpret_cast<const float*>(scratch + r * 128 + (((lane / 4) ^ (r & 7)) << 4) + lane % 4 * 4);
            f[i] = fmaf(v, e.scale, bias);
        }
        if (e.res) {
#pragma unroll
            for (int i = 0; i < kTurn; ++i) res[i] = ahead[i];
            if (r0 + kTurn < rows) fetch(r0 + kTurn);
        }
        if (e.pre) {
            T* at = (T*)e.pre + (int64_t)(row0 + r0) * e.ldp + col;
#pragma unroll
            for (int i = 0; i < kTurn; ++i)
                if (in && r0 + i < rows) at[i * e.ldp] = from_f32<T>(f[i]);
        }
        act_n<T>(f, e.act);
        if (e.drop.thr) {
#pragma unroll
            for (int i = 0; i < kTurn; ++i) {
                const uint32_t bits = __shfl_sync(~0u, keep, i * 4 + lane / 8) >> (r0 + lane % 8);
                f[i] = bits & 1 ? f[i] * e.drop.scale : 0.f;
            }
        }
        if (e.res) {
#pragma unroll
            for (int i = 0; i < kTurn; ++i) f[i] += res[i];
        }
        T* at = (T*)e.out + (int64_t)(row0 + r0) * e.ldo + col;
#pragma unroll
        for (int i = 0; i < kTurn; ++i)
            if (in && r0 + i < rows) at[i * e.ldo] = from_f32<T>(f[i]);
    }
}

// BOXES: results leave as TMA boxes; otherwise as a split's partial tiles, or by
// ragged_slice.  LONG: fp32 with more than kChain blocks of K.
template <typename T, bool PAIR, bool BOXES, bool LONG>
__global__ void __launch_bounds__(kThreads, 1)
gemm_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
            const __grid_constant__ CUtensorMap map_out, const __grid_constant__ CUtensorMap map_pre,
            const __grid_constant__ CUtensorMap map_res, const __grid_constant__ Args a)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    constexpr int CG = PAIR ? 2 : 1;
    const int BN = a.BN, NS = a.NS;
    constexpr int a_bytes = kBM * 128;
    const int b_rows = BN / CG, stage_bytes = a_bytes + b_rows * 128;
    uint8_t* scratch = smem + (size_t)NS * stage_bytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(scratch + kEpiWarps * a.warp_bytes);   // in a pair the leader's count both blocks' bytes
    uint64_t* empty = full + NS;
    uint64_t* tfull = empty + NS;
    uint64_t* tempty = tfull + 2;                                       // in a pair the leader's count both epilogues
    uint64_t* rfull = tempty + 2;                                       // an epilogue warp's residual slice
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(rfull + kEpiWarps);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
    const int rank = PAIR ? (int)(blockIdx.x & 1) : 0, first = (int)blockIdx.x / CG, stride = (int)gridDim.x / CG;
    const int per_split = a.tiles_m * a.tiles_n, tiles = per_split * a.splits;

    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], CG * kEpiWarps);
        }
        for (int i = 0; i < kEpiWarps; ++i) mbar_init(&rfull[i], 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        if constexpr (PAIR) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                             smem_u32(tmem_holder)),
                         "r"(a.tmem_cols)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                             smem_u32(tmem_holder)),
                         "r"(a.tmem_cols)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
    }
    tc_fence_before();
    __syncwarp();
    if constexpr (PAIR) cluster_barrier();   // the other block's barriers are set up too
    else __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;
    pdl_begin(a.overlap);

    if (warp == 0) {
        // -------------------------------------------------------- TMA producer
        int stage = 0, q = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int t = first; ok && t < tiles; t += stride) {
            const int split = a.splits == 1 ? 0 : t / per_split, tt = t - split * per_split;
            const int m0 = (tt / a.tiles_n * CG + rank) * kBM, n0 = tt % a.tiles_n * BN + rank * b_rows;
            const auto [b0, b1] = k_range(a, split);
            for (int p = 0; ok && p < a.pairs; ++p) {
                const int pp = plane_pair(a.pairs, p), pa = pp >> 2, pb = pp & 3;
                for (int kb = b0; kb < b1; ++kb) {
                    ok = __all_sync(~0u, mbar_wait(&empty[stage], phase ^ 1u, abort_flag, a.wait_cycles));
                    if (!ok) break;
                    uint8_t* sa = smem + (size_t)stage * stage_bytes;
                    if (elect_one()) {
                        // the other block's bytes can only be those of this phase: it too waits for the stage
                        if (rank == 0) mbar_expect_tx(&full[stage], (uint32_t)(CG * stage_bytes));
                        const uint32_t bar = PAIR ? peer_u32(&full[stage], 0) : 0;
                        auto load = [&](void* dst, const CUtensorMap* map, int c0, int c1, int c2) {
                            if constexpr (PAIR) tma_load_3d_pair(dst, map, c0, c1, c2, bar);
                            else tma_load_3d(dst, map, c0, c1, c2, &full[stage]);
                        };
                        if (a.a_mn) {
#pragma unroll
                            for (int i = 0; i < kBM / 64; ++i) load(sa + i * 8192, &map_a, m0 + i * 64, kb * kKB, pa);
                        } else {
                            load(sa, &map_a, kb * kKB, m0, pa);
                        }
                        if (a.b_mn) {
                            for (int i = 0; i < b_rows / 64; ++i)
                                load(sa + a_bytes + i * 8192, &map_b, n0 + i * 64, kb * kKB, pb);
                        } else {
                            load(sa + a_bytes, &map_b, kb * kKB, n0, pb);
                        }
                    }
                    __syncwarp();
                    ++q;
                    if (++stage == NS) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
        }
        if (lane == 0) {
            // every copy has been multiplied before the block exits
            for (int j = (q > NS ? q - NS : 0); ok && j < q; ++j)
                ok = mbar_wait(&empty[j % NS], (uint32_t)(j / NS) & 1u, abort_flag, a.wait_cycles);
            if (*abort_flag) {   // the copies already issued must land before the block exits
                if constexpr (PAIR) {
                    // counted together with the other block's, which may have given up before it asked
                    // for them: leave them a thousand times a copy's latency
                    const long long t0 = clock64();
                    while (clock64() - t0 < 2000000) {
                    }
                } else {
                    for (int j = (q > NS ? q - NS : 0); j < q; ++j) mbar_drain(&full[j % NS], (uint32_t)(j / NS) & 1u);
                }
            }
        }
    } else if (warp == 1) {
        if (rank == 0) {
            // ---------------------------------------------------- MMA issuer
            auto commit = [&](uint64_t* bar) {
                if constexpr (PAIR) tc_commit_pair(bar);
                else tc_commit(bar);
            };
            auto mma = [&](uint32_t d, uint64_t ad, uint64_t bd, uint32_t accumulate) {
                if constexpr (PAIR) tc_mma_f16_pair(d, ad, bd, a.idesc, accumulate);
                else tc_mma_f16(d, ad, bd, a.idesc, accumulate);
            };
            // descriptors of stage 0, and what a K step adds to their address field (16-byte units)
            const uint32_t sa = smem_u32(smem), sb = sa + a_bytes;
            const uint64_t ad0 = a.a_mn ? sw128_desc_mn(sa, 8192, 1024) : sw128_desc(sa);
            const uint64_t bd0 = a.b_mn ? sw128_desc_mn(sb, 8192, 1024) : sw128_desc(sb);
            constexpr uint32_t kMajor = 32 / 16, mnMajor = 2048 / 16;
            // A wait that gives up ends the issue at once: a stage whose copies have not
            // landed must not be handed back, as its barrier takes no second request
            // while one is open, and the other block would load on into its own.
            int stage = 0, it = 0;
            uint32_t phase = 0;
            auto issue = [&](auto step_a, auto step_b) {   // the descriptors' steps as constants
            constexpr uint32_t da = decltype(step_a)::value, db = decltype(step_b)::value;
            for (int t = first; t < tiles; t += stride) {
                const Range r = k_range(a, a.splits == 1 ? 0 : t / per_split);
                const Segments sg = segments<LONG>(r);
                bool ok = true;
                for (int s = 0; ok && s < sg.n; ++s) {
                    const int buf = it & 1;
                    ok = __all_sync(~0u, mbar_wait(&tempty[buf], ((uint32_t)(it >> 1) & 1u) ^ 1u, abort_flag, a.wait_cycles));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t d = tmem_base + (uint32_t)(buf * BN);
                    uint32_t accumulate = 0;
                    // the small products all in the first segment, then the first planes' share
                    for (int p = s ? a.pairs - 1 : 0; ok && p < a.pairs; ++p) {
                        const bool last = p == a.pairs - 1;
                        const int b0 = last ? r.b0 + s * sg.len : r.b0, b1 = last ? min(r.b1, b0 + sg.len) : r.b1;
                        for (int kb = b0; kb < b1; ++kb) {
                            ok = __all_sync(~0u, mbar_wait(&full[stage], phase, abort_flag, a.wait_cycles));
                            if (!ok) break;
                            tc_fence_after();
                            const uint64_t ad = ad0 + (uint32_t)(stage * (stage_bytes / 16));
                            const uint64_t bd = bd0 + (uint32_t)(stage * (stage_bytes / 16));
                            if (elect_one()) {
                                if (kb != a.kb - 1 || a.last_steps == 4) {
                                    mma(d, ad, bd, accumulate);
                                    mma(d, ad + da, bd + db, 1);
                                    mma(d, ad + 2 * da, bd + 2 * db, 1);
                                    mma(d, ad + 3 * da, bd + 3 * db, 1);
                                } else {   // the rest of K holds zeros past last_steps
                                    for (int kk = 0; kk < a.last_steps; ++kk)
                                        mma(d, ad + kk * da, bd + kk * db, kk ? 1 : accumulate);
                                }
                                commit(&empty[stage]);
                            }
                            accumulate = 1;
                            if (++stage == NS) {
                                stage = 0;
                                phase ^= 1u;
                            }
                        }
                    }
                    if (!ok) break;
                    __syncwarp();
                    if (elect_one()) commit(&tfull[buf]);
                    __syncwarp();
                    ++it;
                }
                if (!ok) break;
            }
            };
            using K = std::integral_constant<uint32_t, kMajor>;
            using MN = std::integral_constant<uint32_t, mnMajor>;
            if (a.a_mn) issue(MN{}, MN{});
            else if (a.b_mn) issue(K{}, MN{});
            else issue(K{}, K{});
            // MMAs already issued must finish before TMEM is freed; tfull[it & 1] has not been
            // committed to for this segment
            if (__any_sync(~0u, *abort_flag != 0) && elect_one()) {
                commit(&tfull[it & 1]);
                mbar_drain(&tfull[it & 1], (uint32_t)(it >> 1) & 1u);
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue
        const int quarter = warp & 3, part = (warp - 2) / 4;
        uint8_t* mine = scratch + (warp - 2) * a.warp_bytes;   // a box of out, of pre, of the residual
        uint8_t* pre_box = mine + kBoxBytes<T>;
        uint8_t* res_box = pre_box + (a.e.pre ? kBoxBytes<T> : 0);
        uint64_t* rbar = rfull + (warp - 2);
        const DropKey key = drop_key(a.e.drop);
        int it = 0;
        uint32_t asked = 0, used = 0;                          // residual slices asked for, and added
        for (int t = first; t < tiles; t += stride, ++it) {
            const int split = a.splits == 1 ? 0 : t / per_split, tt = t - split * per_split;
            const int row0 = (tt / a.tiles_n * CG + rank) * kBM + 32 * quarter, n0 = tt % a.tiles_n * BN;
            const uint32_t lanes = tmem_base + ((uint32_t)(32 * quarter) << 16);
            const int cols = row0 < a.M ? min(BN, a.N - n0) : 0;   // none of the warp's rows may lie inside
            auto ask = [&](int c0) {   // the residual's slice at c0, ahead of its use
                if (lane == 0) {
                    mbar_expect_tx(rbar, kBoxBytes<T>);
                    tma_load_2d(res_box, &map_res, n0 + c0, row0, rbar);
                }
                ++asked;
            };
            if (BOXES && a.e.res && kSlice * part < cols) ask(kSlice * part);
            auto arrived = [&] {   // the products of buffer it & 1
                const bool in = __all_sync(~0u, mbar_wait(&tfull[it & 1], (uint32_t)(it >> 1) & 1u, abort_flag, a.wait_cycles));
                tc_fence_after();
                return in;
            };
            auto release = [&] {   // the accumulator has been read: the tile or segment after next may overwrite it
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (PAIR) mbar_arrive_cluster(peer_u32(&tempty[it & 1], 0));
                    else mbar_arrive(&tempty[it & 1]);
                }
            };
            const Segments sg = segments<LONG>(k_range(a, split));
            if (sg.n == 1) {
                if (!arrived()) break;
            } else {
                // the segments' sums, then the whole in the last one's place, from where it goes on as any tile
                constexpr int kSlices = 256 / kSliceStep;   // the most a warp has
                float sum[kSlices][kSlice] = {};
                bool in = true;
                for (int s = 0; in && s < sg.n; ++s) {
                    if (s) {
                        release();
                        ++it;
                    }
                    in = arrived();
                    if (!in) break;
#pragma unroll
                    for (int j = 0; j < kSlices; ++j) {
                        const int c0 = kSlice * part + kSliceStep * j;
                        if (c0 < cols) add_slice(lanes + (uint32_t)((it & 1) * BN + c0), sum[j]);
                    }
                }
                if (!in) break;
#pragma unroll
                for (int j = 0; j < kSlices; ++j) {
                    const int c0 = kSlice * part + kSliceStep * j;
                    if (c0 < cols) put_slice(lanes + (uint32_t)((it & 1) * BN + c0), sum[j]);
                }
                tmem_wait_st();
            }
            const uint32_t taddr = lanes + (uint32_t)((it & 1) * BN);
            if (kSlice * part >= cols) {
                release();
                continue;
            }
            bool ok = true;
            for (int c0 = kSlice * part; c0 < cols; c0 += kSliceStep) {
                const bool last = c0 + kSliceStep >= cols;
                if constexpr (BOXES) {
                    float f[kSlice];
                    {
                        uint32_t v[32];
                        tmem_ld_x32(taddr + c0, v);
                        tmem_wait_ld(v);
#pragma unroll
                        for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(v[i]);
                    }
                    if (last) release();
                    if (lane == 0) bulk_wait_read<0>();   // the previous slice's stores have read theirs
                    if (a.e.bias) {                        // the same columns for every lane
                        const float* bias = a.e.bias + n0 + c0;
                        if (a.bias_vec && c0 + kSlice <= cols) {
#pragma unroll
                            for (int i = 0; i < kSlice / 4; ++i) {
                                const float4 b = __ldg(reinterpret_cast<const float4*>(bias) + i);
                                f[4 * i] += b.x, f[4 * i + 1] += b.y, f[4 * i + 2] += b.z, f[4 * i + 3] += b.w;
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < kSlice; ++i) f[i] += c0 + i < cols ? __ldg(bias + i) : 0.f;
                        }
                    } else if (a.e.scale != 1.f) {
#pragma unroll
                        for (int i = 0; i < kSlice; ++i) f[i] *= a.e.scale;
                    }
                    __syncwarp();
                    if (a.e.pre) write_box_row<T>(pre_box, f);
                    act_n<T>(f, a.e.act);
                    if (a.e.drop.thr)
#pragma unroll
                        for (int q = 0; q < kSlice / 8; ++q)
                            drop8(reinterpret_cast<float(&)[8]>(f[8 * q]), a.e.drop, key, (uint32_t)(row0 + lane),
                                  (uint32_t)(n0 + c0) / 8 + q);
                    if (a.e.res) {
                        ok = __all_sync(~0u, mbar_wait(rbar, used & 1u, abort_flag, a.wait_cycles));
                        if (!ok) break;
                        ++used;
                        add_box_row<T>(res_box, f);
                        __syncwarp();
                        if (!last) ask(c0 + kSliceStep);
                    }
                    write_box_row<T>(mine, f);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) {   // rows and columns past the tensor are clipped
                        tma_store_2d(&map_out, n0 + c0, row0, mine);
                        if (a.e.pre) tma_store_2d(&map_pre, n0 + c0, row0, pre_box);
                        bulk_commit();
                    }
                } else {
                    auto loaded = [&] {
                        if (last) release();
                    };
                    if (a.splits > 1) {
                        stage_slice(taddr + c0, mine, loaded);
                        float f[4][8];
                        take_rows(mine, f);
                        const int row = row0 + lane / 4, col = n0 + c0 + 8 * (lane % 4);
                        float4* p = reinterpret_cast<float4*>(a.partial + ((int64_t)split * a.M + row) * a.Np + col);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (row + 8 * i < a.M && col < a.N) {
                                p[2 * i * a.Np] = make_float4(f[i][0], f[i][1], f[i][2], f[i][3]);
                                p[2 * i * a.Np + 1] = make_float4(f[i][4], f[i][5], f[i][6], f[i][7]);
                            }
                    } else {
                        ragged_slice<T>(a.e, key, taddr + c0, mine, row0, a.M, n0 + c0, a.N, loaded);
                    }
                }
            }
            if (!ok) break;
        }
        if (lane == 0) {
            bulk_wait_all();   // the stores are complete, and a slice asked for has landed, before the block exits
            if (used < asked) mbar_drain(rbar, used & 1u);
        }
        __syncwarp();
    }

    tc_fence_before();
    __syncwarp();
    if constexpr (PAIR) cluster_barrier();   // neither block leaves while the other still reads its memory
    else __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        if constexpr (PAIR)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(a.tmem_cols)
                         : "memory");
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(a.tmem_cols)
                         : "memory");
    }
    if (threadIdx.x == 0 && *abort_flag) set_status(a.status, DLRM_STATUS_TIMEOUT);
    pdl_end(a.overlap);
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
    int column;   // cycles an epilogue takes for a tile's column
};

// What the plan takes for it (64K x 1024 outputs: 14 cycles a column of a 128-row
// tile for the stores alone, 14 for dropout, 16 for GELU, 12 for the residual;
// ragged rows 40).  It goes by the sizes alone, which the workspace query has too.
inline int column_cycles(int N, int es, bool layer) { return (N * (int64_t)es % 16 ? 40 : 14) + (layer ? 14 : 0); }

// A TMA store clips at 16 bytes: the last columns of another width would spill past N.
inline bool takes_boxes(const Epilogue& e, int N, int es) { return e.vec && (int64_t)N * es % 16 == 0; }

struct Plan {
    int BN, splits;
    bool pair;
};

// How a product is cut: the plan with the least estimated time, in cycles.
inline Plan plan(const Shape& s)
{
    struct Tile {
        int BN;
        bool pair;
        double block;   // cycles of a 64-wide block of K, measured: bound by the products for the
                        // widest, by the operands' way from L2 for the narrow ones
    };
    constexpr Tile tiles_of[] = {{256, true, 700}, {256, false, 800}, {128, true, 600}, {128, false, 650}, {64, false, 500}};
    const int sms = num_sms();
    const int64_t kb = (s.K + kKB - 1) / kKB;
    Plan best = {};
    double least = 0;
    for (const Tile& t : tiles_of) {
        const int rows = kBM * (t.pair ? 2 : 1), units = t.pair ? sms / 2 : sms;
        const int64_t tiles = (int64_t)((s.M + rows - 1) / rows) * ((s.N + t.BN - 1) / t.BN);
        for (int S = 1; S <= 32 && S <= kb; ++S) {
            if (S > 1 && tiles * S > 4 * (int64_t)units) break;
            const int64_t waves = (tiles * S + units - 1) / units;
            const double products = (double)((kb + S - 1) / S) * s.pairs * t.block;
            const double epilogue = 1500 + (S > 1 ? 20.0 : s.column) * (s.N < t.BN ? s.N : t.BN);
            double cost = waves * (products > epilogue ? products : epilogue) + epilogue;
            // another launch, and the partial tiles' way to memory and back
            if (S > 1) cost += 4000 + (double)s.M * s.N * S * 8 / 4000 + (double)s.M * s.N * s.column / 128 / sms;
            if (least == 0 || cost < least) {
                least = cost;
                best = {t.BN, S, t.pair};
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

// A box map of an output or of the residual.
template <typename T>
dlrm_status make_box_map(const char* fn, CUtensorMap* m, const void* p, int64_t ld, int M, int N)
{
    EncodeTiledFn enc = encode_fn();
    if (!enc) return fail(DLRM_ERR_CUDA, "%s: cuTensorMapEncodeTiled unavailable", fn);
    const cuuint64_t dims[2] = {(cuuint64_t)N, (cuuint64_t)M};
    const cuuint64_t str[1] = {(cuuint64_t)(M > 1 ? ld : padded(N)) * sizeof(T)};
    const cuuint32_t box[2] = {kSlice, 32}, ones[2] = {1, 1};
    const CUtensorMapDataType type = std::is_same_v<T, float>    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                     : std::is_same_v<T, __half> ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                                 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const CUresult r = enc(m, type, 2, const_cast<void*>(p), dims, str, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           sizeof(T) == 2 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(DLRM_ERR_CUDA, "%s: tensor map (%d)", fn, (int)r);
    return DLRM_OK;
}

// out = A B^T and the epilogue; T the type of the epilogue's tensors, bf
// whether the operands are bf16 (fp16 otherwise).  partial: partial_bytes(s);
// finish() has to follow.
template <typename T>
dlrm_status run(const char* fn, const Shape& s, const Operand& A, const Operand& B, bool bf, const Epilogue& e,
                float* partial, uint32_t* status, cudaStream_t st, Overlap overlap = {})
{
    const Plan p = plan(s);
    CUtensorMap ma, mb, mo = {}, mp = {}, mr = {};
    dlrm_status r = make_map(fn, &ma, A, bf, s.M, s.K, kBM);
    if (r == DLRM_OK) r = make_map(fn, &mb, B, bf, s.N, s.K, p.pair ? p.BN / 2 : p.BN);
    if (r != DLRM_OK) return r;
    Args a = {};
    a.M = s.M;
    a.N = s.N;
    a.kb = (s.K + kKB - 1) / kKB;
    a.last_steps = (s.K - (a.kb - 1) * kKB + 15) / 16;
    a.pairs = s.pairs;
    a.splits = p.splits;
    a.BN = p.BN;
    const int CG = p.pair ? 2 : 1, b_rows = p.BN / CG;
    const int64_t tm = (s.M + CG * kBM - 1) / (CG * kBM), tn = (s.N + p.BN - 1) / p.BN;
    if (tm * tn > INT32_MAX / 64) return fail(DLRM_ERR_UNSUPPORTED, "%s: %lld output tiles", fn, (long long)(tm * tn));
    a.tiles_m = (int)tm;
    a.tiles_n = (int)tn;
    a.a_mn = A.mn;
    a.b_mn = B.mn;
    const bool boxes = p.splits == 1 && takes_boxes(e, s.N, sizeof(T));
    a.bias_vec = aligned16(e.bias);
    a.warp_bytes = 32 * 128;   // a split's or a ragged slice's fp32 rows
    if (boxes) {
        a.warp_bytes = kBoxBytes<T> * (1 + (e.pre != nullptr) + (e.res != nullptr));
        r = make_box_map<T>(fn, &mo, e.out, e.ldo, s.M, s.N);
        if (r == DLRM_OK && e.pre) r = make_box_map<T>(fn, &mp, e.pre, e.ldp, s.M, s.N);
        if (r == DLRM_OK && e.res) r = make_box_map<T>(fn, &mr, e.res, e.ldr, s.M, s.N);
        if (r != DLRM_OK) return r;
    }
    a.NS = kMaxStages;
    while (smem_bytes(b_rows, a.NS, a.warp_bytes) > (size_t)kSmemLimit) --a.NS;
    a.idesc = idesc_f16(CG * kBM, p.BN) | (bf ? 1u << 7 | 1u << 10 : 0u) | (A.mn ? 1u << 15 : 0u) | (B.mn ? 1u << 16 : 0u);
    a.tmem_cols = 2 * p.BN;
    a.partial = partial;
    a.Np = padded(s.N);
    a.e = e;
    a.status = status;
    a.wait_cycles = wait_limit_cycles();
    a.overlap = overlap;
    const int64_t tiles = tm * tn * p.splits, units = num_sms() / CG;
    const int grid = (int)(tiles < units ? tiles : units) * CG;
    const size_t smem = smem_bytes(b_rows, a.NS, a.warp_bytes);
    auto pick = [&](auto l) {
        constexpr bool LONG = decltype(l)::value;
        return p.pair ? (boxes ? gemm_kernel<T, true, true, LONG> : gemm_kernel<T, true, false, LONG>)
                      : (boxes ? gemm_kernel<T, false, true, LONG> : gemm_kernel<T, false, false, LONG>);
    };
    auto kern = pick(std::false_type());
    if constexpr (std::is_same_v<T, float>)
        if ((a.kb + p.splits - 1) / p.splits > kChain) kern = pick(std::true_type());
    cudaError_t ce = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (ce != cudaSuccess) return fail(DLRM_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(ce));
    return check_launch_pdl(p.pair ? launch_cluster(kern, dim3(grid), dim3(kThreads), smem, st, 2, ma, mb, mo, mp, mr, a)
                                   : launch_pdl(kern, dim3(grid), dim3(kThreads), smem, st, ma, mb, mo, mp, mr, a),
                            "gemm_kernel");
}

// Adds up a split product's partial tiles.
template <typename T>
dlrm_status finish(const Shape& s, const Epilogue& e, const float* partial, cudaStream_t st)
{
    const Plan p = plan(s);
    if (p.splits == 1) return DLRM_OK;
    const int64_t Np = padded(s.N), runs = Np / 8 * s.M, want = (runs + 255) / 256, most = (int64_t)num_sms() * 8;
    return check_launch_pdl(launch_pdl(finish_kernel<T>, dim3((unsigned)(want < most ? want : most)), dim3(256), 0, st,
                                       partial, p.splits, Np, s.M, s.N, e),
                            "finish_kernel");
}

}  // namespace gemm
}  // namespace dlrm
