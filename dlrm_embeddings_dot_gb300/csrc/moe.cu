// moe.cu -- a mixture-of-experts layer for a few tokens in two kernels.
//
// Bound by the touched experts' weights, each read once from HBM into matrix
// fragments (few_rows.cuh).
//
//   moe_up    routing and the first product.  Every cluster of eight blocks
//             computes the router's logits for itself (each block an eighth
//             of H, the partial sums exchanged through distributed shared
//             memory), so no block waits for another cluster; each block
//             then picks the top k, lists the tokens of each chosen expert and
//             takes its share of the (expert, 16 rows) units.  A unit's K is
//             split over G warps, whose partial tiles meet in shared memory;
//             probs * a(.) goes to the workspace in the tensors' type.
//   moe_down  a cluster owns 16 rows of the output: its warps share out the
//             (expert, run of I) items of all chosen experts, each warp adding
//             all its items into one set of accumulators (an absent token's
//             fragment is zero), and the warps' and blocks' sums are added in a
//             fixed order.  No atomics on floats, no partial outputs in HBM.
#include <map>
#include <mutex>

#include "few_rows.cuh"

namespace dlrm {
namespace {

using namespace few;

constexpr int kThreads = 256, kWarps = kThreads / kWarp;
constexpr int kUpCluster = 8, kMaxSplit = 8;   // blocks of a cluster in moe_up, at most in moe_down
constexpr int kMaxE = DLRM_MOE_MAX_EXPERTS, kMaxK = DLRM_MOE_MAX_TOP_K;

struct MoeArgs {
    const void *x, *wr, *w1, *w2, *res;
    int64_t ldx, ldr, ldy;
    int T, H, I, E, k, act, gated, group;   // group: warps that share a unit of moe_up
    int chunk;                              // values of I in an item of moe_down
    void* y;
    int32_t* ids;
    float* probs;
    void* h;                                // [kTerms][T][k][I]
};

// probs * h enters the second product as the sum of two values of a 2-byte type
// (the rounded value and the rounded rest): the product of the weights with a
// second fragment is free beside the weights' traffic, and y then has one
// rounding, its own.
template <typename T>
constexpr int kTerms = sizeof(T) == 2 ? 2 : 1;

// Which tokens chose which expert, in shared memory.
struct Lists {
    unsigned long long mask[kMaxE];        // bit t: token t chose the expert
    uint16_t entry[kMaxTokens * kMaxK];    // per expert, its tokens ascending: token * kMaxK + slot
    uint16_t first[kMaxE];                 // an expert's first entry
    uint16_t active[kMaxE];                // the chosen experts, ascending
    int n_active;
};

// Builds the lists from id(t, j) (all threads of the block).
template <typename Id>
__device__ __forceinline__ void build_lists(Lists& l, int T, int k, int E, Id&& id)
{
    for (int e = threadIdx.x; e < E; e += kThreads) l.mask[e] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < T * k; i += kThreads) atomicOr(&l.mask[id(i / k, i % k)], 1ull << (i / k));
    __syncthreads();
    if (threadIdx.x < kWarp) {
        const int lane = threadIdx.x;
        int n = 0, used = 0;
        for (int e = lane * 8; e < min(E, lane * 8 + 8); ++e) {
            n += __popcll(l.mask[e]);
            used += l.mask[e] != 0;
        }
        int n0 = n, u0 = used;
#pragma unroll
        for (int d = 1; d < kWarp; d *= 2) {
            const int a = __shfl_up_sync(~0u, n0, d), b = __shfl_up_sync(~0u, u0, d);
            if (lane >= d) {
                n0 += a;
                u0 += b;
            }
        }
        if (lane == kWarp - 1) l.n_active = u0;
        n0 -= n;
        u0 -= used;
        for (int e = lane * 8; e < min(E, lane * 8 + 8); ++e) {
            l.first[e] = (uint16_t)n0;
            if (l.mask[e]) l.active[u0++] = (uint16_t)e;
            n0 += __popcll(l.mask[e]);
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < T * k; i += kThreads) {
        const int t = i / k, j = i % k, e = id(t, j);
        l.entry[l.first[e] + __popcll(l.mask[e] & ((1ull << t) - 1))] = (uint16_t)(t * kMaxK + j);
    }
    __syncthreads();
}

// Order of the logits as integers: NaN above all, -0 equal to 0.
__device__ __forceinline__ uint32_t logit_key(float v)
{
    if (v != v) return 0xffffffffu;
    const uint32_t b = __float_as_uint(v == 0.f ? 0.f : v);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ void group_sync(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads, 2) moe_up_kernel(MoeArgs a)
{
    pdl_wait();
    extern __shared__ float smem[];
    __shared__ Lists lists;
    __shared__ uint8_t ids_s[kMaxTokens * kMaxK];
    __shared__ float probs_s[kMaxTokens * kMaxK];
    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp, g = lane / 4, t4 = lane % 4;
    const T *x = (const T*)a.x, *wr = (const T*)a.wr, *w1 = (const T*)a.w1;

    // ---- the router's logits: this block's eighth of H
    const int e_tiles = (a.E + kRows - 1) / kRows, E16 = e_tiles * kRows;
    const int sub = e_tiles < kWarps ? kWarps / e_tiles : 1;     // warps that split an expert tile's K
    const uint32_t rank = cluster_rank();
    float* lp = smem;                        // [sub][T][E16]: partial logits
    float* lg = smem + sub * a.T * E16;      // [T][E16]: logits
    {
        const int steps = (a.H + kStep<T> - 1) / kStep<T>;
        const int per = (steps + kUpCluster * sub - 1) / (kUpCluster * sub) * kStep<T>;
        for (int i = warp; i < e_tiles * sub; i += kWarps) {
            const int tile = i % e_tiles, s = i / e_tiles;
            const int k0 = ((int)rank * sub + s) * per, k1 = min(a.H, k0 + per);
            const int e0 = tile * kRows + g;
            const T* w[1][2] = {{wr + (int64_t)min(e0, a.E - 1) * a.H, wr + (int64_t)min(e0 + 8, a.E - 1) * a.H}};
            with_token_tiles(a.T, [&](auto nt) {
                constexpr int NT = decltype(nt)::value;
                const T* xp[NT];
#pragma unroll
                for (int j = 0; j < NT; ++j) xp[j] = x + min(j * 8 + g, a.T - 1) * a.ldx;
                float acc[1][NT][4] = {};
                rows_mac<T, 1, NT, VEC>(acc, w, xp, k0, k1);
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int tok = j * 8 + 2 * t4 + (c & 1);
                        if (tok < a.T) lp[(s * a.T + tok) * E16 + tile * kRows + g + (c >> 1) * 8] = acc[0][j][c];
                    }
            });
        }
        if (sub > 1) {   // the block's own sums first: what is read across the cluster is read once
            __syncthreads();
            for (int i = threadIdx.x; i < a.T * E16; i += kThreads) {
                float v = lp[i];
                for (int s = 1; s < sub; ++s) v += lp[s * a.T * E16 + i];
                lp[i] = v;
            }
        }
        cluster_sync();
        // block r adds up every eighth logit and hands it to all
        for (int i = threadIdx.x * kUpCluster + rank; i < a.T * E16; i += kThreads * kUpCluster) {
            float v[kUpCluster];
#pragma unroll
            for (int r = 0; r < kUpCluster; ++r) v[r] = cluster_ld(cluster_map(lp + i, r));
#pragma unroll
            for (int r = 1; r < kUpCluster; ++r) v[0] += v[r];
#pragma unroll
            for (int r = 0; r < kUpCluster; ++r) cluster_st(cluster_map(lg + i, r), v[0]);
        }
        cluster_sync();
    }

    // ---- top k and its softmax, a warp per token
    for (int t = warp; t < a.T; t += kWarps) {
        unsigned long long key[kMaxE / kWarp];
#pragma unroll
        for (int i = 0; i < kMaxE / kWarp; ++i) {
            const int e = i * kWarp + lane;
            key[i] = e < a.E ? (unsigned long long)logit_key(lg[t * E16 + e]) << 32 | (uint32_t)(kMaxE - e) : 0;
        }
        float top = 0.f, mine = 0.f;
        int best = 0;
        for (int j = 0; j < a.k; ++j) {
            unsigned long long m = 0;
#pragma unroll
            for (int i = 0; i < kMaxE / kWarp; ++i) m = key[i] > m ? key[i] : m;
#pragma unroll
            for (int d = 16; d; d /= 2) {
                const unsigned long long o = __shfl_xor_sync(~0u, m, d);
                m = o > m ? o : m;
            }
            const int e = kMaxE - (int)(uint32_t)m;
#pragma unroll
            for (int i = 0; i < kMaxE / kWarp; ++i)
                if (key[i] == m) key[i] = 0;
            const float v = lg[t * E16 + e];
            if (j == 0) top = v;
            if (lane == j) {
                best = e;
                mine = expf(v - top);
            }
        }
        float sum = lane < a.k ? mine : 0.f;
#pragma unroll
        for (int d = 4; d; d /= 2) sum += __shfl_xor_sync(~0u, sum, d);   // lanes 0..7 hold the k <= 8 values
        if (lane < a.k) {
            ids_s[t * kMaxK + lane] = (uint8_t)best;
            probs_s[t * kMaxK + lane] = mine / sum;
            if (blockIdx.x == 0) {
                a.ids[t * a.k + lane] = best;
                a.probs[t * a.k + lane] = mine / sum;
            }
        }
    }
    __syncthreads();
    build_lists(lists, a.T, a.k, a.E, [&](int t, int j) { return (int)ids_s[t * kMaxK + j]; });

    // ---- the first product: units of 16 rows of one chosen expert, G warps each
    const int G = a.group, groups = kWarps / G, mine = warp / G, wg = warp % G;
    const int tiles = (a.I + kRows - 1) / kRows, units = lists.n_active * tiles;
    const int steps = (a.H + kStep<T> - 1) / kStep<T>, per = (steps + G - 1) / G * kStep<T>;
    const int k0 = wg * per, k1 = min(a.H, k0 + per);
    const int nt_max = a.T <= 8 ? 1 : a.T <= 16 ? 2 : a.T <= 32 ? 4 : 8;
    const int tile_floats = nt_max * 8 * kPitch;
    float* red = smem;    // [warp][2][token][kPitch], over the logits
    T* h = (T*)a.h;
    for (int u = blockIdx.x * groups + mine; u < units; u += gridDim.x * groups) {
        const int e = lists.active[u / tiles], row0 = u % tiles * kRows;
        const int n = __popcll(lists.mask[e]);
        const uint16_t* entry = lists.entry + lists.first[e];
        const int64_t base = (int64_t)e * (a.gated ? 2 : 1) * a.I;
        const T* w[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int b = 0; b < 2; ++b)
                w[i][b] = w1 + (base + (int64_t)(a.gated ? i : 0) * a.I + min(row0 + g + 8 * b, a.I - 1)) * a.H;
        with_token_tiles(n, [&](auto nt) {
            constexpr int NT = decltype(nt)::value;
            const T* xp[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j)
                xp[j] = x + (int64_t)(entry[min(j * 8 + g, n - 1)] / kMaxK) * a.ldx;
            if (a.gated) {
                float acc[2][NT][4] = {};
                rows_mac<T, 2, NT, VEC>(acc, w, xp, k0, k1);
                put_partial(red + (warp * 2) * tile_floats, acc[0]);
                put_partial(red + (warp * 2 + 1) * tile_floats, acc[1]);
            } else {
                const T* w0[1][2] = {{w[0][0], w[0][1]}};
                float acc[1][NT][4] = {};
                rows_mac<T, 1, NT, VEC>(acc, w0, xp, k0, k1);
                put_partial(red + (warp * 2) * tile_floats, acc[0]);
            }
        });
        group_sync(1 + mine, G * kWarp);
        for (int i = wg * kWarp + lane; i < n * kRows; i += G * kWarp) {
            const int tok = i / kRows, r = i % kRows;
            const float* p = red + (mine * G * 2) * tile_floats + tok * kPitch + r;
            float z = 0.f, up = 0.f;
            for (int q = 0; q < G; ++q) {
                z += p[q * 2 * tile_floats];
                if (a.gated) up += p[(q * 2 + 1) * tile_floats];
            }
            const int slot = entry[tok];
            float v = act_f(z, a.act);
            if (a.gated) v *= up;
            if (row0 + r < a.I) {
                T* dst = h + ((int64_t)(slot / kMaxK) * a.k + slot % kMaxK) * a.I + row0 + r;
                v *= probs_s[slot];
                const T top = from_f32<T>(v);
                *dst = top;
                if constexpr (kTerms<T> == 2) {
                    const float rest = v - to_f32(top);   // NaN for an infinite v: its rest is zero
                    dst[(int64_t)a.T * a.k * a.I] = from_f32<T>(fabsf(to_f32(top)) <= 3.4e38f ? rest : 0.f);
                }
            }
        }
        group_sync(1 + mine, G * kWarp);
    }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads, 2) moe_down_kernel(MoeArgs a)
{
    pdl_wait();
    extern __shared__ float smem[];   // [warp][token][kPitch]: each warp's sums over its items
    __shared__ Lists lists;
    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp, g = lane / 4, t4 = lane % 4;
    const int S = (int)cluster_size(), rank = (int)cluster_rank();
    const int row0 = (int)(blockIdx.x / S) * kRows;
    float* mine = smem + warp * a.T * kPitch;
    for (int i = lane; i < a.T * kPitch; i += kWarp) mine[i] = 0.f;
    build_lists(lists, a.T, a.k, a.E, [&](int t, int j) { return a.ids[t * a.k + j]; });

    const int chunks = (a.I + a.chunk - 1) / a.chunk, items = lists.n_active * chunks;
    const T *w2 = (const T*)a.w2, *h = (const T*)a.h;
    for (int it = rank * kWarps + warp; it < items; it += S * kWarps) {
        const int e = lists.active[it / chunks], k0 = it % chunks * a.chunk, n = __popcll(lists.mask[e]);
        const uint16_t* entry = lists.entry + lists.first[e];
        const T* w[1][2];
#pragma unroll
        for (int b = 0; b < 2; ++b) w[0][b] = w2 + ((int64_t)e * a.H + min(row0 + g + 8 * b, a.H - 1)) * a.I;
        with_token_tiles(n, [&](auto nt) {
            constexpr int NT = decltype(nt)::value;
            const T* hp[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int slot = entry[min(j * 8 + g, n - 1)];
                hp[j] = h + ((int64_t)(slot / kMaxK) * a.k + slot % kMaxK) * a.I;
            }
            float acc[1][NT][4] = {};
            rows_mac<T, 1, NT, VEC, kTerms<T>>(acc, w, hp, k0, min(a.I, k0 + a.chunk), (int64_t)a.T * a.k * a.I);
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int i = j * 8 + 2 * t4 + (c & 1);
                    if (i < n) mine[entry[i] / kMaxK * kPitch + g + (c >> 1) * 8] += acc[0][j][c];
                }
        });
        __syncwarp();   // another item's token may be another lane's
    }
    __syncthreads();
    // the warps' sums into the first one's place, then the blocks' into the output
    for (int i = threadIdx.x; i < a.T * kRows; i += kThreads) {
        const int at = i / kRows * kPitch + i % kRows;
        float v = smem[at];
#pragma unroll
        for (int q = 1; q < kWarps; ++q) v += smem[q * a.T * kPitch + at];
        smem[at] = v;
    }
    cluster_sync();
    for (int i = threadIdx.x * S + rank; i < a.T * kRows; i += kThreads * S) {
        const int t = i / kRows, r = row0 + i % kRows;
        float v[kMaxSplit];
#pragma unroll
        for (int q = 0; q < kMaxSplit; ++q) v[q] = q < S ? cluster_ld(cluster_map(smem + t * kPitch + i % kRows, q)) : 0.f;
#pragma unroll
        for (int q = 1; q < kMaxSplit; ++q) v[0] += v[q];
        if (r < a.H) {
            if (a.res) v[0] += to_f32(((const T*)a.res)[t * a.ldr + r]);
            ((T*)a.y)[t * a.ldy + r] = from_f32<T>(v[0]);
        }
    }
    cluster_sync();   // no block leaves while another reads its sums
}

// Blocks of moe_up that run at the same time (a multiple of the cluster).
template <typename K>
int resident_blocks(K kern, size_t smem)
{
    static std::mutex mu;
    static std::map<std::pair<int, size_t>, int> known;
    int dev = 0;
    cudaGetDevice(&dev);
    std::lock_guard<std::mutex> lock(mu);
    auto [it, fresh] = known.try_emplace({dev, smem}, kUpCluster);
    if (fresh) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = kUpCluster;
        cfg.blockDim = kThreads;
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim = {kUpCluster, 1, 1};
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) == cudaSuccess && n > 0) it->second = n * kUpCluster;
        else cudaGetLastError();
    }
    return it->second;
}

template <typename T, bool VEC>
dlrm_status launch_moe(MoeArgs a, cudaStream_t st)
{
    const int nt = a.T <= 8 ? 1 : a.T <= 16 ? 2 : a.T <= 32 ? 4 : 8;
    const int e_tiles = (a.E + kRows - 1) / kRows, E16 = e_tiles * kRows, sub = e_tiles < kWarps ? kWarps / e_tiles : 1;
    const size_t logits = (size_t)(sub + 1) * a.T * E16 * 4, red = (size_t)kWarps * 2 * nt * 8 * kPitch * 4;
    const size_t smem = logits > red ? logits : red;
    auto up = moe_up_kernel<T, VEC>;
    cudaError_t e = cudaFuncSetAttribute(up, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return fail(DLRM_ERR_CUDA, "dlrm_moe_fwd: %s", cudaGetErrorString(e));
    const int most = resident_blocks(up, smem);
    const int chosen = a.E < a.T * a.k ? a.E : a.T * a.k;            // experts at most
    const int64_t units = (int64_t)chosen * ((a.I + kRows - 1) / kRows);
    // warps of a unit: as many as leave every group of warps one unit, else the
    // number whose rounds of units cost least (a step of K against a unit's ten steps of overhead)
    const int64_t steps = (a.H + kStep<T> - 1) / kStep<T>;
    int64_t least = 0;
    for (int G = kWarps; G >= 1; G /= 2) {
        const int64_t groups = (int64_t)most * kWarps / G, cost = (units + groups - 1) / groups * ((steps + G - 1) / G + 10);
        if (least == 0 || cost < least) {
            least = cost;
            a.group = G;
        }
    }
    int64_t blocks = (units * a.group + kWarps - 1) / kWarps;
    if (blocks > most) blocks = most;
    blocks = (blocks + kUpCluster - 1) / kUpCluster * kUpCluster;
    e = launch_cluster(up, dim3((unsigned)blocks), dim3(kThreads), smem, st, kUpCluster, a);
    dlrm_status s = check_launch_pdl(e, "moe_up_kernel");
    if (s != DLRM_OK) return s;

    const int row_tiles = (a.H + kRows - 1) / kRows;
    int S = kMaxSplit;
    while (S > 1 && row_tiles * S > 4 * num_sms()) S /= 2;
    const int64_t share = (int64_t)chosen * a.I / (S * kWarps * 2);   // two items a warp where there is that much
    const int chunk = (int)(share < 2048 ? share : 2048) / kStep<T> * kStep<T>;
    a.chunk = chunk < kStep<T> ? kStep<T> : chunk;
    return check_launch_pdl(launch_cluster(moe_down_kernel<T, VEC>, dim3(row_tiles * S), dim3(kThreads),
                                           (size_t)kWarps * a.T * kPitch * 4, st, S, a),
                            "moe_down_kernel");
}

bool moe_sizes_ok(dlrm_dtype dtype, int T, int H, int I, int E, int k)
{
    return dense_dtype_ok(dtype) && T >= 0 && H >= 1 && I >= 1 && E >= 1 && k >= 1 && k <= E;
}

}  // namespace
}  // namespace dlrm

using namespace dlrm;

extern "C" size_t dlrm_moe_fwd_workspace_size(dlrm_dtype dtype, int T, int H, int I, int E, int k)
{
    if (!moe_sizes_ok(dtype, T, H, I, E, k)) return 0;
    return dlrm_ws_align((size_t)T * k * I * 4);   // one fp32 term, or two of 2 bytes
}

extern "C" dlrm_status dlrm_moe_fwd(const void* d_x, int64_t ldx, const void* d_w_router, const void* d_w1,
                                    const void* d_w2, const void* d_residual, int64_t ldr, dlrm_dtype dtype, int T,
                                    int H, int I, int E, int k, dlrm_act act, int gated, void* d_y, int64_t ldy,
                                    int32_t* d_ids, float* d_probs, void* d_workspace, size_t workspace_bytes,
                                    void* stream)
{
    DLRM_API_RANGE("dlrm_moe_fwd");
    clear_error();
    const char* fn = "dlrm_moe_fwd";
    if (!moe_sizes_ok(dtype, T, H, I, E, k) || act < DLRM_ACT_NONE || act > DLRM_ACT_SILU)
        return fail(DLRM_ERR_INVALID_ARG, "%s: need T >= 0, H, I, E >= 1, 1 <= k <= E and a known dtype and activation",
                    fn);
    if (T > DLRM_MOE_MAX_TOKENS || E > kMaxE || k > kMaxK)
        return fail(DLRM_ERR_UNSUPPORTED, "%s: at most %d tokens, %d experts and %d experts a token", fn,
                    DLRM_MOE_MAX_TOKENS, kMaxE, kMaxK);
    if (T == 0) return DLRM_OK;
    const int es = dense_dtype_size(dtype);
    dlrm_status s;
    if ((s = check_matrix(fn, "d_x", d_x, ldx, T, H, es)) != DLRM_OK) return s;
    if ((s = check_matrix(fn, "d_w_router", d_w_router, H, E, H, es)) != DLRM_OK) return s;
    if ((s = check_matrix(fn, "d_w1", d_w1, H, E, H, es)) != DLRM_OK) return s;
    if ((s = check_matrix(fn, "d_w2", d_w2, I, E, I, es)) != DLRM_OK) return s;
    if (d_residual && (s = check_matrix(fn, "d_residual", d_residual, ldr, T, H, es)) != DLRM_OK) return s;
    if ((s = check_matrix(fn, "d_y", d_y, ldy, T, H, es)) != DLRM_OK) return s;
    if ((s = check_matrix(fn, "d_ids", d_ids, k, T, k, 4)) != DLRM_OK) return s;
    if ((s = check_matrix(fn, "d_probs", d_probs, k, T, k, 4)) != DLRM_OK) return s;
    const size_t need = dlrm_moe_fwd_workspace_size(dtype, T, H, I, E, k);
    if (!d_workspace || workspace_bytes < need)
        return fail(DLRM_ERR_WORKSPACE, "%s: workspace %zu bytes < %zu", fn, d_workspace ? workspace_bytes : 0, need);
    if (reinterpret_cast<uintptr_t>(d_workspace) & 255u)
        return fail(DLRM_ERR_INVALID_ARG, "%s: the workspace must be 256-byte aligned", fn);
    MoeArgs a = {d_x, d_w_router, d_w1, d_w2, d_residual, ldx, ldr, ldy, T,     H,       I,          E, k, (int)act,
                 gated != 0, 0, 0, d_y, d_ids, d_probs, d_workspace};
    // the workspace's planes start on the grid where I keeps its rows there
    const bool vec = rows_aligned16(d_x, ldx, T, es) && rows_aligned16(d_w_router, H, E, es) &&
                     rows_aligned16(d_w1, H, 2, es) && rows_aligned16(d_w2, I, 2, es);
    return with_type(dtype, [&](auto t) {
        using T_ = decltype(t);
        return vec ? launch_moe<T_, true>(a, as_stream(stream)) : launch_moe<T_, false>(a, as_stream(stream));
    });
}
