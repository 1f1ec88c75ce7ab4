// experts.cu -- a mixture of experts in training: the choice of experts and its
// gradient, the order of the choices by expert, and the rows' way to their
// experts and back.  Each is bound by memory, or by latency where there are few tokens.
#include "dlrm_block.h"
#include "row_units.cuh"
#include "sort_layout.h"

namespace dlrm {
namespace {

// ------------------------------------------------------------ choice of experts
// A logit and its expert as one unsigned number, so that the largest is the choice: the value's
// bits made to order as numbers do (a NaN above all, -0 as 0), below them 255 - e, so that equal
// ones go by lower index.  2-byte types fit 32 bits.  0 stands for no logit; expert() and
// value() give the parts back.
template <typename T>
struct Key {
    using Word = uint32_t;
    static constexpr uint32_t kInf = std::is_same_v<T, __half> ? 0x7c00u : 0x7f80u;
    static constexpr Word kClosed = (Word)(0xffffu & ~(0x8000u | kInf)) << 16 | 0xffffu;   // -infinity, whichever expert
    static __device__ __forceinline__ Word make(T v, int e)
    {
        uint16_t h;
        memcpy(&h, &v, 2);
        const uint32_t b = h == 0x8000u ? 0u : h;
        const uint32_t o = (b & 0x7fffu) > kInf ? 0xffffu : b & 0x8000u ? ~b & 0xffffu : b | 0x8000u;
        return o << 16 | (255 - e);
    }
    static __device__ __forceinline__ float value(Word k)
    {
        const uint32_t o = k >> 16;
        const uint16_t h = (uint16_t)(o == 0xffffu ? 0x7fffu : o & 0x8000u ? o ^ 0x8000u : ~o);
        T v;
        memcpy(&v, &h, 2);
        return to_f32(v);
    }
    static __device__ __forceinline__ int expert(Word k) { return 255 - (int)(k & 0xffu); }
};

template <>
struct Key<float> {
    using Word = unsigned long long;
    static constexpr Word kClosed = (Word)0x007fffffu << 32 | 0xffffffffu;
    static __device__ __forceinline__ Word make(float v, int e)
    {
        const uint32_t b = v == 0.f ? 0u : __float_as_uint(v);
        const uint32_t o = v != v ? 0xffffffffu : b & 0x80000000u ? ~b : b | 0x80000000u;
        return (Word)o << 32 | (uint32_t)(255 - e);
    }
    static __device__ __forceinline__ float value(Word k)
    {
        const uint32_t o = (uint32_t)(k >> 32);
        return __uint_as_float(o == 0xffffffffu ? 0x7fffffffu : o & 0x80000000u ? o ^ 0x80000000u : ~o);
    }
    static __device__ __forceinline__ int expert(Word k) { return 255 - (int)((uint32_t)k & 0xffu); }
};

// The largest of L lanes' keys, in all of them.
template <int L, typename Word>
__device__ __forceinline__ Word largest(Word k)
{
    if constexpr (L == kWarp && sizeof(Word) == 4) {
        return __reduce_max_sync(~0u, k);
    } else if constexpr (L == kWarp) {
        const uint32_t hi = __reduce_max_sync(~0u, (uint32_t)(k >> 32));
        return (Word)hi << 32 | __reduce_max_sync(~0u, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
    } else {
#pragma unroll
        for (int m = L / 2; m; m /= 2) k = max(k, __shfl_xor_sync(~0u, k, m));
        return k;
    }
}

// Eight keys in descending order (a network of 19 exchanges, the fewest there are).
template <typename Word>
__device__ __forceinline__ void sort8(Word (&k)[8])
{
    auto order = [&](int i, int j) {
        const Word a = k[i], b = k[j];
        k[i] = max(a, b);
        k[j] = min(a, b);
    };
    order(0, 2); order(1, 3); order(4, 6); order(5, 7);
    order(0, 4); order(1, 5); order(2, 6); order(3, 7);
    order(0, 1); order(2, 3); order(4, 5); order(6, 7);
    order(2, 4); order(3, 5);
    order(1, 4); order(3, 6);
    order(1, 2); order(3, 4); order(5, 6);
}

// L lanes take a token, eight logits each, which they sort; k rounds of the largest of the lanes'
// first keys, whose lane drops it.  Its whole cost is instructions and their latency, so a warp
// takes 32 / L tokens (65536 of 64 experts, 4 of them, bf16: a warp a token and searched anew each
// round 33 us, sorted 9; of 256 experts, 8 of them, fp32: searched anew 77 us).
template <typename T, bool VEC, int L>
__global__ void __launch_bounds__(256)
route_fwd_kernel(const T* __restrict__ logits, int64_t ldl, int tokens, int E, int k, int32_t* __restrict__ ids,
                 float* __restrict__ probs)
{
    using K = Key<T>;
    using Word = typename K::Word;
    pdl_wait();
    const int lane = threadIdx.x % kWarp, l = lane % L, n = E - l * 8;
    const int64_t step = (int64_t)gridDim.x * (256 / L);
    for (int64_t t0 = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / kWarp * (kWarp / L); t0 < tokens; t0 += step) {
        const int64_t t = t0 + lane / L;
        const bool here = t < tokens;
        Word key[8];
        {
            T v[8];
            if (here && n > 0) {
                const Raw8<T> raw = load8<T, VEC>(logits + t * ldl + l * 8, n);
                memcpy(v, &raw, sizeof(raw));
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) key[i] = here && i < n ? K::make(v[i], l * 8 + i) : 0;
        }
        sort8(key);
        Word mine = 0;       // lane j of the token's: choice j
        for (int j = 0; j < k; ++j) {
            const Word best = largest<L>(key[0]);
            if (key[0] == best) {
#pragma unroll
                for (int i = 0; i < 7; ++i) key[i] = key[i + 1];
                key[7] = 0;
            }
            if (l == j) mine = best;
        }
        const bool open = mine > K::kClosed;
        const float logit = K::value(mine), top = __shfl_sync(~0u, logit, 0, L);
        const float e = open ? expf(logit - top) : 0.f;
        float sum = e;
#pragma unroll
        for (int m = 4; m; m /= 2) sum += __shfl_xor_sync(~0u, sum, m);   // the first eight lanes have the choices
        if (here && l < k) {
            ids[t * k + l] = open ? K::expert(mine) : -1;
            probs[t * k + l] = open ? e / sum : 0.f;
        }
    }
}

// L lanes take a token's row of grad_logits: zeros, eight columns each, then lane j < k writes choice j.
template <typename T, bool VEC, int L>
__global__ void __launch_bounds__(256)
route_bwd_kernel(const float* __restrict__ grad_probs, const int32_t* __restrict__ ids, const float* __restrict__ probs,
                 int tokens, int E, int k, T* __restrict__ grad, int64_t ldgl)
{
    pdl_wait();
    const int lane = threadIdx.x % kWarp, l = lane % L;
    const int64_t step = (int64_t)gridDim.x * (256 / L);
    for (int64_t t0 = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / kWarp * (kWarp / L); t0 < tokens; t0 += step) {
        const int64_t t = t0 + lane / L;
        T* row = grad + t * ldgl;
        int id = -1;
        float p = 0.f, g = 0.f;
        if (t < tokens && l < k) {
            id = __ldg(ids + t * k + l);
            p = __ldg(probs + t * k + l);
            g = __ldg(grad_probs + t * k + l);
        }
        if (t < tokens) {
            if constexpr (VEC) {
                for (int c = l * (16 / (int)sizeof(T)); c < E; c += L * (16 / (int)sizeof(T)))
                    *reinterpret_cast<uint4*>(row + c) = make_uint4(0, 0, 0, 0);
            } else {
                for (int c = l; c < E; c += L) row[c] = from_f32<T>(0.f);
            }
        }
        if (id < 0 || id >= E) {
            id = -1;
            p = g = 0.f;
        }
        float dot = g * p;
#pragma unroll
        for (int m = 4; m; m /= 2) dot += __shfl_xor_sync(~0u, dot, m);
        const float d = p * (g - __shfl_sync(~0u, dot, 0, L));
        // of a token's equal ids the last one's lane; the zeros are in place for all lanes
        const uint32_t same = __match_any_sync(~0u, lane / L << 16 | (id & 0xffff));
        __syncwarp();
        if (id >= 0 && same >> lane == 1) row[id] = from_f32<T>(d);
    }
}

// fn(the lanes of a token as a constant)
template <typename Fn>
dlrm_status with_lanes(int E, Fn&& fn)
{
    if (E <= 64) return fn(std::integral_constant<int, 8>());
    if (E <= 128) return fn(std::integral_constant<int, 16>());
    return fn(std::integral_constant<int, 32>());
}

// ------------------------------------------------------------- order by expert
// A counting sort that keeps the order of equal experts.  A block takes a chunk of the choices,
// its warps contiguous parts of it; a warp counts and places 32 choices at a time, those of
// one expert found by match.any, in counters of its own in shared memory.  Choices without
// expert count as expert E.  With one block that is all; with more, expert_count_kernel writes
// the chunks' counts and their warps' first, and a block of expert_place_kernel adds up those of the
// blocks before it (and all of them: where an expert begins).  Both wait for what is before them on the stream
// before they read a choice.  The steps are chains of latencies: a warp's choices are
// loaded kBatch rounds at a time, and the counts' sums are shared out over all threads
// (sort_layout.h).  (us in a graph; the warps counted a second time while the counts were written / counts
// read back: 9000 choices of 16 4.9 / 5.6, 65536 x 4 of 64 8.9 / 9.3, 65536 x 8 of 256 19.8 / 19.4, 300000 x 8 of 33
// 42.0 / 31.8.  The former read choices ahead of its own wait.)
constexpr int kBatch = 8;
constexpr int kBins = DLRM_ROUTE_MAX_EXPERTS + 1;
static_assert(kBins <= kSortThreads, "a thread for each bin");

// A warp's part [from, to) of the choices, the first kBatch rounds of it in registers.
struct Part {
    const int32_t* ids;
    int64_t from, to;
    int id[kBatch];
    __device__ Part(const int32_t* p, int64_t n, int64_t chunk) : ids(p)
    {
        const int64_t part = chunk / kSortWarps, first = blockIdx.x * chunk;
        from = min(n, first + threadIdx.x / kWarp * part);
        to = min(n, from + part);
        load(from, id);
    }
    __device__ __forceinline__ void load(int64_t c0, int (&v)[kBatch]) const
    {
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int64_t c = c0 + b * kWarp + threadIdx.x % kWarp;
            v[b] = c < to ? __ldg(ids + c) : 0;
        }
    }
    // each(choice, id, bin, rank among the 32 of its bin, how many of them); bin kBins: past the part's end
    template <typename Each>
    __device__ __forceinline__ void walk(int E, Each each) const
    {
        const int lane = threadIdx.x % kWarp;
        auto rounds = [&](int64_t c0, const int (&v)[kBatch]) {
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const int64_t c = c0 + b * kWarp + lane;
                if (c0 + b * kWarp >= to) break;
                const int bin = c >= to ? kBins : v[b] >= 0 && v[b] < E ? v[b] : E;
                const uint32_t same = __match_any_sync(~0u, bin);
                each(c, v[b], bin, __popc(same & ((1u << lane) - 1)), __popc(same));
                __syncwarp();
            }
        };
        rounds(from, id);
        for (int64_t c0 = from + kBatch * kWarp; c0 < to; c0 += kBatch * kWarp) {
            int v[kBatch];
            load(c0, v);
            rounds(c0, v);
        }
    }
};

// Counts the warps' parts of the block's chunk into warps[warp][bin].
__device__ __forceinline__ void count_parts(const Part& part, int E, int (*warps)[kBins])
{
    int* mine = warps[threadIdx.x / kWarp];
    for (int e = threadIdx.x % kWarp; e <= E; e += kWarp) mine[e] = 0;
    __syncwarp();
    part.walk(E, [&](int64_t, int, int bin, int rank, int many) {
        if (rank == 0 && bin < kBins) mine[bin] += many;
    });
    __syncthreads();
}

__global__ void __launch_bounds__(kSortThreads)
expert_count_kernel(const int32_t* __restrict__ ids, int64_t n, int64_t chunk, int E, int32_t* __restrict__ counts,
                    int32_t* __restrict__ parts)
{
    pdl_wait();
    __shared__ int warps[kSortWarps][kBins];
    const Part part(ids, n, chunk);
    count_parts(part, E, warps);
    for (int e = threadIdx.x; e <= E; e += kSortThreads) {
        int s = 0;
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) {
            s += warps[w][e];
            parts[((int)blockIdx.x * kSortWarps + w) * (E + 1) + e] = warps[w][e];
        }
        counts[blockIdx.x * (E + 1) + e] = s;
    }
}

// MANY: more than one block, whose counts expert_count_kernel has written.
template <bool MANY>
__global__ void __launch_bounds__(kSortThreads)
expert_place_kernel(const int32_t* __restrict__ ids, int64_t n, int64_t chunk, int E, const int32_t* __restrict__ counts,
                    const int32_t* __restrict__ parts, int32_t* __restrict__ offsets, int32_t* __restrict__ slots,
                    int32_t* __restrict__ order, uint32_t* __restrict__ status)
{
    __shared__ int warps[kSortWarps][kBins];
    __shared__ int total[MANY ? kBins : 1], before[MANY ? kBins : 1], scan[kSortWarps];
    const int bins = E + 1, tid = threadIdx.x;
    pdl_wait();
    const Part part(ids, n, chunk);
    if constexpr (!MANY) {
        count_parts(part, E, warps);
    } else {
        const int w = tid / kWarp;
        const int32_t* own = parts + ((int)blockIdx.x * kSortWarps + w) * bins;
#pragma unroll 4
        for (int e = tid % kWarp; e < bins; e += kWarp) warps[w][e] = __ldcg(own + e);
        for (int e = tid; e < bins; e += kSortThreads) total[e] = before[e] = 0;
        __syncthreads();
        const CountShare share = count_share(tid, bins, (int)gridDim.x, (int)blockIdx.x);
        if (share.rows > 0) {
            int all = 0, ahead = 0;
#pragma unroll 8
            for (int i = 0; i < share.rows; ++i) {
                const int b = share.block(i), v = __ldcg(counts + b * bins + share.bin);
                all += v;
                ahead += b < (int)blockIdx.x ? v : 0;
            }
            atomicAdd(&total[share.bin], all);      // whole numbers: the same in any order
            atomicAdd(&before[share.bin], ahead);
        }
        __syncthreads();
    }
    // where each expert's places begin: an exclusive scan of the totals over the bins
    {
        const int e = tid, lane = e % kWarp;
        int mine[kSortWarps], v = 0;
        if (e < bins) {
#pragma unroll
            for (int w = 0; w < kSortWarps; ++w) mine[w] = warps[w][e];
            if constexpr (MANY) {
                v = total[e];
            } else {
#pragma unroll
                for (int w = 0; w < kSortWarps; ++w) v += mine[w];
            }
        }
        int s = v;
#pragma unroll
        for (int m = 1; m < kWarp; m *= 2) {
            const int o = __shfl_up_sync(~0u, s, m);
            if (lane >= m) s += o;
        }
        if (lane == kWarp - 1) scan[e / kWarp] = s;
        __syncthreads();
        if (e < bins) {
            for (int w = 0; w < e / kWarp; ++w) s += scan[w];
            int at = s - v;
            if (blockIdx.x == 0) offsets[e] = at;   // offsets[E]: how many have a place
            if constexpr (MANY) at += before[e];
#pragma unroll
            for (int w = 0; w < kSortWarps; ++w) {
                warps[w][e] = at;
                at += mine[w];
            }
        }
    }
    __syncthreads();
    int* mine = warps[tid / kWarp];
    bool bad = false;
    part.walk(E, [&](int64_t c, int id, int bin, int rank, int many) {
        const int at = bin < kBins ? mine[bin] + rank : 0;
        __syncwarp();
        if (rank == 0 && bin < kBins) mine[bin] += many;
        if (c < part.to) {
            slots[c] = bin < E ? at : -1;
            if (order) order[at] = bin < E ? (int32_t)c : -1;
            bad = bad || id >= E;
        }
    });
    if (bad) set_status(status, DLRM_STATUS_OOB_INDEX);
}

// -------------------------------------------------- rows to their experts and back
constexpr int kMaxK = DLRM_ROUTE_MAX_TOP_K;

// The slots of a token; those without a row as -1.
template <int K>
__device__ __forceinline__ void load_slots(const int32_t* slots, int64_t t, int k, int R, int (&s)[K], bool& bad)
{
#pragma unroll
    for (int j = 0; j < K; ++j) s[j] = j < k ? __ldg(slots + t * k + j) : -1;
#pragma unroll
    for (int j = 0; j < K; ++j)
        if (s[j] >= R) {
            bad = true;
            s[j] = -1;
        }
}

// xs[slots[t][j]] = x[t]: a row is read once and written k times.
template <typename T, int LAY>
__global__ void __launch_bounds__(256)
dispatch_kernel(const T* __restrict__ x, int64_t ldx, const int32_t* __restrict__ slots, int tokens, int k, int H, int R,
                int lanes, T* __restrict__ xs, int64_t ldxs, uint32_t* __restrict__ status)
{
    constexpr int U = kRuns<T, LAY, 2>;
    pdl_wait();
    bool bad = false;
    const Unit unit(lanes);
    for (Items it(unit, H, U); it.row < tokens; it.next()) {
        int s[kMaxK];
        Raw8<T> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (u < it.per)
                v[u] = load_cols<T, LAY>(x + it.row * ldx, unit.first<LAY, sizeof(T)>(it.run(u)), H, lanes);
        load_slots(slots, it.row, k, R, s, bad);
#pragma unroll
        for (int j = 0; j < kMaxK; ++j)
            if (s[j] >= 0)
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (u < it.per)
                        store_raw<T, LAY>(xs + s[j] * ldxs, unit.first<LAY, sizeof(T)>(it.run(u)), H, lanes, v[u]);
    }
    if (bad) set_status(status, DLRM_STATUS_OOB_INDEX);
}

// y[t] = residual[t] + sum over j of probs[t][j] ys[slots[t][j]]; probs NULL: the plain sum.  k <= K.
template <typename T, int LAY, int K>
__global__ void __launch_bounds__(256)
combine_kernel(const T* __restrict__ ys, int64_t ldys, const int32_t* __restrict__ slots, const float* __restrict__ probs,
               const T* __restrict__ res, int64_t ldres, int tokens, int k, int H, int R, int lanes, T* __restrict__ y,
               int64_t ldy, uint32_t* __restrict__ status)
{
    constexpr int U = kRuns<T, LAY, K>;
    pdl_wait();
    bool bad = false;
    const Unit unit(lanes);
    for (Items it(unit, H, U); it.row < tokens; it.next()) {
        int s[K];
        float p[K];
        load_slots(slots, it.row, k, R, s, bad);
#pragma unroll
        for (int j = 0; j < K; ++j) p[j] = probs && j < k ? __ldg(probs + it.row * k + j) : 1.f;
        Raw8<T> v[U][K], vr[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (u >= it.per) break;
            const int c = unit.first<LAY, sizeof(T)>(it.run(u));
#pragma unroll
            for (int j = 0; j < K; ++j)
                if (s[j] >= 0) v[u][j] = load_cols<T, LAY>(ys + s[j] * ldys, c, H, lanes);
            if (res) vr[u] = load_cols<T, LAY>(res + it.row * ldres, c, H, lanes);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (u >= it.per) break;
            float f[8] = {}, w[8];
#pragma unroll
            for (int j = 0; j < K; ++j)
                if (s[j] >= 0) {
                    widen8<T>(v[u][j], w);
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] = fmaf(p[j], w[i], f[i]);
                }
            if (res) {
                widen8<T>(vr[u], w);
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] += w[i];
            }
            store_cols<T, LAY>(y + it.row * ldy, unit.first<LAY, sizeof(T)>(it.run(u)), H, lanes, f);
        }
    }
    if (bad) set_status(status, DLRM_STATUS_OOB_INDEX);
}

struct CombineBwd {
    const void *gy, *ys;
    int64_t ldgy, ldys;
    const int32_t* slots;
    const float* probs;
    int tokens, k, H, R, lanes;
    void* gys;          // may be NULL
    int64_t ldgys;
    float* gp;          // may be NULL
    uint32_t* status;
};

// A unit takes a token, or with W = 8 warps a whole block does: grad_y once, and for each choice its
// row of ys in and of grad_ys out.  k <= K.
template <typename T, int LAY, int K, int W>
__global__ void __launch_bounds__(256) combine_bwd_kernel(const __grid_constant__ CombineBwd a)
{
    constexpr int U = kRuns<T, LAY, K>;
    __shared__ float red[W > 1 ? 8 * K : 1];
    pdl_wait();
    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp, H = a.H;
    const Unit unit(W > 1 ? kWarp : a.lanes);
    const int lanes = unit.lanes;
    bool bad = false;
    // a token's slots and shares, on the grid loaded a token ahead (40000 x 515 bf16, off it: 82 us so, 62
    // without: the registers)
    int next[K];
    float next_p[K];
    auto fetch = [&](int64_t t) {
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const bool has = j < a.k && t < a.tokens;
            next[j] = has ? __ldg(a.slots + t * a.k + j) : -1;
            next_p[j] = has && a.gys ? __ldg(a.probs + t * a.k + j) : 0.f;
        }
    };
    const int64_t first = W > 1 ? blockIdx.x : unit.unit - lane / lanes, step = W > 1 ? gridDim.x : unit.units;
    if (LAY == kOnGrid) fetch(W > 1 ? first : first + lane / lanes);
    // all units of a warp go through the loop together
    for (int64_t t0 = first; t0 < a.tokens; t0 += step) {
        const int64_t t = W > 1 ? t0 : t0 + lane / lanes;
        const bool here = t < a.tokens;
        int s[K];
        float p[K], dot[K];
        if (LAY != kOnGrid) fetch(t);
#pragma unroll
        for (int j = 0; j < K; ++j) {
            s[j] = next[j];
            if (s[j] >= a.R) {
                bad = true;
                s[j] = -1;
            }
            p[j] = next_p[j];
            dot[j] = 0.f;
        }
        if (LAY == kOnGrid) fetch(t + step);
        for (int run = W > 1 ? warp * U : 0; here && run * lanes * 8 < H; run += W * U) {
            Raw8<T> vg[U], v[U][K];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = unit.first<LAY, sizeof(T)>(run + u);
                vg[u] = load_cols<T, LAY>((const T*)a.gy + t * a.ldgy, c, H, lanes);
                if (a.gp)
#pragma unroll
                    for (int j = 0; j < K; ++j)
                        if (s[j] >= 0) v[u][j] = load_cols<T, LAY>((const T*)a.ys + s[j] * a.ldys, c, H, lanes);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = unit.first<LAY, sizeof(T)>(run + u);
                float g[8];
                widen8<T>(vg[u], g);
#pragma unroll
                for (int j = 0; j < K; ++j)
                    if (s[j] >= 0) {
                        if (a.gp) {
                            float w[8];
                            widen8<T>(v[u][j], w);
#pragma unroll
                            for (int i = 0; i < 8; ++i) dot[j] = fmaf(g[i], w[i], dot[j]);
                        }
                        if (a.gys) {
                            float o[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) o[i] = p[j] * g[i];
                            store_cols<T, LAY>((T*)a.gys + s[j] * a.ldgys, c, H, lanes, o);
                        }
                    }
            }
        }
        if (!a.gp) continue;
#pragma unroll
        for (int j = 0; j < K; ++j)
            if (j < a.k)
                for (int m = lanes / 2; m; m /= 2) dot[j] += __shfl_xor_sync(~0u, dot[j], m);
        if constexpr (W > 1) {
            static_assert(W == 8, "the block's barrier");
            __syncthreads();
            if (lane == 0)
#pragma unroll
                for (int j = 0; j < K; ++j) red[warp * K + j] = dot[j];
            __syncthreads();
            if (threadIdx.x < (unsigned)a.k) {
                float sum = red[threadIdx.x];
#pragma unroll
                for (int w = 1; w < W; ++w) sum += red[w * K + threadIdx.x];
                a.gp[t * a.k + threadIdx.x] = sum;
            }
        } else if (here && unit.l == 0) {
#pragma unroll
            for (int j = 0; j < K; ++j)
                if (j < a.k) a.gp[t * a.k + j] = dot[j];
        }
    }
    if (bad) set_status(a.status, DLRM_STATUS_OOB_INDEX);
}

// ------------------------------------------------------------------- checks
dlrm_status check_route(const char* fn, dlrm_dtype dtype, int T, int E, int k)
{
    if (!dense_dtype_ok(dtype)) return fail(DLRM_ERR_INVALID_ARG, "%s: bad dtype", fn);
    if (T < 0 || E < 1 || k < 1) return fail(DLRM_ERR_INVALID_ARG, "%s: need T >= 0, E >= 1 and k >= 1", fn);
    if (k > E) return fail(DLRM_ERR_INVALID_ARG, "%s: k is more than E", fn);
    if (E > DLRM_ROUTE_MAX_EXPERTS || k > DLRM_ROUTE_MAX_TOP_K || T > kMaxSize)
        return fail(DLRM_ERR_UNSUPPORTED, "%s: up to %d tokens, %d experts and %d of them a token", fn, kMaxSize,
                    DLRM_ROUTE_MAX_EXPERTS, DLRM_ROUTE_MAX_TOP_K);
    return DLRM_OK;
}

// An array of 4-byte elements that has to be there.
dlrm_status check_words(const char* fn, const char* name, const void* p)
{
    if (!p) return fail(DLRM_ERR_INVALID_ARG, "%s: %s is NULL", fn, name);
    if (reinterpret_cast<uintptr_t>(p) & 3u)
        return fail(DLRM_ERR_INVALID_ARG, "%s: %s is not aligned to its element size", fn, name);
    return DLRM_OK;
}

dlrm_status check_rows(const char* fn, dlrm_dtype dtype, int T, int k, int H, int R)
{
    if (!dense_dtype_ok(dtype)) return fail(DLRM_ERR_INVALID_ARG, "%s: bad dtype", fn);
    if (T < 0 || k < 1 || H < 1 || R < 0)
        return fail(DLRM_ERR_INVALID_ARG, "%s: need T >= 0, k >= 1, H >= 1 and R >= 0", fn);
    if (k > DLRM_ROUTE_MAX_TOP_K || T > kMaxSize || H > kMaxSize || R > kMaxSize)
        return fail(DLRM_ERR_UNSUPPORTED, "%s: sizes up to %d and %d places a token", fn, kMaxSize, DLRM_ROUTE_MAX_TOP_K);
    return DLRM_OK;
}

// fn(the layout as a constant)
template <typename Fn>
dlrm_status with_layout(int lay, Fn&& fn)
{
    if (lay == kOnGrid) return fn(std::integral_constant<int, kOnGrid>());
    if (lay == kFewLanes) return fn(std::integral_constant<int, kFewLanes>());
    return fn(std::integral_constant<int, kOffGrid>());
}

// fn(k rounded up to 2, 4 or 8 as a constant)
template <typename Fn>
dlrm_status with_choices(int k, Fn&& fn)
{
    if (k <= 2) return fn(std::integral_constant<int, 2>());
    if (k <= 4) return fn(std::integral_constant<int, 4>());
    return fn(std::integral_constant<int, 8>());
}

// Blocks of 256 threads where `lanes` take a token.
inline unsigned token_blocks(int64_t tokens, int lanes, const void* kern)
{
    return grid_blocks((tokens * lanes + 255) / 256, kern);
}

dlrm_status run_combine(const char* fn, const void* ys, int64_t ldys, const int32_t* slots, const float* probs,
                        const void* res, int64_t ldres, dlrm_dtype dtype, int T, int k, int H, int R, void* y, int64_t ldy,
                        uint32_t* status, void* stream)
{
    const int es = dense_dtype_size(dtype);
    const bool vec = H % 8 == 0 && rows_aligned16(ys, ldys, R, es) && (!res || rows_aligned16(res, ldres, T, es)) &&
                     rows_aligned16(y, ldy, T, es);
    return with_type(dtype, [&](auto t) {
        using E = decltype(t);
        return with_layout(row_layout(vec, H), [&](auto l) {
            constexpr int LAY = decltype(l)::value;
            return with_choices(k, [&](auto kk) {
                constexpr int K = decltype(kk)::value;
                const int lanes = unit_lanes(H, LAY);
                auto kern = combine_kernel<E, LAY, K>;
                const unsigned blocks = item_blocks(T, H, lanes, kRuns<E, LAY, K>, (const void*)kern);
                return check_launch_pdl(launch_pdl(kern, dim3(blocks), dim3(256), 0, as_stream(stream), (const E*)ys, ldys, slots,
                                                   probs, (const E*)res, ldres, T, k, H, R, lanes, (E*)y, ldy, status),
                                        fn);
            });
        });
    });
}

}  // namespace
}  // namespace dlrm

using namespace dlrm;

extern "C" dlrm_status dlrm_route_fwd(const void* d_logits, int64_t ldl, dlrm_dtype dtype, int T, int E, int k,
                                      int32_t* d_ids, float* d_probs, void* stream)
{
    DLRM_API_RANGE("dlrm_route_fwd");
    clear_error();
    const char* fn = "dlrm_route_fwd";
    dlrm_status s = check_route(fn, dtype, T, E, k);
    if (s != DLRM_OK || T == 0) return s;
    if ((s = check_matrix(fn, "d_logits", d_logits, ldl, T, E, dense_dtype_size(dtype))) != DLRM_OK) return s;
    if ((s = check_words(fn, "d_ids", d_ids)) != DLRM_OK) return s;
    if ((s = check_words(fn, "d_probs", d_probs)) != DLRM_OK) return s;
    return with_type(dtype, [&](auto t) {
        using X = decltype(t);
        return with_lanes(E, [&](auto l) {
            constexpr int L = decltype(l)::value;
            auto kern = E % 8 == 0 && rows_aligned16(d_logits, ldl, T, sizeof(X)) ? route_fwd_kernel<X, true, L>
                                                                                  : route_fwd_kernel<X, false, L>;
            return check_launch_pdl(launch_pdl(kern, dim3(token_blocks(T, L, (const void*)kern)), dim3(256), 0, as_stream(stream),
                                               (const X*)d_logits, ldl, T, E, k, d_ids, d_probs),
                                    "route_fwd_kernel");
        });
    });
}

extern "C" dlrm_status dlrm_route_bwd(const float* d_grad_probs, const int32_t* d_ids, const float* d_probs,
                                      dlrm_dtype dtype, int T, int E, int k, void* d_grad_logits, int64_t ldgl,
                                      void* stream)
{
    DLRM_API_RANGE("dlrm_route_bwd");
    clear_error();
    const char* fn = "dlrm_route_bwd";
    dlrm_status s = check_route(fn, dtype, T, E, k);
    if (s != DLRM_OK || T == 0) return s;
    if ((s = check_words(fn, "d_grad_probs", d_grad_probs)) != DLRM_OK) return s;
    if ((s = check_words(fn, "d_ids", d_ids)) != DLRM_OK) return s;
    if ((s = check_words(fn, "d_probs", d_probs)) != DLRM_OK) return s;
    if ((s = check_matrix(fn, "d_grad_logits", d_grad_logits, ldgl, T, E, dense_dtype_size(dtype))) != DLRM_OK) return s;
    return with_type(dtype, [&](auto t) {
        using X = decltype(t);
        return with_lanes(E, [&](auto l) {
            constexpr int L = decltype(l)::value;
            auto kern = E % 8 == 0 && rows_aligned16(d_grad_logits, ldgl, T, sizeof(X)) ? route_bwd_kernel<X, true, L>
                                                                                        : route_bwd_kernel<X, false, L>;
            return check_launch_pdl(launch_pdl(kern, dim3(token_blocks(T, L, (const void*)kern)), dim3(256), 0, as_stream(stream),
                                               d_grad_probs, d_ids, d_probs, T, E, k, (X*)d_grad_logits, ldgl),
                                    "route_bwd_kernel");
        });
    });
}

static bool sort_sizes_ok(int T, int k, int E)
{
    return T >= 0 && k >= 1 && k <= DLRM_ROUTE_MAX_TOP_K && E >= 1 && E <= DLRM_ROUTE_MAX_EXPERTS &&
           (int64_t)T * k <= kMaxSize;
}

extern "C" size_t dlrm_expert_sort_workspace_size(int T, int k, int E)
{
    if (!sort_sizes_ok(T, k, E)) return 0;
    const SortShape z = sort_shape((int64_t)T * k);
    return z.blocks > 1 ? dlrm_ws_align((size_t)z.blocks * (1 + kSortWarps) * (E + 1) * 4) : 0;
}

extern "C" dlrm_status dlrm_expert_sort(const int32_t* d_ids, int T, int k, int E, int32_t* d_offsets, int32_t* d_slots,
                                        int32_t* d_order, void* d_workspace, size_t workspace_bytes, uint32_t* d_status,
                                        void* stream)
{
    DLRM_API_RANGE("dlrm_expert_sort");
    clear_error();
    const char* fn = "dlrm_expert_sort";
    if (T < 0 || k < 1 || E < 1) return fail(DLRM_ERR_INVALID_ARG, "%s: need T >= 0, k >= 1 and E >= 1", fn);
    if (!sort_sizes_ok(T, k, E))
        return fail(DLRM_ERR_UNSUPPORTED, "%s: up to %d choices, %d experts and %d of them a token", fn, kMaxSize,
                    DLRM_ROUTE_MAX_EXPERTS, DLRM_ROUTE_MAX_TOP_K);
    dlrm_status s = check_words(fn, "d_offsets", d_offsets);
    if (s != DLRM_OK) return s;
    if (T > 0 && (s = check_words(fn, "d_ids", d_ids)) != DLRM_OK) return s;
    if (T > 0 && (s = check_words(fn, "d_slots", d_slots)) != DLRM_OK) return s;
    if (d_order && (s = check_words(fn, "d_order", d_order)) != DLRM_OK) return s;
    const size_t need = dlrm_expert_sort_workspace_size(T, k, E);
    if (need && (!d_workspace || workspace_bytes < need))
        return fail(DLRM_ERR_WORKSPACE, "%s: workspace %zu bytes < %zu", fn, d_workspace ? workspace_bytes : 0, need);
    if (need && (reinterpret_cast<uintptr_t>(d_workspace) & 255u))
        return fail(DLRM_ERR_INVALID_ARG, "%s: the workspace must be 256-byte aligned", fn);
    const int64_t n = (int64_t)T * k;
    const SortShape z = sort_shape(n);
    const cudaStream_t st = as_stream(stream);
    int32_t *const counts = (int32_t*)d_workspace, *const parts = counts + (z.blocks > 1 ? z.blocks * (E + 1) : 0);
    if (z.blocks > 1) {
        s = check_launch_pdl(launch_pdl(expert_count_kernel, dim3(z.blocks), dim3(kSortThreads), 0, st, d_ids, n, z.chunk, E,
                                        counts, parts),
                             "expert_count_kernel");
        if (s != DLRM_OK) return s;
    }
    auto place = z.blocks > 1 ? expert_place_kernel<true> : expert_place_kernel<false>;
    return check_launch_pdl(launch_pdl(place, dim3(z.blocks), dim3(kSortThreads), 0, st, d_ids, n, z.chunk, E,
                                       (const int32_t*)counts, (const int32_t*)parts, d_offsets, d_slots, d_order, d_status),
                            "expert_place_kernel");
}

extern "C" dlrm_status dlrm_dispatch_fwd(const void* d_x, int64_t ldx, const int32_t* d_slots, dlrm_dtype dtype, int T,
                                         int k, int H, int R, void* d_xs, int64_t ldxs, uint32_t* d_status, void* stream)
{
    DLRM_API_RANGE("dlrm_dispatch_fwd");
    clear_error();
    const char* fn = "dlrm_dispatch_fwd";
    dlrm_status s = check_rows(fn, dtype, T, k, H, R);
    if (s != DLRM_OK || T == 0) return s;
    const int es = dense_dtype_size(dtype);
    if ((s = check_matrix(fn, "d_x", d_x, ldx, T, H, es)) != DLRM_OK) return s;
    if ((s = check_words(fn, "d_slots", d_slots)) != DLRM_OK) return s;
    if (R > 0 && (s = check_matrix(fn, "d_xs", d_xs, ldxs, R, H, es)) != DLRM_OK) return s;
    const bool vec = H % 8 == 0 && rows_aligned16(d_x, ldx, T, es) && rows_aligned16(d_xs, ldxs, R, es);
    return with_type(dtype, [&](auto t) {
        using X = decltype(t);
        return with_layout(row_layout(vec, H), [&](auto l) {
            constexpr int LAY = decltype(l)::value;
            const int lanes = unit_lanes(H, LAY);
            return check_launch_pdl(launch_pdl(dispatch_kernel<X, LAY>, dim3(item_blocks(T, H, lanes, kRuns<X, LAY, 2>, nullptr)),
                                               dim3(256), 0, as_stream(stream), (const X*)d_x, ldx, d_slots, T, k, H, R, lanes,
                                               (X*)d_xs, ldxs, d_status),
                                    "dispatch_kernel");
        });
    });
}

extern "C" dlrm_status dlrm_dispatch_bwd(const void* d_grad_xs, int64_t ldgxs, const int32_t* d_slots, dlrm_dtype dtype,
                                         int T, int k, int H, int R, void* d_grad_x, int64_t ldgx, uint32_t* d_status,
                                         void* stream)
{
    DLRM_API_RANGE("dlrm_dispatch_bwd");
    clear_error();
    const char* fn = "dlrm_dispatch_bwd";
    dlrm_status s = check_rows(fn, dtype, T, k, H, R);
    if (s != DLRM_OK || T == 0) return s;
    const int es = dense_dtype_size(dtype);
    if (R > 0 && (s = check_matrix(fn, "d_grad_xs", d_grad_xs, ldgxs, R, H, es)) != DLRM_OK) return s;
    if ((s = check_words(fn, "d_slots", d_slots)) != DLRM_OK) return s;
    if ((s = check_matrix(fn, "d_grad_x", d_grad_x, ldgx, T, H, es)) != DLRM_OK) return s;
    return run_combine("dispatch_bwd's combine_kernel", d_grad_xs, ldgxs, d_slots, nullptr, nullptr, 0, dtype, T, k, H, R,
                       d_grad_x, ldgx, d_status, stream);
}

extern "C" dlrm_status dlrm_combine_fwd(const void* d_ys, int64_t ldys, const int32_t* d_slots, const float* d_probs,
                                        const void* d_residual, int64_t ldres, dlrm_dtype dtype, int T, int k, int H,
                                        int R, void* d_y, int64_t ldy, uint32_t* d_status, void* stream)
{
    DLRM_API_RANGE("dlrm_combine_fwd");
    clear_error();
    const char* fn = "dlrm_combine_fwd";
    dlrm_status s = check_rows(fn, dtype, T, k, H, R);
    if (s != DLRM_OK || T == 0) return s;
    const int es = dense_dtype_size(dtype);
    if (R > 0 && (s = check_matrix(fn, "d_ys", d_ys, ldys, R, H, es)) != DLRM_OK) return s;
    if ((s = check_words(fn, "d_slots", d_slots)) != DLRM_OK) return s;
    if ((s = check_words(fn, "d_probs", d_probs)) != DLRM_OK) return s;
    if (d_residual && (s = check_matrix(fn, "d_residual", d_residual, ldres, T, H, es)) != DLRM_OK) return s;
    if ((s = check_matrix(fn, "d_y", d_y, ldy, T, H, es)) != DLRM_OK) return s;
    return run_combine("combine_kernel", d_ys, ldys, d_slots, d_probs, d_residual, ldres, dtype, T, k, H, R, d_y, ldy,
                       d_status, stream);
}

extern "C" dlrm_status dlrm_combine_bwd(const void* d_grad_y, int64_t ldgy, const void* d_ys, int64_t ldys,
                                        const int32_t* d_slots, const float* d_probs, dlrm_dtype dtype, int T, int k,
                                        int H, int R, void* d_grad_ys, int64_t ldgys, float* d_grad_probs,
                                        uint32_t* d_status, void* stream)
{
    DLRM_API_RANGE("dlrm_combine_bwd");
    clear_error();
    const char* fn = "dlrm_combine_bwd";
    dlrm_status s = check_rows(fn, dtype, T, k, H, R);
    if (s != DLRM_OK || T == 0) return s;
    const int es = dense_dtype_size(dtype);
    if (!d_grad_ys && !d_grad_probs && R > 0) return fail(DLRM_ERR_INVALID_ARG, "%s: neither d_grad_ys nor d_grad_probs", fn);
    if ((s = check_matrix(fn, "d_grad_y", d_grad_y, ldgy, T, H, es)) != DLRM_OK) return s;
    if ((s = check_words(fn, "d_slots", d_slots)) != DLRM_OK) return s;
    if (R > 0 && d_grad_probs && (s = check_matrix(fn, "d_ys", d_ys, ldys, R, H, es)) != DLRM_OK) return s;
    if (d_grad_ys && (s = check_words(fn, "d_probs", d_probs)) != DLRM_OK) return s;
    if (R > 0 && d_grad_ys && (s = check_matrix(fn, "d_grad_ys", d_grad_ys, ldgys, R, H, es)) != DLRM_OK) return s;
    if (d_grad_probs && (s = check_words(fn, "d_grad_probs", d_grad_probs)) != DLRM_OK) return s;
    const bool vec = H % 8 == 0 && rows_aligned16(d_grad_y, ldgy, T, es) &&
                     (!d_grad_probs || rows_aligned16(d_ys, ldys, R, es)) &&
                     (!d_grad_ys || rows_aligned16(d_grad_ys, ldgys, R, es));
    // a block a token where those would leave SMs idle.  In a graph, us, a warp / a block a token, fp16 of 2 and 8:
    // 16 tokens x 768 2.7 / 2.2 and 6.3 / 2.9, x 4096 6.5 / 2.3 and 21 / 4.0; 600 x 768 2.8 / 3.7 and 6.6 / 5.7, x 4096
    // 6.7 / 4.2 and 24 / 10; 1200 x 768 2.8 / 6.3 and 6.5 / 9.9, x 4096 6.9 / 7.3 and 37 / 28; fp32 16 x 768 of 8
    // 8.0 / 3.7, 1200 8.9 / 14
    const bool wide = T < num_sms() * 4 && H > 512;
    const int lay = row_layout(vec, H), lanes = unit_lanes(H, lay);
    const CombineBwd a = {d_grad_y, d_ys, ldgy, ldys, d_slots, d_probs, T, k, H, R, lanes, d_grad_ys, ldgys, d_grad_probs,
                          d_status};
    const int64_t blocks = wide ? T : ((int64_t)T * lanes + 255) / 256;
    return with_type(dtype, [&](auto t) {
        using X = decltype(t);
        return with_layout(lay, [&](auto l) {
            constexpr int LAY = decltype(l)::value;
            return with_choices(k, [&](auto kk) {
                constexpr int K = decltype(kk)::value;
                auto kern = combine_bwd_kernel<X, LAY, K, 1>;
                if constexpr (LAY != kFewLanes)
                    if (wide) kern = combine_bwd_kernel<X, LAY, K, 8>;
                return check_launch_pdl(launch_pdl(kern, dim3(grid_blocks(blocks, (const void*)kern)), dim3(256), 0,
                                                   as_stream(stream), a),
                                        "combine_bwd_kernel");
            });
        });
    });
}
