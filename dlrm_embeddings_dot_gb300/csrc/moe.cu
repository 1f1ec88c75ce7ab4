// moe.cu -- a mixture-of-experts layer for a few tokens in two kernels.
//
// Bound by the touched experts' weights, each read once from HBM.  A weight goes
// by TMA into shared memory and from there into the fragments of one warp: each
// of 8 warps has a ring of two stages of 8 KB that it asks for itself, on into its
// next units, so that 128 KB an SM are on the way without a register (weights
// loaded straight into registers, two blocks of 8 warps with 128 of them, reached
// 3.2 TB/s).  A box is 16 rows by 256 or 512 bytes (TMA takes rows at a fixed
// rate: rows of 64 bytes brought 3.2 TB/s at most); lane (g, t) = (lane / 4,
// lane % 4) reads chunk t of row g of a 64-byte step, a two-way bank conflict that
// is hidden behind HBM, and takes the same 16 bytes of its token.
//
//   moe_up    routing and the first product.  Every cluster of four blocks
//             computes the router's logits for itself (each block a quarter
//             of H, the partial sums exchanged through distributed shared
//             memory), so no block waits for another cluster; each block
//             then picks the top k, lists the tokens of each chosen expert and
//             takes its share of the (expert, 16 rows) units.  A unit's K is
//             split over G warps, whose partial tiles meet in shared memory;
//             probs * a(.) goes to the workspace.
//   moe_down  a cluster owns 16 rows of the output: its warps share out the
//             (expert, run of I) items of all chosen experts, each warp adding
//             its items into its own per-token sums in shared memory, and the
//             warps' and blocks' sums are added in a fixed order.  No atomics on
//             floats, no partial outputs in HBM.
#include "few_rows.cuh"
#include "memo.h"
#include "moe_layout.h"
#include "tcgen05.cuh"

namespace dlrm {
namespace {

using namespace few;
using moe::kRing, moe::kStage, moe::kStages, moe::kSteps, moe::kThreads, moe::kWarps;
static_assert(moe::kRows == few::kRows && moe::kPitch == few::kPitch);

constexpr int kUpCluster = 4, kMaxSplit = 8;   // blocks of a cluster in moe_up, at most in moe_down
constexpr int64_t kOwnRouter = 32 << 10;
// Weights past this leave L2 first (half of L2: less may stay there from call to
// call).  Streaming 805 MB so took 160 us instead of 181: the tokens, the
// intermediate rows and the code itself stay in L2.
constexpr int64_t kOnce = 64 << 20;
constexpr int kMaxE = DLRM_MOE_MAX_EXPERTS, kMaxK = DLRM_MOE_MAX_TOP_K;
constexpr int kGroup = 32;                     // tokens of an expert that are multiplied together
constexpr int kMaxGroups = kMaxTokens * kMaxK / kGroup + kMaxE;

template <typename T>
constexpr int kQ = 16 / (int)sizeof(T);        // values of a lane's chunk
template <typename T>
constexpr int kStepK = 4 * kQ<T>;              // K of a step

// probs * h enters the second product with 22 bits or more: the products of the
// weights with further fragments are free beside the weights' traffic, and y then
// has one rounding, its own.
//   fp32  as it is
//   bf16  as the sum of three values (split1)
//   fp16  as the sum of two, divided by a power of two, so that none overflows and none
//         is lost below 2^-14, whatever the size of the activations.  Each run of 16
//         values of a token (a unit's rows) has its own: 2^kPower where the run's
//         largest is in [2^kPowerLow, 2^kPowerHigh) (no fewer than 21 bits of it), as
//         activations mostly are, else what brings that into [2^14, 2^15).  Where
//         all are 2^kPower moe_down has no more to do than to multiply its sums.
//         Otherwise it brings the runs of an item to the largest power among them
//         (times 1 or less) before the products (48 tokens, 64 experts, 182 us where
//         that took 172).
template <typename T>
constexpr int kTerms = std::is_same_v<T, float> ? 1 : std::is_same_v<T, bf16> ? 3 : 2;
template <typename T>
constexpr bool kScaled = std::is_same_v<T, __half>;
constexpr int kPower = -11, kPowerLow = -15, kPowerHigh = 4;
constexpr int kLeastPower = -80, kMostPower = 113;   // of the others (values below 2^-66 are nothing to any fp16 y)
constexpr int kMaxUpBlocks = kThreads;               // blocks of moe_up: a thread of moe_down reads one's report

struct MoeArgs {
    const void *x, *wr, *w1, *w2, *res;
    int64_t ldx, ldr, ldy;
    int T, H, I, E, k, act, gated, group;   // group: warps that share a unit of moe_up
    int chunk;                              // values of I in an item of moe_down
    void* y;
    int32_t* ids;
    float* probs;
    void* h;                                // [kTerms][T][k][I]
    uint8_t* other;                         // fp16: [up_blocks]: 1 where a block had runs of another power than kPower
    int8_t* powers;                         // fp16: [T][k][runs of 16 in I]: what their values were divided by, log2
    int up_blocks;
    uint32_t* status;
    long long wait_cycles;
    int once;                               // the weights are more than L2 keeps from call to call
};

// Which tokens chose which expert, in shared memory.
struct Lists {
    unsigned long long mask[kMaxE];        // bit t: token t chose the expert
    uint16_t entry[kMaxTokens * kMaxK];    // per expert, its tokens ascending: token * kMaxK + slot
    uint16_t first[kMaxE];                 // an expert's first entry
    uint16_t active[kMaxGroups];           // the chosen experts, ascending: expert + kMaxE * (group of tokens)
    int n_active;
};

// One entry of `active`.
struct Choice {
    int e, n;                // the expert, and how many tokens
    const uint16_t* entry;   // theirs
};

__device__ __forceinline__ Choice choice(const Lists& l, int i)
{
    const int e = l.active[i] % kMaxE, grp = l.active[i] / kMaxE;
    return {e, min(kGroup, __popcll(l.mask[e]) - grp * kGroup), l.entry + l.first[e] + grp * kGroup};
}

// Builds the lists from id(t, j) (all threads of the block; the masks are zero).
// The last entries are in place after the caller's next __syncthreads.
template <typename Id>
__device__ __forceinline__ void build_lists(Lists& l, int T, int k, int E, Id&& id)
{
    for (int i = threadIdx.x; i < T * kMaxK; i += kThreads)
        if (i % kMaxK < k) atomicOr(&l.mask[id(i / kMaxK, i % kMaxK)], 1ull << (i / kMaxK));
    __syncthreads();
    if (threadIdx.x < kWarp) {
        const int lane = threadIdx.x, per = (E + kWarp - 1) / kWarp, e0 = lane * per, e1 = min(E, e0 + per);
        int n = 0, used = 0;
        for (int e = e0; e < e1; ++e) {
            const int c = __popcll(l.mask[e]);
            n += c;
            used += (c + kGroup - 1) / kGroup;
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
        for (int e = e0; e < e1; ++e) {
            const int c = __popcll(l.mask[e]);
            l.first[e] = (uint16_t)n0;
            for (int grp = 0; grp * kGroup < c; ++grp) l.active[u0++] = (uint16_t)(e + kMaxE * grp);
            n0 += c;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < T * kMaxK; i += kThreads) {
        const int t = i / kMaxK, j = i % kMaxK;
        if (j >= k) continue;
        const int e = id(t, j);
        l.entry[l.first[e] + __popcll(l.mask[e] & ((1ull << t) - 1))] = (uint16_t)(t * kMaxK + j);
    }
}

// Order of the logits as integers: NaN above all, -0 equal to 0.
__device__ __forceinline__ uint32_t logit_key(float v)
{
    if (v != v) return 0xffffffffu;
    const uint32_t b = __float_as_uint(v == 0.f ? 0.f : v);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// fn(std::integral_constant<int, NT>) with the least NT of 1, 2, 4 that covers n <= 32 tokens.
template <typename Fn>
__device__ __forceinline__ void with_group_tiles(int n, Fn&& fn)
{
    if (n <= 8) fn(std::integral_constant<int, 1>{});
    else if (n <= 16) fn(std::integral_constant<int, 2>{});
    else fn(std::integral_constant<int, 4>{});
}

__device__ __forceinline__ void group_sync(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

struct Rings {
    uint64_t full[kWarps * kStages];
    int abort_flag;
};

// Sets up the barriers; the caller synchronises.
__device__ __forceinline__ void init_rings(Rings& r)
{
    if (threadIdx.x == 0) {
        for (int i = 0; i < kWarps * kStages; ++i) tc::mbar_init(&r.full[i], 1);
        r.abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
}

// What a warp asks for: of items first, first + stride, ... below `items`, K from
// k0(item) to k1(item) of the WT tiles of 16 rows at row(item) and tile_rows
// further; a stage holds WT boxes of 16 rows by 512 / WT bytes.
template <typename T, int WT, typename Row, typename K0, typename K1>
struct Ring {
    const CUtensorMap* map;
    uint8_t* mem;
    uint64_t* full;
    volatile int* abort_flag;
    long long wait_cycles;
    int item, stride, items, tile_rows;
    Row row;
    K0 k0;
    K1 k1;
    int k, end, at;
    uint32_t asked, taken;
    uint64_t policy;   // 0: none

    __device__ __forceinline__ void start()
    {
        asked = taken = 0;
        if (item < items) enter();
        for (int i = 0; i < kStages; ++i) ask();
    }
    __device__ __forceinline__ void enter()
    {
        k = k0(item);
        end = k1(item);
        at = row(item);
        if (k >= end) items = 0;   // the warp's share of K is empty
    }
    __device__ __forceinline__ void ask()
    {
        // after a wait gave up a stage may be asked for already: no barrier takes two requests
        if (item >= items || *abort_flag) return;
        const uint32_t s = asked++ % kStages;
        if (threadIdx.x % kWarp == 0) {
            tc::mbar_expect_tx(&full[s], kStage);
#pragma unroll
            for (int i = 0; i < WT; ++i) {
                uint8_t* dst = mem + s * kStage + i * (kStage / WT);
                if (policy) tc::tma_load_2d_hint(dst, map, k, at + i * tile_rows, &full[s], policy);
                else tc::tma_load_2d(dst, map, k, at + i * tile_rows, &full[s]);
            }
        }
        k += kSteps / WT * kStepK<T>;
        if (k >= end) {
            item += stride;
            if (item < items) enter();
        }
    }
    __device__ __forceinline__ const uint8_t* take()
    {
        const uint32_t s = taken % kStages;
        tc::mbar_wait(&full[s], (taken / kStages) & 1u, abort_flag, wait_cycles);
        __syncwarp();
        return mem + s * kStage;
    }
    // The taken stage has been read: ask for another in its place.
    __device__ __forceinline__ void give_back()
    {
        __syncwarp();
        ++taken;
        ask();
    }
    // Reports a wait that gave up; every copy has then landed (or was waited for).
    __device__ __forceinline__ void finish(uint32_t* status)
    {
        if (threadIdx.x % kWarp == 0 && *abort_flag) {
            for (uint32_t i = asked > kStages ? asked - kStages : 0; i < asked; ++i)
                tc::mbar_drain(&full[i % kStages], (i / kStages) & 1u);
            set_status(status, DLRM_STATUS_TIMEOUT);
        }
        __syncwarp();
    }
};

template <typename T, int WT, typename Row, typename K0, typename K1>
__device__ __forceinline__ Ring<T, WT, Row, K0, K1> make_ring(Rings& r, uint8_t* rings, const CUtensorMap* map,
                                                              const MoeArgs& a, int first, int stride, int items,
                                                              int tile_rows, Row row, K0 k0, K1 k1)
{
    const int warp = threadIdx.x / kWarp;
    return {map,  rings + warp * kStages * kStage, r.full + warp * kStages, &r.abort_flag, a.wait_cycles, first, stride, items,
            tile_rows, row, k0, k1, 0, 0, 0, 0, 0, a.once ? tc::l2_evict_first() : 0};
}

__device__ __forceinline__ uint8_t* shared_area(uint8_t* raw)
{
    return reinterpret_cast<uint8_t*>(moe::area(reinterpret_cast<uintptr_t>(raw)));
}

// fp16's runs of one item where not all have the same power, for the lane's token 8 j + g of each j.
template <int NT>
struct RunScale {
    const int8_t* at[NT];   // the runs' powers from the item's first value on
    int top[NT];            // their largest

    // powers(token): the powers of a token's row
    template <typename Powers>
    __device__ __forceinline__ void load(Powers&& powers, int n, int k0, int k1)
    {
        const int lane = threadIdx.x % kWarp, g = lane / 4, t = lane % 4;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            at[j] = powers(min(j * 8 + g, n - 1)) + k0 / kRows;
            int m = kLeastPower;
            for (int i = t; k0 + i * kRows < k1; i += 4) m = max(m, (int)__ldg(at[j] + i));
            m = max(m, __shfl_xor_sync(~0u, m, 1));
            top[j] = max(m, __shfl_xor_sync(~0u, m, 2));
        }
    }
    // What a run is multiplied with, twice in a word: 2^(power - top).
    __device__ __forceinline__ uint32_t factor(int j, int power) const
    {
        const int d = power - top[j];
        return (d >= -14 ? (uint32_t)(15 + d) << 10 : d >= -24 ? 1u << (24 + d) : 0u) * 0x10001u;
    }
    static __device__ __forceinline__ void apply(uint4& v, uint32_t f)
    {
        __half2 h[4], s;
        memcpy(h, &v, 16);
        memcpy(&s, &f, 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __hmul2(h[i], s);
        memcpy(&v, h, 16);
    }
    // The sums of tokens 8 j + 2 t and 8 j + 2 t + 1 are to be multiplied with these (all lanes).
    __device__ __forceinline__ float2 of_sums(int j) const
    {
        const int t = threadIdx.x % 4;
        const int a = __shfl_sync(~0u, top[j], 8 * t), b = __shfl_sync(~0u, top[j], 8 * t + 4);
        return make_float2(__int_as_float((a + 127) << 23), __int_as_float((b + 127) << 23));
    }
};

__device__ __forceinline__ uint4 lds16(const uint8_t* p) { return *reinterpret_cast<const uint4*>(p); }

// The sums of WT tiles of 16 weight rows with tokens [0, n) over [k0, k1) of K
// (k0 a multiple of a stage's), the weights taken from the ring stage by stage.
// out(i, token, row, value) gets every sum (zero for an empty range).  token(j):
// the row of token j; its values past K are not read, and the boxes hold zeros
// there.  SCALED: powers(j) has the powers of two of its runs.
struct NoPowers {
};
template <typename T, int WT, int XP, typename R, typename Token, typename Out, typename Powers = NoPowers>
__device__ __forceinline__ void ring_times_tokens(R& ring, Token&& token, int n, int k0, int k1, int K, int64_t xplane,
                                                  Out&& out, Powers&& powers = Powers())
{
    constexpr bool SCALED = !std::is_same_v<std::decay_t<Powers>, NoPowers>;
    constexpr int ST = kSteps / WT, kRow = ST * 64;   // steps in a stage, bytes of a row in a box
    const int lane = threadIdx.x % kWarp, g = lane / 4, t = lane % 4;
    // mul(x, w, ahead): the products of one step of each tile (row g at w) with the tokens'
    // chunks x[N]; at(j): where token chunk j begins; also(d, k): anything else to load
    // for the step that begins at k.  The chunks of the next D
    // steps are on their way while one step is multiplied; no more than D steps are
    // unrolled, because a block runs this code for a few units only and has to
    // fetch every instruction of it.
    auto run = [&](auto nn, auto dd, auto&& at, auto&& also, auto&& mul) {
        constexpr int N = decltype(nn)::value, D = decltype(dd)::value;
        const T* x[N];
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] = at(j) + k0 + t * kQ<T>;
        int left = K - k0 - t * kQ<T>;   // of the token's row, from this step's chunk on
        uint4 b[D][N];
        auto fetch = [&](uint4 (&c)[N], int ahead) {
#pragma unroll
            for (int j = 0; j < N; ++j)
                c[j] = left > ahead * kStepK<T> ? ldg_nc_l1_v4(x[j] + ahead * kStepK<T>) : make_uint4(0, 0, 0, 0);
        };
#pragma unroll
        for (int d = 0; d < D; ++d) {
            fetch(b[d], d);
            also(d, k0 + d * kStepK<T>);
        }
        const uint8_t* w = nullptr;
        int in = 0;   // steps left in the stage
#pragma unroll 1
        for (int k = k0; k < k1; k += D * kStepK<T>) {
            if (in == 0) {
                w = ring.take() + g * kRow + t * 16;
                in = ST;
            }
#pragma unroll
            for (int d = 0; d < D; ++d) {
                mul(b[d], w + d * 64, d);
                fetch(b[d], D + d);
                also(d, k + (D + d) * kStepK<T>);
            }
#pragma unroll
            for (int j = 0; j < N; ++j) x[j] += D * kStepK<T>;
            left -= D * kStepK<T>;
            w += D * 64;
            in -= D;
            if (in == 0 || k + D * kStepK<T> >= k1) {
                in = 0;
                ring.give_back();
            }
        }
    };
    if (std::is_same_v<T, float> && n <= 8) {
        // fp32, few tokens: fp32 products; a lane has all the tokens for its share of K
        auto with = [&](auto nn) {
            constexpr int NX = decltype(nn)::value;
            float acc[WT][NX][2] = {};
            run(nn, std::integral_constant<int, NX <= 2 ? 4 : 2>{}, [&](int j) { return token(min(j, n - 1)); },
                [](int, int) {},
                [&](uint4 (&x)[NX], const uint8_t* w, int) {
#pragma unroll
                    for (int i = 0; i < WT; ++i)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float4 a = u4_as_f4(lds16(w + i * (kStage / WT) + h * (8 * kRow)));
#pragma unroll
                            for (int j = 0; j < NX; ++j) {
                                const float4 v = u4_as_f4(x[j]);
                                float& d = acc[i][j][h];
                                d = fmaf(a.x, v.x, d);
                                d = fmaf(a.y, v.y, d);
                                d = fmaf(a.z, v.z, d);
                                d = fmaf(a.w, v.w, d);
                            }
                        }
                });
#pragma unroll
            for (int i = 0; i < WT; ++i)
#pragma unroll
                for (int j = 0; j < NX; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float v = acc[i][j][h];   // the four lanes of a row add up their shares
                        v += __shfl_xor_sync(~0u, v, 1);
                        v += __shfl_xor_sync(~0u, v, 2);
                        if (t == 0 && j < n) out(i, j, g + 8 * h, v);
                    }
        };
        if (n <= 2) with(std::integral_constant<int, 2>{});
        else if (n <= 4) with(std::integral_constant<int, 4>{});
        else with(std::integral_constant<int, 8>{});
    } else {
        auto with = [&](auto nn) {
            constexpr int NT = decltype(nn)::value, D = NT * XP <= 3 ? 4 : 2;
            float acc[WT][NT][4] = {};
            RunScale<NT> scale;
            if constexpr (SCALED) scale.load(powers, n, k0, k1);
            int power[D][NT];
            run(std::integral_constant<int, NT * XP>{}, std::integral_constant<int, D>{},
                [&](int j) { return token(min(j / XP * 8 + g, n - 1)) + j % XP * xplane; },
                [&](int d, int k) {
                    if constexpr (SCALED) {
                        const int c = k + t * kQ<T>;   // the lane's chunk lies within one run
#pragma unroll
                        for (int j = 0; j < NT; ++j)
                            power[d][j] = c < k1 ? __ldg(scale.at[j] + (c - k0) / kRows) : kLeastPower;
                    }
                },
                [&](uint4 (&x)[NT * XP], const uint8_t* w, int d) {
                    if constexpr (SCALED) {
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            const uint32_t f = scale.factor(j, power[d][j]);
#pragma unroll
                            for (int q = 0; q < XP; ++q) scale.apply(x[j * XP + q], f);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < WT; ++i) {
                        const uint4 lo = lds16(w + i * (kStage / WT)), hi = lds16(w + i * (kStage / WT) + 8 * kRow);
#pragma unroll
                        for (int j = 0; j < NT * XP; ++j) mac16<T>(acc[i][j / XP], lo, hi, x[j]);
                    }
                });
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                float2 f = make_float2(1.f, 1.f);
                if constexpr (SCALED) f = scale.of_sums(j);
#pragma unroll
                for (int i = 0; i < WT; ++i)
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                        const int tok = j * 8 + 2 * t + (d & 1);
                        if (tok < n) out(i, tok, g + 8 * (d >> 1), acc[i][j][d] * (d & 1 ? f.y : f.x));
                    }
            }
        };
        if constexpr (std::is_same_v<T, float>) {
            if (n <= 16) with(std::integral_constant<int, 2>{});
            else with(std::integral_constant<int, 4>{});
        } else {
            with_group_tiles(n, with);
        }
    }
}

// 16 experts' logits of n <= 8 NT tokens over [k0, k1) of H.  Short loops: a block
// runs this once, and what takes its time is fetching the code.
template <typename T, int NT, bool VEC, typename Token, typename Out>
__device__ __forceinline__ void router_tile(const T* w0, const T* w8, Token&& token, int n, int k0, int k1, Out&& out)
{
    const int lane = threadIdx.x % kWarp, g = lane / 4, t = lane % 4;
    const T* x[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) x[j] = token(min(j * 8 + g, n - 1));
    auto chunk = [&](const T* p, int at) {
        if constexpr (VEC) {
            return at < k1 ? ldg_nc_l1_v4(p + at) : make_uint4(0, 0, 0, 0);
        } else {
            T e[kQ<T>];
#pragma unroll
            for (int i = 0; i < kQ<T>; ++i) e[i] = at + i < k1 ? __ldg(p + at + i) : from_f32<T>(0.f);
            uint4 v;
            memcpy(&v, e, 16);
            return v;
        }
    };
    float acc[NT][4] = {};
#pragma unroll 1
    for (int at = k0 + t * kQ<T>; at - t * kQ<T> < k1; at += kStepK<T>) {
        const uint4 lo = chunk(w0, at), hi = chunk(w8, at);
        uint4 b[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) b[j] = chunk(x[j], at);
#pragma unroll
        for (int j = 0; j < NT; ++j) mac16<T>(acc[j], lo, hi, b[j]);
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const int tok = j * 8 + 2 * t + (d & 1);
            if (tok < n) out(tok, g + 8 * (d >> 1), acc[j][d]);
        }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads, 1) moe_up_kernel(const __grid_constant__ CUtensorMap map, MoeArgs a)
{
    extern __shared__ uint8_t raw[];
    uint8_t* rings = shared_area(raw);
    float* smem = reinterpret_cast<float*>(rings);
    __shared__ Lists lists;
    __shared__ uint8_t ids_s[kMaxTokens * kMaxK];
    __shared__ uint32_t keys_s[kWarps][kMaxE];
    __shared__ float probs_s[kMaxTokens * kMaxK];
    __shared__ Rings sync;
    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp, g = lane / 4;
    const T *x = (const T*)a.x, *wr = (const T*)a.wr, *w1 = (const T*)a.w1;
    init_rings(sync);
    for (int e = threadIdx.x; e < a.E; e += kThreads) lists.mask[e] = 0;
    pdl_wait();

    // ---- the router's logits: this block's share of H
    const int e_tiles = moe::expert_tiles(a.E), E16 = e_tiles * kRows;
    const int sub = moe::router_split(a.E);
    const int C = (int)cluster_size(), rank = (int)cluster_rank();
    float* lp = smem;                        // [sub][T][E16]: partial logits
    float* lg = smem + sub * a.T * E16;      // [T][E16]: logits
    {
        const int steps = (a.H + kStepK<T> - 1) / kStepK<T>;
        const int per = (steps + C * sub - 1) / (C * sub) * kStepK<T>;
        for (int i = warp; i < e_tiles * sub; i += kWarps) {
            const int tile = i % e_tiles, s = i / e_tiles;
            const int k0 = (rank * sub + s) * per, k1 = min(a.H, k0 + per);
            const T* w0 = wr + (int64_t)min(tile * kRows + g, a.E - 1) * a.H;
            const T* w8 = wr + (int64_t)min(tile * kRows + g + 8, a.E - 1) * a.H;
            for (int t0 = 0; t0 < a.T; t0 += kGroup) {
                const int n = min(kGroup, a.T - t0);
                with_group_tiles(n, [&](auto nt) {
                    router_tile<T, decltype(nt)::value, VEC>(
                        w0, w8, [&](int t) { return x + (t0 + t) * a.ldx; }, n, k0, k1,
                        [&](int t, int r, float v) { lp[(s * a.T + t0 + t) * E16 + tile * kRows + r] = v; });
                });
            }
        }
        __syncthreads();
        float* own = C > 1 ? lp : lg;   // the block's own sums first: what is read across the cluster is read once
        for (int i = threadIdx.x; i < a.T * E16; i += kThreads) {
            float v = lp[i];
            for (int s = 1; s < sub; ++s) v += lp[s * a.T * E16 + i];
            own[i] = v;
        }
        if (C > 1) {
            cluster_sync();
            // block r adds up every C-th logit and hands it to all
            for (int i = threadIdx.x * C + rank; i < a.T * E16; i += kThreads * C) {
                float v[kUpCluster];
#pragma unroll
                for (int r = 0; r < kUpCluster; ++r) v[r] = cluster_ld(cluster_map(lp + i, r));
#pragma unroll
                for (int r = 1; r < kUpCluster; ++r) v[0] += v[r];
#pragma unroll
                for (int r = 0; r < kUpCluster; ++r) cluster_st(cluster_map(lg + i, r), v[0]);
            }
            cluster_sync();
        } else {
            __syncthreads();
        }
    }

    // ---- top k and its softmax, a warp per token
    uint32_t* keys = keys_s[warp];
    for (int t = warp; t < a.T; t += kWarps) {
        for (int e = lane; e < a.E; e += kWarp) keys[e] = logit_key(lg[t * E16 + e]);
        float top = 0.f, mine = 0.f;
        int best = 0;
#pragma unroll 1
        for (int j = 0; j < a.k; ++j) {
            uint32_t m = 0, at = kMaxE;    // a lane's largest key and its lowest expert (no logit's key is 0)
#pragma unroll 1
            for (int e = lane; e < a.E; e += kWarp)
                if (keys[e] > m) m = keys[e], at = e;
            const uint32_t most = __reduce_max_sync(~0u, m);
            const int e = (int)__reduce_min_sync(~0u, m == most ? at : kMaxE);
            if (e % kWarp == lane) keys[e] = 0;
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
    const int tiles = (a.I + kRows - 1) / kRows, units = lists.n_active * tiles, stride = gridDim.x * groups;
    const int WT = a.gated ? 2 : 1, stage_k = kSteps / WT * kStepK<T>;
    const int per = ((a.H + stage_k - 1) / stage_k + G - 1) / G * stage_k;
    const int k0 = wg * per, k1 = min(a.H, k0 + per);
    const int tile_floats = moe::token_tiles(a.T) * 8 * kPitch;
    float* red = reinterpret_cast<float*>(rings + (VEC ? kRing : 0));   // [warp][2][token][kPitch]
    T* h = (T*)a.h;
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the rings were the logits' memory
    __syncthreads();
    bool other = false;   // fp16: a run had another power than kPower
    // One unit: products(put) brings the warp's partial sums, which meet in shared memory.
    auto unit = [&](const Choice& c, int row0, auto&& products) {
        products([&](int i, int tok, int r, float v) { red[(warp * 2 + i) * tile_floats + tok * kPitch + r] = v; });
        group_sync(1 + mine, G * kWarp);
        for (int i0 = wg * kWarp; i0 < c.n * kRows; i0 += G * kWarp) {   // a token's 16 rows are 16 neighbouring lanes'
            const int tok = min((i0 + lane) / kRows, c.n - 1), r = lane % kRows;
            const bool token = i0 + lane < c.n * kRows, in = token && row0 + r < a.I;
            const float* p = red + (mine * G * 2) * tile_floats + tok * kPitch + r;
            float z = 0.f, up = 0.f;
            for (int q = 0; q < G; ++q) {
                z += p[q * 2 * tile_floats];
                if (a.gated) up += p[(q * 2 + 1) * tile_floats];
            }
            const int slot = c.entry[tok];
            float v = act_f<T>(z, a.act);
            if (a.gated) v *= up;
            v *= probs_s[slot];
            const int64_t row = (int64_t)(slot / kMaxK) * a.k + slot % kMaxK, plane = (int64_t)a.T * a.k * a.I;
            T* dst = h + row * a.I + row0 + r;
            if constexpr (kScaled<T>) {
                float m = in ? fabsf(v) : 0.f;   // a NaN stays one whatever the power
#pragma unroll
                for (int d = 8; d; d /= 2) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
                const int e = (int)(__float_as_uint(m) >> 23) - 127;
                const bool usual = e >= kPowerLow && e < kPowerHigh;
                const int power = usual ? kPower : min(max(e - 14, kLeastPower), kMostPower);
                other |= token && !usual && m != 0.f;   // (a run of zeros goes with any power)
                if (token && r == 0) a.powers[row * tiles + row0 / kRows] = (int8_t)power;
                v *= __int_as_float((127 - power) << 23);
                const T top = from_f32<T>(v);
                const float rest = v - to_f32(top);   // NaN for an infinite v: its rest is zero
                if (in) {
                    dst[0] = top;
                    dst[plane] = from_f32<T>(fabsf(to_f32(top)) <= 65504.f ? rest : 0.f);
                }
            } else if constexpr (kTerms<T> == 3) {
                uint32_t hi, mid;
                float lo;
                split1(v, hi, mid, lo);
                if (in) {
                    dst[0] = from_f32<T>(__uint_as_float(hi));
                    dst[plane] = from_f32<T>(__uint_as_float(mid));
                    dst[2 * plane] = from_f32<T>(lo);
                }
            } else if (in) {
                dst[0] = v;
            }
        }
        group_sync(1 + mine, G * kWarp);
    };
    const int first = blockIdx.x * groups + mine;
    if constexpr (VEC) {
        auto all = [&](auto wt) {
            constexpr int W = decltype(wt)::value;
            auto ring = make_ring<T, W>(
                sync, rings, &map, a, first, stride, units, a.I,
                [&](int u) { return (lists.active[u / tiles] % kMaxE) * W * a.I + u % tiles * kRows; }, [&](int) { return k0; },
                [&](int) { return k1; });
            ring.start();
            for (int u = first; u < units; u += stride) {
                const Choice c = choice(lists, u / tiles);
                unit(c, u % tiles * kRows, [&](auto&& put) {
                    ring_times_tokens<T, W, 1>(
                        ring, [&](int i) { return x + (int64_t)(c.entry[i] / kMaxK) * a.ldx; }, c.n, k0, k1, a.H, 0, put);
                });
            }
            ring.finish(a.status);
        };
        if (a.gated) all(std::integral_constant<int, 2>{});
        else all(std::integral_constant<int, 1>{});
    } else {
        for (int u = first; u < units; u += stride) {
            const Choice c = choice(lists, u / tiles);
            const int row0 = u % tiles * kRows;
            unit(c, row0, [&](auto&& put) {
                for (int i = 0; i < WT; ++i) {
                    const T* base = w1 + ((int64_t)c.e * WT * a.I + (int64_t)i * a.I) * a.H;
                    const T* w[1][2] = {{base + (int64_t)min(row0 + g, a.I - 1) * a.H,
                                         base + (int64_t)min(row0 + g + 8, a.I - 1) * a.H}};
                    with_group_tiles(c.n, [&](auto nt) {
                        rows_times_tokens<T, 1, decltype(nt)::value, 0>(
                            w, [&](int t) { return x + (int64_t)(c.entry[t] / kMaxK) * a.ldx; }, c.n, k0, k1, 0,
                            [&](int, int tok, int r, float v) { put(i, tok, r, v); });
                    });
                }
            });
        }
    }
    if constexpr (kScaled<T>) {
        other = __syncthreads_or(other);
        if (threadIdx.x == 0) a.other[blockIdx.x] = other;
    }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads, 1) moe_down_kernel(const __grid_constant__ CUtensorMap map, MoeArgs a)
{
    extern __shared__ uint8_t raw[];
    uint8_t* rings = shared_area(raw);
    float* smem = reinterpret_cast<float*>(rings + (VEC ? kRing : 0));   // [warp][token][kPitch]: each warp's sums
    __shared__ Lists lists;
    __shared__ Rings sync;
    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp, g = lane / 4;
    const int S = (int)cluster_size(), rank = (int)cluster_rank();
    const int row0 = (int)(blockIdx.x / S) * kRows;
    init_rings(sync);
    for (int e = threadIdx.x; e < a.E; e += kThreads) lists.mask[e] = 0;
    for (int i = threadIdx.x; i < kWarps * a.T * kPitch; i += kThreads) smem[i] = 0.f;
    __syncthreads();
    pdl_wait();
    uint8_t other = 0;
    if constexpr (kScaled<T>)
        if (threadIdx.x < a.up_blocks) other = __ldg(a.other + threadIdx.x);
    build_lists(lists, a.T, a.k, a.E, [&](int t, int j) { return a.ids[t * a.k + j]; });
    const bool scaled = __syncthreads_or(other != 0);   // fp16: the runs' powers differ

    const int chunks = (a.I + a.chunk - 1) / a.chunk, items = lists.n_active * chunks, stride = S * kWarps;
    const T *w2 = (const T*)a.w2, *h = (const T*)a.h;
    const int first = rank * kWarps + warp;
    float* mine = smem + warp * a.T * kPitch;
    const int64_t plane = (int64_t)a.T * a.k * a.I;
    auto k0 = [&](int i) { return i % chunks * a.chunk; };
    auto k1 = [&](int i) { return min(a.I, i % chunks * a.chunk + a.chunk); };
    const int runs = (a.I + kRows - 1) / kRows;
    auto all = [&](auto&& products) {
        for (int it = first; it < items; it += stride) {
            const Choice c = choice(lists, it / chunks);
            auto row = [&](int i) { return (int64_t)(c.entry[i] / kMaxK) * a.k + c.entry[i] % kMaxK; };
            products(c, it, [&](int i) { return h + row(i) * a.I; }, [&](int i) { return a.powers + row(i) * runs; },
                     [&](int, int i, int r, float v) {
                         if constexpr (kScaled<T>) v = scaled ? v : v * (1.f / (1 << -kPower));
                         mine[c.entry[i] / kMaxK * kPitch + r] += v;
                     });
            __syncwarp();   // another item's token may be another lane's
        }
    };
    if constexpr (VEC) {
        auto ring = make_ring<T, 1>(sync, rings, &map, a, first, stride, items, 0,
                                    [&](int i) { return (lists.active[i / chunks] % kMaxE) * a.H + row0; }, k0, k1);
        ring.start();
        if (kScaled<T> && scaled)
            all([&](const Choice& c, int it, auto&& token, auto&& powers, auto&& add) {
                ring_times_tokens<T, 1, kTerms<T>>(ring, token, c.n, k0(it), k1(it), a.I, plane, add, powers);
            });
        else
            all([&](const Choice& c, int it, auto&& token, auto&& powers, auto&& add) {
                ring_times_tokens<T, 1, kTerms<T>>(ring, token, c.n, k0(it), k1(it), a.I, plane, add);
            });
        ring.finish(a.status);
    } else {
        all([&](const Choice& c, int it, auto&& token, auto&& powers, auto&& add) {
            const T* base = w2 + (int64_t)c.e * a.H * a.I;
            const T* w[1][2] = {{base + (int64_t)min(row0 + g, a.H - 1) * a.I,
                                 base + (int64_t)min(row0 + g + 8, a.H - 1) * a.I}};
            with_group_tiles(c.n, [&](auto nt) {
                constexpr int NT = decltype(nt)::value;
                if (kScaled<T> && scaled) {
                    RunScale<NT> scale;
                    scale.load(powers, c.n, k0(it), k1(it));
                    float2 f[NT];
#pragma unroll
                    for (int j = 0; j < NT; ++j) f[j] = scale.of_sums(j);
                    rows_times_tokens<T, 1, NT, 0, kTerms<T>>(
                        w, token, c.n, k0(it), k1(it), plane,
                        [&](int i, int tok, int r, float v) {
                            float2 s = f[0];
#pragma unroll
                            for (int j = 1; j < NT; ++j)
                                if (tok / 8 == j) s = f[j];
                            add(i, tok, r, v * (tok & 1 ? s.y : s.x));
                        },
                        [&](int j, int k, Chunk& x) {   // k: of the lane's 16 values, one run, from the item's first on
                            const uint32_t s = scale.factor(j, k + k0(it) < k1(it) ? __ldg(scale.at[j] + k / kRows) : kLeastPower);
                            scale.apply(x.v[0], s);
                            scale.apply(x.v[1], s);
                        });
                } else {
                    rows_times_tokens<T, 1, NT, 0, kTerms<T>>(w, token, c.n, k0(it), k1(it), plane, add);
                }
            });
        });
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

// Blocks of a kernel that run at the same time in clusters of `cluster`.
template <typename K>
int resident_blocks(K kern, size_t smem, int cluster)
{
    const int one_each = num_sms() / cluster * cluster;
    if (cluster == 1) return one_each;
    int dev = 0;
    cudaGetDevice(&dev);
    static KernelMemo memo;   // one for all kernels of the type K: the key says which
    return memo.get({reinterpret_cast<const void*>(kern), dev, cluster, smem}, [&] {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = cluster;
        cfg.blockDim = kThreads;
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = cluster;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) == cudaSuccess && n > 0) return n * cluster;
        cudaGetLastError();
        return one_each;
    });
}

// Boxes of 16 rows by `steps` steps of a [rows][cols] matrix of weights.
template <typename T>
dlrm_status weight_map(CUtensorMap* m, const void* p, int64_t rows, int cols, int steps)
{
    tc::EncodeTiledFn enc = tc::encode_fn();
    if (!enc) return fail(DLRM_ERR_CUDA, "dlrm_moe_fwd: cuTensorMapEncodeTiled unavailable");
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, str[1] = {(cuuint64_t)cols * sizeof(T)};
    const cuuint32_t box[2] = {(cuuint32_t)(steps * kStepK<T>), kRows}, ones[2] = {1, 1};
    const CUtensorMapDataType type = std::is_same_v<T, float>    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                     : std::is_same_v<T, __half> ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                                 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const CUresult r = enc(m, type, 2, const_cast<void*>(p), dims, str, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(DLRM_ERR_CUDA, "dlrm_moe_fwd: tensor map (%d)", (int)r);
    return DLRM_OK;
}

template <typename T, bool VEC>
dlrm_status launch_moe(MoeArgs a, cudaStream_t st)
{
    CUtensorMap m1 = {}, m2 = {};
    dlrm_status s;
    if (VEC) {
        s = weight_map<T>(&m1, a.w1, (int64_t)a.E * (a.gated ? 2 : 1) * a.I, a.H, kSteps / (a.gated ? 2 : 1));
        if (s == DLRM_OK) s = weight_map<T>(&m2, a.w2, (int64_t)a.E * a.H, a.I, kSteps);
        if (s != DLRM_OK) return s;
    }
    const size_t smem = moe::asked(moe::up_used(a.T, a.E, VEC));
    auto up = moe_up_kernel<T, VEC>;
    cudaError_t e = cudaFuncSetAttribute(up, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return fail(DLRM_ERR_CUDA, "dlrm_moe_fwd: %s", cudaGetErrorString(e));
    // a cluster shares the router's product out; a router of a few kilobytes is read sooner by every block for itself
    const int C = (int64_t)a.E * a.H * (int64_t)sizeof(T) <= kOwnRouter ? 1 : kUpCluster;
    const int most = resident_blocks(up, smem, C);
    const int chosen = a.E < a.T * a.k ? a.E : a.T * a.k;            // experts at most
    const int64_t units = (int64_t)chosen * ((a.I + kRows - 1) / kRows);
    // warps of a unit: the number with the least time in stages, a unit's overhead
    // (its meeting in shared memory) being one
    const int stage_k = kSteps / (a.gated ? 2 : 1) * kStepK<T>;
    const int64_t stages = (a.H + stage_k - 1) / stage_k;
    int64_t least = 0;
    for (int G = kWarps; G >= 1; G /= 2) {
        const int64_t groups = (int64_t)most * kWarps / G, cost = (units + groups - 1) / groups * ((stages + G - 1) / G + 1);
        if (least == 0 || cost < least) {
            least = cost;
            a.group = G;
        }
    }
    int64_t blocks = (units * a.group + kWarps - 1) / kWarps;
    if (blocks > most) blocks = most;
    if (blocks > kMaxUpBlocks) blocks = kMaxUpBlocks;
    blocks = (blocks + C - 1) / C * C;   // C divides kMaxUpBlocks
    a.up_blocks = (int)blocks;
    e = launch_cluster(up, dim3((unsigned)blocks), dim3(kThreads), smem, st, C, m1, a);
    s = check_launch_pdl(e, "moe_up_kernel");
    if (s != DLRM_OK) return s;

    const int row_tiles = (a.H + kRows - 1) / kRows;
    const size_t down = moe::asked(moe::down_used(a.T, VEC));
    auto kern = moe_down_kernel<T, VEC>;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)down);
    if (e != cudaSuccess) return fail(DLRM_ERR_CUDA, "dlrm_moe_fwd: %s", cudaGetErrorString(e));
    // blocks that share 16 rows of the output: the number with the least time, in
    // nanoseconds (an SM's share of HBM is 45 bytes each; 2 us for a round of blocks)
    int S = 1;
    double best = 0;
    for (int c = 1; c <= kMaxSplit; c *= 2) {
        const int at_once = resident_blocks(kern, down, c);
        const double rounds = ((int64_t)row_tiles * c + at_once - 1) / at_once;
        const double cost = rounds * ((double)chosen * kRows * a.I * sizeof(T) / c / 45 + 2000) + (c > 1 ? 500 : 0);
        if (best == 0 || cost < best) {
            best = cost;
            S = c;
        }
    }
    // an item: as long as leaves every warp four
    const int down_k = kSteps * kStepK<T>;
    const int64_t share = (int64_t)chosen * a.I / (S * kWarps * 4) / down_k * down_k;
    a.chunk = share < down_k ? down_k : share > 8 * down_k ? 8 * down_k : (int)share;
    return check_launch_pdl(launch_cluster(kern, dim3(row_tiles * S), dim3(kThreads), down, st, S, m2, a),
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
    if (!moe_sizes_ok(dtype, T, H, I, E, k) || T == 0) return 0;
    // the terms of probs * h, and fp16's reports and powers of two
    const size_t bytes = dtype == DLRM_BF16 ? 6 : 4;
    return dlrm_ws_align((size_t)T * k * I * bytes +
                         (dtype == DLRM_F16 ? kMaxUpBlocks + (size_t)T * k * (((size_t)I + 15) / 16) : 0));
}

extern "C" dlrm_status dlrm_moe_fwd(const void* d_x, int64_t ldx, const void* d_w_router, const void* d_w1,
                                    const void* d_w2, const void* d_residual, int64_t ldr, dlrm_dtype dtype, int T,
                                    int H, int I, int E, int k, dlrm_act act, int gated, void* d_y, int64_t ldy,
                                    int32_t* d_ids, float* d_probs, void* d_workspace, size_t workspace_bytes,
                                    uint32_t* d_status, void* stream)
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
    if (H > kMaxSize || I > kMaxSize) return fail(DLRM_ERR_UNSUPPORTED, "%s: sizes up to %d", fn, kMaxSize);
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
    if ((int64_t)E * 2 * I > INT32_MAX || (int64_t)E * H > INT32_MAX)
        return fail(DLRM_ERR_UNSUPPORTED, "%s: more than 2^31 weight rows", fn);
    MoeArgs a = {};
    a.x = d_x, a.wr = d_w_router, a.w1 = d_w1, a.w2 = d_w2, a.res = d_residual;
    a.ldx = ldx, a.ldr = ldr, a.ldy = ldy;
    a.T = T, a.H = H, a.I = I, a.E = E, a.k = k, a.act = act, a.gated = gated != 0;
    a.y = d_y, a.ids = d_ids, a.probs = d_probs, a.h = d_workspace;
    a.other = (uint8_t*)d_workspace + (size_t)T * k * I * 4;
    a.powers = (int8_t*)a.other + kMaxUpBlocks;
    a.status = d_status, a.wait_cycles = wait_limit_cycles();
    a.once = (int64_t)E * (gated ? 3 : 2) * I * H * es > kOnce;
    // TMA and 16-byte loads where every row is on the grid (the workspace's are where I's are)
    const bool vec = rows_aligned16(d_x, ldx, T, es) && rows_aligned16(d_w_router, H, E, es) &&
                     rows_aligned16(d_w1, H, 2, es) && rows_aligned16(d_w2, I, 2, es) && H * es % 16 == 0 && I * es % 16 == 0;
    return with_type(dtype, [&](auto t) {
        using T_ = decltype(t);
        return vec ? launch_moe<T_, true>(a, as_stream(stream)) : launch_moe<T_, false>(a, as_stream(stream));
    });
}
