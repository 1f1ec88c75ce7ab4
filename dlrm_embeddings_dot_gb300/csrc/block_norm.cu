// block_norm.cu -- the norms after a block and before the next one, with the
// block's gate and residual scale:
//
//   u = norm(y) w_post + b_post;  r = residual + scale gate(g) u;  h = norm(r) w_pre + b_pre
//
// and its gradient.  Both are bound by memory: every matrix goes once, a row stays in
// registers between its sums.
//
// A row is taken by W warps, eight columns a lane, which holds its part of the vectors in
// registers.  The next rows are on their way meanwhile: a ring of rows in shared
// memory, each thread copying its own columns (cp.async), so that no thread waits for
// another's copies.  Sums of a row go by shuffles, then over its warps by shared memory.
//
//   forward    the statistics are taken in two passes over the registers (mean, then
//              squares about it)
//   backward   a lane also adds up its columns' sums over rows.  Blocks' sums go to `partial`
//              and block_norm_sum_kernel adds them in order
//
// Nothing here depends on which columns a lane has.  On the 16-byte grid they are eight
// neighbours.  Off it a warp copies the aligned 16-byte words that hold its 256 columns and a
// lane has every 32nd column, or pair of them, which shared memory gives without conflicts.
#include "dlrm_block.h"
#include "row_units.cuh"

namespace dlrm {
namespace {

// ------------------------------------------------------------- runs of a row
// The first column of a lane's run where a warp has 256 columns of a row; run_col has the others.
template <bool VEC, int ES>
__device__ __forceinline__ int run_first(int warp, int lane)
{
    return warp * 256 + lane * (VEC ? 16 / ES : ES == 2 ? 2 : 1);
}

// A tensor's row that a group of warps is at, stepped from one of its rows to the next.
template <typename T>
struct Cursor {
    const T *base, *row;
    int64_t inc;
    __device__ Cursor(const void* p, int64_t ld, int64_t row0, int64_t step)
        : base((const T*)p), row((const T*)p + row0 * ld), inc(step * ld)
    {
    }
    __device__ __forceinline__ const T* ahead(int rows) const { return row + rows * inc; }
    __device__ __forceinline__ T* out() const { return const_cast<T*>(row); }
    __device__ __forceinline__ void next() { row += inc; }
};

// The rows to come: kAhead rows of NT tensors, three where the blocks that share an SM (two of
// 256 threads, one of more) have the memory.  Columns past the row's end are 0.
template <int STAGE, int THREADS>
constexpr int kRowsAhead = (THREADS > 256 ? 224 << 10 : 110 << 10) / STAGE < 3 ? (THREADS > 256 ? 224 << 10 : 110 << 10) / STAGE : 3;

__device__ __forceinline__ void copy16(uint32_t to, const void* from, uint32_t bytes)   // the rest of the word becomes 0
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}

// On the grid: each thread copies and reads its own eight columns.
template <typename T, bool VEC, int NT, int THREADS>
struct Ring {
    static constexpr int kWords = sizeof(T) / 2, kSlot = kWords * THREADS * 16, kStage = NT * kSlot;
    static constexpr int kAhead = kRowsAhead<kStage, THREADS>;
    static_assert(kAhead >= 1, "a row fits");
    static constexpr size_t kBytes = (size_t)kAhead * kStage;
    uint8_t* mine;    // word 0 of slot 0 of stage 0
    uint32_t at;      // its shared address
    int N, first;

    __device__ Ring(uint8_t* smem, int n, int f, int) : mine(smem + threadIdx.x * 16), N(n), first(f)
    {
        at = (uint32_t)__cvta_generic_to_shared(mine);
        for (int i = 0; i < kAhead * NT * kWords; ++i)
            *reinterpret_cast<uint4*>(mine + i * THREADS * 16) = make_uint4(0, 0, 0, 0);
    }
    // Starts the copy of a tensor's row `rows` ahead to a slot.  inner: words that hold a part of the
    // row are in the matrix as a whole.
    __device__ __forceinline__ void fetch(int stage, int slot, const Cursor<T>& c, int rows, bool) const
    {
        const T* row = c.ahead(rows);
        const uint32_t to = at + stage * kStage + slot * kSlot;
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            if (first + i * 128 < N) copy16(to + i * THREADS * 16, row + first + i * 128, 16);
    }
    static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    // The oldest row's copies are complete.
    static __device__ __forceinline__ void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory"); }
    static __device__ __forceinline__ void done() {}
    __device__ __forceinline__ void read(int stage, int slot, const T*, float2 (&f)[4]) const
    {
        Raw8<T> r;
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            r.w[i] = *reinterpret_cast<const uint4*>(mine + stage * kStage + slot * kSlot + i * THREADS * 16);
        float v[8];
        widen8<T>(r, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = make_float2(v[2 * i], v[2 * i + 1]);
    }
};

// Off the grid: a warp's 256 columns lie in 16 ES + 1 aligned words at most, which its lanes copy.
// Near the matrix's ends the last word is cut there, and one that begins before the matrix is put
// together from its elements.
template <typename T, int NT, int THREADS>
struct Ring<T, false, NT, THREADS> {
    static constexpr int kES = sizeof(T), kWords = 16 * kES + 1, kSlot = THREADS / kWarp * kWords * 16, kStage = NT * kSlot;
    static constexpr int kAhead = kRowsAhead<kStage, THREADS>;
    static_assert(kAhead >= 1, "a row fits");
    static constexpr size_t kBytes = (size_t)kAhead * kStage;
    uint8_t* mine;    // the warp's word 0
    uint32_t at;
    int N, first, from, bytes;   // from: the warp's first column; bytes of its columns, 0 or less: none

    // f0: the row's warp's number times 256
    __device__ Ring(uint8_t* smem, int n, int f, int f0) : N(n), first(f), from(f0)
    {
        mine = smem + __shfl_sync(~0u, (int)threadIdx.x / kWarp, 0) * kWords * 16;
        at = (uint32_t)__cvta_generic_to_shared(mine);
        bytes = min(256, N - from) * kES;
    }
    __device__ __forceinline__ void fetch(int stage, int slot, const Cursor<T>& c, int rows, bool inner) const
    {
        const int lane = threadIdx.x % kWarp;
        const uint32_t to = at + stage * kStage + slot * kSlot + lane * 16;
        const uint8_t* p = reinterpret_cast<const uint8_t*>(c.ahead(rows) + from);
        const int off = (int)((uintptr_t)p & 15), end = off + bytes;
        const uint8_t* word = p - off + lane * 16;
        if (inner) {
#pragma unroll
            for (int i = 0; i < (kWords + kWarp - 1) / kWarp; ++i)
                if ((lane + kWarp * i) * 16 < end) copy16(to + kWarp * 16 * i, word + kWarp * 16 * i, 16);
        } else if (bytes > 0) {
            const bool cut = (uintptr_t)(p - off) < (uintptr_t)c.base;
            for (int w = lane; w * 16 < end; w += kWarp)
                if (w > 0 || !cut) copy16(to + (w - lane) * 16, p - off + w * 16, min(16, end - w * 16));
            if (cut && lane >= off / kES && lane < min(16, end) / kES)
                reinterpret_cast<T*>(mine + stage * kStage + slot * kSlot)[lane] = __ldg(reinterpret_cast<const T*>(p) + lane - off / kES);
        }
    }
    static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    static __device__ __forceinline__ void wait()
    {
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
        __syncwarp();   // the other lanes' copies too
    }
    static __device__ __forceinline__ void done() { __syncwarp(); }   // all lanes have read the row
    __device__ __forceinline__ void read(int stage, int slot, const T* row, float2 (&f)[4]) const
    {
        const uint8_t* p = mine + stage * kStage + slot * kSlot + ((uintptr_t)(row + from) & 15) + (first - from) * kES;
        const T* e = reinterpret_cast<const T*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = make_float2(to_f32(e[run_col<false, kES>(0, 2 * i)]), to_f32(e[run_col<false, kES>(0, 2 * i + 1)]));
        if (bytes < 256 * kES) {   // what is left there from other rows
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[i].x = run_col<false, kES>(first, 2 * i) < N ? f[i].x : 0.f;
                f[i].y = run_col<false, kES>(first, 2 * i + 1) < N ? f[i].y : 0.f;
            }
        }
    }
};

template <typename T, bool VEC>
__device__ __forceinline__ void store_run(T* row, int first, int N, bool full, const float2 (&v)[4])
{
    if constexpr (VEC) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = v[i].x;
            f[2 * i + 1] = v[i].y;
        }
        if constexpr (sizeof(T) == 2) {
            if (first < N) store8<T, true>(row + first, 8, f);
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (first + i * 128 < N)
                    *reinterpret_cast<float4*>(row + first + i * 128) = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
        }
    } else if constexpr (sizeof(T) == 2) {
        T* const p = row + first;
        if (full && row_of_words(row)) {
            float f[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = v[i].x;
                f[2 * i + 1] = v[i].y;
            }
            const uint4 w = pack8<T>(f);
            uint32_t* const q = reinterpret_cast<uint32_t*>(p);
            q[0] = w.x;
            q[32] = w.y;
            q[64] = w.z;
            q[96] = w.w;
        } else if (full) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p[64 * i] = from_f32<T>(v[i].x);
                p[64 * i + 1] = from_f32<T>(v[i].y);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (first + 64 * i < N) p[64 * i] = from_f32<T>(v[i].x);
                if (first + 64 * i + 1 < N) p[64 * i + 1] = from_f32<T>(v[i].y);
            }
        }
    } else {
        T* const p = row + first;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (full || first + 64 * i < N) p[64 * i] = v[i].x;
            if (full || first + 64 * i + 32 < N) p[64 * i + 32] = v[i].y;
        }
    }
}

// The run's part of a vector: `fill` everywhere where there is none, 0 past the row's end; and of an fp32 output.
template <bool VEC, int ES>
__device__ __forceinline__ void load_vector(const float* p, int first, int N, float fill, float2 (&f)[4])
{
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int c = run_col<VEC, ES>(first, i);
        v[i] = c >= N ? 0.f : p ? __ldg(p + c) : fill;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = make_float2(v[2 * i], v[2 * i + 1]);
}

template <bool VEC, int ES>
__device__ __forceinline__ void store_vector(float* p, int first, int N, const float2 (&v)[4])
{
    if constexpr (VEC) {   // N is a multiple of eight
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (run_col<VEC, ES>(first, 4 * i) < N)
                *reinterpret_cast<float4*>(p + run_col<VEC, ES>(first, 4 * i)) = make_float4(v[2 * i].x, v[2 * i].y, v[2 * i + 1].x, v[2 * i + 1].y);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = run_col<VEC, ES>(first, 2 * i), d = run_col<VEC, ES>(first, 2 * i + 1);
            if (c < N) p[c] = v[i].x;
            if (d < N) p[d] = v[i].y;
        }
    }
}

// Sums of V (1 or 2) values over the W warps of a row, the same in all of them.  red: two areas
// that take turns, so that one barrier a sum is enough.
template <int W, int V>
__device__ __forceinline__ void row_sum(float (&v)[V], float* red, int& turn, int warp)
{
    const int lane = threadIdx.x % kWarp;
    float s = v[0];
    if constexpr (V == 2) {   // each half of the warp goes on with one of the two
        const bool up = lane & 16;
        s = (up ? v[1] : v[0]) + __shfl_xor_sync(~0u, up ? v[0] : v[1], 16);
    } else {
        s += __shfl_xor_sync(~0u, s, 16);
    }
#pragma unroll
    for (int m = 8; m; m /= 2) s += __shfl_xor_sync(~0u, s, m);
    if constexpr (W == 1) {
        if constexpr (V == 2) {
            const float o = __shfl_xor_sync(~0u, s, 16);
            v[0] = lane & 16 ? o : s;
            v[1] = lane & 16 ? s : o;
        } else {
            v[0] = s;
        }
    } else {
        constexpr int kWarps = W > 8 ? W : 8;
        float* area = red + turn * kWarps * 2;   // [row][2 values][warp]: rows' sums of one and two values may meet
        turn ^= 1;
        if (V == 2 ? lane % 16 == 0 : lane == 0) area[(warp / W * 2 + lane / 16) * W + warp % W] = s;
        if constexpr (W >= 8) __syncthreads();
        else asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / W), "r"(W * 32) : "memory");
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float* p = area + (warp / W * 2 + i) * W;
            if constexpr (W == 2) {
                const float2 q = *reinterpret_cast<const float2*>(p);
                v[i] = q.x + q.y;
            } else {
                v[i] = 0.f;
#pragma unroll
                for (int w = 0; w < W; w += 4) {
                    const float4 q = *reinterpret_cast<const float4*>(p + w);
                    v[i] += (q.x + q.y) + (q.z + q.w);
                }
            }
        }
    }
}

// (s, s) and sums of pairs
__device__ __forceinline__ float2 both(float s) { return make_float2(s, s); }
__device__ __forceinline__ float add_up(const float2 (&v)[4])
{
    const float2 a = __fadd2_rn(__fadd2_rn(v[0], v[1]), __fadd2_rn(v[2], v[3]));
    return a.x + a.y;
}

// gate(g), and gate'(g): with s the sigmoid, SIGMOID s and s (1 - s), SILU s g and s (1 + g (1 - s)).
template <typename T>
__device__ __forceinline__ float gate_f(float g, int act)
{
    if (act == DLRM_GATE_NONE) return g;
    return sigmoid<T>(g) * (act == DLRM_GATE_SIGMOID ? 1.f : g);
}

template <typename T>
__device__ __forceinline__ void gate_both(float& g, int act, float& slope)
{
    slope = 1.f;
    if (act == DLRM_GATE_NONE) return;
    const float s = sigmoid<T>(g), m = act == DLRM_GATE_SIGMOID ? 1.f : g;
    g = s * m;
    slope = s * fmaf(m, 1.f - s, act == DLRM_GATE_SIGMOID ? 0.f : 1.f);
}

// Blocks of at least 256 threads, G rows at a time.
template <int W>
struct Group {
    static constexpr int kWarps = W > 8 ? W : 8, kThreads = kWarps * 32, kRows = kWarps / W;
};

// ------------------------------------------------------------------- forward
struct NormFwd {
    const void *y, *gate, *res;
    int64_t ldy, ldg, ldres;
    int gate_cols;                   // 0: no gate
    const float *w_post, *b_post, *scale, *w_pre, *b_pre;
    int M, N, margin, layer, gate_act;   // margin: rows at the matrices' ends that do not have 16 bytes of them beyond
    float eps, inv_n;
    void *r, *h;
    int64_t ldr, ldh;
    float4* stats;
};

// (mean, 1 / sqrt(mean square + eps)) of a row; f becomes what is left without the mean, 0 past the end
template <bool VEC, int ES, int W>
__device__ __forceinline__ float2 centre(float2 (&f)[4], int first, bool full, const NormFwd& a, float* red, int& turn, int warp)
{
    float s[1], mean = 0.f;
    if (a.layer) {
        s[0] = add_up(f);
        row_sum<W>(s, red, turn, warp);
        mean = s[0] * a.inv_n;
        if (full) {
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = __fadd2_rn(f[i], both(-mean));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[i].x = run_col<VEC, ES>(first, 2 * i) < a.N ? f[i].x - mean : 0.f;
                f[i].y = run_col<VEC, ES>(first, 2 * i + 1) < a.N ? f[i].y - mean : 0.f;
            }
        }
    }
    float2 q = __fmul2_rn(f[0], f[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) q = __ffma2_rn(f[i], f[i], q);
    s[0] = q.x + q.y;
    row_sum<W>(s, red, turn, warp);
    return make_float2(mean, 1.f / sqrtf(fmaf(s[0], a.inv_n, a.eps)));
}

template <typename T, bool VEC, int W>
__global__ void __launch_bounds__(Group<W>::kThreads, W > 8 ? 1 : 2)
block_norm_fwd_kernel(const __grid_constant__ NormFwd a)
{
    constexpr int kWarps = Group<W>::kWarps, G = Group<W>::kRows;
    using R = Ring<T, VEC, 3, Group<W>::kThreads>;
    constexpr int kAhead = R::kAhead;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float red[W > 1 ? 4 * kWarps : 1];
    // the same in all lanes, so that what depends on the row alone takes the uniform datapath
    const int warp = __shfl_sync(~0u, (int)threadIdx.x / kWarp, 0), lane = threadIdx.x % kWarp, N = a.N;
    const bool full = warp % W * 256 + 256 <= N;   // all columns of the warp are in the row
    const int first = run_first<VEC, sizeof(T)>(warp % W, lane);
    int turn = 0;
    const R ring(smem, N, first, warp % W * 256);
    pdl_wait();
    const int64_t step = (int64_t)gridDim.x * G;
    const int64_t row0 = (int64_t)blockIdx.x * G + warp / W;
    Cursor<T> cy(a.y, a.ldy, row0, step), cg(a.gate, a.ldg, row0, step), cres(a.res, a.ldres, row0, step),
        cr(a.r, a.ldr, row0, step), ch(a.h, a.ldh, row0, step);
    auto fetch = [&](int stage, int64_t row, int rows) {
        const int64_t at = row + rows * step;
        if (at < a.M) {
            const bool inner = at >= a.margin && at < a.M - a.margin;
            if (a.y) ring.fetch(stage, 0, cy, rows, inner);
            if (a.gate_cols > 1) ring.fetch(stage, 1, cg, rows, inner);
            if (a.res) ring.fetch(stage, 2, cres, rows, inner);
        }
        R::commit();
    };
#pragma unroll
    for (int k = 0; k < kAhead - 1; ++k) fetch(k, row0, k);
    float2 aw[4], ab[4], wp[4], bp[4];   // scale w_post, scale b_post, w_pre, b_pre
    load_vector<VEC, sizeof(T)>(a.scale, first, N, 1.f, wp);
    load_vector<VEC, sizeof(T)>(a.w_post, first, N, 1.f, aw);
    load_vector<VEC, sizeof(T)>(a.b_post, first, N, 0.f, ab);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        aw[i] = __fmul2_rn(aw[i], wp[i]);
        ab[i] = __fmul2_rn(ab[i], wp[i]);
    }
    load_vector<VEC, sizeof(T)>(a.w_pre, first, N, 1.f, wp);
    load_vector<VEC, sizeof(T)>(a.b_pre, first, N, 0.f, bp);
    int stage = 0;
    for (int64_t row = row0; row < a.M; row += step) {
        fetch(stage == 0 ? kAhead - 1 : stage - 1, row, kAhead - 1);
        R::wait();
        float4 st = make_float4(0.f, 0.f, 0.f, 0.f);
        float2 r[4];
        if (a.res) ring.read(stage, 2, cres.row, r);
        else
#pragma unroll
            for (int i = 0; i < 4; ++i) r[i] = both(0.f);
        if (a.y) {
            float2 f[4], g[4];
            ring.read(stage, 0, cy.row, f);
            if (a.gate_cols > 1) {
                ring.read(stage, 1, cg.row, g);
                if (a.gate_act != DLRM_GATE_NONE)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        g[i].x = gate_f<T>(g[i].x, a.gate_act);
                        g[i].y = gate_f<T>(g[i].y, a.gate_act);
                    }
            } else {
                const float g1 = a.gate_cols == 1 ? gate_f<T>(to_f32(__ldg(cg.row)), a.gate_act) : 1.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) g[i] = both(g1);
            }
            const float2 s = centre<VEC, sizeof(T), W>(f, first, full, a, red, turn, warp);
            st.x = s.x;
            st.y = s.y;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 u = __ffma2_rn(__fmul2_rn(f[i], both(s.y)), aw[i], ab[i]);   // scale u
                r[i] = __ffma2_rn(u, g[i], r[i]);
            }
            store_run<T, VEC>(cr.out(), first, N, full, r);
        }
        if (a.h) {
            const float2 s = centre<VEC, sizeof(T), W>(r, first, full, a, red, turn, warp);
            st.z = s.x;
            st.w = s.y;
#pragma unroll
            for (int i = 0; i < 4; ++i) r[i] = __ffma2_rn(__fmul2_rn(r[i], both(s.y)), wp[i], bp[i]);
            store_run<T, VEC>(ch.out(), first, N, full, r);
        }
        if (a.stats && warp % W == 0 && lane == 0) a.stats[row] = st;
        R::done();
        cy.next();
        cg.next();
        cres.next();
        cr.next();
        ch.next();
        stage = stage == kAhead - 1 ? 0 : stage + 1;
    }
}

// Warps of a row, a power of two, and the blocks of a call.
int norm_warps(int N)
{
    int w = 1;
    while (w * 256 < N) w *= 2;
    return w;
}

int norm_blocks(int M, int N)
{
    const int w = norm_warps(N), rows = w > 8 ? 1 : 8 / w;
    const int64_t want = ((int64_t)M + rows - 1) / rows, most = (int64_t)num_sms() * (w > 8 ? 1 : 2);
    return (int)(want < most ? want : most);
}

// fn(the warps of a row as a constant)
template <typename Fn>
dlrm_status with_warps(int N, Fn&& fn)
{
    using std::integral_constant;
    switch (norm_warps(N)) {
    case 1: return fn(integral_constant<int, 1>());
    case 2: return fn(integral_constant<int, 2>());
    case 4: return fn(integral_constant<int, 4>());
    case 8: return fn(integral_constant<int, 8>());
    case 16: return fn(integral_constant<int, 16>());
    default: return fn(integral_constant<int, 32>());
    }
}

template <typename K, typename A>
dlrm_status launch_norm(const char* what, K kern, const A& a, int threads, size_t smem, cudaStream_t st)
{
    const cudaError_t e =   // the first 48 KB need no leave
        smem > 46 << 10 ? cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) : cudaSuccess;
    if (e != cudaSuccess) return fail(DLRM_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
    return check_launch_pdl(launch_pdl(kern, dim3(norm_blocks(a.M, a.N)), dim3(threads), smem, st, a), what);
}

template <typename T, bool VEC>
dlrm_status launch_fwd(const NormFwd& a, cudaStream_t st)
{
    return with_warps(a.N, [&](auto w) {
        constexpr int W = decltype(w)::value, kThreads = Group<W>::kThreads;
        return launch_norm("block_norm_fwd_kernel", block_norm_fwd_kernel<T, VEC, W>, a, kThreads,
                           Ring<T, VEC, 3, kThreads>::kBytes, st);
    });
}

// ------------------------------------------------------------------ backward
struct NormBwd {
    const void *gr, *gh, *y, *gate, *r;
    int64_t ldgr, ldgh, ldy, ldg, ldr;
    int gate_cols;
    const float4* stats;
    const float *w_post, *b_post, *scale, *w_pre;
    int M, N, margin, layer, gate_act;
    float inv_n;
    void *gy, *gg, *gres;
    int64_t ldgy, ldgg, ldgres;
    float* partial;   // [gridDim.x][4][Np]: sums of dr gate norm(y), dr gate, grad_h norm(r), grad_h; or NULL
    int64_t Np;
};

template <typename T, bool VEC, int W, bool POST, bool PRE>
__global__ void __launch_bounds__(Group<W>::kThreads, W > 8 ? 1 : 2)
block_norm_bwd_kernel(const __grid_constant__ NormBwd a)
{
    constexpr int kWarps = Group<W>::kWarps, G = Group<W>::kRows;
    constexpr int kGr = 0, kGh = 1, kR = 2, kY = PRE ? 3 : 1, kGate = kY + 1;   // slots
    using Rg = Ring<T, VEC, POST && PRE ? 5 : 3, Group<W>::kThreads>;
    constexpr int kAhead = Rg::kAhead;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float red[W > 1 ? 4 * kWarps : 1];
    // the same in all lanes, so that what depends on the row alone takes the uniform datapath
    const int warp = __shfl_sync(~0u, (int)threadIdx.x / kWarp, 0), lane = threadIdx.x % kWarp, N = a.N;
    const bool full = warp % W * 256 + 256 <= N;   // all columns of the warp are in the row
    const int first = run_first<VEC, sizeof(T)>(warp % W, lane);
    int turn = 0;
    const Rg ring(smem, N, first, warp % W * 256);
    pdl_wait();
    const int64_t step = (int64_t)gridDim.x * G, row0 = (int64_t)blockIdx.x * G + warp / W;
    Cursor<T> cgr(a.gr, a.ldgr, row0, step), cgh(a.gh, a.ldgh, row0, step), cr(a.r, a.ldr, row0, step),
        cy(a.y, a.ldy, row0, step), cg(a.gate, a.ldg, row0, step), cgy(a.gy, a.ldgy, row0, step), cgg(a.gg, a.ldgg, row0, step),
        cgres(a.gres, a.ldgres, row0, step);
    auto fetch = [&](int stage, int64_t row, int rows) {
        const int64_t at = row + rows * step;
        if (at < a.M) {
            const bool inner = at >= a.margin && at < a.M - a.margin;
            if (a.gr) ring.fetch(stage, kGr, cgr, rows, inner);
            if (PRE) {
                ring.fetch(stage, kGh, cgh, rows, inner);
                ring.fetch(stage, kR, cr, rows, inner);
            }
            if (POST) {
                ring.fetch(stage, kY, cy, rows, inner);
                if (a.gate_cols > 1) ring.fetch(stage, kGate, cg, rows, inner);
            }
        }
        Rg::commit();
    };
#pragma unroll
    for (int k = 0; k < kAhead - 1; ++k) fetch(k, row0, k);
    float2 aw[4], ab[4], wp[4];   // scale w_post, scale b_post, w_pre; 0 past the row's end
    load_vector<VEC, sizeof(T)>(a.scale, first, N, 1.f, wp);
    load_vector<VEC, sizeof(T)>(a.w_post, first, N, 1.f, aw);
    load_vector<VEC, sizeof(T)>(a.b_post, first, N, 0.f, ab);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        aw[i] = __fmul2_rn(aw[i], wp[i]);
        ab[i] = __fmul2_rn(ab[i], wp[i]);
    }
    load_vector<VEC, sizeof(T)>(a.w_pre, first, N, 1.f, wp);
    float2 sum[4][4] = {};
    // what a row has one of is loaded a row ahead
    float4 st_next = row0 < a.M ? __ldg(a.stats + row0) : make_float4(0, 0, 0, 0);
    float g_next = a.gate_cols == 1 && row0 < a.M ? to_f32(__ldg(cg.row)) : 1.f;
    int stage = 0;
    for (int64_t row = row0; row < a.M; row += step) {
        fetch(stage == 0 ? kAhead - 1 : stage - 1, row, kAhead - 1);
        const float4 st = st_next;
        float g1 = g_next, slope1 = 1.f;
        if (row + step < a.M) {
            st_next = __ldg(a.stats + row + step);
            if (a.gate_cols == 1) g_next = to_f32(__ldg(cg.ahead(1)));
        }
        Rg::wait();
        float2 dr[4];
        if (a.gr) ring.read(stage, kGr, cgr.row, dr);
        else
#pragma unroll
            for (int i = 0; i < 4; ++i) dr[i] = both(0.f);
        if (PRE) {
            float2 d[4], x[4], p, q;
            ring.read(stage, kGh, cgh.row, d);
            ring.read(stage, kR, cr.row, x);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = __fmul2_rn(__fadd2_rn(x[i], both(-st.z)), both(st.w));
                sum[2][i] = __ffma2_rn(d[i], x[i], sum[2][i]);
                sum[3][i] = __fadd2_rn(sum[3][i], d[i]);
                d[i] = __fmul2_rn(d[i], wp[i]);
                p = i ? __ffma2_rn(d[i], x[i], p) : __fmul2_rn(d[i], x[i]);
                q = i ? __fadd2_rn(d[i], q) : d[i];
            }
            float c0, c1 = 0.f;
            if (a.layer) {
                float c[2] = {p.x + p.y, q.x + q.y};
                row_sum<W>(c, red, turn, warp);
                c0 = c[0] * -a.inv_n;
                c1 = c[1] * -a.inv_n;
            } else {
                float c[1] = {p.x + p.y};
                row_sum<W>(c, red, turn, warp);
                c0 = c[0] * -a.inv_n;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                dr[i] = __ffma2_rn(__ffma2_rn(x[i], both(c0), __fadd2_rn(d[i], both(c1))), both(st.w), dr[i]);
        }
        if (a.gres) store_run<T, VEC>(cgres.out(), first, N, full, dr);
        if (POST) {
            float2 x[4], g[4], k[4], p, q, t = both(0.f);
            ring.read(stage, kY, cy.row, x);
            if (a.gate_cols > 1) {
                ring.read(stage, kGate, cg.row, g);
                if (a.gate_act != DLRM_GATE_NONE)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        gate_both<T>(g[i].x, a.gate_act, k[i].x);
                        gate_both<T>(g[i].y, a.gate_act, k[i].y);
                    }
                else
#pragma unroll
                    for (int i = 0; i < 4; ++i) k[i] = both(1.f);
            } else {
                if (a.gate_cols == 1) gate_both<T>(g1, a.gate_act, slope1);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    g[i] = both(g1);
                    k[i] = both(1.f);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = __fmul2_rn(__fadd2_rn(x[i], both(-st.x)), both(st.y));
                const float2 su = __ffma2_rn(x[i], aw[i], ab[i]);   // scale u
                t = __ffma2_rn(dr[i], su, t);
                k[i] = __fmul2_rn(__fmul2_rn(dr[i], su), k[i]);
                dr[i] = __fmul2_rn(dr[i], g[i]);
                sum[0][i] = __ffma2_rn(dr[i], x[i], sum[0][i]);
                sum[1][i] = __fadd2_rn(sum[1][i], dr[i]);
                dr[i] = __fmul2_rn(dr[i], aw[i]);
                p = i ? __ffma2_rn(dr[i], x[i], p) : __fmul2_rn(dr[i], x[i]);
                q = i ? __fadd2_rn(dr[i], q) : dr[i];
            }
            if (a.gg && a.gate_cols > 1) store_run<T, VEC>(cgg.out(), first, N, full, k);
            float c0, c1 = 0.f;
            if (a.layer) {
                float c[2] = {p.x + p.y, q.x + q.y};
                row_sum<W>(c, red, turn, warp);
                c0 = c[0] * -a.inv_n;
                c1 = c[1] * -a.inv_n;
            } else {
                float c[1] = {p.x + p.y};
                row_sum<W>(c, red, turn, warp);
                c0 = c[0] * -a.inv_n;
            }
            if (a.gg && a.gate_cols == 1) {
                float c[1] = {t.x + t.y};
                row_sum<W>(c, red, turn, warp);
                if (warp % W == 0 && lane == 0) *cgg.out() = from_f32<T>(c[0] * slope1);
            }
            if (a.gy) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    dr[i] = __fmul2_rn(__ffma2_rn(x[i], both(c0), __fadd2_rn(dr[i], both(c1))), both(st.y));
                store_run<T, VEC>(cgy.out(), first, N, full, dr);
            }
        }
        Rg::done();
        cgr.next();
        cgh.next();
        cr.next();
        cy.next();
        cg.next();
        cgy.next();
        cgg.next();
        cgres.next();
        stage = stage == kAhead - 1 ? 0 : stage + 1;
    }
    if (!a.partial) return;
    // the rows' sums of a block: its groups one after another, by way of the ring's memory
    float2* const tile = reinterpret_cast<float2*>(smem);
    asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        if (s < 2 ? !POST : !PRE) continue;
        if constexpr (G > 1) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 4; ++i) tile[i * 256 + threadIdx.x] = sum[s][i];
            __syncthreads();
            if (warp < W) {
#pragma unroll
                for (int g = 1; g < G; ++g)
#pragma unroll
                    for (int i = 0; i < 4; ++i) sum[s][i] = __fadd2_rn(sum[s][i], tile[i * 256 + g * W * 32 + threadIdx.x]);
            }
        }
        if (warp < W) store_vector<VEC, sizeof(T)>(a.partial + ((int64_t)blockIdx.x * 4 + s) * a.Np, first, N, sum[s]);
    }
}

struct NormSum {
    const float* partial;
    int64_t Np;
    int blocks, N;
    const float *w_post, *b_post, *scale;
    float *gw_post, *gb_post, *gscale, *gw_pre, *gb_pre;
};

// The vectors' gradients: kSumCols columns a block, a sector of each block's sums, 128 threads a column;
// blockIdx.y 0 the side of the norm after the block, 1 that of the norm before the next.
constexpr int kSumCols = 8, kSumRows = 128;

__global__ void __launch_bounds__(kSumCols * kSumRows) block_norm_sum_kernel(const __grid_constant__ NormSum a)
{
    pdl_wait();
    __shared__ float red[2][kSumRows / 4][kSumCols];
    const int tx = threadIdx.x % kSumCols, ty = threadIdx.x / kSumCols, n = blockIdx.x * kSumCols + tx;
    const bool pre = blockIdx.y == 1;
    if (pre ? !a.gw_pre && !a.gb_pre : !a.gw_post && !a.gb_post && !a.gscale) return;
    float s = 0.f, t = 0.f;
    if (n < a.N) {
        const float* p = a.partial + (pre ? 2 * a.Np : 0) + n;
#pragma unroll 4
        for (int b = ty; b < a.blocks; b += kSumRows) {
            s += p[(int64_t)b * 4 * a.Np];
            t += p[(int64_t)b * 4 * a.Np + a.Np];
        }
    }
#pragma unroll
    for (int m = 16; m >= kSumCols; m /= 2) {   // a warp's four rows
        s += __shfl_xor_sync(~0u, s, m);
        t += __shfl_xor_sync(~0u, t, m);
    }
    if (ty % 4 == 0) {
        red[0][ty / 4][tx] = s;
        red[1][ty / 4][tx] = t;
    }
    __syncthreads();
    if (ty || n >= a.N) return;
#pragma unroll
    for (int y = 1; y < kSumRows / 4; ++y) {
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

template <typename T, bool VEC, bool POST, bool PRE>
dlrm_status launch_bwd(const NormBwd& a, cudaStream_t st)
{
    return with_warps(a.N, [&](auto w) {
        constexpr int W = decltype(w)::value, kThreads = Group<W>::kThreads;
        return launch_norm("block_norm_bwd_kernel", block_norm_bwd_kernel<T, VEC, W, POST, PRE>, a, kThreads,
                           Ring<T, VEC, POST && PRE ? 5 : 3, kThreads>::kBytes, st);
    });
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

// Checks fp32 vectors of N elements, each of which may be NULL; *vec: whether all start on 16-byte boundaries.
dlrm_status check_vectors(const char* fn, std::initializer_list<const void*> v, bool* vec)
{
    for (const void* p : v) {
        if (reinterpret_cast<uintptr_t>(p) & 3u)
            return fail(DLRM_ERR_INVALID_ARG, "%s: a vector is not aligned to its element size", fn);
        *vec = *vec && aligned16(p);
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
        return vec ? launch_fwd<T, true>(a, as_stream(stream)) : launch_fwd<T, false>(a, as_stream(stream));
    });
}

extern "C" size_t dlrm_block_norm_bwd_workspace_size(int M, int N)
{
    if (M < 1 || N < 1 || M > kMaxSize || N > DLRM_BLOCK_MAX_WIDTH) return 0;
    return dlrm_ws_align((size_t)norm_blocks(M, N) * 4 * ((N + 7) / 8 * 8) * 4);
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
    bool vec = N % 8 == 0, grads_vec = true;
    float* const grads[5] = {d_grad_w_post, d_grad_b_post, d_grad_scale, d_grad_w_pre, d_grad_b_pre};
    if ((s = check_vectors(fn, {d_w_post, d_b_post, d_scale, d_w_pre}, &vec)) != DLRM_OK) return s;
    if ((s = check_vectors(fn, {grads[0], grads[1], grads[2], grads[3], grads[4]}, &grads_vec)) != DLRM_OK) return s;
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
                       (const float4*)d_stats, d_w_post, d_b_post, d_scale, d_w_pre, M, N, end_rows(N, es), norm == DLRM_NORM_LAYER,
                       (int)gate_act, (float)(1.0 / N), d_grad_y, d_grad_gate, d_grad_residual, ldgy, ldgg, ldgres,
                       sums ? (float*)d_workspace : nullptr, Np};
    s = with_type(dtype, [&](auto t) {
        using T = decltype(t);
        auto go = [&](auto v) {
            constexpr bool VEC = decltype(v)::value;
            return !d_y ? launch_bwd<T, VEC, false, true>(a, st) : d_grad_h ? launch_bwd<T, VEC, true, true>(a, st)
                                                                           : launch_bwd<T, VEC, true, false>(a, st);
        };
        return vec ? go(std::true_type()) : go(std::false_type());
    });
    if (s != DLRM_OK || !sums) return s;
    const NormSum q = {a.partial, Np, norm_blocks(M, N), N, d_w_post, d_b_post, d_scale,
                       d_grad_w_post, d_grad_b_post, d_grad_scale, d_grad_w_pre, d_grad_b_pre};
    return check_launch_pdl(launch_pdl(block_norm_sum_kernel, dim3((N + kSumCols - 1) / kSumCols, 2), dim3(kSumCols * kSumRows), 0, st, q),
                            "block_norm_sum_kernel");
}
