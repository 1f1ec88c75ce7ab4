// dense_epilogue.cuh -- what follows a product of the dense layer, on eight
// consecutive columns of a row: bias, activation, dropout, residual, stores.
#pragma once

#include "dense_ops.cuh"

namespace dlrm {

struct Epilogue {
    const float* bias;   // may be NULL
    const void* res;     // may be NULL
    int64_t ldr;
    void* pre;           // may be NULL
    int64_t ldp;
    void* out;
    int64_t ldo;
    int act;
    int vec;             // rows of res, pre and out all start on 16-byte boundaries
    Drop drop;
    float scale = 1.f;   // of the product (1 where there is a bias)
};

inline int epilogue_vec(const Epilogue& e, int M, int es)
{
    return rows_aligned16(e.out, e.ldo, M, es) && (!e.res || rows_aligned16(e.res, e.ldr, M, es)) &&
           (!e.pre || rows_aligned16(e.pre, e.ldp, M, es));
}

// a(.) of n values: one branch for all of them.
template <typename T, int n>
__device__ __forceinline__ void act_n(float (&f)[n], int act)
{
    if (act == DLRM_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < n; ++i) f[i] = act_f<T>(f[i], DLRM_ACT_RELU);
    } else if (act == DLRM_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < n; ++i) f[i] = act_f<T>(f[i], DLRM_ACT_GELU);
    } else if (act == DLRM_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < n; ++i) f[i] = act_f<T>(f[i], DLRM_ACT_SILU);
    }
}

// f *= a'(z)
template <typename T>
__device__ __forceinline__ void slope8(float (&f)[8], const float (&z)[8], int act)
{
    if (act == DLRM_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = z[i] <= 0.f ? 0.f : f[i];
    } else if (act == DLRM_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= act_slope<T>(z[i], DLRM_ACT_GELU);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= act_slope<T>(z[i], DLRM_ACT_SILU);
    }
}

// The bias of columns col .. col + 7 (zeros past N or without a bias).
__device__ __forceinline__ void bias8(const float* bias, int col, int N, float (&b)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = bias && col + i < N ? __ldg(bias + col + i) : 0.f;
}

// f: the product's columns col .. col + 7 of a row, n of them inside; r: the
// residual's, loaded before (unused without one).
template <typename T, bool VEC>
__device__ __forceinline__ void finish8(const Epilogue& e, const DropKey& key, int row, int col, int n, float (&f)[8],
                                        const float (&b)[8], const Raw8<T>& r)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = fmaf(f[i], e.scale, b[i]);   // zeros without a bias
    if (e.pre) store8<T, VEC>((T*)e.pre + row * e.ldp + col, n, f);
    act_n<T>(f, e.act);
    if (e.drop.thr) drop8(f, e.drop, key, (uint32_t)row, (uint32_t)col >> 3);
    if (e.res) {
        float g[8];
        widen8<T>(r, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] += g[i];
    }
    store8<T, VEC>((T*)e.out + row * e.ldo + col, n, f);
}

// finish8 for a run that may be short or off the 16-byte grid.
template <typename T>
__device__ __forceinline__ void finish8_any(const Epilogue& e, const DropKey& key, int row, int col, int n,
                                            float (&f)[8], const float (&b)[8])
{
    Raw8<T> r = {};
    if (e.vec && n >= 8) {
        if (e.res) r = load8<T, true>((const T*)e.res + row * e.ldr + col, 8);
        finish8<T, true>(e, key, row, col, 8, f, b, r);
    } else {
        if (e.res) r = load8<T, false>((const T*)e.res + row * e.ldr + col, n);
        finish8<T, false>(e, key, row, col, n, f, b, r);
    }
}

}  // namespace dlrm
