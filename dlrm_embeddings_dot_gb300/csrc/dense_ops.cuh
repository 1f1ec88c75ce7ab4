// dense_ops.cuh -- what the kernels of the dense network share: element types,
// activations and their slopes, the counter-based generator, and access to
// runs of eight columns of a row (the unit of the generator).
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"
#include "dlrm_dense.h"

namespace dlrm {

using bf16 = __nv_bfloat16;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(bf16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v)
{
    if constexpr (std::is_same_v<T, float>) return v;
    else if constexpr (std::is_same_v<T, __half>) return __float2half_rn(v);
    else return __float2bfloat16_rn(v);
}

// Eight consecutive elements at a 16-byte aligned address.
template <typename T>
__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8])
{
    static_assert(sizeof(T) == 2);
    if constexpr (std::is_same_v<T, __half>) {
        h8_to_f8(v, f);
    } else {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}

template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&f)[8])
{
    static_assert(sizeof(T) == 2);
    if constexpr (std::is_same_v<T, __half>) {
        return f8_to_h8(f);
    } else {
        uint4 v;
        __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&v);
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        return v;
    }
}

// Eight columns of a row as raw words, so that a load can be issued long before
// its values are used: one 16-byte word for 2-byte types, two for fp32.
template <typename T>
struct Raw8 {
    uint4 w[sizeof(T) / 2];
};

// Columns [0, n) of the run at p (n <= 8; the others read as zero).  VEC: the
// run is 16-byte aligned and has all eight columns.
template <typename T, bool VEC>
__device__ __forceinline__ Raw8<T> load8(const T* p, int n)
{
    Raw8<T> r;
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < (int)(sizeof(T) / 2); ++i) r.w[i] = ldg_nc_v4(reinterpret_cast<const uint4*>(p) + i);
    } else {
        T e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = i < n ? __ldg(p + i) : from_f32<T>(0.f);
        memcpy(&r, e, sizeof(r));
    }
    return r;
}

// The same for a run that starts anywhere: the 16-byte words that it lies in, shifted into
// place, where those are inside the matrix [lo, hi) (nearly everywhere), else element by
// element.  Columns from n on hold anything.  n >= 1.  A third of the instructions of
// eight single loads, and each reads whole sectors.
template <typename T>
__device__ __forceinline__ Raw8<T> load8_shifted(const T* p, int n, const T* lo, const T* hi)
{
    constexpr int kWords = 2 * sizeof(T), kLoads = kWords / 4 + 1;   // 32-bit words of a run; 16-byte words it can touch
    const uint32_t off = (uint32_t)(uintptr_t)p & 15u;
    const uint4* base = reinterpret_cast<const uint4*>((const char*)p - off);
    const int last = (int)(off + min(n, 8) * (int)sizeof(T) - 1) / 16;   // the last word with a column of the run
    if ((uintptr_t)base < (uintptr_t)lo || (uintptr_t)(base + last + 1) > (uintptr_t)hi) return load8<T, false>(p, n);
    uint32_t w[4 * kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const uint4 v = ldg_nc_v4(base + min(i, last));
        w[4 * i] = v.x;
        w[4 * i + 1] = v.y;
        w[4 * i + 2] = v.z;
        w[4 * i + 3] = v.w;
    }
    if (off & 8u)
#pragma unroll
        for (int i = 0; i < kWords + 2; ++i) w[i] = w[i + 2];
    if (off & 4u)
#pragma unroll
        for (int i = 0; i < kWords + 1; ++i) w[i] = w[i + 1];
    Raw8<T> r;
    uint32_t* out = &r.w[0].x;
#pragma unroll
    for (int i = 0; i < kWords; ++i) out[i] = sizeof(T) == 2 ? __funnelshift_r(w[i], w[i + 1], (off & 2u) * 8) : w[i];
    return r;
}

template <typename T>
__device__ __forceinline__ void widen8(const Raw8<T>& r, float (&f)[8])
{
    if constexpr (std::is_same_v<T, float>) {
        const float4 a = u4_as_f4(r.w[0]), b = u4_as_f4(r.w[1]);
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
        unpack8<T>(r.w[0], f);
    }
}

// Stores columns [0, n) of the run at p, rounding each once.
template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* p, int n, const float (&f)[8])
{
    if constexpr (VEC) {
        if constexpr (std::is_same_v<T, float>) {
            reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
            reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
        } else {
            *reinterpret_cast<uint4*>(p) = pack8<T>(f);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = from_f32<T>(f[i]);
    }
}

// Three bf16 parts of a float: hi and mid as the upper halves of words, lo as a
// float that has at most eight bits left.  hi and mid are cut, not rounded, so
// none overflows, and lo holds the rest exactly.  An infinity or NaN goes whole
// into lo, which meets only the other side's hi: no 0 * inf turns an infinity
// into a NaN.
__device__ __forceinline__ void split1(float v, uint32_t& hi, uint32_t& mid, float& lo)
{
    const bool wild = (__float_as_uint(v) & 0x7f800000u) == 0x7f800000u;
    hi = wild ? 0u : __float_as_uint(v) & 0xffff0000u;
    const float r = v - __uint_as_float(hi);
    mid = wild ? 0u : __float_as_uint(r) & 0xffff0000u;
    lo = r - __uint_as_float(mid);
}

// A gradient as the sum of two values of a 2-byte type: hi rounded, kept finite, and the
// rest.  An infinity or NaN goes whole into lo.  fp16 gets 7/8 of it: a slope of up to
// 1.13 (GELU) times any fp16 number then is in range, and no more than a fifth of a
// bit is lost at the range's other end.
template <typename T>
constexpr float kFit = std::is_same_v<T, __half> ? 0.875f : 1.f;

template <typename T>
__device__ __forceinline__ void split2(float v, float& hi, float& lo)
{
    constexpr float kMost = std::is_same_v<T, __half> ? 65504.f : 3.38953139e38f;
    v *= kFit<T>;
    hi = to_f32(from_f32<T>(fmaxf(fminf(v, kMost), -kMost)));
    lo = v - hi;
}

// -------------------------------------------------------------- activations
// The functions of the header's definitions, for results of type T.  NaN passes
// through each.
//   fp32  GELU by the library's erf and exp, SILU with a reciprocal rounded by one
//         Newton step: the error of the definition computed in 32 bits (GELU over -3 to
//         3: half that of the other form).  65536 x 1024 outputs, K = 64: GELU 99 us
//         against 80, 5000 x 512 outputs, K = 512: 30 us against 29
//   2-byte types, whose own rounding is 2,000 times as large: the hardware's
//         exponential and reciprocal, and Abramowitz and Stegun 7.1.26 for the tail of
//         the normal distribution.  There the epilogue is bound by the instructions it
//         issues, and with the library's functions an activation had two to four
//         times as many (the same outputs: GELU 166 us against 61, SILU 184 us against
//         44, other changes of the epilogue included)
__device__ __forceinline__ float exp2_fast(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float rcp_fast(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 1 / (1 + e^-z), and 1 less that: near 1 the difference has none of its digits left, so above 0 it is a product
template <typename T>
__device__ __forceinline__ float sigmoid(float z, float& rest)
{
    const float e = exp2_fast(z * -1.44269504f), d = 1.f + e, r = rcp_fast(d);
    float s = r;
    if constexpr (std::is_same_v<T, float>) s = d < 0x1p126f ? fmaf(fmaf(-d, r, 1.f), r, r) : r;
    rest = z > 0.f ? e * s : 1.f - s;
    return s;
}

template <typename T>
__device__ __forceinline__ float sigmoid(float z)
{
    float rest;
    return sigmoid<T>(z, rest);
}

// exp(-z^2 / 2)
template <typename T>
__device__ __forceinline__ float normal_exp(float z)
{
    if constexpr (std::is_same_v<T, float>) return expf(-0.5f * z * z);
    else return exp2_fast(z * z * -0.72134752f);
}

// The normal distribution function of |z|'s sign and size; e = exp(-z^2 / 2) (unused in
// fp32).  The tail's error is below 7.5e-8.
template <typename T>
__device__ __forceinline__ float normal_cdf(float z, float e)
{
    if constexpr (std::is_same_v<T, float>) {
        return fmaf(0.5f, erff(z * 0.70710678f), 0.5f);
    } else {
        const float t = rcp_fast(fmaf(fabsf(z), 0.3275911f * 0.70710678f, 1.f));
        float p = fmaf(t, 1.061405429f, -1.453152027f);
        p = fmaf(t, p, 1.421413741f);
        p = fmaf(t, p, -0.284496736f);
        p = fmaf(t, p, 0.254829592f);
        const float tail = 0.5f * p * t * e;
        return z >= 0.f ? 1.f - tail : tail;
    }
}

template <typename T>
__device__ __forceinline__ float act_f(float z, int act)
{
    switch (act) {
    case DLRM_ACT_RELU: {
        float r;
        asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(z));
        return r;
    }
    case DLRM_ACT_GELU: return z * normal_cdf<T>(z, std::is_same_v<T, float> ? 0.f : normal_exp<T>(z));
    case DLRM_ACT_SILU: return z * sigmoid<T>(z);
    default: return z;
    }
}

// a'(z)
template <typename T>
__device__ __forceinline__ float act_slope(float z, int act)
{
    switch (act) {
    case DLRM_ACT_RELU: return z <= 0.f ? 0.f : 1.f;
    case DLRM_ACT_GELU: {
        const float e = normal_exp<T>(z);
        return fmaf(z * 0.39894228f, e, normal_cdf<T>(z, e));
    }
    case DLRM_ACT_SILU: {
        const float s = sigmoid<T>(z);
        return s * fmaf(z, 1.f - s, 1.f);
    }
    default: return 1.f;
    }
}

// ------------------------------------------------------------------ dropout
// Philox4x32-10 (Salmon et al., SC 2011): ten rounds of two 32 x 32 -> 64 bit
// products on a 128-bit counter, the key stepping by two Weyl constants.
__device__ __forceinline__ uint4 philox4x32(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, uint32_t k0,
                                            uint32_t k1)
{
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
        c1 = (uint32_t)b;
        c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
        c3 = (uint32_t)a;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(c0, c1, c2, c3);
}

// What a kernel needs to drop elements.  thr == 0: no dropout, rng unread.
struct Drop {
    const uint64_t* rng;
    uint32_t thr;    // floor(65536 p + 0.5), below 65536
    float scale;     // 65536 / (65536 - thr)
};

struct DropKey {
    uint32_t k0, k1, o0, o1;
};

__device__ __forceinline__ DropKey drop_key(const Drop& d)
{
    DropKey k = {0, 0, 0, 0};
    if (d.thr) {
        const uint64_t a = __ldg(d.rng), b = __ldg(d.rng + 1);
        k = {(uint32_t)a, (uint32_t)(a >> 32), (uint32_t)b, (uint32_t)(b >> 32)};
    }
    return k;
}

// Drops and scales the eight columns 8 * group .. 8 * group + 7 of a row.  A
// number has 16 bits: one Philox call (about 60 instructions) serves eight
// columns, where 32-bit numbers take two calls for them; the rate in force is
// the multiple of 2^-16 nearest to p and the scale goes by it.
__device__ __forceinline__ void drop8(float (&f)[8], const Drop& d, const DropKey& k, uint32_t row, uint32_t group)
{
    const uint4 u = philox4x32(group, row, k.o0, k.o1, k.k0, k.k1);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w}, t = d.thr << 16;   // numbers compared in the upper half
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = (w[i] << 16) >= t ? f[2 * i] * d.scale : 0.f;
        f[2 * i + 1] = w[i] >= t ? f[2 * i + 1] * d.scale : 0.f;
    }
}

// The eight columns of a group that are kept, a bit each.
__device__ __forceinline__ uint32_t keep8(const Drop& d, const DropKey& k, uint32_t row, uint32_t group)
{
    const uint4 u = philox4x32(group, row, k.o0, k.o1, k.k0, k.k1);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w}, t = d.thr << 16;
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) bits |= ((w[i] << 16) >= t ? 1u << 2 * i : 0u) | (w[i] >= t ? 2u << 2 * i : 0u);
    return bits;
}

// ---------------------------------------------------------------- host side
constexpr int kMaxSize = INT32_MAX - (1 << 20);   // tiles and chunks that start below it end below 2^31

inline bool dense_dtype_ok(dlrm_dtype dt) { return dt == DLRM_F32 || dt == DLRM_F16 || dt == DLRM_BF16; }
inline int dense_dtype_size(dlrm_dtype dt) { return dt == DLRM_F32 ? 4 : 2; }

// Whether a matrix's rows of `width` elements all start on 16-byte boundaries.
inline bool rows_aligned16(const void* p, int64_t ld, int rows, int es)
{
    return aligned16(p) && (rows <= 1 || ld * es % 16 == 0);
}

// fn(T()) for the element type of dt.
template <typename Fn>
auto with_type(dlrm_dtype dt, Fn&& fn)
{
    if (dt == DLRM_F32) return fn(float());
    if (dt == DLRM_F16) return fn(__half());
    return fn(bf16());
}

// Checks p and rng; fills *d.
inline dlrm_status make_drop(const char* fn, double p, const uint64_t* rng, Drop* d)
{
    if (!(p >= 0.0 && p * 65536.0 < 65535.5))
        return fail(DLRM_ERR_INVALID_ARG, "%s: p must be in [0, 1) with 65536 p below 65535.5 (got %g)", fn, p);
    d->thr = (uint32_t)(p * 65536.0 + 0.5);
    d->scale = (float)(65536.0 / (65536.0 - d->thr));
    d->rng = rng;
    if (p > 0.0 && !rng) return fail(DLRM_ERR_INVALID_ARG, "%s: p > 0 needs d_rng", fn);
    if (p > 0.0 && (reinterpret_cast<uintptr_t>(rng) & 7u))
        return fail(DLRM_ERR_INVALID_ARG, "%s: d_rng must be 8-byte aligned", fn);
    return DLRM_OK;
}

// Checks one matrix argument of a call (rows > 0).
inline dlrm_status check_matrix(const char* fn, const char* name, const void* p, int64_t ld, int rows, int cols, int es)
{
    if (!p) return fail(DLRM_ERR_INVALID_ARG, "%s: %s is NULL", fn, name);
    if (reinterpret_cast<uintptr_t>(p) % es)
        return fail(DLRM_ERR_INVALID_ARG, "%s: %s is not aligned to its element size", fn, name);
    if (rows > 1 && (ld < cols || ld > (INT64_C(1) << 40)))
        return fail(DLRM_ERR_INVALID_ARG, "%s: row distance of %s (%lld) must be in [%d, 2^40]", fn, name,
                    (long long)ld, cols);
    return DLRM_OK;
}

}  // namespace dlrm
