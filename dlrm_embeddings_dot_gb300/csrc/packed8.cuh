// packed8.cuh -- matrices in 8 bits (include/dlrm_block.h): eight columns read back.
#pragma once

#include "dense_ops.cuh"

namespace dlrm {

constexpr int kBlock8 = 32;   // columns that share an exponent byte

struct Packed8 {
    const uint8_t* q;
    int64_t ld;
    const uint8_t* exps;      // [rows][blocks]
    int blocks;
    const uint8_t* end;       // behind the last row
};

inline int blocks8(int cols) { return (cols - 1) / kBlock8 + 1; }

inline Packed8 packed8(const uint8_t* q, int64_t ld, const uint8_t* exps, int rows, int cols)
{
    return {q, ld, exps, blocks8(cols), q + (rows > 0 ? (rows - 1) * (rows > 1 ? ld : 0) + cols : 0)};
}

// Eight columns as they lie in memory, and their block's exponent byte.
struct Run8 {
    uint2 q;
    uint32_t e;
};

// VEC: the run starts on an 8-byte boundary and has all eight columns; the others read as 0.
// scaled: with the exponent.
template <bool VEC>
__device__ __forceinline__ Run8 load_run8(const Packed8& m, int64_t row, int col, int n, bool scaled = true)
{
    Run8 r;
    const uint8_t* p = m.q + row * m.ld + col;
    if constexpr (VEC) {
        r.q = __ldg(reinterpret_cast<const uint2*>(p));
    } else {
        const uint32_t off = (uint32_t)(uintptr_t)p & 3u;
        const uint32_t* w = reinterpret_cast<const uint32_t*>(p - off);
        if (n >= 8 && (uintptr_t)w >= (uintptr_t)m.q && (uintptr_t)(w + 3) <= (uintptr_t)m.end) {
            const uint32_t a = __ldg(w), b = __ldg(w + 1), c = __ldg(w + 2);   // the words that it lies in
            r.q = make_uint2(__funnelshift_r(a, b, off * 8), __funnelshift_r(b, c, off * 8));
        } else {
            uint8_t b[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) b[i] = i < n ? __ldg(p + i) : 0;
            memcpy(&r.q, b, 8);
        }
    }
    r.e = scaled ? __ldg(m.exps + row * m.blocks + col / kBlock8) : 0;
    return r;
}

// The largest size a value read back has as a T (fp32: bf16's).
template <typename T>
constexpr float kMost8 = std::is_same_v<T, __half> ? 65504.f : 3.3895313892515355e38f;

// 2^(e - 127), below fp32's normal numbers too
__device__ __forceinline__ float scale8(uint32_t e) { return __uint_as_float(e ? e << 23 : 0x00400000u); }

// The largest scale under which no value passes kMost8: 448 2^7, or 448 2^119.
template <typename T>
constexpr float kSafe8 = std::is_same_v<T, __half> ? 128.f : 0x1p119f;

// q scale, exact in fp32, a scale for each pair of columns
template <typename T>
__device__ __forceinline__ void widen_codes8(const uint2& q, const float (&scale)[4], float (&f)[8])
{
    const uint32_t w[2] = {q.x, q.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(w[i / 2] >> 16 * (i % 2))));
        __half2 v;
        memcpy(&v, &h, 4);
        const float2 g = __half22float2(v);
        f[2 * i] = g.x * scale[i];
        f[2 * i + 1] = g.y * scale[i];
    }
    if (fmaxf(fmaxf(scale[0], scale[1]), fmaxf(scale[2], scale[3])) > kSafe8<T>)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (fabsf(f[i]) > kMost8<T>) f[i] = copysignf(kMost8<T>, f[i]);
}

template <typename T>
__device__ __forceinline__ void widen_run8(const Run8& r, float (&f)[8])
{
    const float s = scale8(r.e), scale[4] = {s, s, s, s};
    widen_codes8<T>(r.q, scale, f);
}

// One column: a code and its block's exponent byte.
template <typename T>
__device__ __forceinline__ float value8(uint32_t code, uint32_t e)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)code));
    const float f = __half2float(__ushort_as_half((uint16_t)h)) * scale8(e);
    return fabsf(f) > kMost8<T> ? copysignf(kMost8<T>, f) : f;
}

// Whether runs of eight columns start on 8-byte boundaries in every row.
inline bool rows_aligned8(const void* p, int64_t ld, int rows)
{
    return (reinterpret_cast<uintptr_t>(p) & 7u) == 0 && (rows <= 1 || ld % 8 == 0);
}

// Checks a matrix in 8 bits (rows > 0).
inline dlrm_status check_packed(const char* fn, const char* name, const uint8_t* q, int64_t ld, const uint8_t* exps, int rows,
                                int cols)
{
    const dlrm_status s = check_matrix(fn, name, q, ld, rows, cols, 1);
    if (s != DLRM_OK) return s;
    if (!exps) return fail(DLRM_ERR_INVALID_ARG, "%s: %s has no exponents", fn, name);
    return DLRM_OK;
}

}  // namespace dlrm
