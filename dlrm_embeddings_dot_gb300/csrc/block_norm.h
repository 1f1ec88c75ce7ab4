// block_norm.h -- the norms' kernels as the entry points call them: block_norm.cu has the checks, and a
// file for each type its kernels (block_norm.cuh), which are compiled side by side.
#pragma once

#include "dense_ops.cuh"
#include "dlrm_block.h"

namespace dlrm {
namespace norms {

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

// Rows of up to 128 columns are a few lanes' each, longer ones take warps, a power of two.  Measured, us, few lanes / a
// warp a row, 65536 rows, bf16: forward of 16 columns 10 / 26, 64 14 / 26, 128 24 / 27, 99 (off the grid) 31 / 41;
// gradient 17 / 41, 24 / 41, 37 / 42, 52 / 74.
inline int norm_lanes(int N) { return N <= 32 ? 4 : N <= 64 ? 8 : N <= 128 ? 16 : 32; }

inline int norm_warps(int N)
{
    int w = 1;
    while (w * 256 < N) w *= 2;
    return w;
}

inline int norm_blocks(int M, int N)
{
    const int w = norm_warps(N), rows = w > 8 ? 1 : 8 / w * (kWarp / norm_lanes(N));
    const int64_t want = ((int64_t)M + rows - 1) / rows, most = (int64_t)num_sms() * (w > 8 ? 1 : 2);
    return (int)(want < most ? want : most);
}

// vec: rows and vectors are on the 16-byte grid
template <typename T>
dlrm_status forward(const NormFwd& a, bool vec, cudaStream_t st);
template <typename T>
dlrm_status backward(const NormBwd& a, bool vec, cudaStream_t st);

}  // namespace norms
}  // namespace dlrm
