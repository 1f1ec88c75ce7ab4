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

// Rows of up to 128 columns are a few lanes' each, a power of two; longer ones take warps (norm_warps).  Measured, us, few
// lanes / a warp a row, 65536 rows, bf16: forward of 16 columns 10 / 26, 64 14 / 26, 128 24 / 27, 99 (off the grid) 31 / 41;
// gradient 17 / 41, 24 / 41, 37 / 42, 52 / 74.
inline int norm_lanes(int N) { return N <= 32 ? 4 : N <= 64 ? 8 : N <= 128 ? 16 : 32; }

// Warps of a row, 256 columns each: every number to 8, then in steps that leave a fifth idle at most up to 24.  (Powers of two
// only, us: 40000 x 1280 fp16 forward 135, so 98 and gradient 209, 143; 10000 x 4500 bf16 gradient 522, 297.)
inline int norm_warps(int N)
{
    const int w = (N + 255) / 256;
    return w <= 8 ? w : w <= 12 ? (w + 1) / 2 * 2 : w <= 24 ? (w + 3) / 4 * 4 : 32;
}

// Blocks of an SM and rows of a block where W warps take a row: blocks of eight warps, or of one group where W is more,
// or one block of as many groups as fit where eight are no whole number of groups.  From 16 warps on an SM has one
// row at a time, in the gradient of both norms from 10 on (bwd_warps).
constexpr bool norm_eights(int W) { return W <= 8 && 8 % W == 0; }
constexpr int norm_per_sm(int W, int warps) { return norm_eights(W) ? warps / 8 : W > 8 && warps >= 2 * W ? warps / W : 1; }
constexpr int norm_groups(int W, int warps) { return W > 8 ? 1 : norm_eights(W) ? 8 / W : warps / W; }

// Warps an SM at most.  More hide more of a row's chain of sums, at fewer registers each.  Measured, us, 16 / 24 warps:
// forward 22924 x 2272 fp16 201 / 141, 40000 x 1536 bf16 125 / 107; in blocks of eight warps on the grid 65536 x 1024 bf16
// 111 / 117, off it (any) 40000 x 771 bf16 141 / 123, 40000 x 201 37 / 41.  Gradient on the grid of the norm before the
// next block alone 16000 x 2904 bf16 145 / 90, 65536 x 1024 117 / 98; of that after the block 22924 x 2272 149 / 121 and
// the same with 20; of both 219 / 244; off the grid 30000 x 1700 109 / 115, a few lanes a row 12 / 14.
constexpr int fwd_warps(int W, bool any) { return norm_eights(W) && (W == 1 || !any) ? 16 : 24; }
constexpr int bwd_warps(bool post, bool pre, bool grid) { return !grid || (post && pre) ? 16 : pre ? 24 : 20; }

inline bool on_grid(bool vec, int N) { return vec && norm_lanes(N) == kWarp; }

inline int norm_blocks(int M, int N, int warps)
{
    const int w = norm_warps(N), rows = norm_groups(w, warps) * (kWarp / norm_lanes(N));
    const int64_t want = ((int64_t)M + rows - 1) / rows, most = (int64_t)num_sms() * norm_per_sm(w, warps);
    return (int)(want < most ? want : most);
}

// vec: rows and vectors are on the 16-byte grid
template <typename T>
dlrm_status forward(const NormFwd& a, bool vec, cudaStream_t st);
template <typename T>
dlrm_status backward(const NormBwd& a, bool vec, cudaStream_t st);

}  // namespace norms
}  // namespace dlrm
