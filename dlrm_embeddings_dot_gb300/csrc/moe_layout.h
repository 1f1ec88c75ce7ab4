/*
 * moe_layout.h -- the dynamic shared memory of the mixture's two kernels: what the
 * host asks for and what the kernels use, from the same functions.  Plain C++,
 * so that a host compiler can check the sizes.
 */
#pragma once

#include <stddef.h>
#include <stdint.h>

#ifdef __CUDACC__
#define DLRM_LAYOUT __host__ __device__ constexpr
#else
#define DLRM_LAYOUT constexpr
#endif

namespace dlrm {
namespace moe {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kRows = 16;        // weight rows of a tile
constexpr int kPitch = 20;       // floats between tokens of a partial tile
constexpr int kStages = 2, kSteps = 8, kStage = kSteps * 1024;   // a step: 16 rows by 64 bytes
constexpr size_t kRing = (size_t)kWarps * kStages * kStage;

// The kernels' area begins at the next 128-byte boundary (TMA's) behind their static
// arrays, wherever those end.
constexpr size_t kAlign = 128;
DLRM_LAYOUT uintptr_t area(uintptr_t raw) { return (raw + kAlign - 1) & ~(uintptr_t)(kAlign - 1); }
DLRM_LAYOUT size_t asked(size_t used) { return used + kAlign; }

// The experts' rows in tiles, and the warps that split a tile's K.
DLRM_LAYOUT int expert_tiles(int E) { return (E + kRows - 1) / kRows; }
DLRM_LAYOUT int router_split(int E) { return expert_tiles(E) < kWarps ? kWarps / expert_tiles(E) : 1; }

// moe_up: the rings (rows on the 16-byte grid only), which the logits use first (2 x
// 64 x 256 floats at most, which fit), then the partial tiles of nt times eight
// tokens.  Without rings the partial tiles lie over the logits.
DLRM_LAYOUT int token_tiles(int T) { return T <= 8 ? 1 : T <= 16 ? 2 : 4; }
DLRM_LAYOUT size_t logit_bytes(int T, int E) { return (size_t)(router_split(E) + 1) * T * expert_tiles(E) * kRows * 4; }
DLRM_LAYOUT size_t tile_bytes(int T) { return (size_t)kWarps * 2 * token_tiles(T) * 8 * kPitch * 4; }
DLRM_LAYOUT size_t up_used(int T, int E, bool rings)
{
    return rings ? kRing + tile_bytes(T) : logit_bytes(T, E) > tile_bytes(T) ? logit_bytes(T, E) : tile_bytes(T);
}

// moe_down: the rings, then each warp's sums of every token.
DLRM_LAYOUT size_t sum_bytes(int T) { return (size_t)kWarps * T * kPitch * 4; }
DLRM_LAYOUT size_t down_used(int T, bool rings) { return (rings ? kRing : 0) + sum_bytes(T); }

}  // namespace moe
}  // namespace dlrm
