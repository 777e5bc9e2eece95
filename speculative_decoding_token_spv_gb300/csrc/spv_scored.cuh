// spv_scored.cuh -- arguments of the attention kernels of calls with scores.
#pragma once

#include "spv_attention.cuh"
#include "spv_scores.cuh"

namespace spv {

// The arguments of a call with scores.
struct ScoredParams : AttParams {
    ScoresView sc;
};
ScoredParams scored_params(const AttentionLaunch &L);
__device__ __forceinline__ const Work &work_of(const AttParams &p) { return p.w; }
__host__ __device__ __forceinline__ ScoredWork work_of(const ScoredParams &p)
{
    ScoredWork w;
    static_cast<Work &>(w) = p.w;
    w.sc = p.sc;
    return w;
}

// Attention in tiles of 128 or 256 query rows: spv_prompt_attention, and
// spv_paged_attention_scored of many rows a key head.  `pairs`: two tiles of 128
// rows at a time (head_dim up to 128; the workspace has to have room for pieces
// of so many).
cudaError_t launch_tiles(const ScoredParams &p, const KvLaunch &L, bool pairs, cudaStream_t st);
constexpr int TILES_PAIR_ROWS = 256;  // of a piece then

}  // namespace spv
