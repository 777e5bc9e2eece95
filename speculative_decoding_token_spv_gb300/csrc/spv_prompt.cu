// spv_prompt.cu -- spv_prompt_attention, and which kernel takes a call of many
// rows a key head.
#include "spv_scored.cuh"
#include "spv_tiles.cuh"

namespace spv {

cudaError_t launch_tiles_bf16(const TilesParams &p, const KvLaunch &L, bool pairs, cudaStream_t st);
cudaError_t launch_tiles_f16(const TilesParams &p, const KvLaunch &L, bool pairs, cudaStream_t st);
cudaError_t launch_tiles_e4m3(const TilesParams &p, const KvLaunch &L, bool pairs, cudaStream_t st);

cudaError_t launch_tiles(const ScoredParams &scored, const KvLaunch &L, bool pairs, cudaStream_t st)
{
    TilesParams p{};
    static_cast<ScoredParams &>(p) = scored;
    p.timeouts = L.row_status;
    p.q_bf16 = L.dtype == SPV_BF16;
    if (L.cache.dtype == SPV_E4M3) return launch_tiles_e4m3(p, L, pairs, st);
    return L.cache.dtype == SPV_BF16 ? launch_tiles_bf16(p, L, pairs, st) : launch_tiles_f16(p, L, pairs, st);
}

size_t prompt_ws_bytes(int, int, int, int, int head_dim)
{
    const int rows = head_dim == 256 ? 128 : TILES_PAIR_ROWS;
    return ATT_PARTS_AT + static_cast<size_t>(ATT_SMS) * 2 * rows * (head_dim + 2) * sizeof(float);
}

cudaError_t launch_prompt(const AttentionLaunch &L, cudaStream_t st)
{
    const KvLaunch &k = L.kv;
    const ScoredParams p = scored_params(L);
    if (k.row_status) {
        const cudaError_t e = launch_scored_status(p.c, work_of(p), k.row_status, st);
        if (e != cudaSuccess) return e;
    }
    return launch_tiles(p, k, p.rows > 128 && k.cache.head_dim <= 128, st);
}

}  // namespace spv
