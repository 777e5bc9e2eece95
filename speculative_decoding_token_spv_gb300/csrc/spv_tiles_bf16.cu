// spv_tiles_bf16.cu -- attention in tiles of query rows, bf16 cache.
#include "spv_tiles.cuh"

namespace spv {

cudaError_t launch_tiles_bf16(const TilesParams &p, const KvLaunch &L, bool pairs, cudaStream_t st)
{
    return launch_tiles_types<__nv_bfloat16>(p, L, pairs, st);
}

}  // namespace spv
