// spv_tiles_f16.cu -- attention in tiles of query rows, f16 cache.
#include "spv_tiles.cuh"

namespace spv {

cudaError_t launch_tiles_f16(const TilesParams &p, const KvLaunch &L, bool pairs, cudaStream_t st)
{
    return launch_tiles_types<__half>(p, L, pairs, st);
}

}  // namespace spv
