// spv_tiles_e4m3.cu -- attention in tiles of query rows, e4m3 cache.
#include "spv_tiles.cuh"

namespace spv {

cudaError_t launch_tiles_e4m3(const TilesParams &p, const KvLaunch &L, bool pairs, cudaStream_t st)
{
    return launch_tiles_types<__nv_fp8_e4m3>(p, L, pairs, st);
}

}  // namespace spv
