// spv_mass.cu -- spv_attention_mass.
#include "spv_mass.cuh"

namespace spv {

cudaError_t launch_mass(const MassLaunch &L, cudaStream_t st)
{
    MassParams p{};
    mass_params(p, L);
    return launch_params(p, L.kv, st);
}

}  // namespace spv
