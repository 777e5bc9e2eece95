// spv_mass_scored.cu -- spv_attention_mass_scored.
#include "spv_mass.cuh"

namespace spv {

cudaError_t launch_mass_scored(const MassLaunch &L, cudaStream_t st)
{
    ScoredMassParams p{};
    mass_params(p, L);
    p.sc = scores_view(L.scores);
    return launch_params(p, L.kv, st);
}

}  // namespace spv
