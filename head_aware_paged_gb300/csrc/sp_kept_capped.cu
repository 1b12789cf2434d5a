// sp_kept_capped.cu -- the instances of k_kept (sp_kept.cuh) for scores capped by a
// tanh.
#include "sp_kept.cuh"

namespace sp {

cudaError_t launch_kept_capped(const KeptParams& p, cudaStream_t s) { return launch_kept_any<true>(p, s); }

}  // namespace sp
