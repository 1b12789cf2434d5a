// sp_kept_capped.cu -- the instances of k_kept (sp_kept.cuh) for bf16 pages and scores capped
// by a tanh.
#include "sp_kept.cuh"

namespace sp {

cudaError_t launch_kept_bf16_capped(KeptParams& p, const KeptLoad& load, bool& serves, cudaStream_t s) {
    return launch_kept_bf16<true>(p, load, serves, s);
}

}  // namespace sp
