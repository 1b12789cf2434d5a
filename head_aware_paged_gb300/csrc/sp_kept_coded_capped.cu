// sp_kept_coded_capped.cu -- the instances of k_kept (sp_kept.cuh) for FP8 and 4-bit pages and scores
// capped by a tanh.
#include "sp_kept.cuh"

namespace sp {

cudaError_t launch_kept_coded_capped(KeptParams& p, const KeptLoad& load, bool& serves, cudaStream_t s) {
    return launch_kept_coded<true>(p, load, serves, s);
}

}  // namespace sp
