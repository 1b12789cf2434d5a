// sp_kept_coded.cu -- the instances of k_kept (sp_kept.cuh) for FP8 and 4-bit pages.
#include "sp_kept.cuh"

namespace sp {

cudaError_t launch_kept_coded_plain(KeptParams& p, const KeptLoad& load, bool& serves, cudaStream_t s) {
    return launch_kept_coded<false>(p, load, serves, s);
}

}  // namespace sp
