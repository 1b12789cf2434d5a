// sp_kept.cu -- the instances of k_kept (sp_kept.cuh) for bf16 pages and scores as they
// are.
#include "sp_kept.cuh"

namespace sp {

cudaError_t launch_kept_bf16_plain(KeptParams& p, const KeptLoad& load, bool& serves, cudaStream_t s) {
    return launch_kept_bf16<false>(p, load, serves, s);
}

}  // namespace sp
