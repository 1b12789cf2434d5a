// sp_decode4_capped.cu -- the instances of k_decode4 (sp_decode4.cuh) for scores
// capped by a tanh.
#include "sp_decode4.cuh"

namespace sp {

cudaError_t launch_decode4_capped(const sp_cache* c, DecodeParams& p, int grid, cudaStream_t s) {
    return launch_decode4_any<true>(c, p, grid, s);
}

}  // namespace sp
