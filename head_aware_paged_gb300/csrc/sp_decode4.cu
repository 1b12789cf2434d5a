// sp_decode4.cu -- the instances of k_decode4 (sp_decode4.cuh) for scores
// as they are.
#include "sp_decode4.cuh"

namespace sp {

cudaError_t launch_decode4(const sp_cache* c, DecodeParams& p, int grid, cudaStream_t s) {
    return launch_decode4_any<false>(c, p, grid, s);
}

}  // namespace sp
