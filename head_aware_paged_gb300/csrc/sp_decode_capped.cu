// sp_decode_capped.cu -- the instances of k_decode (sp_decode.cuh) for scores
// capped by a tanh.
#include "sp_decode.cuh"

namespace sp {

cudaError_t launch_decode_capped(const sp_cache* c, DecodeParams& p, int grid, cudaStream_t s) {
    return launch_decode_any<true>(c, p, grid, s);
}

}  // namespace sp
