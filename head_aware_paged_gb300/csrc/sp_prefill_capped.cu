// sp_prefill_capped.cu -- the instances of k_prefill (sp_prefill.cuh) for
// scores capped by a tanh: one per page type and head_dim, whatever the page
// size.
#include "sp_prefill.cuh"

namespace sp {

cudaError_t launch_prefill_capped(sp_cache* c, const PrefillParams& p, int grid, bool two,
                                  const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                  cudaStream_t s) {
    if (c->geo.fp8) return launch_prefill_t<128, 0, true, false, false, true>(c, p, grid, tq, tk, tv, s);
    if (c->geo.fp4 && two) return launch_prefill_t<128, 0, false, true, false, true, true>(c, p, grid, tq, tk, tv, s);
    if (c->geo.fp4) return launch_prefill_t<128, 0, false, false, false, true, true>(c, p, grid, tq, tk, tv, s);
    if (two) return launch_prefill_t<128, 0, false, true, false, true>(c, p, grid, tq, tk, tv, s);
    if (c->geo.d == 128) return launch_prefill_t<128, 0, false, false, false, true>(c, p, grid, tq, tk, tv, s);
    return launch_prefill_t<64, 0, false, false, false, true>(c, p, grid, tq, tk, tv, s);
}

}  // namespace sp
