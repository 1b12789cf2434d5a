// sp_prefill_rows.cu -- the instances of k_prefill (sp_prefill.cuh) whose
// history is the bf16 rows made from 4-bit pages (sp_dequant.cu), whatever the
// page size.
#include "sp_prefill.cuh"

namespace sp {

cudaError_t launch_prefill_rows(sp_cache* c, const PrefillParams& p, int grid, bool two, bool spec,
                                const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                cudaStream_t s) {
    if (spec) return launch_prefill_t<128, 0, false, true, true, false, true>(c, p, grid, tq, tk, tv, s);
    if (two) return launch_prefill_t<128, 0, false, true, false, false, true>(c, p, grid, tq, tk, tv, s);
    return launch_prefill_t<128, 0, false, false, false, false, true>(c, p, grid, tq, tk, tv, s);
}

}  // namespace sp
