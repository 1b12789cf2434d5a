// sp_decode.cu -- decode launches: the grid, and the instances of k_decode
// (sp_decode.cuh) for scores as they are.
#include "sp_decode.cuh"

namespace sp {

cudaError_t launch_decode(const sp_cache* c, DecodeParams& p, cudaStream_t s) {
    // Persistent grid, but at least kMinItemsPerCta pages per CTA: a small batch
    // then spreads one head over a few CTAs instead of dozens (fewer partials
    // to merge).
    constexpr int64_t kMinItemsPerCta = 8;
    int grid = c->decode_ctas;
    const int64_t want = (p.total_items + kMinItemsPerCta - 1) / kMinItemsPerCta;
    if (want < grid) grid = (int)(want > 0 ? want : 1);
    if (c->geo.fp4) return p.cap.on ? launch_decode4_capped(c, p, grid, s) : launch_decode4(c, p, grid, s);
    return p.cap.on ? launch_decode_capped(c, p, grid, s) : launch_decode_any<false>(c, p, grid, s);
}

}  // namespace sp
