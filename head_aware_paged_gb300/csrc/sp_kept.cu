// sp_kept.cu -- launches of the decode over chosen pages in one kernel
// (sp_kept.cuh), and its instances for scores as they are.
#include "sp_kept.cuh"

namespace sp {

cudaError_t launch_kept(const sp_cache* c, KeptParams& p, cudaStream_t s) {
    // Blocks a unit: enough to fill the GPU.
    const int units = p.n_seqs * c->geo.hkv;
    p.log_ranks = 0;
    while (p.log_ranks < 4 && (units << (p.log_ranks + 1)) <= 2 * c->num_sms) ++p.log_ranks;
    return p.score_cap.on ? launch_kept_capped(p, s) : launch_kept_any<false>(p, s);
}

}  // namespace sp
