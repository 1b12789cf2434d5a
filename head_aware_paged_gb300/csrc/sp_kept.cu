// sp_kept.cu -- launches of the decode over chosen pages in one kernel
// (sp_kept.cuh), and its instances for scores as they are.
#include "sp_kept.cuh"

namespace sp {

cudaError_t launch_kept(const sp_cache* c, KeptParams& p, cudaStream_t s) {
    // Blocks a unit (a power of two, 16 at most): as many as run at once, three an SM
    // less what clusters cannot use of a group of SMs.  Twice as many, and some units
    // start when others have ended: 45 units of 64 pages with 8 blocks each 17.3 us,
    // 16 each 30.7 us; 128 units with 2 and 4 each 27.7 and 40 us.  Half as many:
    // 20.5 us with 4 each, 42.5 us with 1 each.
    const int units = p.n_seqs * c->geo.hkv;
    p.log_ranks = 0;
    while (p.log_ranks < 4 && 2 * (units << (p.log_ranks + 1)) <= 5 * c->num_sms) ++p.log_ranks;
    return p.score_cap.on ? launch_kept_capped(p, s) : launch_kept_any<false>(p, s);
}

}  // namespace sp
