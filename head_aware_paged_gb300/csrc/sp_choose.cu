// sp_choose.cu -- the pages that a decode query keeps of each GLOBAL head: its
// first and its newest ones, and of the others those with the highest scores
// (sp_bounds.cuh), ties to the lower page; for a decode in a launch of its own.
//
// One launch: the blocks of a unit score its candidates, and the last of them to
// finish (an atomic ticket, no waiting) finds the `top` highest scores and lays the
// kept pages' places in the pool end to end for the decode, which then streams them
// as if they were the whole unit.  The decode is launched early and waits for the
// table where it needs it (its start costs as much as the choice).
//
// Bound by the bounds' bytes (2 d + 4 a candidate) when there are many units, by its
// chain of look-ups, barriers and passes when there are few.  Scores by dp4a, one
// 16-byte piece a lane and five shuffles a head: 24.1 us for 256 units of 504
// candidates (33 MB), 9.3 us for 8 units of 61; by integer products 18.9 and 7 us.
#include <algorithm>

#include "sp_choose.cuh"

namespace sp {

namespace {

constexpr int kChooseThreads = 256;
constexpr int kChooseWarps = kChooseThreads / 32;
static_assert(kListKeys <= 17 * kChooseThreads, "a block's registers hold the list");

// NH: steps of 8 query heads (group <= 8 NH).
template <int D, int NH>
__global__ void __launch_bounds__(kChooseThreads) k_choose(const __grid_constant__ ChooseParams p) {
    __shared__ QueryCodes<D, NH> qc;
    __shared__ ChooseShared<kChooseWarps> sh;
    __shared__ uint32_t list[kListKeys];
    __shared__ int32_t last;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Geo& g = p.geo;
    const int u = blockIdx.x, b = u / g.hkv, h = u - b * g.hkv, tid = threadIdx.x;
    const int64_t row = g.unit_row(p.seq[b], p.layer, h);
    int32_t* pages = p.pages ? p.pages + (int64_t)u * p.cap : nullptr;
    if (p.meta.pol[row].kind != kGlobal) {
        if (blockIdx.y == 0 && pages)
            for (int j = tid; j < p.cap; j += kChooseThreads) pages[j] = -1;
        return;
    }
    const int nb = (p.n[b] + g.page - 1) / g.page;
    const int32_t* tab = p.meta.ptab + row * g.max_pages_unit;
    int32_t* kept = p.kept + (int64_t)u * g.max_pages_unit;
    if (nb <= p.cap) {                                // all of them
        if (blockIdx.y != 0) return;
        for (int j = tid; j < nb; j += kChooseThreads) kept[j] = tab[j];
        if (pages)
            for (int j = tid; j < p.cap; j += kChooseThreads) pages[j] = j < nb ? j : -1;
        return;
    }
    const int m = nb - p.first - p.newest;            // candidates, more than p.top
    const int c0 = blockIdx.y * p.chunk, c1 = min(c0 + p.chunk, m);
    if (p.top > 0 ? c0 >= m : c0 > 0) return;
    if (c0 == 0)
        for (int j = tid; j < p.first + p.newest; j += kChooseThreads) {
            const int at = j < p.first ? j : j + p.top, pg = j < p.first ? j : nb - p.newest + (j - p.first);
            kept[at] = tab[pg];
            if (pages) pages[at] = pg;
        }
    if (p.top == 0) return;
    const bool alone = m <= p.chunk, listed = m <= kListKeys;
    uint32_t* key = p.score + (int64_t)u * g.max_pages_unit;
    int32_t id[kTiles];
    first_pages<kChooseWarps>(tab, p.first, c0, c1, id);
    score_pages<D, NH, kChooseWarps>(p, qc, tab, p.q + ((int64_t)b * g.hq + h * g.group) * D, c0, c1, id, [] {},
                                     [&](int c, uint32_t k, int half) {
                                         if (half == 0) (alone && listed ? list : key)[c] = k;
                                     });
    if (!alone) {
        __threadfence();
        __syncthreads();
        if (tid == 0) {
            last = atomicAdd(&p.tickets[u], 1) == (m + p.chunk - 1) / p.chunk - 1;
            if (last) p.tickets[u] = 0;
        }
        __syncthreads();
        if (!last) return;
        __threadfence();
        if (listed)
            for (int c = tid; c < m; c += kChooseThreads) list[c] = __ldcg(key + c);
    }
    __syncthreads();
    auto take = [&](int at, int c) { kept[p.first + at] = p.first + c; };
    if (listed) choose_top<17, kChooseWarps>(sh, m, p.top, [&](int c) { return list[c]; }, take);
    else choose_top<0, kChooseWarps>(sh, m, p.top, [&](int c) { return __ldcg(key + c); }, take);
    __syncthreads();
    for (int i = p.first + tid; i < p.first + p.top; i += kChooseThreads) {      // page numbers to places
        const int pg = kept[i];
        kept[i] = tab[pg];
        if (pages) pages[i] = pg;
    }
}

}  // namespace

cudaError_t launch_choose(const sp_cache* c, ChooseParams& p, cudaStream_t s) {
    // Candidates of the longest unit, a block's share of them
    int64_t most = 1;
    for (int b = 0; b < p.n_seqs; ++b)
        most = std::max<int64_t>(most, cdiv64(p.n[b], c->geo.page) - p.first - p.newest);
    const int64_t tile = kChooseWarps * kTilePages, most_blocks = 65535;
    p.chunk = (int32_t)(tile * cdiv64(most, tile * most_blocks));
    const dim3 grid((unsigned)(p.n_seqs * c->geo.hkv), (unsigned)((most + p.chunk - 1) / p.chunk));
    const bool wide = c->geo.group > 8;
    if (c->geo.d == 128) {
        if (wide) k_choose<128, 2><<<grid, kChooseThreads, 0, s>>>(p);
        else k_choose<128, 1><<<grid, kChooseThreads, 0, s>>>(p);
    } else {
        if (wide) k_choose<64, 2><<<grid, kChooseThreads, 0, s>>>(p);
        else k_choose<64, 1><<<grid, kChooseThreads, 0, s>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace sp
