// sp_choose.cu -- the pages that a decode query keeps of each GLOBAL head: its
// first and its newest ones, and of the others those with the highest scores
// (sp_bounds.cuh), ties to the lower page.
//
// One launch: the blocks of a unit score its candidates, and the last of them to
// finish (an atomic ticket, no waiting) finds the `top`-th highest score digit by
// digit and lays the kept pages' places in the pool end to end for the decode,
// which then streams them as if they were the whole unit.
#include <algorithm>

#include "sp_bounds.cuh"
#include "sp_device.cuh"
#include "sp_internal.h"

namespace sp {

namespace {

constexpr int kChooseThreads = 256;
constexpr int kChooseWarps = kChooseThreads / 32;

// Order-preserving key of a score (never NaN).
__device__ __forceinline__ uint32_t score_key(float x) {
    const uint32_t u = __float_as_uint(x);
    return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

template <int D>
__global__ void __launch_bounds__(kChooseThreads) k_choose(const __grid_constant__ ChooseParams p) {
    constexpr int T = 2 * D / 16;                     // lanes of a page: 16 bytes of bounds each
    __shared__ __align__(16) uint32_t qw[16][2 * D / 4];   // a head's codes >= 0, then those <= 0
    __shared__ float qstep[16];
    __shared__ int32_t hist[256], warp_sum[2][kChooseWarps], found[2], last;
    const Geo& g = p.geo;
    const int u = blockIdx.x, b = u / g.hkv, h = u - b * g.hkv, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
    uint32_t* key = p.score + (int64_t)u * g.max_pages_unit;
    if (p.top > 0) {
        const int c0 = blockIdx.y * p.chunk, c1 = min(c0 + p.chunk, m);
        if (c0 >= m) return;
        // the query heads' codes
        for (int r = warp; r < g.group; r += kChooseWarps) {
            const __nv_bfloat16* q = p.q + ((int64_t)b * g.hq + h * g.group + r) * D;
            float x[D / 32], top = 0.f;
            #pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                x[i] = __bfloat162float(q[lane * (D / 32) + i]);
                top = fmaxf(top, fabsf(x[i]));
            }
            #pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const int e = grid_exponent(top);
            const float up = grid_step(-e);
            int8_t* pos = reinterpret_cast<int8_t*>(qw[r]);
            #pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const int code = (int)rintf(fminf(fmaxf(x[i] * up, -127.f), 127.f));
                pos[lane * (D / 32) + i] = (int8_t)max(code, 0);
                pos[D + lane * (D / 32) + i] = (int8_t)min(code, 0);
            }
            if (lane == 0) qstep[r] = grid_step(e);
        }
        __syncthreads();
        const int li = tid % T;
        for (int base = c0; base < c1; base += kChooseThreads / T) {      // (the same trips for every lane of a warp)
            const int c = base + tid / T;
            const bool live = c < c1;
            int32_t page = live ? tab[p.first + c] : 0;
            if (page < 0 || page >= g.num_pages) {
                atomicOr(p.meta.status, kStatusBadPage);
                page = 0;
            }
            const int4 w = __ldg(reinterpret_cast<const int4*>(p.codes + (int64_t)page * 2 * D) + li);
            float best = -INFINITY;
            for (int r = 0; r < g.group; ++r) {
                const int4 x = *reinterpret_cast<const int4*>(&qw[r][li * 4]);
                int s = __dp4a(w.x, x.x, 0);
                s = __dp4a(w.y, x.y, s);
                s = __dp4a(w.z, x.z, s);
                s = __dp4a(w.w, x.w, s);
                #pragma unroll
                for (int o = 1; o < T; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                best = fmaxf(best, (float)s * qstep[r]);
            }
            if (live && li == 0) key[c] = score_key(best * p.step[page]);
        }
        __threadfence();
        __syncthreads();
        if (tid == 0) {
            const int blocks = (m + p.chunk - 1) / p.chunk;
            last = atomicAdd(&p.tickets[u], 1) == blocks - 1;
            if (last) p.tickets[u] = 0;
        }
        __syncthreads();
        if (!last) return;
        __threadfence();
    } else if (blockIdx.y != 0) {
        return;
    }
    for (int j = tid; j < p.first + p.newest; j += kChooseThreads) {
        const int at = j < p.first ? j : j + p.top, pg = j < p.first ? j : nb - p.newest + (j - p.first);
        kept[at] = tab[pg];
        if (pages) pages[at] = pg;
    }
    if (p.top == 0) return;
    // The top-th highest key, eight bits at a time: `want` of the keys that start
    // with `prefix` are among the highest.
    uint32_t prefix = 0;
    int want = p.top;
    for (int shift = 24; shift >= 0; shift -= 8) {
        hist[tid] = 0;
        __syncthreads();
        for (int c = tid; c < m; c += kChooseThreads) {
            const uint32_t k = __ldcg(key + c);
            if (shift == 24 || (k >> (shift + 8)) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1);
        }
        __syncthreads();
        // keys in this and higher bins: a suffix sum over the 256 bins
        int x = hist[tid];
        const int mine = x;
        #pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_down_sync(0xffffffffu, x, o);
            if (lane + o < 32) x += y;
        }
        if (lane == 0) warp_sum[0][warp] = x;
        __syncthreads();
        for (int w = warp + 1; w < kChooseWarps; ++w) x += warp_sum[0][w];
        if (x >= want && x - mine < want) {
            found[0] = tid;
            found[1] = want - (x - mine);
        }
        __syncthreads();
        prefix = (prefix << 8) | (uint32_t)found[0];
        want = found[1];
        __syncthreads();
    }
    // Thread t's run of candidates: how many lie above the key, and on it; then
    // all above and the first `want` on it, in order.
    const int per = (m + kChooseThreads - 1) / kChooseThreads, r0 = min(tid * per, m), r1 = min(r0 + per, m);
    int above = 0, on = 0;
    for (int c = r0; c < r1; ++c) {
        const uint32_t k = __ldcg(key + c);
        above += k > prefix;
        on += k == prefix;
    }
    int sa = above, so = on;
    #pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int ya = __shfl_up_sync(0xffffffffu, sa, o), yo = __shfl_up_sync(0xffffffffu, so, o);
        if (lane >= o) { sa += ya; so += yo; }
    }
    if (lane == 31) { warp_sum[0][warp] = sa; warp_sum[1][warp] = so; }
    __syncthreads();
    for (int w = 0; w < warp; ++w) { sa += warp_sum[0][w]; so += warp_sum[1][w]; }
    sa -= above;
    so -= on;
    for (int c = r0; c < r1; ++c) {
        const uint32_t k = __ldcg(key + c);
        const bool take = k > prefix || (k == prefix && so < want);
        if (take) {
            const int at = p.first + sa + min(so, want);
            kept[at] = tab[p.first + c];
            if (pages) pages[at] = p.first + c;
        }
        sa += k > prefix;
        so += k == prefix;
    }
}

}  // namespace

cudaError_t launch_choose(const sp_cache* c, ChooseParams& p, cudaStream_t s) {
    // Candidates of the longest unit, a block's share of them
    int64_t most = 1;
    for (int b = 0; b < p.n_seqs; ++b)
        most = std::max<int64_t>(most, cdiv64(p.n[b], c->geo.page) - p.first - p.newest);
    p.chunk = 128;
    const dim3 grid((unsigned)(p.n_seqs * c->geo.hkv), (unsigned)((most + p.chunk - 1) / p.chunk));
    if (c->geo.d == 128) k_choose<128><<<grid, kChooseThreads, 0, s>>>(p);
    else k_choose<64><<<grid, kChooseThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace sp
