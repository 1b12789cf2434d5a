// sp_choose.cuh -- scores of pages and the choice of the best ones (definitions:
// sp_bounds.cuh), as parts of a block: of k_choose (sp_choose.cu), which chooses for
// a decode that follows, and of k_kept (sp_kept.cuh), which reads the pages itself.
//
// Scores: pages are the M side of 8-bit integer products (exact), query heads the N
// side, two products of 32 bytes for every 64 of a page's bounds.  A lane reads 16
// bytes of each 64 of its two pages, so the order of the dimensions inside a product
// is permuted, the same way for pages and queries.
#pragma once
#include "sp_bounds.cuh"
#include "sp_device.cuh"
#include "sp_internal.h"

namespace sp {

namespace {

constexpr int kTilePages = 16;                        // pages of a warp's tile
constexpr int kListKeys = 4096;                       // keys that a block holds in shared memory

// Order-preserving key of a score (never NaN).
__device__ __forceinline__ uint32_t score_key(float x) {
    const uint32_t u = __float_as_uint(x);
    return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ void mma_s8_16832(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int D, int NH>
struct QueryCodes {
    __align__(16) uint8_t code[8 * NH][2 * D];        // a head's codes >= 0, then those <= 0
    float step[8 * NH];
};

// Physical pages of this lane's candidates in its warp's first kTiles tiles of
// [c0, c1) (candidate c is page first + c of the unit).
constexpr int kTiles = 2;
template <int WARPS>
__device__ __forceinline__ void first_pages(const int32_t* tab, int first, int c0, int c1, int32_t (&id)[kTiles]) {
    #pragma unroll
    for (int t = 0; t < kTiles; ++t) {
        const int c = c0 + ((threadIdx.x >> 5) + t * WARPS) * kTilePages + (threadIdx.x & 15);
        id[t] = c < c1 ? tab[first + c] : 0;
    }
}

// Keys of candidates [c0, c1): a warp takes every WARPS-th tile, kTiles of them in
// flight, the first ones' pages given.  emit(c, key, half) is called for each by
// two lanes, half 0 and 1; ready() once before the first.  NH: steps of 8 query
// heads.  Every thread of the block takes part (one barrier).
template <int D, int NH, int WARPS, typename P, typename G, typename F>
__device__ __forceinline__ void score_pages(const P& p, QueryCodes<D, NH>& qc, const int32_t* tab, const __nv_bfloat16* q,
                                            int c0, int c1, int32_t (&id)[kTiles], G&& ready, F&& emit) {
    constexpr int NC = 2 * D / 64;                    // 64-byte pieces of a page's bounds
    constexpr int kStep = WARPS * kTilePages;
    const Geo& g = p.geo;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gl = lane >> 2, j = lane & 3;
    struct Tile { uint4 x[NC][2]; float st[2]; };
    auto page_of = [&](int base) {                    // of this lane's candidate of a tile
        const int c = base + (lane & 15);
        return c < c1 ? tab[p.first + c] : 0;
    };
    auto load = [&](Tile& t, int32_t page) {
        if (page < 0 || page >= g.num_pages) {
            atomicOr(p.meta.status, kStatusBadPage);
            page = 0;
        }
        #pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int32_t pg = __shfl_sync(0xffffffffu, page, gl + 8 * r);
            const uint4* src = reinterpret_cast<const uint4*>(p.codes + (int64_t)pg * 2 * D) + j;
            #pragma unroll
            for (int i = 0; i < NC; ++i) t.x[i][r] = __ldg(src + 4 * i);
            t.st[r] = __ldg(p.step + pg);
        }
    };
    Tile tile[kTiles];
    const int base0 = c0 + warp * kTilePages;
    // the query heads' codes (a head that is not there: whatever the memory held, not used)
    float v[(8 * NH + WARPS - 1) / WARPS][D / 32];
    #pragma unroll
    for (int k = 0; k * WARPS < 8 * NH; ++k)
        #pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            const int r = warp + k * WARPS;
            v[k][i] = r < g.group ? __bfloat162float(q[r * D + lane * (D / 32) + i]) : 0.f;
        }
    #pragma unroll
    for (int t = 0; t < kTiles; ++t) {
        if (base0 + t * kStep < c1) load(tile[t], id[t]);
        id[t] = page_of(base0 + (t + kTiles) * kStep);
    }
    #pragma unroll
    for (int k = 0; k * WARPS < 8 * NH; ++k) {
        const int r = warp + k * WARPS;
        if (r >= g.group) break;
        float top = 0.f;
        #pragma unroll
        for (int i = 0; i < D / 32; ++i) top = fmaxf(top, fabsf(v[k][i]));
        // (of floats that are not negative, the largest is the largest pattern)
        top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
        const int e = grid_exponent(top);
        const float up = grid_step(-e);
        #pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            const int code = (int)rintf(fminf(fmaxf(v[k][i] * up, -127.f), 127.f));
            qc.code[r][lane * (D / 32) + i] = (uint8_t)max(code, 0);
            qc.code[r][D + lane * (D / 32) + i] = (uint8_t)min(code, 0);
        }
        if (lane == 0) qc.step[r] = grid_step(e);
    }
    __syncthreads();
    uint4 qb[NH][NC];
    float qs[NH][2];
    #pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
        #pragma unroll
        for (int i = 0; i < NC; ++i) qb[nh][i] = *reinterpret_cast<const uint4*>(&qc.code[8 * nh + gl][64 * i + 16 * j]);
        #pragma unroll
        for (int e = 0; e < 2; ++e) qs[nh][e] = qc.step[8 * nh + 2 * j + e];
    }
    ready();
    auto score = [&](const Tile& t, int base) {
        float best[2] = {-INFINITY, -INFINITY};
        #pragma unroll
        for (int nh = 0; nh < NH; ++nh) {
            int s[4] = {0, 0, 0, 0};
            #pragma unroll
            for (int i = 0; i < NC; ++i) {
                mma_s8_16832(s, t.x[i][0].x, t.x[i][1].x, t.x[i][0].y, t.x[i][1].y, qb[nh][i].x, qb[nh][i].y);
                mma_s8_16832(s, t.x[i][0].z, t.x[i][1].z, t.x[i][0].w, t.x[i][1].w, qb[nh][i].z, qb[nh][i].w);
            }
            #pragma unroll
            for (int e = 0; e < 4; ++e)
                if (8 * nh + 2 * j + (e & 1) < g.group)
                    best[e >> 1] = fmaxf(best[e >> 1], (float)s[e] * (qs[nh][e & 1] * t.st[e >> 1]));
        }
        #pragma unroll
        for (int r = 0; r < 2; ++r) {
            best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], 1));
            best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], 2));
        }
        const int c = base + gl + 8 * (j & 1);
        if (c < c1) emit(c, score_key((j & 1) ? best[1] : best[0]), j >> 1);
    };
    for (int base = base0; base < c1; base += kTiles * kStep)
        #pragma unroll
        for (int t = 0; t < kTiles; ++t) {
            const int at = base + t * kStep, next = at + kTiles * kStep;
            if (at >= c1) break;
            score(tile[t], at);
            if (next < c1) load(tile[t], id[t]);
            id[t] = page_of(next + kTiles * kStep);
        }
}

template <int WARPS>
struct ChooseShared {
    __align__(16) int32_t hist[WARPS * 128];
    uint32_t warp_min[WARPS], warp_max[WARPS];
    int32_t warp_sum[2][WARPS], found[3];
};

// The `top` highest of keys 0 .. m - 1 (top < m; ties: the lower index): calls
// emit(rank in order of index, index) for each.  Every thread of the block takes
// part; the keys are in place before the call.  A thread's run of neighbouring keys
// is held in registers, K of them (m <= 32 WARPS K, K odd), or read again for every
// pass (K = 0).
//
// Keys at or above `cut` are taken, and of those in [low, cut) the first `want`
// (once they are all equal).  A pass counts a range's keys in bins and keeps the one
// that the want-th highest lies in; the first spans the keys' own range, so that few
// share a bin and one pass mostly does.
template <int K, int WARPS, typename G, typename F>
__device__ __forceinline__ void choose_top(ChooseShared<WARPS>& sh, int m, int top, G&& key_at, F&& emit) {
    constexpr int T = WARPS * 32, kBinBits = WARPS == 8 ? 10 : 9;
    static_assert(4 * T == 1 << kBinBits, "four bins a thread");
    static_assert(K == 0 || K % 2 == 1, "odd runs: no two lanes on one bank");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = ((m + T - 1) / T) | 1, r0 = min(tid * per, m), r1 = min(r0 + per, m);
    uint32_t held[K > 0 ? K : 1];
    if constexpr (K > 0) {
        #pragma unroll
        for (int i = 0; i < K; ++i) held[i] = r0 + i < r1 ? key_at(r0 + i) : 0u;
    }
    // f(key, index) for this thread's keys, in order
    auto each = [&](auto&& f) {
        if constexpr (K > 0) {
            #pragma unroll
            for (int i = 0; i < K; ++i)
                if (r0 + i < r1) f(held[i], r0 + i);
        } else {
            for (int c = r0; c < r1; ++c) f(key_at(c), c);
        }
    };
    uint32_t lo = 0xFFFFFFFFu, hi = 0u;
    each([&](uint32_t k, int) {
        lo = min(lo, k);
        hi = max(hi, k);
    });
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) { sh.warp_min[warp] = lo; sh.warp_max[warp] = hi; }
    *reinterpret_cast<int4*>(&sh.hist[4 * tid]) = make_int4(0, 0, 0, 0);
    __syncthreads();
    #pragma unroll
    for (int w = 0; w < WARPS; ++w) { lo = min(lo, sh.warp_min[w]); hi = max(hi, sh.warp_max[w]); }
    uint32_t low = lo, wide = hi - lo, cut;           // the range is [low, low + wide]
    int want = top, shift = max(0, 32 - __clz(hi - lo) - kBinBits);
    while (true) {
        each([&](uint32_t k, int) {
            if (k >= low && k - low <= wide) atomicAdd(&sh.hist[(k - low) >> shift], 1);
        });
        __syncthreads();
        const int4 f = *reinterpret_cast<const int4*>(&sh.hist[4 * tid]);
        int s = f.x + f.y + f.z + f.w;                // of this thread's bins and all above
        const int own = s;
        #pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_down_sync(0xffffffffu, s, o);
            if (lane + o < 32) s += y;
        }
        if (lane == 0) sh.warp_sum[0][warp] = s;
        *reinterpret_cast<int4*>(&sh.hist[4 * tid]) = make_int4(0, 0, 0, 0);
        __syncthreads();
        #pragma unroll
        for (int w = 1; w < WARPS; ++w) s += w > warp ? sh.warp_sum[0][w] : 0;
        if (s >= want && s - own < want) {            // the bin is one of these four
            const int n4[4] = {f.x, f.y, f.z, f.w};
            int above = s - own;
            #pragma unroll
            for (int i = 3; i >= 0; --i) {
                if (above < want && above + n4[i] >= want) {
                    sh.found[0] = 4 * tid + i;
                    sh.found[1] = want - above;
                    sh.found[2] = n4[i];
                }
                above += n4[i];
            }
        }
        __syncthreads();
        low += (uint32_t)sh.found[0] << shift;
        want = sh.found[1];
        cut = low + (1u << shift);
        if (want == sh.found[2]) {                    // the whole bin
            cut = low;
            want = 0;
            break;
        }
        if (shift == 0) break;
        wide = (1u << shift) - 1;
        shift = max(0, shift - kBinBits);
    }
    // How many keys of the run are at or above the cut, how many on the bin below it;
    // then all of the former and the first `want` of the latter, in order.
    int above = 0, on = 0;
    each([&](uint32_t k, int) {
        above += k >= cut;
        on += k >= low && k < cut;
    });
    int sa = above, so = on;
    #pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int ya = __shfl_up_sync(0xffffffffu, sa, o), yo = __shfl_up_sync(0xffffffffu, so, o);
        if (lane >= o) { sa += ya; so += yo; }
    }
    if (lane == 31) { sh.warp_sum[0][warp] = sa; sh.warp_sum[1][warp] = so; }
    __syncthreads();
    #pragma unroll
    for (int w = 0; w < WARPS - 1; ++w)
        if (w < warp) { sa += sh.warp_sum[0][w]; so += sh.warp_sum[1][w]; }
    sa -= above;
    so -= on;
    each([&](uint32_t k, int c) {
        const bool up = k >= cut, tie = !up && k >= low;
        if (up || (tie && so < want)) emit(sa + min(so, want), c);
        sa += up;
        so += tie;
    });
}

}  // namespace

}  // namespace sp
