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

// Keys of candidates [c0, c1) (page first + c of the unit), kTilePages a warp and
// pass; emit(c, key) is called by one lane each.  NH: steps of 8 query heads.  Every
// thread of the block takes part (one barrier).
template <int D, int NH, int WARPS, typename P, typename F>
__device__ __forceinline__ void score_pages(const P& p, QueryCodes<D, NH>& qc, const int32_t* tab, const __nv_bfloat16* q,
                                            int c0, int c1, F&& emit) {
    constexpr int NC = 2 * D / 64;                    // 64-byte pieces of a page's bounds
    const Geo& g = p.geo;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gl = lane >> 2, j = lane & 3;
    uint4 x[NC][2];
    float st[2];
    auto load = [&](int base) {
        const int c = base + warp * kTilePages + (lane & 15);
        int32_t page = c < c1 ? tab[p.first + c] : 0;
        if (page < 0 || page >= g.num_pages) {
            atomicOr(p.meta.status, kStatusBadPage);
            page = 0;
        }
        #pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int32_t pg = __shfl_sync(0xffffffffu, page, gl + 8 * r);
            const uint4* src = reinterpret_cast<const uint4*>(p.codes + (int64_t)pg * 2 * D) + j;
            #pragma unroll
            for (int i = 0; i < NC; ++i) x[i][r] = __ldg(src + 4 * i);
            st[r] = __ldg(p.step + pg);
        }
    };
    load(c0);
    for (int r = warp; r < 8 * NH; r += WARPS) {      // the query heads' codes
        float v[D / 32], top = 0.f;
        #pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            v[i] = r < g.group ? __bfloat162float(q[r * D + lane * (D / 32) + i]) : 0.f;
            top = fmaxf(top, fabsf(v[i]));
        }
        #pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const int e = grid_exponent(top);
        const float up = grid_step(-e);
        #pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            const int code = (int)rintf(fminf(fmaxf(v[i] * up, -127.f), 127.f));
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
    for (int base = c0; base < c1; base += WARPS * kTilePages) {
        float best[2] = {-INFINITY, -INFINITY};
        #pragma unroll
        for (int nh = 0; nh < NH; ++nh) {
            int s[4] = {0, 0, 0, 0};
            #pragma unroll
            for (int i = 0; i < NC; ++i) {
                mma_s8_16832(s, x[i][0].x, x[i][1].x, x[i][0].y, x[i][1].y, qb[nh][i].x, qb[nh][i].y);
                mma_s8_16832(s, x[i][0].z, x[i][1].z, x[i][0].w, x[i][1].w, qb[nh][i].z, qb[nh][i].w);
            }
            #pragma unroll
            for (int e = 0; e < 4; ++e)
                if (8 * nh + 2 * j + (e & 1) < g.group)
                    best[e >> 1] = fmaxf(best[e >> 1], (float)s[e] * (qs[nh][e & 1] * st[e >> 1]));
        }
        if (base + WARPS * kTilePages < c1) load(base + WARPS * kTilePages);
        #pragma unroll
        for (int r = 0; r < 2; ++r) {
            best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], 1));
            best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], 2));
        }
        const int c = base + warp * kTilePages + gl + 8 * j;
        if (j < 2 && c < c1) emit(c, score_key(j ? best[1] : best[0]));
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
// part; the keys are in place before the call.
//
// Keys at or above `cut` are taken, and of those in [low, cut) the first `want`
// (once they are all equal).  A pass counts a range's keys in bins and keeps the one
// that the want-th highest lies in; the first spans the keys' own range, so that few
// share a bin and one pass mostly does.
template <int WARPS, typename K, typename F>
__device__ __forceinline__ void choose_top(ChooseShared<WARPS>& sh, int m, int top, K&& key_at, F&& emit) {
    constexpr int T = WARPS * 32, kBinBits = WARPS == 8 ? 10 : 9;
    static_assert(4 * T == 1 << kBinBits, "four bins a thread");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t lo = 0xFFFFFFFFu, hi = 0u;
    for (int c = tid; c < m; c += T) {
        const uint32_t k = key_at(c);
        lo = min(lo, k);
        hi = max(hi, k);
    }
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
        for (int c = tid; c < m; c += T) {
            const uint32_t k = key_at(c);
            if (k >= low && k - low <= wide) atomicAdd(&sh.hist[(k - low) >> shift], 1);
        }
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
    // Thread t's run of keys (an odd number of them: no two lanes on one bank): how
    // many are at or above the cut, how many below it; then all of the former and
    // the first `want` of the latter, in order.
    const int per = ((m + T - 1) / T) | 1, r0 = min(tid * per, m), r1 = min(r0 + per, m);
    int above = 0, on = 0;
    for (int c = r0; c < r1; ++c) {
        const uint32_t k = key_at(c);
        above += k >= cut;
        on += k >= low && k < cut;
    }
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
    for (int c = r0; c < r1; ++c) {
        const uint32_t k = key_at(c);
        const bool up = k >= cut, tie = !up && k >= low;
        if (up || (tie && so < want)) emit(sa + min(so, want), c);
        sa += up;
        so += tie;
    }
}

}  // namespace

}  // namespace sp
