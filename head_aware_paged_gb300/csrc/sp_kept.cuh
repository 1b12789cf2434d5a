// sp_kept.cuh -- choice and attention of a decode over chosen pages in one launch.
//
// A unit (sequence, KV head) reads a few dozen pages here, so what costs time is not
// the stream but everything around it: a second launch, the look-ups, the merge.
// A cluster of blocks therefore takes one unit from its query to its output:
//   1. scores: the blocks share the candidates and write each key into every block's
//      shared memory; after one cluster barrier all make the same choice
//      (sp_choose.cuh), so no list has to travel back;
//   2. attention: the unit's visible slots in groups of 16 (a group lies inside a page
//      whatever the page size), a neighbouring run of them per warp.  There is no
//      staging: a lane loads its operands' bytes of K and V straight into registers,
//      the next step's K as soon as the scores are taken and its V after the products;
//   3. merge: the warps' (o, m, l) meet in shared memory, the blocks' sums are written
//      to the block that finishes them (each a part of the output): one barrier.
// LOCAL and RETRIEVAL heads, and GLOBAL ones that keep everything, skip the first step.
//
// Keys are the M side of m16n8k16 and the query heads the N side, as in
// sp_decode4.cuh:
//     S^T = K Q^T      16 keys x 8 heads per group, D / 16 steps
//     O^T = V^T P^T    16 dimensions x 8 heads, D / 16 tiles
// The reduction over dimensions may run in any order, so a lane's 16-byte pieces of a
// key's row serve as they come; V's rows of two keys are interleaved by byte
// permutations.  P^T goes through two 8 x 8 register transposes.
//
// Scores, maxima, sums and partials are fp32.  P is rounded to V's type, for a product
// takes both operands in one: bf16 (2^-8 of a weight; it brings a row's error against 64
// bits from 0.0017, the output's own rounding, to 0.0019 .. 0.0023 of its norm), or f16 for
// FP8 and 4-bit pages (2^-11, nothing to see); the query under channel scales to f16.  A score's
// tanh is CUDA's (relative to the score it is exact to fp32; the difference of two
// numbers of the cap's size that k_decode takes, which is shorter, was 9e-6 off at a cap
// of 50 and showed in the lse of few keys; no difference in time).
//
// What it takes (8 KV heads of 4 query heads, d 128, page 64; with a launch for the
// choice in brackets): 1 x 4K, 16 of 64 pages 8.5 us (23); 1 x 128K, two heads GLOBAL,
// 128 of 2,048 pages 15.4 (40); 32 x 32K, all GLOBAL, 32 of 512 pages 61 (72): 9 us of
// it reading 34 MB of bounds, 2.5 until the stream starts, 43 streaming 268 MB at 6.2 TB/s.  Small
// calls are bound by their chain: look-ups, three barriers and about 1.1 us a step of
// 16 bf16 keys a warp.
//
// Measured and not kept: three tiles of bounds in flight (spills: 32 x 32K 63 us); the
// other blocks' keys read after the barrier instead of pushed before it (1 x 128K 3 us
// more); the choice by every warp alone, bisecting keys in registers (504 keys: 7 to 17
// us against 2); at 8 warps a block two steps in flight, or twice the keys a step (no
// change: a step's own chain of products, votes and exponentials decides).
#pragma once
#include <algorithm>
#include <mutex>

#include "sp_choose.cuh"
#include "sp_decode4.cuh"

namespace sp {

namespace {

static_assert(kKeptCandidates <= 33 * 128 && kKeptCandidates <= 17 * 256, "a block's registers hold the keys");

constexpr int kMaxKeptDevices = 64;

enum { kRowsBf16, kRowsFp8, kRowsFp4 };

template <int N>
struct Count { static constexpr int value = N; };

// What a lane holds of a step's NG groups, and the products' operands from it.
// Lane (gl, j): slots gl and gl + 8 of K, slots 2 j, 2 j + 1, 2 j + 8, 2 j + 9 of V.
template <int KV, int D>
struct Rows;

__device__ __forceinline__ uint4 ld_stream16(const void* p) {
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}
__device__ __forceinline__ uint2 ld_stream8(const void* p) {
    uint2 r;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
    return r;
}
__device__ __forceinline__ uint32_t ld_stream4(const void* p) {
    uint32_t r;
    asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(r) : "l"(p));
    return r;
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// bf16: a row in 64-byte pieces, 16 bytes of each a lane.
template <int D>
struct Rows<kRowsBf16, D> {
    static constexpr int NP = D * 2 / 64, NG = 4 / NP, NS = D / 128 ? 2 : 1;   // pieces, groups a step, chunk sets of V
    static constexpr int kGroupBytes = 16 * D * 2;
    uint4 k[NG][2][NP], v[NG][4][NS];
    __device__ __forceinline__ void load_k(int q, const uint8_t* grp, int gl, int j) {
        #pragma unroll
        for (int r = 0; r < 2; ++r)
            #pragma unroll
            for (int i = 0; i < NP; ++i) k[q][r][i] = ld_stream16(grp + (gl + 8 * r) * (D * 2) + 64 * i + 16 * j);
    }
    __device__ __forceinline__ void load_v(int q, const uint8_t* grp, int gl, int j) {
        #pragma unroll
        for (int r = 0; r < 4; ++r)
            #pragma unroll
            for (int i = 0; i < NS; ++i)
                v[q][r][i] = ld_stream16(grp + (2 * j + (r & 1) + 8 * (r >> 1)) * (D * 2) + (gl + 8 * i) * 16);
    }
    __device__ __forceinline__ void clear_k(int q) {
        #pragma unroll
        for (int r = 0; r < 2; ++r)
            #pragma unroll
            for (int i = 0; i < NP; ++i) k[q][r][i] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void clear_v(int q) {
        #pragma unroll
        for (int r = 0; r < 4; ++r)
            #pragma unroll
            for (int i = 0; i < NS; ++i) v[q][r][i] = make_uint4(0, 0, 0, 0);
    }
    // dimension of element e of step s's operand registers (0, 1: the first, 2, 3: the second)
    __device__ static int q_dim(int s, int e, int j) { return 32 * (s >> 1) + 8 * j + 4 * (s & 1) + e; }
    __device__ __forceinline__ void k_step(int q, int s, uint32_t (&a)[4]) const {
        const uint4 &x = k[q][0][s >> 1], &y = k[q][1][s >> 1];
        a[0] = (s & 1) ? x.z : x.x;
        a[1] = (s & 1) ? y.z : y.x;
        a[2] = (s & 1) ? x.w : x.y;
        a[3] = (s & 1) ? y.w : y.y;
    }
    // dimension of tile t, row half i
    __device__ static int v_dim(int t, int i, int gl) { return 8 * (gl + 8 * (t >> 2)) + 2 * (t & 3) + i; }
    template <typename F>
    __device__ __forceinline__ void v_tiles(int q, int, int, F&& f) const {
        #pragma unroll
        for (int t = 0; t < D / 16; ++t) {
            uint32_t w[4];
            #pragma unroll
            for (int r = 0; r < 4; ++r) w[r] = word(v[q][r][t >> 2], t & 3);
            const uint32_t a[4] = {prmt(w[0], w[1], 0x5410u), prmt(w[0], w[1], 0x7632u), prmt(w[2], w[3], 0x5410u),
                                   prmt(w[2], w[3], 0x7632u)};
            f(t, a);
        }
    }
    // slots of this lane's rows of S^T
    __device__ static int slot_a(int gl) { return gl; }
};

// FP8: codes become f16 (exact).
template <>
struct Rows<kRowsFp8, 128> {
    static constexpr int NG = 2;
    static constexpr int kGroupBytes = 16 * 128;
    uint4 k[NG][2][2], v[NG][4];
    __device__ __forceinline__ void load_k(int q, const uint8_t* grp, int gl, int j) {
        #pragma unroll
        for (int r = 0; r < 2; ++r)
            #pragma unroll
            for (int i = 0; i < 2; ++i) k[q][r][i] = ld_stream16(grp + (gl + 8 * r) * 128 + 64 * i + 16 * j);
    }
    __device__ __forceinline__ void load_v(int q, const uint8_t* grp, int gl, int j) {
        #pragma unroll
        for (int r = 0; r < 4; ++r) v[q][r] = ld_stream16(grp + (2 * j + (r & 1) + 8 * (r >> 1)) * 128 + gl * 16);
    }
    __device__ __forceinline__ void clear_k(int q) {
        #pragma unroll
        for (int r = 0; r < 2; ++r) k[q][r][0] = k[q][r][1] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void clear_v(int q) {
        #pragma unroll
        for (int r = 0; r < 4; ++r) v[q][r] = make_uint4(0, 0, 0, 0);
    }
    __device__ static int q_dim(int s, int e, int j) { return 64 * (s >> 2) + 16 * j + 4 * (s & 3) + e; }
    __device__ __forceinline__ void k_step(int q, int s, uint32_t (&a)[4]) const {
        f16x2x2_of_e4m3x4(word(k[q][0][s >> 2], s & 3), a[0], a[2]);
        f16x2x2_of_e4m3x4(word(k[q][1][s >> 2], s & 3), a[1], a[3]);
    }
    __device__ static int v_dim(int t, int i, int gl) { return 16 * gl + 2 * t + i; }
    template <typename F>
    __device__ __forceinline__ void v_tiles(int q, int, int, F&& f) const {
        #pragma unroll
        for (int w = 0; w < 4; ++w) {
            uint32_t x[4];
            #pragma unroll
            for (int r = 0; r < 4; ++r) x[r] = word(v[q][r], w);
            uint32_t a[4], b[4];
            f16x2x2_of_e4m3x4(prmt(x[0], x[1], 0x5140u), a[0], a[1]);
            f16x2x2_of_e4m3x4(prmt(x[2], x[3], 0x5140u), a[2], a[3]);
            f16x2x2_of_e4m3x4(prmt(x[0], x[1], 0x7362u), b[0], b[1]);
            f16x2x2_of_e4m3x4(prmt(x[2], x[3], 0x7362u), b[2], b[3]);
            f(2 * w, a);
            f(2 * w + 1, b);
        }
    }
    __device__ static int slot_a(int gl) { return gl; }
};

// 4-bit pages: the places of sp_fp4.cuh are those that these operands want.
template <>
struct Rows<kRowsFp4, 128> {
    static constexpr int NG = 4;
    static constexpr int kGroupBytes = kFp4GroupBytes;
    uint4 k[NG][2];
    uint2 v[NG][4];
    uint32_t ks[NG], vs[NG];
    __device__ __forceinline__ void load_k(int q, const uint8_t* grp, int gl, int j) {
        k[q][0] = ld_stream16(grp + gl * 64 + j * 16);
        k[q][1] = ld_stream16(grp + (gl + 8) * 64 + j * 16);
        ks[q] = ld_stream4(grp + kFp4ScaleOff + (gl * 4 + j) * 4);
    }
    __device__ __forceinline__ void load_v(int q, const uint8_t* grp, int gl, int j) {
        #pragma unroll
        for (int t = 0; t < 4; ++t) v[q][t] = ld_stream8(grp + (j + 4 * t) * 64 + (gl ^ ((j & 2) << 1)) * 8);
        vs[q] = ld_stream4(grp + kFp4ScaleOff + gl * 16 + j * 4);
    }
    __device__ __forceinline__ void clear_k(int q) {
        k[q][0] = k[q][1] = make_uint4(0, 0, 0, 0);
        ks[q] = 0;
    }
    __device__ __forceinline__ void clear_v(int q) {
        #pragma unroll
        for (int t = 0; t < 4; ++t) v[q][t] = make_uint2(0, 0);
        vs[q] = 0;
    }
    __device__ static int q_dim(int s, int e, int j) { return 32 * j + 4 * s + e; }
    __device__ __forceinline__ void k_step(int q, int s, uint32_t (&a)[4]) const {
        // word s / 2 of both rows: 8 dimensions, two steps; the scale of its block as f16, twice
        const uint32_t fa = prmt(ks[q], 0u, (s >> 2) ? 0x4141u : 0x4040u) << 7;
        const uint32_t fb = prmt(ks[q], 0u, (s >> 2) ? 0x4343u : 0x4242u) << 7;
        uint32_t x[4], y[4];
        fp4_word_f16(word(k[q][0], s >> 1), x[0], x[1], x[2], x[3]);
        fp4_word_f16(word(k[q][1], s >> 1), y[0], y[1], y[2], y[3]);
        a[0] = hmul2(x[2 * (s & 1)], fa);
        a[1] = hmul2(y[2 * (s & 1)], fb);
        a[2] = hmul2(x[2 * (s & 1) + 1], fa);
        a[3] = hmul2(y[2 * (s & 1) + 1], fb);
    }
    __device__ static int v_dim(int t, int i, int gl) { return 16 * gl + 2 * t + i; }
    template <typename F>
    __device__ __forceinline__ void v_tiles(int q, int, int, F&& f) const {
        const uint32_t f0 = prmt(vs[q], 0u, 0x4140u) << 7, f1 = prmt(vs[q], 0u, 0x4342u) << 7;
        constexpr uint32_t kLow = 0x0F0F0F0Fu;
        #pragma unroll
        for (int w = 0; w < 2; ++w) {
            uint32_t x[4];
            #pragma unroll
            for (int t = 0; t < 4; ++t) x[t] = w ? v[q][t].y : v[q][t].x;
            uint32_t a0[4], a1[4], a2[4], a3[4];
            fp4_word_f16((x[0] & kLow) | ((x[1] << 4) & ~kLow), a0[0], a0[1], a0[2], a0[3]);
            fp4_word_f16(((x[0] >> 4) & kLow) | (x[1] & ~kLow), a1[0], a1[1], a1[2], a1[3]);
            fp4_word_f16((x[2] & kLow) | ((x[3] << 4) & ~kLow), a2[0], a2[1], a2[2], a2[3]);
            fp4_word_f16(((x[2] >> 4) & kLow) | (x[3] & ~kLow), a3[0], a3[1], a3[2], a3[3]);
            #pragma unroll
            for (int t = 0; t < 4; ++t) {
                const uint32_t a[4] = {hmul2(a0[t], f0), hmul2(a1[t], f0), hmul2(a2[t], f1), hmul2(a3[t], f1)};
                f(4 * w + t, a);
            }
        }
    }
    __device__ static int slot_a(int gl) { return (gl >> 1) + 4 * (gl & 1); }
};

// A cluster's barrier; the first one only says that every block runs (its shared
// memory may be written from then on).
__device__ __forceinline__ void cluster_started() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Stores to shared memory of block `rank` of the cluster, at this block's address.
__device__ __forceinline__ uint32_t peer_smem(const void* local, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(local)), "r"(rank));
    return r;
}
__device__ __forceinline__ void st_peer(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// A block of W warps a cluster rank.  Registers: three blocks of 4 warps an SM at
// NH = 1 (two at NH = 2), or one of 8, for few units.
template <int KV, int D, int NH, int W, bool CAP>
__global__ void __launch_bounds__(W * 32, W == 8 ? 1 : NH == 1 ? 3 : 2) k_kept(const __grid_constant__ KeptParams p) {
    using R = Rows<KV, D>;
    constexpr int T = W * 32;
    constexpr int NG = R::NG, MT = D / 16, KS = D / 16, HF = D + 8;   // groups a step, tiles, steps, a head's floats
    extern __shared__ __align__(16) float parts[];    // [warps][group][HF], then the blocks' sums and all (m, l)
    __shared__ QueryCodes<D, NH> qc;
    __shared__ ChooseShared<W> sh;
    __shared__ uint32_t list[kKeptCandidates];
    __shared__ int32_t kept[kKeptPages];
    __shared__ __align__(8) float score_scale[8 * NH];
    __shared__ int32_t range_lo[3], range_hi[3], range_groups[3];    // visible slots, and the groups they touch
    const Geo& g = p.geo;
    const int group = g.group, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gl = lane >> 2, j = lane & 3;
    if (p.log_ranks > 0) cluster_started();
    const int u = (int)(blockIdx.x >> p.log_ranks), ranks = 1 << p.log_ranks, rank = blockIdx.x & (ranks - 1);
    const int b = u / g.hkv, h = u - b * g.hkv, seq = p.seq[b], lp = 31 - __clz(g.page);
    const int64_t row = g.unit_row(seq, p.layer, h);
    const UnitPol pol = p.meta.pol[row];
    const int32_t* tab = p.meta.ptab + row * g.max_pages_unit;
    const __nv_bfloat16* q0 = p.q + ((int64_t)b * g.hq + h * group) * D;
    int32_t* pages = p.pages && rank == 0 ? p.pages + (int64_t)u * p.cap : nullptr;
    const int n = p.n[b], nb = (n + g.page - 1) >> lp;
    // candidates (more than p.top), this block's share of them, and its first ones'
    // pages, looked up before the head's class is known
    const int m = nb - p.first - p.newest;
    const int per = ((m + ranks - 1) / ranks + kTilePages - 1) & ~(kTilePages - 1);
    const int c0 = min(rank * per, m), c1 = min(c0 + per, m);
    int32_t id[kTiles] = {};
    if (nb > p.cap && p.top > 0) first_pages<W>(tab, p.first, c0, c1, id);
    const bool chosen = pol.kind == kGlobal && nb > p.cap;

    // The query as the products' operand.  bf16 pages: as it is.  Others: f16, times a
    // power of two per head that takes the largest |q * channel scale| to 2^14 .. 2^15
    // (sp_decode4.cuh says why); the scores are multiplied back in fp32.
    const float* kscale = p.meta.kscale + ((int64_t)p.layer * g.hkv + h) * D;
    const float unit_scale = CAP ? p.scale_log2 / p.score_cap.a : p.scale_log2;      // (to score / cap, or to log2 units)
    uint32_t qb[NH][KS][2];
    #pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
        const int head = 8 * nh + gl;
        float top = 0.f;
        #pragma unroll
        for (int s = 0; s < KS; ++s)
            #pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t w = head < group
                    ? *reinterpret_cast<const uint32_t*>(q0 + head * D + R::q_dim(s, 2 * e, j)) : 0u;
                qb[nh][s][e] = w;
                if constexpr (KV != kRowsBf16) {
                    const __nv_bfloat162 v2 = *reinterpret_cast<const __nv_bfloat162*>(&w);
                    float x = __low2float(v2), y = __high2float(v2);
                    if (p.scaled) {
                        const float2 f = __ldg(reinterpret_cast<const float2*>(kscale + R::q_dim(s, 2 * e, j)));
                        x *= f.x;
                        y *= f.y;
                    }
                    top = fmax3_abs(top, x, y);
                }
            }
        float factor = 1.f;
        if constexpr (KV != kRowsBf16) {
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int ex = min(max(__float_as_int(top) >> 23, 15), 254);     // 2^(ex - 127) <= top
            const float up = __int_as_float((268 - ex) << 23);
            factor = __int_as_float((ex - 14) << 23);
            #pragma unroll
            for (int s = 0; s < KS; ++s)
                #pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const __nv_bfloat162 v2 = *reinterpret_cast<const __nv_bfloat162*>(&qb[nh][s][e]);
                    float x = __low2float(v2), y = __high2float(v2);
                    if (p.scaled) {
                        const float2 f = __ldg(reinterpret_cast<const float2*>(kscale + R::q_dim(s, 2 * e, j)));
                        x *= f.x;
                        y *= f.y;
                    }
                    qb[nh][s][e] = pack_f16(x * up, y * up);
                }
        }
        // (this lane's query is head gl, its scores are heads 2 j and 2 j + 1's)
        if (warp == 0 && j == 0) score_scale[head] = factor * unit_scale;
    }

    if (warp == W - 1 && lane == 0) {
        const int64_t t = chosen ? kept_slots(n, g.page, p.cap) - 1 : n - 1;
        const SlotRanges rg = decode_ranges(pol, p.meta.idx + (int64_t)seq * g.max_idx_per_seq + pol.idx_off, t, g.page);
        #pragma unroll
        for (int i = 0; i < 3; ++i) {
            range_lo[i] = (int32_t)rg.lo[i];
            range_hi[i] = (int32_t)rg.hi[i];
            range_groups[i] = rg.hi[i] > rg.lo[i] ? (int32_t)(((rg.hi[i] - 1) >> 4) - (rg.lo[i] >> 4) + 1) : 0;
        }
    }
    if (chosen) {
        for (int i = tid; i < p.first + p.newest; i += T) {
            const int at = i < p.first ? i : i + p.top, pg = i < p.first ? i : nb - p.newest + (i - p.first);
            kept[at] = tab[pg];
            if (pages) pages[at] = pg;
        }
        if (p.top > 0) {
            score_pages<D, NH, W>(p, qc, tab, q0, c0, c1, id, [&] { if (ranks > 1) cluster_wait(); },
                                  [&](int c, uint32_t k, int half) {
                                      if (ranks == 1) list[c] = k;               // (both halves the same)
                                      else for (int r = half; r < ranks; r += 2) st_peer(peer_smem(&list[c], r), k);
                                  });
            if (ranks > 1) { cluster_arrive(); cluster_wait(); } else __syncthreads();
            auto take = [&](int at, int c) { kept[p.first + at] = p.first + c; };
            auto key_at = [&](int c) { return list[c]; };
            if (m <= 5 * T) choose_top<5, W>(sh, m, p.top, key_at, take);
            else if (m <= 9 * T) choose_top<9, W>(sh, m, p.top, key_at, take);
            else if (m <= 17 * T) choose_top<17, W>(sh, m, p.top, key_at, take);
            else if constexpr (W == 4) choose_top<33, W>(sh, m, p.top, key_at, take);
            // page numbers to places: one look-up a thread, not one after another where
            // a thread's run holds several
            __syncthreads();
            for (int i = p.first + tid; i < p.first + p.top; i += T) {
                const int pg = kept[i];
                kept[i] = tab[pg];
                if (pages) pages[i] = pg;
            }
        }
    } else if (pages) {
        for (int i = tid; i < p.cap; i += T) pages[i] = pol.kind == kGlobal && i < nb ? i : -1;
    }

    __syncthreads();

    // The unit's visible slots are read in groups of 16; this warp's run [w0, w1) of them.
    const int total = range_groups[0] + range_groups[1] + range_groups[2];
    const int runs = ranks * W, run = rank * W + warp;
    const int w0 = (int)((int64_t)total * run / runs), w1 = (int)((int64_t)total * (run + 1) / runs);
    // Lane i of a batch of 32: group w0 + batch + i's place in the pool (in groups)
    // and its visible slots, low | high << 8 (0: none).
    uint32_t place = 0, seen = 0;
    int batch = -32;
    auto look_up = [&](int i) {
        int at = i;
        place = seen = 0;
        #pragma unroll
        for (int r = 0; r < 3; ++r) {
            if (at >= 0 && at < range_groups[r]) {
                const int32_t lo = range_lo[r], slot = ((lo >> 4) + at) << 4, pg = slot >> lp;
                const int32_t page = chosen ? kept[pg] : tab[pg];
                if (page < 0 || page >= g.num_pages) {
                    atomicOr(p.meta.status, kStatusBadPage);
                } else {
                    place = (((uint32_t)page << lp) + (uint32_t)(slot & (g.page - 1))) >> 4;
                    seen = (uint32_t)max(lo - slot, 0) | ((uint32_t)min(range_hi[r] - slot, 16) << 8);
                }
            }
            at -= range_groups[r];
        }
    };
    R rows;
    uint32_t vis[NG], vat[NG];                        // visible slots; places, for V
    auto take = [&](int i) {                          // groups w0 + i ...: look-ups, loads of K
        if (i >= batch + 32) {
            batch += 32;
            if (w0 + batch + lane < w1) look_up(w0 + batch + lane); else place = seen = 0;
        }
        #pragma unroll
        for (int q = 0; q < NG; ++q) {
            vis[q] = __shfl_sync(0xffffffffu, seen, i + q - batch);
            vat[q] = __shfl_sync(0xffffffffu, place, i + q - batch);
            if (vis[q]) rows.load_k(q, p.kpool + (int64_t)vat[q] * R::kGroupBytes, gl, j);
            else rows.clear_k(q);
        }
    };
    auto take_v = [&] {
        #pragma unroll
        for (int q = 0; q < NG; ++q) {
            if (vis[q]) rows.load_v(q, p.vpool + (int64_t)vat[q] * R::kGroupBytes, gl, j);
            else rows.clear_v(q);                     // (weight 0 times what the registers held would not do)
        }
    };
    float o[NH][MT][4], m_run[NH][2], l_run[NH][2];
    #pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
        m_run[nh][0] = m_run[nh][1] = -INFINITY;
        l_run[nh][0] = l_run[nh][1] = 0.f;
        #pragma unroll
        for (int t = 0; t < MT; ++t)
            #pragma unroll
            for (int e = 0; e < 4; ++e) o[nh][t][e] = 0.f;
    }
    const int mine = w1 - w0;
    if (mine > 0) { take(0); take_v(); }
    for (int i = 0; i < mine; i += NG) {
        float sc[NG][NH][4];
        #pragma unroll
        for (int q = 0; q < NG; ++q) {
            #pragma unroll
            for (int nh = 0; nh < NH; ++nh)
                #pragma unroll
                for (int e = 0; e < 4; ++e) sc[q][nh][e] = 0.f;
            #pragma unroll
            for (int s = 0; s < KS; ++s) {
                uint32_t a[4];
                rows.k_step(q, s, a);
                #pragma unroll
                for (int nh = 0; nh < NH; ++nh) {
                    if constexpr (KV == kRowsBf16) mma_bf16_16816(sc[q][nh], a, qb[nh][s][0], qb[nh][s][1]);
                    else mma_f16_16816(sc[q][nh], a, qb[nh][s][0], qb[nh][s][1]);
                }
            }
        }
        uint32_t now[NG];
        #pragma unroll
        for (int q = 0; q < NG; ++q) now[q] = vis[q];
        const bool more = i + NG < mine;
        if (more) take(i + NG);
        const int sa = R::slot_a(gl), sb = sa + 8;
        float mx[NH][2];
        bool grew = false;
        #pragma unroll
        for (int nh = 0; nh < NH; ++nh) {
            const float2 f = *reinterpret_cast<const float2*>(&score_scale[8 * nh + 2 * j]);
            #pragma unroll
            for (int e = 0; e < 2; ++e) mx[nh][e] = -INFINITY;
            #pragma unroll
            for (int q = 0; q < NG; ++q) {
                const int from = now[q] & 0xFF, to = now[q] >> 8;
                const bool in_a = sa >= from && sa < to, in_b = sb >= from && sb < to;
                #pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float x = sc[q][nh][e] * ((e & 1) ? f.y : f.x);
                    if constexpr (CAP) x = p.score_cap.a * tanhf(x);
                    x = (e < 2 ? in_a : in_b) ? x : -INFINITY;
                    sc[q][nh][e] = x;
                    mx[nh][e & 1] = fmaxf(mx[nh][e & 1], x);
                }
            }
            #pragma unroll
            for (int e = 0; e < 2; ++e) grew = grew || mx[nh][e] > m_run[nh][e] + kRefAbove;
        }
        // the exponentials' reference, raised only when a score passes it by kRefAbove
        if (__any_sync(0xffffffffu, grew)) {
            #pragma unroll
            for (int nh = 0; nh < NH; ++nh)
                #pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = mx[nh][e];
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                    const float m_new = fmaxf(m_run[nh][e], x - kRefBelow);
                    const float alpha = fast_exp2(m_run[nh][e] - (m_new == -INFINITY ? 0.f : m_new));
                    m_run[nh][e] = m_new;
                    l_run[nh][e] *= alpha;
                    #pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        o[nh][t][e] *= alpha;
                        o[nh][t][2 + e] *= alpha;
                    }
                }
        }
        uint32_t pb[NG][NH][2];
        #pragma unroll
        for (int q = 0; q < NG; ++q)
            #pragma unroll
            for (int nh = 0; nh < NH; ++nh) {
                float w[4];
                #pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float ref = m_run[nh][e & 1] == -INFINITY ? 0.f : m_run[nh][e & 1];
                    w[e] = fast_exp2(sc[q][nh][e] - ref);
                    l_run[nh][e & 1] += w[e];
                }
                if constexpr (KV == kRowsBf16) {
                    pb[q][nh][0] = transpose8x8(pack_bf16(w[0], w[1]));
                    pb[q][nh][1] = transpose8x8(pack_bf16(w[2], w[3]));
                } else {
                    pb[q][nh][0] = transpose8x8(pack_f16(w[0], w[1]));
                    pb[q][nh][1] = transpose8x8(pack_f16(w[2], w[3]));
                }
            }
        #pragma unroll
        for (int q = 0; q < NG; ++q)
            rows.v_tiles(q, gl, j, [&](int t, const uint32_t (&a)[4]) {
                #pragma unroll
                for (int nh = 0; nh < NH; ++nh) {
                    if constexpr (KV == kRowsBf16) mma_bf16_16816(o[nh][t], a, pb[q][nh][0], pb[q][nh][1]);
                    else mma_f16_16816(o[nh][t], a, pb[q][nh][0], pb[q][nh][1]);
                }
            });
        if (more) take_v();
    }

    // ------------------------------- merge -------------------------------
    // A head's sums lie in the tiles' order: dimension v_dim(t, i, gl) at 16 t + 2 gl + i.
    float* mine_o = parts + warp * group * HF;
    float* sums = parts + W * group * HF;                  // [ranks][group * D / ranks]
    float2* warp_ml = reinterpret_cast<float2*>(sums + group * D);  // [warps][group]
    float2* rank_ml = warp_ml + W * group;                 // [ranks][group]
    const float* vscale = p.meta.vscale + ((int64_t)p.layer * g.hkv + h) * D;
    #pragma unroll
    for (int nh = 0; nh < NH; ++nh)
        #pragma unroll
        for (int e = 0; e < 2; ++e) {
            float l = l_run[nh][e];
            l += __shfl_xor_sync(0xffffffffu, l, 4);
            l += __shfl_xor_sync(0xffffffffu, l, 8);
            l += __shfl_xor_sync(0xffffffffu, l, 16);
            const int head = 8 * nh + 2 * j + e;
            if (head >= group) continue;
            #pragma unroll
            for (int t = 0; t < MT; ++t)
                *reinterpret_cast<float2*>(mine_o + head * HF + 16 * t + 2 * gl) = make_float2(o[nh][t][e], o[nh][t][2 + e]);
            if (gl == 0) warp_ml[warp * group + head] = make_float2(m_run[nh][e], l);
        }
    if (ranks > 1 && !(chosen && p.top > 0)) cluster_wait();         // every block runs
    __syncthreads();
    __nv_bfloat16* out = p.out + ((int64_t)b * g.hq + h * group) * D;
    float* lse = p.lse ? p.lse + (int64_t)b * g.hq + h * group : nullptr;
    // a unit without a visible token: O = 0, LSE = -inf
    auto finish = [&](int r, int at, float acc, float m, float l) {
        const int c = R::v_dim(at >> 4, at & 1, (at >> 1) & 7);
        if (KV != kRowsBf16 && p.scaled) acc *= __ldg(vscale + c);
        out[r * D + c] = __float2bfloat16(l == 0.f ? 0.f : acc / l);
        if (at == 0 && lse) lse[r] = (m + __log2f(l)) * 0.69314718055994531f;
    };
    const int part = (group * D) >> p.log_ranks;                    // outputs that a block finishes
    for (int e = tid; e < group * D; e += T) {
        const int r = e / D, at = e % D;
        float m = -INFINITY, l = 0.f, acc = 0.f;
        float2 ml[W];
        #pragma unroll
        for (int w = 0; w < W; ++w) {
            ml[w] = warp_ml[w * group + r];
            m = fmaxf(m, ml[w].x);
        }
        const float ref = m == -INFINITY ? 0.f : m;
        #pragma unroll
        for (int w = 0; w < W; ++w) {
            const float f = fast_exp2(ml[w].x - ref);
            l += f * ml[w].y;
            acc += f * parts[(w * group + r) * HF + at];
        }
        if (ranks == 1) {
            finish(r, at, acc, m, l);
        } else {
            const int owner = e / part;
            st_peer(peer_smem(&sums[rank * part + (e - owner * part)], owner), __float_as_uint(acc));
            if (at < ranks) {                                       // (D >= ranks) lanes share the blocks to tell
                const uint32_t to = peer_smem(&rank_ml[rank * group + r], at);
                st_peer(to, __float_as_uint(m));
                st_peer(to + 4, __float_as_uint(l));
            }
        }
    }
    if (ranks == 1) return;
    cluster_arrive();
    cluster_wait();
    auto join = [&](auto count) {
        constexpr int N = decltype(count)::value;
        for (int e = tid; e < part; e += T) {
            const int r = (rank * part + e) / D, at = (rank * part + e) % D;
            float2 ml[N];
            float x[N], m = -INFINITY, l = 0.f, acc = 0.f;
            #pragma unroll
            for (int i = 0; i < N; ++i) {
                ml[i] = rank_ml[i * group + r];
                x[i] = sums[i * part + e];
            }
            #pragma unroll
            for (int i = 0; i < N; ++i) m = fmaxf(m, ml[i].x);
            const float ref = m == -INFINITY ? 0.f : m;
            #pragma unroll
            for (int i = 0; i < N; ++i) {
                const float f = fast_exp2(ml[i].x - ref);
                l += f * ml[i].y;
                acc += f * x[i];
            }
            finish(r, at, acc, m, l);
        }
    };
    if (ranks == 2) join(Count<2>());
    else if (ranks == 4) join(Count<4>());
    else if (ranks == 8) join(Count<8>());
    else join(Count<16>());
}

// An instance's launches, on the current device.
template <int KV, int D, int NH, int W, bool CAP>
struct KeptLaunch {
    static int bytes(int heads) { return (W * heads * (D + 8) + heads * D + 2 * (W + 16) * heads) * 4; }
    static void fill(cudaLaunchConfig_t& cfg, cudaLaunchAttribute& at, int units, int log_ranks, int heads, cudaStream_t s) {
        at.id = cudaLaunchAttributeClusterDimension;
        at.val.clusterDim.x = 1u << log_ranks;
        at.val.clusterDim.y = at.val.clusterDim.z = 1;
        cfg.gridDim = dim3((unsigned)units << log_ranks);
        cfg.blockDim = dim3(W * 32);
        cfg.dynamicSmemBytes = (size_t)bytes(heads);
        cfg.stream = s;
        cfg.attrs = &at;
        cfg.numAttrs = 1;
    }
    // Units of 1 << log_ranks blocks that run at once; asked for once per device.
    struct Fit { bool known; int units[5]; };
    static cudaError_t fit(Fit& f) {
        static std::mutex mu;
        static Fit of[kMaxKeptDevices];
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        if (dev >= kMaxKeptDevices) return cudaErrorInvalidDevice;
        std::lock_guard<std::mutex> lock(mu);
        if (!of[dev].known) {
            auto kernel = k_kept<KV, D, NH, W, CAP>;
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes(8 * NH));
            if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            for (int r = 0; r < 5 && e == cudaSuccess; ++r) {
                cudaLaunchConfig_t cfg{};
                cudaLaunchAttribute at{};
                fill(cfg, at, 1, r, 8 * NH, 0);
                e = cudaOccupancyMaxActiveClusters(&of[dev].units[r], kernel, &cfg);
            }
            if (e != cudaSuccess) return e;
            of[dev].known = true;
        }
        f = of[dev];
        return cudaSuccess;
    }
    static cudaError_t run(KeptParams& p, int log_ranks, cudaStream_t s) {
        cudaLaunchConfig_t cfg{};
        cudaLaunchAttribute at{};
        p.log_ranks = log_ranks;
        fill(cfg, at, p.n_seqs * p.geo.hkv, log_ranks, p.geo.group, s);
        return cudaLaunchKernelEx(&cfg, k_kept<KV, D, NH, W, CAP>, static_cast<const KeptParams&>(p));
    }
};

// Microseconds until the last of the units ends, of which `at_once` run side by side
// and the others in turn: a start and a merge, a choice where there is one, and the
// steps of a unit's warps (measured on bf16 pages of d 128: 6.5, 4 and 1.1 us; other
// types take the same numbers).
inline float kept_span(const KeptLoad& load, int at_once, int groups_a_step) {
    float busy[kKeptLoads] = {};
    const int n = at_once < kKeptLoads ? at_once : kKeptLoads;
    float end = 0.f;
    for (int u = 0; u < load.n; ++u) {
        int first = 0;
        for (int i = 1; i < n; ++i) first = busy[i] < busy[first] ? i : first;
        const int steps = (load.groups[u] + groups_a_step - 1) / groups_a_step;
        busy[first] += 6.5f + (load.chosen[u] ? 4.f : 0.f) + 1.1f * (float)steps;
        end = std::max(end, busy[first]);
    }
    return end;
}

// Warps a block and blocks a unit: the most warps a unit with which all units still
// run at once (three blocks of 4 warps an SM, or one of 8; clusters cannot use all SMs
// of a group).  45 units of 64 pages, FP8, 4 warps: 8 blocks each 16.3 us, 4 each
// 20.5, 16 each (more than run at once) 30.7; 128 units, 4-bit: 2 each 25.2, 4 each 40;
// 32 units: 8 warps in 4 blocks each 15.3, 4 warps in 8 each 16.5.  A few units may
// differ much (one sequence's GLOBAL heads and its LOCAL ones): then the largest
// clusters can end first although some units wait (1 x 128K, two of eight heads
// GLOBAL, while a choice took longer: 17.5 us against 22.3; 1 x 4K, all GLOBAL: 18
// against 10).
//
// A unit is one cluster's work, so many pages of few units, or of some among many
// light ones, leave most of the GPU waiting for them, and k_decode, which shares all
// pages out evenly, is ahead although it starts after the choice.  What decides is the
// groups a warp of the longest unit, and how much of the work is the longest units'
// kind.  Microseconds in one launch / in two, L2 flushed, 8 KV heads of 4 query heads,
// d 128, at that many groups a warp:
//   largest clusters (16 blocks a unit, a few units), whatever the other units are: of 8
//     warps to 64, of 4 to 48.  1 x 128K, one head of eight GLOBAL, 56: bf16 81 / 116, FP8
//     68 / 153, 4 bits 60 / 70, bf16 of d 64 capped 66 / 81; two heads 81 / 98, 67 / 143,
//     60 / 92, 66 / 75; 2 x 64K, one head (4 warps), 40: 60 / 63, 52 / 77, 42 / 44,
//     50 / 47, 48: 69 / 65, 58 / 85, 48 / 47, 56 / 50, 56: 78 / 67, 66 / 94, 52 / 50, 62 / 51.
//   the longest units' kind is half of the work or more: to 48.  Four heads of eight
//     GLOBAL, 48: 4 x 64K 76 / 73, 62 / 69, 56 / 49; 16 x 32K 76 / 79, 64 / 67, 52 / 49;
//     32 x 32K 85 / 94, 72 / 78, 60 / 59.  All eight, 1 x 128K 76 / 76, 64 / 71, 56 / 55.
//   less: to 24.  One head of eight, 4 x 64K 24: 46 / 43, 40 / 43, 36 / 36, 32: 55 / 49,
//     47 / 51, 42 / 37; 8 x 64K 16: 40 / 39, 37 / 47, 31 / 35, 24: 49 / 40, 44 / 50, 36 / 36;
//     32 x 32K 24: 56 / 59, 48 / 51, 42 / 42, 48: 83 / 65, 70 / 54, 58 / 44.
// d 64 and capped scores cross a little earlier (bf16, d 64, capped, four heads of eight, 40:
// 16 x 32K 54 / 52, 32 x 32K 58 / 57; 8 x 64K one head 16: 33 / 34, 24: 41 / 33); they
// take the same limits.  Of 630 calls around the limits (15 shapes, 16 to 62 groups, six
// types) the way taken was 1.6 % behind the better one on average; to 48 groups 26 % at
// most (capped scores on 4-bit pages), above 41 % (FP8, largest clusters of 4 warps).
// Units of about the same length on blocks of 4 warps bear more (32K tokens a sequence:
// bf16, 32 sequences, 64: 107 / 136, 128: 194 / 210, 256: 369 / 359; 16 sequences, 128:
// 192 / 190; FP8, 32 sequences, 64: 81 / 105, 128: 143 / 144; 4 bits, 64: 64 / 82, 128:
// 109 / 105).
template <int KV, int D, int NH, bool CAP>
cudaError_t launch_kept_heads(KeptParams& p, const KeptLoad& load, bool& serves, cudaStream_t s) {
    typedef KeptLaunch<KV, D, NH, 8, CAP> Eight;
    typedef KeptLaunch<KV, D, NH, 4, CAP> Four;
    typename Eight::Fit eight;
    typename Four::Fit four;
    cudaError_t e = Eight::fit(eight);
    if (e == cudaSuccess) e = Four::fit(four);
    if (e != cudaSuccess) return e;
    const int units = p.n_seqs * p.geo.hkv;
    constexpr int NG = Rows<KV, D>::NG;
    int ranks = 0, warps = 4;                         // (the former as a power of two)
    if (units <= eight.units[4]) {
        ranks = 4;
        warps = 8;
    } else if (units <= eight.units[3]) {
        const bool largest = load.n == units && eight.units[4] > 0 &&
                             kept_span(load, eight.units[4], 128 * NG) < kept_span(load, eight.units[3], 64 * NG);
        ranks = largest ? 4 : 3;
        warps = 8;
    } else if (units <= four.units[4]) {
        ranks = 4;
    } else if (units <= eight.units[2]) {
        ranks = 2;
        warps = 8;
    } else {
        for (int r = 3; r > 0 && ranks == 0; --r)
            if (units <= four.units[r]) ranks = r;
    }
    const int64_t per_warp = cdiv64(load.longest, warps << ranks), full = load.longest * units;
    const bool half = 2 * load.total >= full, even = 4 * load.total >= 3 * full;
    const int limit = ranks == 4 ? (warps == 8 ? 64 : 48) : half ? 48 : 24;
    serves = per_warp <= limit || (warps == 4 && even && per_warp <= (KV == kRowsBf16 ? 128 : 64));
    if (!serves) return cudaSuccess;
    return warps == 8 ? Eight::run(p, ranks, s) : Four::run(p, ranks, s);
}

template <int KV, int D, bool CAP>
cudaError_t launch_kept_type(KeptParams& p, const KeptLoad& load, bool& serves, cudaStream_t s) {
    return p.geo.group > 8 ? launch_kept_heads<KV, D, 2, CAP>(p, load, serves, s)
                           : launch_kept_heads<KV, D, 1, CAP>(p, load, serves, s);
}
template <bool CAP>
cudaError_t launch_kept_bf16(KeptParams& p, const KeptLoad& load, bool& serves, cudaStream_t s) {
    return p.geo.d == 128 ? launch_kept_type<kRowsBf16, 128, CAP>(p, load, serves, s)
                          : launch_kept_type<kRowsBf16, 64, CAP>(p, load, serves, s);
}
template <bool CAP>
cudaError_t launch_kept_coded(KeptParams& p, const KeptLoad& load, bool& serves, cudaStream_t s) {
    return p.geo.fp4 ? launch_kept_type<kRowsFp4, 128, CAP>(p, load, serves, s)
                     : launch_kept_type<kRowsFp8, 128, CAP>(p, load, serves, s);
}

}  // namespace

}  // namespace sp
