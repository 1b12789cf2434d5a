// sp_decode4.cuh -- split-KV decode over 4-bit pages (format: sp_fp4.cuh).
//
// All visible slots of the call are one list of work items, split evenly over
// a persistent grid, and a unit spread over several CTAs is merged by the last
// of them, as in k_decode (sp_decode.cuh).  What 4 bits change:
//
//   * 144 bytes a key instead of 512, so arithmetic and latency decide.  Keys
//     are the M side of the matrix instructions and the query heads the N side
//     (8 of them, or 16 in two steps), so no row is padding:
//         S^T = K Q^T      16 keys x 8 heads, 8 steps of 16 dimensions
//         O^T = V^T P^T    16 dimensions x 8 heads, 8 tiles, K = 16 keys
//     P^T goes from the accumulator to the operand layout by two 8 x 8
//     register transposes (movmatrix).
//   * An item is a run of 64 slots of a unit whatever the page size (four groups
//     of 16; a group that no query sees is loaded too, or a neighbour in its
//     place).
//   * There is no producer and no barrier in the stream: each warp takes a run
//     of neighbouring items (mostly of one unit), owns one stage and refills
//     its K half as soon as the scores are taken and its V half after the
//     products.  The lanes look up the pages of the warp's next 32 items at once
//     and hand them out by shuffle.  A unit that lies inside a warp's run is
//     finished by that warp; a run's first and last units leave a partial (o, m,
//     l) in shared memory, merged once when the CTA's warps are done.
//   * Codes become f16 by the hardware's conversion, one instruction per two,
//     and times their block's scale exactly (6 significant bits); a lane's
//     codes of a K fragment lie in two blocks and of a V fragment in one, so
//     one 32-bit word holds its scales of a group.  V codes of two keys are
//     interleaved by two bit selects per eight pairs before the conversion.
//   * Channel scales: K's are folded into the query, V's into the finished
//     sums.  Scores, maxima, sums and outputs are fp32; what the matrix
//     instructions take is f16, rounded once (2^-11 relative at most, next to
//     the bf16 output's 2^-8): P, and the query under channel scales that are
//     not powers of two.  A power of two per head keeps the query in f16's range.
#pragma once
#include <algorithm>

#include "sp_decode.cuh"

namespace sp {

namespace {

constexpr int kD4Warps = 8;
constexpr int kD4Threads = kD4Warps * 32;
constexpr int kD4TileBytes = kFp4ItemSlots * kFp4RowBytes;
constexpr int kD4StageBytes = 2 * kD4TileBytes;      // K, then V
constexpr int kD4Dim = 128;
// The reference of the exponentials is set kRefBelow under a maximum and
// raised when a score passes it by kRefAbove, so P lies between 2^7 (at first)
// and 2^15 at its largest: f16 then holds weights down to 2^-31 of it.
constexpr float kRefBelow = 7.f, kRefAbove = 15.f;
// A partial's head in shared memory: dimension 16 gl + 2 mt + i at 16 mt + 2 gl +
// i, heads 132 floats apart (a half warp's 8-byte stores then meet no bank twice).
constexpr int kD4HeadFloats = 132;
__device__ __forceinline__ int d4_dim(int at) { return ((at >> 1) & 7) * 16 + (at >> 4) * 2 + (at & 1); }
static_assert(16 * kD4HeadFloats * 4 <= kD4StageBytes, "16 heads fit a warp's stages");
constexpr int kD4Groups = kFp4ItemSlots / kFp4Group;
static_assert(kD4Groups == 4, "an item is four groups of 16 slots");

// CTA whose share of the items holds item x.
__device__ __forceinline__ int cta_of(const DecodeParams& p, int32_t x) {
    const int32_t more = p.rem * (p.per + 1);        // items of the CTAs that take one more
    return x < more ? x / (p.per + 1) : p.rem + (x - more) / p.per;
}
// Transpose of an 8x8 f16 matrix held as one pair a lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// A work item: its groups' places in the pool (in groups), and its visible
// slots [lo, hi) as lo | hi << 8.
struct Item4 { uint32_t g[kD4Groups], visible; };

// Item j of unit u (positions and slots are below 2^31).
__device__ __forceinline__ Item4 find_item4(const DecodeParams& p, int u, int32_t j) {
    const Geo& g = p.geo;
    const uint32_t P = (uint32_t)g.page, lp = 31 - __clz(P);
    const int b = u / g.hkv, h = u - b * g.hkv;
    const int seq = p.seq[b];
    const int32_t t = p.tq[b];
    const int64_t row = g.unit_row(seq, p.layer, h);
    const UnitPol pol = p.meta.pol[row];
    // the visible ranges of decode_ranges (sp_rules.h), in 32 bits
    int32_t lo[3] = {0, 0, 0}, hi[3] = {0, 0, 0};
    if (pol.kind == kGlobal) {
        hi[0] = t + 1;
    } else if (pol.kind == kLocal) {
        const int32_t sink_end = min(pol.sink, t + 1);
        hi[0] = sink_end;
        const int32_t w0 = max(max(t - pol.window + 1, 0), sink_end);
        if (w0 <= t) {
            const int32_t base = pol.sink_pages << lp, ring = pol.ring << lp, len = t - w0 + 1;
            const int32_t q0 = (int32_t)((uint32_t)(w0 - pol.sink) % (uint32_t)ring);
            lo[1] = base + q0;
            hi[1] = base + min(q0 + len, ring);
            lo[2] = base;
            hi[2] = base + max(q0 + len - ring, 0);
        }
    } else {
        const int32_t* idx = p.meta.idx + (int64_t)seq * g.max_idx_per_seq + pol.idx_off;
        hi[0] = (int32_t)count_below(idx, pol.n_idx, (int64_t)t + 1);
    }
    int32_t w = 0, l = 0, e = 1;                      // window, visible slots [l, e) in it
    #pragma unroll
    for (int q = 0; q < 3; ++q) {
        if (hi[q] <= lo[q]) continue;
        const int32_t first = lo[q] / kFp4ItemSlots, n = (hi[q] - 1) / kFp4ItemSlots - first + 1;
        if (j >= 0 && j < n) {
            w = (first + j) * kFp4ItemSlots;
            l = max(lo[q] - w, 0);
            e = min(hi[q] - w, kFp4ItemSlots);
        }
        j -= n;
    }
    // a group without a visible slot may have no page: its nearest neighbour
    // that has one is read in its place
    Item4 it;
    it.visible = (uint32_t)l | ((uint32_t)e << 8);
    const int32_t* tab = p.meta.ptab + row * g.max_pages_unit;
    #pragma unroll
    for (int k = 0; k < kD4Groups; ++k) {
        if (P >= kFp4ItemSlots && k > 0) { it.g[k] = it.g[0] + k; continue; }   // one page holds the item
        const int near = P >= kFp4ItemSlots ? 0 : min(max(k, l >> 4), (e - 1) >> 4);
        const uint32_t slot = (uint32_t)w + 16 * near;
        const int32_t page = tab[slot >> lp];
        it.g[k] = 0;                                  // a bad page: load something harmless
        if (page < 0 || page >= g.num_pages) atomicOr(p.meta.status, kStatusBadPage);
        else it.g[k] = (((uint32_t)page << lp) + (slot & (P - 1))) >> 4;
    }
    return it;
}

// NH: 8-head steps (group <= 8 * NH).  Two CTAs of 8 warps share an SM at
// NH = 1 (at most 128 registers a thread); NH = 2 holds twice the output and
// runs one.
template <int NH, bool CAP>
__global__ void __launch_bounds__(kD4Threads, NH == 1 ? 2 : 1)
k_decode4(const __grid_constant__ DecodeParams p, const uint8_t* __restrict__ kpool,
          const uint8_t* __restrict__ vpool) {
    constexpr int D = kD4Dim;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    const Geo& g = p.geo;
    const int group = g.group;
    uint8_t* stages = smem_raw;
    // A warp's first and last partials are entries 2 w and 2 w + 1: (m, l) and
    // unit here, outputs in its slot and in its stages.
    float* slots = reinterpret_cast<float*>(stages + kD4Warps * kD4StageBytes);     // [warps][group][kD4HeadFloats]
    float2* entry_ml = reinterpret_cast<float2*>(slots + p.merge_floats);           // [2 warps][group]
    float2* unit_ml = entry_ml + 2 * kD4Warps * group;                              // [2 warps][group]
    float* entry_weight = reinterpret_cast<float*>(unit_ml + 2 * kD4Warps * group); // [2 warps][group]
    __shared__ uint64_t full[2 * kD4Warps];          // K and V of each warp's stage landed
    __shared__ __align__(8) float score_scale[kD4Warps][8 * NH];   // each head's factor of its products
    __shared__ int abort_word, flag_last[2], entry_unit[2 * kD4Warps], list[2 * kD4Warps], n_list;
    volatile int* abort_flag = &abort_word;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = gridDim.x, c = blockIdx.x;
    // CTA c takes p.per items, one more if c < p.rem (per >= 1)
    const int32_t x0 = c * p.per + min(c, p.rem), x1 = x0 + p.per + (c < p.rem ? 1 : 0);

    if (threadIdx.x == 0) {
        for (int s = 0; s < 2 * kD4Warps; ++s) mbar_init(&full[s], 1);
        for (int e = 0; e < 2 * kD4Warps; ++e) entry_unit[e] = -1;
        abort_word = 0;
        fence_mbar_init();
    }
    __syncthreads();

    const int ctid = threadIdx.x;
    constexpr int CT = kD4Threads;
    // Units with no visible token: O = 0, LSE = -inf (one CTA each).
    for (int u = c; u < p.n_units; u += G) {
        if (p.item_off[u + 1] != p.item_off[u]) continue;
        const int b = u / g.hkv, h = u % g.hkv;
        for (int e = ctid; e < group * D; e += CT) {
            const int r = e / D, col = e % D;
            p.out[((int64_t)b * g.hq + h * group + r) * D + col] = __float2bfloat16(0.f);
            if (col == 0 && p.lse) p.lse[(int64_t)b * g.hq + h * group + r] = -INFINITY;
        }
    }
    if (p.total_items == 0) return;

    // This warp's items [wx0, wx1) of the CTA's.  The lanes hold 32 of them,
    // [batch, batch + 32).
    const int32_t wx0 = x0 + (x1 - x0) * warp / kD4Warps, wx1 = x0 + (x1 - x0) * (warp + 1) / kD4Warps;
    const int mine = wx1 - wx0;
    uint8_t* my_stages = stages + warp * kD4StageBytes;
    uint64_t* my_full = full + warp * 2;
    int u_first = 0;                                 // first unit with an item >= wx0
    for (int u_hi = p.n_units - 1; u_first < u_hi;) {
        const int mid = (u_first + u_hi) >> 1;
        if (p.item_off[mid + 1] <= wx0) u_first = mid + 1; else u_hi = mid;
    }
    Item4 held{}, next{};
    int batch = -32, u_batch = u_first;
    uint32_t visible = 0;                            // slots of the item in the stage
    const bool one_page = g.page >= kFp4ItemSlots;
    int issued[2] = {0, 0};                          // K and V loads
    // take(i): item i's description into `next`
    auto take = [&](int i) {
        if (i >= batch + 32) {
            // the units of 32 items: walk their ends together (each end is one
            // uniform load), every lane stepping over those before its item
            batch += 32;
            const int32_t x = wx0 + batch + lane, last = min(wx0 + batch + 31, wx1 - 1);
            int u = u_batch;
            int32_t start = p.item_off[u_batch];
            for (; u_batch + 1 < p.n_units; ++u_batch) {
                const int32_t end = p.item_off[u_batch + 1];
                if (end > last) break;
                if (end <= x) { u = u_batch + 1; start = end; }
            }
            if (batch + lane < mine) held = find_item4(p, u, x - start);
        }
        next.visible = __shfl_sync(0xffffffffu, held.visible, i - batch);
        next.g[0] = __shfl_sync(0xffffffffu, held.g[0], i - batch);
        if (!one_page) {
            #pragma unroll
            for (int k = 1; k < kD4Groups; ++k) next.g[k] = __shfl_sync(0xffffffffu, held.g[k], i - batch);
        }
    };
    // lane 0: K (kv = 0) or V of the taken item into the stage
    auto load = [&](int kv) {
        ++issued[kv];
        if (lane != 0) return;
        uint64_t* bar = &my_full[kv];
        uint8_t* dst = my_stages + kv * kD4TileBytes;
        const uint8_t* pool = kv ? vpool : kpool;
        mbar_arrive_expect_tx(bar, kD4TileBytes);
        if (one_page) {
            bulk_load(dst, pool + (int64_t)next.g[0] * kFp4GroupBytes, kD4TileBytes, bar);
            return;
        }
        #pragma unroll
        for (int k = 0; k < kD4Groups; ++k)
            bulk_load(dst + k * kFp4GroupBytes, pool + (int64_t)next.g[k] * kFp4GroupBytes, kFp4GroupBytes, bar);
    };
    const int gl = lane >> 2, j = lane & 3;          // fragment row, column pair
    // raw query words of a unit's heads; the first unit's travel while the
    // first item is looked up
    uint32_t qraw[NH][8][2];
    auto load_q = [&](int u) {
        const int b = u / g.hkv, h = u - b * g.hkv;
        #pragma unroll
        for (int nh = 0; nh < NH; ++nh) {
            const int head = nh * 8 + gl;
            const __nv_bfloat16* qr = p.q + ((int64_t)b * g.hq + h * group + head) * D + j * 32;
            #pragma unroll
            for (int kk = 0; kk < 8; ++kk)
                #pragma unroll
                for (int e = 0; e < 2; ++e)
                    qraw[nh][kk][e] = head < group ? *reinterpret_cast<const uint32_t*>(qr + kk * 4 + 2 * e) : 0u;
        }
    };
    if (mine > 0) { load_q(u_first); take(0); load(0); load(1); }

    // slots of this lane's rows of S^T in a group (positions gl and gl + 8)
    const int slot_a = (gl >> 1) + 4 * (gl & 1), slot_b = slot_a + 8;
    uint32_t qb[NH][8][2];
    float m_run[NH][2], l_run[NH][2], o[NH][8][4];
    int it = 0;                                      // next item of this warp
    bool dead = false;
    for (int u = u_first; it < mine; ++u) {
        const int32_t u_begin = p.item_off[u], u_end = p.item_off[u + 1];
        if (u_end <= wx0 + it) continue;             // no items, or before this run
        const int stop = min(mine, u_end - wx0);
        const int b = u / g.hkv, h = u - b * g.hkv;
        const float* ks = p.meta.kscale + ((int64_t)p.layer * g.hkv + h) * D;
        const float* vs = p.meta.vscale + ((int64_t)p.layer * g.hkv + h) * D;
        if (it > 0) load_q(u);
        // The query enters the products as f16, times a power of two per head
        // that takes the largest |q * channel scale| to 2^14 .. 2^15: exactly
        // where the product has f16's bits and lies within 2^-28 of it, however
        // small or large the scales and the query are; the scores are multiplied
        // back in fp32.
        #pragma unroll
        for (int nh = 0; nh < NH; ++nh) {
            float x[8][2][2], top = 0.f;
            #pragma unroll
            for (int kk = 0; kk < 8; ++kk)
                #pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const __nv_bfloat162 v2 = *reinterpret_cast<const __nv_bfloat162*>(&qraw[nh][kk][e]);
                    x[kk][e][0] = __low2float(v2);
                    x[kk][e][1] = __high2float(v2);
                    if (p.scaled) {
                        const float2 f = __ldg(reinterpret_cast<const float2*>(ks + j * 32 + kk * 4 + 2 * e));
                        x[kk][e][0] *= f.x;
                        x[kk][e][1] *= f.y;
                    }
                    top = fmax3_abs(top, x[kk][e][0], x[kk][e][1]);
                }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int ex = min(max(__float_as_int(top) >> 23, 15), 254);     // 2^(ex - 127) <= top
            const float up = __int_as_float((268 - ex) << 23), down = __int_as_float((ex - 14) << 23);
            #pragma unroll
            for (int kk = 0; kk < 8; ++kk)
                #pragma unroll
                for (int e = 0; e < 2; ++e) qb[nh][kk][e] = pack_f16(x[kk][e][0] * up, x[kk][e][1] * up);
            // (this lane's query is head gl, its scores are heads 2 j and 2 j + 1's)
            if (j == 0) score_scale[warp][nh * 8 + gl] = down * (CAP ? p.cap.k1 : p.scale_log2);
            m_run[nh][0] = m_run[nh][1] = -INFINITY;
            l_run[nh][0] = l_run[nh][1] = 0.f;
            #pragma unroll
            for (int mt = 0; mt < 8; ++mt)
                #pragma unroll
                for (int e = 0; e < 4; ++e) o[nh][mt][e] = 0.f;
        }
        __syncwarp();
        for (; it < stop; ++it) {
            if (dead) continue;
            const uint32_t parity = it & 1;
            dead = __any_sync(0xffffffffu, !mbar_wait(&my_full[0], parity, abort_flag, p.meta.status));
            if (dead) continue;
            visible = next.visible;
            const int lo = visible & 0xFF, hi = visible >> 8;
            const uint8_t* tk = my_stages;
            const uint8_t* tv = tk + kD4TileBytes;
            float sc[kD4Groups][NH][4];              // [group][heads][accumulator]
            #pragma unroll
            for (int q = 0; q < kD4Groups; ++q) {
                #pragma unroll
                for (int nh = 0; nh < NH; ++nh)
                    #pragma unroll
                    for (int e = 0; e < 4; ++e) sc[q][nh][e] = 0.f;
                const uint8_t* gk = tk + q * kFp4GroupBytes;
                const uint4 ca = *reinterpret_cast<const uint4*>(gk + gl * 64 + j * 16);
                const uint4 cb = *reinterpret_cast<const uint4*>(gk + (gl + 8) * 64 + j * 16);
                const uint32_t sw = *reinterpret_cast<const uint32_t*>(gk + kFp4ScaleOff + (gl * 4 + j) * 4);
                const uint32_t wa[4] = {ca.x, ca.y, ca.z, ca.w}, wb[4] = {cb.x, cb.y, cb.z, cb.w};
                #pragma unroll
                for (int w = 0; w < 4; ++w) {        // 8 dimensions: two steps
                    // this block's scale of both rows, twice in a word, as f16
                    const uint32_t fa = prmt(sw, 0u, (w >> 1) ? 0x4141u : 0x4040u) << 7;
                    const uint32_t fb = prmt(sw, 0u, (w >> 1) ? 0x4343u : 0x4242u) << 7;
                    uint32_t a[4], bb[4];
                    fp4_word_f16(wa[w], a[0], a[1], a[2], a[3]);
                    fp4_word_f16(wb[w], bb[0], bb[1], bb[2], bb[3]);
                    #pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t af[4] = {hmul2(a[2 * e], fa), hmul2(bb[2 * e], fb),
                                                hmul2(a[2 * e + 1], fa), hmul2(bb[2 * e + 1], fb)};
                        #pragma unroll
                        for (int nh = 0; nh < NH; ++nh)
                            mma_f16_16816(sc[q][nh], af, qb[nh][2 * w + e][0], qb[nh][2 * w + e][1]);
                    }
                }
            }
            // K's half is read: refill it with the next item's
            const bool more = it + 1 < mine;
            __syncwarp();
            if (more) { take(it + 1); load(0); }
            #pragma unroll
            for (int nh = 0; nh < NH; ++nh) {
                const float2 f = *reinterpret_cast<const float2*>(&score_scale[warp][nh * 8 + 2 * j]);
                #pragma unroll
                for (int q = 0; q < kD4Groups; ++q)
                    #pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float x = sc[q][nh][e] * ((e & 1) ? f.y : f.x);
                        sc[q][nh][e] = CAP ? capped_log2(x, p.cap) : x;
                    }
            }
            if (lo > 0 || hi < kFp4ItemSlots) {
                #pragma unroll
                for (int q = 0; q < kD4Groups; ++q) {
                    const bool in_a = 16 * q + slot_a >= lo && 16 * q + slot_a < hi;
                    const bool in_b = 16 * q + slot_b >= lo && 16 * q + slot_b < hi;
                    #pragma unroll
                    for (int nh = 0; nh < NH; ++nh)
                        #pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (!(e < 2 ? in_a : in_b)) sc[q][nh][e] = -INFINITY;
                }
            }
            // Running reference, raised only when a score passes it by kRefAbove
            // (or the unit has none yet): a warp agrees by one vote instead of
            // exchanging its rows' maxima for every item.
            float mx[NH][2];
            bool grew = false;
            #pragma unroll
            for (int nh = 0; nh < NH; ++nh)
                #pragma unroll
                for (int e = 0; e < 2; ++e) {
                    mx[nh][e] = fmaxf(sc[0][nh][e], sc[0][nh][2 + e]);
                    #pragma unroll
                    for (int q = 1; q < kD4Groups; ++q)
                        mx[nh][e] = fmaxf(mx[nh][e], fmaxf(sc[q][nh][e], sc[q][nh][2 + e]));
                    grew = grew || mx[nh][e] > m_run[nh][e] + kRefAbove;
                }
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
                        for (int mt = 0; mt < 8; ++mt) {
                            o[nh][mt][e] *= alpha;
                            o[nh][mt][2 + e] *= alpha;
                        }
                    }
            }
            uint32_t pb[kD4Groups][NH][2];
            #pragma unroll
            for (int q = 0; q < kD4Groups; ++q)
                #pragma unroll
                for (int nh = 0; nh < NH; ++nh) {
                    float pv[4];
                    #pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float mb = m_run[nh][e & 1] == -INFINITY ? 0.f : m_run[nh][e & 1];
                        pv[e] = fast_exp2(sc[q][nh][e] - mb);
                        l_run[nh][e & 1] += pv[e];
                    }
                    pb[q][nh][0] = transpose8x8(pack_f16(pv[0], pv[1]));
                    pb[q][nh][1] = transpose8x8(pack_f16(pv[2], pv[3]));
                }
            dead = __any_sync(0xffffffffu, !mbar_wait(&my_full[1], parity, abort_flag, p.meta.status));
            if (dead) continue;
            #pragma unroll
            for (int q = 0; q < kD4Groups; ++q) {
                // V: the codes of block gl of slots j, j+4, j+8, j+12
                const uint8_t* gv = tv + q * kFp4GroupBytes;
                const int unit = (gl ^ ((j & 2) << 1)) * 8;
                uint2 cv[4];
                #pragma unroll
                for (int t = 0; t < 4; ++t)
                    cv[t] = *reinterpret_cast<const uint2*>(gv + (j + 4 * t) * 64 + unit);
                const uint32_t sw = *reinterpret_cast<const uint32_t*>(gv + kFp4ScaleOff + gl * 16 + j * 4);
                const uint32_t f0 = prmt(sw, 0u, 0x4140u) << 7, f1 = prmt(sw, 0u, 0x4342u) << 7;
                #pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const uint32_t v0 = w ? cv[0].y : cv[0].x, v1 = w ? cv[1].y : cv[1].x;
                    const uint32_t v2 = w ? cv[2].y : cv[2].x, v3 = w ? cv[3].y : cv[3].x;
                    constexpr uint32_t kLow = 0x0F0F0F0Fu;
                    // bytes (first key low, second key high) of dimensions 0,2,4,6 and 1,3,5,7
                    const uint32_t e0 = (v0 & kLow) | ((v1 << 4) & ~kLow), d0 = ((v0 >> 4) & kLow) | (v1 & ~kLow);
                    const uint32_t e1 = (v2 & kLow) | ((v3 << 4) & ~kLow), d1 = ((v2 >> 4) & kLow) | (v3 & ~kLow);
                    uint32_t a0[4], a1[4], a2[4], a3[4];
                    fp4_word_f16(e0, a0[0], a0[1], a0[2], a0[3]);
                    fp4_word_f16(d0, a1[0], a1[1], a1[2], a1[3]);
                    fp4_word_f16(e1, a2[0], a2[1], a2[2], a2[3]);
                    fp4_word_f16(d1, a3[0], a3[1], a3[2], a3[3]);
                    #pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const uint32_t af[4] = {hmul2(a0[t], f0), hmul2(a1[t], f0), hmul2(a2[t], f1), hmul2(a3[t], f1)};
                        #pragma unroll
                        for (int nh = 0; nh < NH; ++nh)
                            mma_f16_16816(o[nh][4 * w + t], af, pb[q][nh][0], pb[q][nh][1]);
                    }
                }
            }
            __syncwarp();
            if (more) load(1);
        }

        // after an abort: nothing may land in this warp's stages any more (bounded)
        if (dead && lane == 0)
            for (int kv = 0; kv < 2; ++kv)
                mbar_wait(&my_full[kv], (issued[kv] - 1) & 1, nullptr, nullptr);
        __syncwarp();

        // The unit's sums of this run: the result itself if the run holds the
        // whole unit, else a partial, in this warp's slot (the run goes on) or
        // in its stages (it ends here, and nothing is in flight).
        if (p.scaled) {
            #pragma unroll
            for (int mt = 0; mt < 8; ++mt) {
                const float v0 = __ldg(vs + gl * 16 + 2 * mt), v1 = __ldg(vs + gl * 16 + 2 * mt + 1);
                #pragma unroll
                for (int nh = 0; nh < NH; ++nh) {
                    o[nh][mt][0] *= v0; o[nh][mt][1] *= v0;
                    o[nh][mt][2] *= v1; o[nh][mt][3] *= v1;
                }
            }
        }
        const bool complete = u_begin >= wx0 && u_end <= wx1;
        const int entry = 2 * warp + (it < mine ? 0 : 1);
        float* po = it < mine ? slots + warp * group * kD4HeadFloats : reinterpret_cast<float*>(my_stages);
        if (!complete && lane == 0) entry_unit[entry] = u;
        #pragma unroll
        for (int nh = 0; nh < NH; ++nh)
            #pragma unroll
            for (int e = 0; e < 2; ++e) {
                float l = l_run[nh][e];
                l += __shfl_xor_sync(0xffffffffu, l, 4);
                l += __shfl_xor_sync(0xffffffffu, l, 8);
                l += __shfl_xor_sync(0xffffffffu, l, 16);
                const int head = nh * 8 + 2 * j + e;
                if (head >= group) continue;
                if (complete) {
                    const float inv = 1.f / l;
                    const int64_t orow = (int64_t)b * g.hq + h * group + head;
                    uint32_t* out = reinterpret_cast<uint32_t*>(p.out + orow * D + gl * 16);
                    #pragma unroll
                    for (int mt = 0; mt < 8; ++mt)
                        out[mt] = pack_bf16(o[nh][mt][e] * inv, o[nh][mt][2 + e] * inv);
                    if (gl == 0 && p.lse) p.lse[orow] = (m_run[nh][e] + __log2f(l)) * 0.69314718055994531f;
                } else {
                    #pragma unroll
                    for (int mt = 0; mt < 8; ++mt)
                        *reinterpret_cast<float2*>(po + head * kD4HeadFloats + mt * 16 + gl * 2) =
                            make_float2(o[nh][mt][e], o[nh][mt][2 + e]);
                    if (gl == 0) entry_ml[entry * group + head] = make_float2(m_run[nh][e], l);
                }
            }
    }
    __syncthreads();

    // ------------- merge the partials of the CTA, unit by unit -------------
    // The entries in use, in order (units ascend), and every entry's weight
    // 2^(m - m*) in its unit's sum; a unit's (m*, l*) go to all its entries.
    if (warp == 0) {
        const int u = lane < 2 * kD4Warps ? entry_unit[lane] : -1;
        const uint32_t used = __ballot_sync(0xffffffffu, u >= 0);
        if (u >= 0) list[__popc(used & ((1u << lane) - 1u))] = lane;
        if (lane == 0) n_list = __popc(used);
    }
    for (int e = ctid; e < 2 * kD4Warps * group; e += CT) {
        const int w = e / group, r = e - w * group, u = entry_unit[w];
        if (u < 0) continue;
        float mst = -INFINITY, lst = 0.f;
        #pragma unroll
        for (int x = 0; x < 2 * kD4Warps; ++x)
            mst = fmaxf(mst, entry_unit[x] == u ? entry_ml[x * group + r].x : -INFINITY);
        const float ref = mst == -INFINITY ? 0.f : mst;
        #pragma unroll
        for (int x = 0; x < 2 * kD4Warps; ++x)
            lst += entry_unit[x] == u ? fast_exp2(entry_ml[x * group + r].x - ref) * entry_ml[x * group + r].y : 0.f;
        entry_weight[e] = fast_exp2(entry_ml[e].x - ref);
        unit_ml[e] = make_float2(mst, lst);
    }
    __syncthreads();
    // Thread e holds output (head e / 128, place e % 128 of the slots' order).
    int split_unit[2] = {-1, -1};                    // units that other CTAs share
    for (int i = 0; i < n_list;) {
        const int u = entry_unit[list[i]];
        int k = i + 1;
        while (k < n_list && entry_unit[list[k]] == u) ++k;
        const int b = u / g.hkv, h = u - b * g.hkv;
        const bool whole = p.item_off[u] >= x0 && p.item_off[u + 1] <= x1;
        if (!whole) split_unit[split_unit[0] < 0 ? 0 : 1] = u;
        for (int e = ctid; e < group * D; e += CT) {
            const int r = e / D, at = e % D;
            float ost = 0.f;
            #pragma unroll 4
            for (int y = i; y < k; ++y) {
                const int w = list[y];
                const float* po = (w & 1) ? reinterpret_cast<const float*>(stages + (w >> 1) * kD4StageBytes)
                                          : slots + (w >> 1) * group * kD4HeadFloats;
                ost += entry_weight[w * group + r] * po[r * kD4HeadFloats + at];
            }
            const float2 ml = unit_ml[list[i] * group + r];
            if (whole) {
                const int64_t orow = (int64_t)b * g.hq + h * group + r;
                p.out[orow * D + d4_dim(at)] = __float2bfloat16(ost / ml.y);
                if (at == 0 && p.lse) p.lse[orow] = (ml.x + __log2f(ml.y)) * 0.69314718055994531f;
            } else {
                const int64_t part = (int64_t)u + c;
                p.part_o[(part * group + r) * D + at] = ost;
                if (at == 0) {
                    p.part_ml[(part * group + r) * 2] = ml.x;
                    p.part_ml[(part * group + r) * 2 + 1] = ml.y;
                }
            }
        }
        i = k;
    }
    if (split_unit[0] < 0) return;                    // the same for every thread
    __threadfence();
    __syncthreads();
    if (ctid < 2 && split_unit[ctid] >= 0) {
        // every CTA of the grid holds an item, so a unit's CTAs are neighbours
        const int u = split_unit[ctid];
        const int n = cta_of(p, p.item_off[u + 1] - 1) - cta_of(p, p.item_off[u]) + 1;
        flag_last[ctid] = atomicAdd(&p.counters[u], 1) == n - 1;
    }
    __syncthreads();
    for (int q = 0; q < 2; ++q) {
        if (split_unit[q] < 0 || !flag_last[q]) continue;
        // the last CTA of the unit: weights 2^(m - m*) of the parts, then the
        // weighted sum of their outputs
        __threadfence();
        const int u = split_unit[q];
        const int b = u / g.hkv, h = u - b * g.hkv;
        const int c_first = cta_of(p, p.item_off[u]);
        const int nseg = cta_of(p, p.item_off[u + 1] - 1) - c_first + 1;
        float* wts = slots;                            // [nseg][group] weights
        float* mls = slots + p.merge_floats / 2;       // [nseg][group] l
        for (int e = ctid; e < nseg * group; e += CT) {
            const int64_t pi = (int64_t)u + c_first + e / group;
            wts[e] = __ldcg(&p.part_ml[(pi * group + e % group) * 2]);
            mls[e] = __ldcg(&p.part_ml[(pi * group + e % group) * 2 + 1]);
        }
        __syncthreads();
        if (ctid < group) {
            const int r = ctid;
            float mst = -INFINITY;
            for (int sg = 0; sg < nseg; ++sg) mst = fmaxf(mst, wts[sg * group + r]);
            float lst = 0.f;
            for (int sg = 0; sg < nseg; ++sg) {
                const float w = fast_exp2(wts[sg * group + r] - (mst == -INFINITY ? 0.f : mst));
                wts[sg * group + r] = w;
                lst += w * mls[sg * group + r];
            }
            unit_ml[r] = make_float2(mst, lst);
        }
        __syncthreads();
        for (int e = ctid; e < group * D; e += CT) {
            const int r = e / D, at = e % D;
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
            const float* po = p.part_o + (((int64_t)u + c_first) * group + r) * D + at;
            const int64_t step = (int64_t)group * D;
            int sg = 0;
            for (; sg + 4 <= nseg; sg += 4) {
                float v4[4];
                #pragma unroll
                for (int t = 0; t < 4; ++t) v4[t] = __ldcg(po + (sg + t) * step);
                #pragma unroll
                for (int t = 0; t < 4; ++t) acc[t] += wts[(sg + t) * group + r] * v4[t];
            }
            for (; sg < nseg; ++sg) acc[0] += wts[sg * group + r] * __ldcg(po + sg * step);
            const float ost = (acc[0] + acc[1]) + (acc[2] + acc[3]);
            const float2 ml = unit_ml[r];
            const int64_t orow = (int64_t)b * g.hq + h * group + r;
            p.out[orow * D + d4_dim(at)] = __float2bfloat16(ost / ml.y);
            if (at == 0 && p.lse) p.lse[orow] = (ml.x + __log2f(ml.y)) * 0.69314718055994531f;
        }
        if (ctid == 0) p.counters[u] = 0;
        __syncthreads();
    }
}

template <int NH, bool CAP>
cudaError_t launch_decode4_t(const sp_cache* c, DecodeParams& p, int grid, cudaStream_t s) {
    // merge buffer: the warps' first partials, or two [grid][group] arrays
    // for the merge across CTAs, whichever is larger (a multiple of 4)
    constexpr int kCap = (NH == 1 ? 113 : 227) * 1024 - 1024;   // static shared memory besides
    const int group = c->geo.group;
    const int mo = std::max(kD4Warps * group * kD4HeadFloats, 2 * grid * group);
    p.merge_floats = (mo + 3) & ~3;
    const int merge_bytes = (p.merge_floats + 2 * kD4Warps * group * 5) * 4;
    p.per = (int32_t)(p.total_items / grid);
    p.rem = (int32_t)(p.total_items % grid);
    const int smem = kD4Warps * kD4StageBytes + merge_bytes;
    if (smem > kCap) return cudaErrorInvalidConfiguration;
    cudaError_t e = cudaFuncSetAttribute(k_decode4<NH, CAP>, cudaFuncAttributeMaxDynamicSharedMemorySize, kCap);
    if (e == cudaSuccess && NH == 1)
        e = cudaFuncSetAttribute(k_decode4<NH, CAP>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                 (int)cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    k_decode4<NH, CAP><<<grid, kD4Threads, smem, s>>>(p, reinterpret_cast<const uint8_t*>(c->kpool),
                                                      reinterpret_cast<const uint8_t*>(c->vpool));
    return cudaGetLastError();
}

template <bool CAP>
cudaError_t launch_decode4_any(const sp_cache* c, DecodeParams& p, int grid, cudaStream_t s) {
    return c->geo.group <= 8 ? launch_decode4_t<1, CAP>(c, p, grid, s) : launch_decode4_t<2, CAP>(c, p, grid, s);
}

}  // namespace

}  // namespace sp
