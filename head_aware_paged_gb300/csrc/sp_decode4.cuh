// sp_decode4.cuh -- split-KV decode over 4-bit pages (format: sp_fp4.cuh).
//
// The same stream as k_decode (sp_decode.cuh): all visible slots of the call
// are one list of work items, split evenly over a persistent grid; a producer
// warp copies them into a ring of shared-memory stages, consumer warps own the
// stages round robin, and a unit spread over several CTAs is merged by the
// last of them.  What 4 bits change:
//
//   * An item is a run of 64 slots of a unit whatever the page size, two
//     stages of 32; a stage is one or two groups of 16 slots, each a 1152-byte
//     bulk copy of K and one of V, and groups that no query sees are not read.
//   * 144 bytes a key instead of 512, so the arithmetic decides.  Keys are the
//     M side of the matrix instructions and the query heads the N side (8 of
//     them, or 16 in two steps), so no row is padding:
//         S^T = K Q^T      16 keys x 8 heads, 8 steps of 16 dimensions
//         O^T = V^T P^T    16 dimensions x 8 heads, 8 tiles, K = 16 keys
//     P^T goes from the accumulator to the operand layout by two 8 x 8
//     register transposes (movmatrix).
//   * Codes become f16 by the hardware's conversion, one instruction per two,
//     and times their block's scale exactly (6 significant bits); a lane's
//     codes of a K fragment lie in two blocks and of a V fragment in one, so
//     one 32-bit word holds its scales of a group.  V codes of two keys are
//     interleaved by two bit selects per eight pairs before the conversion.
//   * Channel scales: K's are folded into the query (as f16), V's into the
//     finished sums.  Scores, maxima, sums and outputs are fp32; P and the
//     scaled queries are rounded to f16 once (2^-12 relative, next to the
//     output's 2^-9).
#pragma once
#include <algorithm>

#include "sp_decode.cuh"

namespace sp {

namespace {

constexpr int kD4Warps = 8;                          // consumer warps
constexpr int kD4Threads = (kD4Warps + 1) * 32;
constexpr int kD4StageKeys = 32;
constexpr int kD4Sub = kFp4ItemSlots / kD4StageKeys; // stages per item
constexpr int kD4TileBytes = kD4StageKeys * kFp4RowBytes;
constexpr int kD4StageBytes = 2 * kD4TileBytes;      // K, then V
constexpr int kD4Dim = 128;

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

// NH: 8-head steps (group <= 8 * NH).  Two CTAs of 9 warps share an SM at
// NH = 1 (at most 112 registers a thread); NH = 2 holds twice the output and
// runs one.
template <int NH, bool CAP>
__global__ void __launch_bounds__(kD4Threads, NH == 1 ? 2 : 1)
k_decode4(const __grid_constant__ DecodeParams p, const uint8_t* __restrict__ kpool,
          const uint8_t* __restrict__ vpool) {
    constexpr int D = kD4Dim;
    const int NST = p.nst;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* stages = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
    float* merge_o = reinterpret_cast<float*>(stages + NST * kD4StageBytes);   // [warps][group][D]
    float* merge_ml = merge_o + p.merge_floats;                               // [warps][group][2]
    uint64_t* full = reinterpret_cast<uint64_t*>(
        (reinterpret_cast<uintptr_t>(merge_ml + kD4Warps * p.geo.group * 2) + 15) & ~uintptr_t(15));
    uint64_t* empty = full + NST;
    int2* desc = reinterpret_cast<int2*>(empty + NST);          // {unit, lo | hi << 16} of a stage
    volatile int* abort_flag = reinterpret_cast<volatile int*>(desc + NST);
    int* flag_last = const_cast<int*>(abort_flag) + 1;
    int4* batch = reinterpret_cast<int4*>(const_cast<int*>(abort_flag) + 4);  // [32][2] producer batch

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = gridDim.x, c = blockIdx.x;
    const int64_t T = p.total_items;
    const int64_t x0 = T * c / G, x1 = T * (c + 1) / G;
    const Geo& g = p.geo;
    const int group = g.group, P = g.page;

    if (threadIdx.x == 0) {
        for (int s = 0; s < NST; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
        *abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();

    if (warp == kD4Warps) {
        // ---------------- producer: stream this CTA's items ----------------
        if (x0 < x1) {
            int issued = 0, ps = 0;
            uint32_t pk = 0;
            bool stop = false;
            for (int64_t base = x0; base < x1 && !stop; base += 32) {
                const int64_t x = base + lane;
                if (x < x1) {
                    int lo_u = 0, hi_u = p.n_units - 1;      // unit holding item x
                    while (lo_u < hi_u) {
                        const int mid = (lo_u + hi_u) >> 1;
                        if (p.item_off[mid + 1] <= x) lo_u = mid + 1; else hi_u = mid;
                    }
                    const int u = lo_u;
                    const int b = u / g.hkv, h = u % g.hkv;
                    const int seq = p.seq[b];
                    const int64_t row = g.unit_row(seq, p.layer, h);
                    const UnitPol pol = p.meta.pol[row];
                    const int32_t* idx = p.meta.idx + (int64_t)seq * g.max_idx_per_seq + pol.idx_off;
                    const SlotRanges rg = decode_ranges(pol, idx, p.tq[b], P);
                    int64_t j = x - p.item_off[u];
                    int64_t w = 0, lo = 0, hi = 0;           // 64-slot window, visible slots in it
                    for (int q = 0; q < rg.count; ++q) {
                        const int64_t np = range_pages(rg.lo[q], rg.hi[q], kFp4ItemSlots);
                        if (j < np) {
                            w = rg.lo[q] / kFp4ItemSlots + j;
                            lo = max64(rg.lo[q], w * kFp4ItemSlots) - w * kFp4ItemSlots;
                            hi = min64(rg.hi[q], (w + 1) * kFp4ItemSlots) - w * kFp4ItemSlots;
                            break;
                        }
                        j -= np;
                    }
                    // first group row (in groups of the pool) of each group of 16 slots
                    int32_t gr[4];
                    #pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        gr[q] = 0;
                        if (16 * q + 16 <= lo || 16 * q >= hi) continue;
                        const int64_t slot = w * kFp4ItemSlots + 16 * q;
                        const int32_t page = p.meta.ptab[row * g.max_pages_unit + slot / P];
                        if (page < 0 || page >= g.num_pages) {
                            atomicOr(p.meta.status, kStatusBadPage);
                            continue;                        // load something harmless
                        }
                        gr[q] = (int32_t)(((int64_t)page * P + slot % P) >> 4);
                    }
                    batch[2 * lane] = make_int4(u, (int)lo | ((int)hi << 16), 0, 0);
                    batch[2 * lane + 1] = make_int4(gr[0], gr[1], gr[2], gr[3]);
                }
                __syncwarp();
                const int n = (int)min64(32, x1 - base);
                for (int i = 0; i < n && !stop; ++i) {
                    const int4 bi = batch[2 * i];
                    const int lo = bi.y & 0xFFFF, hi = bi.y >> 16;
                    #pragma unroll
                    for (int sub = 0; sub < kD4Sub; ++sub) {
                        if (stop) break;
                        const bool ok = pk == 0 || mbar_wait(&empty[ps], (pk - 1) & 1, abort_flag, p.meta.status);
                        if (__any_sync(0xffffffffu, !ok)) { stop = true; break; }
                        const int k0 = sub * kD4StageKeys;
                        const int slo = max(lo - k0, 0), shi = min(hi - k0, kD4StageKeys);
                        const int g0 = slo >> 4, ng = slo < shi ? ((shi + 15) >> 4) - g0 : 0;
                        if (lane == 0) {
                            desc[ps] = make_int2(bi.x, slo < shi ? slo | (shi << 16) : 0);
                            if (ng > 0) mbar_arrive_expect_tx(&full[ps], 2 * ng * kFp4GroupBytes);
                            else mbar_arrive(&full[ps]);
                        }
                        __syncwarp();
                        // lanes 0..3: (group, K or V) of the stage
                        const int q = lane & 1, kv = lane >> 1;
                        if (lane < 4 && q >= g0 && q < g0 + ng) {
                            const int32_t gr = reinterpret_cast<const int32_t*>(&batch[2 * i + 1])[2 * sub + q];
                            bulk_load(stages + ps * kD4StageBytes + kv * kD4TileBytes + q * kFp4GroupBytes,
                                      (kv ? vpool : kpool) + (int64_t)gr * kFp4GroupBytes, kFp4GroupBytes,
                                      &full[ps]);
                        }
                        ++issued;
                        if (++ps == NST) { ps = 0; ++pk; }
                    }
                }
                __syncwarp();
            }
            // leave only after every load this CTA issued has landed (bounded)
            if (lane == 0)
                for (int s = 0; s < NST && s < issued; ++s)
                    mbar_wait(&full[s], (uint32_t)(((issued - 1 - s) / NST) & 1), nullptr, nullptr);
        }
        return;
    }

    // ------------------------------ consumers ------------------------------
    const int ctid = threadIdx.x;
    constexpr int CT = kD4Warps * 32;
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
    if (x0 >= x1) return;

    const int gl = lane >> 2, j = lane & 3;          // fragment row, column pair
    // slots of this lane's rows of S^T in a group (positions gl and gl + 8)
    const int slot_a = (gl >> 1) + 4 * (gl & 1), slot_b = slot_a + 8;
    uint32_t qb[NH][8][2];
    float m_run[NH][2], l_run[NH][2], o[NH][8][4];
    int xi = warp, s = warp;                         // next stage fill of this warp, its stage
    uint32_t rounds = 0;
    bool dead = false;
    int u_lo = 0, u_hi = p.n_units - 1;              // first unit with an item >= x0
    while (u_lo < u_hi) {
        const int mid = (u_lo + u_hi) >> 1;
        if (p.item_off[mid + 1] <= x0) u_lo = mid + 1; else u_hi = mid;
    }
    for (int u = u_lo; u < p.n_units && p.item_off[u] < x1; ++u) {
        const int64_t ua = max64(p.item_off[u], x0), ub = min64(p.item_off[u + 1], x1);
        if (ua >= ub) continue;
        const int b = u / g.hkv, h = u - b * g.hkv;
        const float* ks = p.meta.kscale + ((int64_t)p.layer * g.hkv + h) * D;
        const float* vs = p.meta.vscale + ((int64_t)p.layer * g.hkv + h) * D;
        #pragma unroll
        for (int nh = 0; nh < NH; ++nh) {
            const int head = nh * 8 + gl;
            const __nv_bfloat16* qr = p.q + ((int64_t)b * g.hq + h * group + head) * D + j * 32;
            #pragma unroll
            for (int kk = 0; kk < 8; ++kk)
                #pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int cc = kk * 4 + 2 * e;
                    uint32_t w = 0;
                    if (head < group) w = *reinterpret_cast<const uint32_t*>(qr + cc);
                    const __nv_bfloat162 v2 = *reinterpret_cast<const __nv_bfloat162*>(&w);
                    qb[nh][kk][e] = pack_f16(__low2float(v2) * __ldg(ks + j * 32 + cc),
                                             __high2float(v2) * __ldg(ks + j * 32 + cc + 1));
                }
            m_run[nh][0] = m_run[nh][1] = -INFINITY;
            l_run[nh][0] = l_run[nh][1] = 0.f;
            #pragma unroll
            for (int mt = 0; mt < 8; ++mt)
                #pragma unroll
                for (int e = 0; e < 4; ++e) o[nh][mt][e] = 0.f;
        }
        for (; x0 * kD4Sub + xi < ub * kD4Sub; xi += kD4Warps) {
            if (!dead && !mbar_wait(&full[s], rounds & 1, abort_flag, p.meta.status)) dead = true;
            if (dead) continue;
            const int2 dd = desc[s];
            const int lo = dd.y & 0xFFFF, hi = dd.y >> 16;
            if (dd.x != u && lane == 0) atomicOr(p.meta.status, kStatusBadState);
            const uint8_t* tk = stages + s * kD4StageBytes;
            const uint8_t* tv = tk + kD4TileBytes;
            if (lo < hi) {
                float sc[2][NH][4];                  // [group][heads][accumulator]
                float mx[NH][2];
                #pragma unroll
                for (int nh = 0; nh < NH; ++nh) mx[nh][0] = mx[nh][1] = -INFINITY;
                #pragma unroll
                for (int q = 0; q < 2; ++q) {
                    #pragma unroll
                    for (int nh = 0; nh < NH; ++nh)
                        #pragma unroll
                        for (int e = 0; e < 4; ++e) sc[q][nh][e] = 0.f;
                    if (16 * q + 16 <= lo || 16 * q >= hi) {
                        #pragma unroll
                        for (int nh = 0; nh < NH; ++nh)
                            #pragma unroll
                            for (int e = 0; e < 4; ++e) sc[q][nh][e] = -INFINITY;
                        continue;
                    }
                    const uint8_t* gk = tk + q * kFp4GroupBytes;
                    const uint4 ca = *reinterpret_cast<const uint4*>(gk + gl * 64 + j * 16);
                    const uint4 cb = *reinterpret_cast<const uint4*>(gk + (gl + 8) * 64 + j * 16);
                    const uint32_t sw = *reinterpret_cast<const uint32_t*>(gk + kFp4ScaleOff + (gl * 4 + j) * 4);
                    const uint32_t wa[4] = {ca.x, ca.y, ca.z, ca.w}, wb[4] = {cb.x, cb.y, cb.z, cb.w};
                    #pragma unroll
                    for (int w = 0; w < 4; ++w) {    // 8 dimensions: two steps
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
                    const bool cut = 16 * q < lo || 16 * q + 16 > hi;
                    const bool in_a = !cut || (16 * q + slot_a >= lo && 16 * q + slot_a < hi);
                    const bool in_b = !cut || (16 * q + slot_b >= lo && 16 * q + slot_b < hi);
                    #pragma unroll
                    for (int nh = 0; nh < NH; ++nh)
                        #pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float v = CAP ? capped_log2(sc[q][nh][e], p.cap) : sc[q][nh][e] * p.scale_log2;
                            if (!(e < 2 ? in_a : in_b)) v = -INFINITY;
                            sc[q][nh][e] = v;
                            mx[nh][e & 1] = fmaxf(mx[nh][e & 1], v);
                        }
                }
                bool grew = false;
                #pragma unroll
                for (int nh = 0; nh < NH; ++nh)
                    #pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        mx[nh][e] = fmaxf(mx[nh][e], __shfl_xor_sync(0xffffffffu, mx[nh][e], 4));
                        mx[nh][e] = fmaxf(mx[nh][e], __shfl_xor_sync(0xffffffffu, mx[nh][e], 8));
                        mx[nh][e] = fmaxf(mx[nh][e], __shfl_xor_sync(0xffffffffu, mx[nh][e], 16));
                        grew = grew || mx[nh][e] > m_run[nh][e];
                    }
                if (__any_sync(0xffffffffu, grew)) {
                    #pragma unroll
                    for (int nh = 0; nh < NH; ++nh)
                        #pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float m_new = fmaxf(m_run[nh][e], mx[nh][e]);
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
                #pragma unroll
                for (int q = 0; q < 2; ++q) {
                    if (16 * q + 16 <= lo || 16 * q >= hi) continue;
                    uint32_t pb[NH][2];
                    #pragma unroll
                    for (int nh = 0; nh < NH; ++nh) {
                        float pv[4];
                        #pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float mb = m_run[nh][e & 1] == -INFINITY ? 0.f : m_run[nh][e & 1];
                            pv[e] = fast_exp2(sc[q][nh][e] - mb);
                            l_run[nh][e & 1] += pv[e];
                        }
                        pb[nh][0] = transpose8x8(pack_f16(pv[0], pv[1]));
                        pb[nh][1] = transpose8x8(pack_f16(pv[2], pv[3]));
                    }
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
                                mma_f16_16816(o[nh][4 * w + t], af, pb[nh][0], pb[nh][1]);
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[s]);
            s += kD4Warps;
            if (s >= NST) { s -= NST; ++rounds; }
        }

        // ------------- merge the warps' partial states -------------
        #pragma unroll
        for (int nh = 0; nh < NH; ++nh)
            #pragma unroll
            for (int e = 0; e < 2; ++e) {
                float l = l_run[nh][e];
                l += __shfl_xor_sync(0xffffffffu, l, 4);
                l += __shfl_xor_sync(0xffffffffu, l, 8);
                l += __shfl_xor_sync(0xffffffffu, l, 16);
                const int head = nh * 8 + 2 * j + e;
                if (head < group) {
                    float* mo = merge_o + ((size_t)warp * group + head) * D + gl * 16;
                    #pragma unroll
                    for (int mt = 0; mt < 8; ++mt)
                        *reinterpret_cast<float2*>(mo + 2 * mt) =
                            make_float2(o[nh][mt][e] * __ldg(vs + gl * 16 + 2 * mt),
                                        o[nh][mt][2 + e] * __ldg(vs + gl * 16 + 2 * mt + 1));
                    if (gl == 0) {
                        merge_ml[(warp * group + head) * 2] = m_run[nh][e];
                        merge_ml[(warp * group + head) * 2 + 1] = l;
                    }
                }
            }
        asm volatile("bar.sync 1, %0;" ::"n"(CT));

        const int64_t ia = p.item_off[u], ib = p.item_off[u + 1];
        const int c_first = (int)cta_of_item(ia, T, G), c_last = (int)cta_of_item(ib - 1, T, G);
        const bool whole = c_first == c_last;
        const int64_t part = (int64_t)u + c;
        for (int e = ctid; e < group * D; e += CT) {
            const int r = e / D, col = e % D;
            float mst = -INFINITY;
            #pragma unroll
            for (int w = 0; w < kD4Warps; ++w) mst = fmaxf(mst, merge_ml[(w * group + r) * 2]);
            float lst = 0.f, ost = 0.f;
            #pragma unroll
            for (int w = 0; w < kD4Warps; ++w) {
                const float sc_w = fast_exp2(merge_ml[(w * group + r) * 2] - mst);
                lst += sc_w * merge_ml[(w * group + r) * 2 + 1];
                ost += sc_w * merge_o[((size_t)w * group + r) * D + col];
            }
            const int64_t orow = (int64_t)b * g.hq + h * group + r;
            if (whole) {
                p.out[orow * D + col] = __float2bfloat16(ost / lst);
                if (col == 0 && p.lse) p.lse[orow] = (mst + __log2f(lst)) * 0.69314718055994531f;
            } else {
                p.part_o[(part * group + r) * D + col] = ost;
                if (col == 0) {
                    p.part_ml[(part * group + r) * 2] = mst;
                    p.part_ml[(part * group + r) * 2 + 1] = lst;
                }
            }
        }
        if (!whole) {
            __threadfence();
            asm volatile("bar.sync 1, %0;" ::"n"(CT));
            if (ctid == 0) {
                int target = 0;
                for (int cc = c_first; cc <= c_last; ++cc)
                    target += (T * cc / G) < (T * (cc + 1) / G) ? 1 : 0;
                const int old = atomicAdd(&p.counters[u], 1);
                *flag_last = (old == target - 1) ? 1 : 0;
            }
            asm volatile("bar.sync 1, %0;" ::"n"(CT));
            if (*flag_last) {
                // the last CTA of the unit: weights 2^(m - m*) of the parts, then
                // the weighted sum of their outputs
                __threadfence();
                const int nseg = c_last - c_first + 1;
                float* wts = merge_o;                          // [nseg][group] weights
                float* mls = merge_o + p.merge_floats / 2;     // [nseg][group] l
                float* mstar = merge_ml;                       // [group] m*, l*
                for (int e = ctid; e < nseg * group; e += CT) {
                    const int sg = e / group, r = e % group;
                    const int cc = c_first + sg;
                    const bool live = (T * cc / G) < (T * (cc + 1) / G);
                    const int64_t pi = (int64_t)u + cc;
                    wts[e] = live ? __ldcg(&p.part_ml[(pi * group + r) * 2]) : -INFINITY;
                    mls[e] = live ? __ldcg(&p.part_ml[(pi * group + r) * 2 + 1]) : 0.f;
                }
                asm volatile("bar.sync 1, %0;" ::"n"(CT));
                if (ctid < group) {
                    const int r = ctid;
                    float mst = -INFINITY;
                    for (int sg = 0; sg < nseg; ++sg) mst = fmaxf(mst, wts[sg * group + r]);
                    float lst = 0.f;
                    for (int sg = 0; sg < nseg; ++sg) {
                        const float w = fast_exp2(wts[sg * group + r] - mst);
                        wts[sg * group + r] = w;
                        lst += w * mls[sg * group + r];
                    }
                    mstar[2 * r] = mst;
                    mstar[2 * r + 1] = lst;
                }
                asm volatile("bar.sync 1, %0;" ::"n"(CT));
                for (int e = ctid; e < group * D; e += CT) {
                    const int r = e / D, col = e % D;
                    float acc[4] = {0.f, 0.f, 0.f, 0.f};
                    int sg = 0;
                    for (; sg + 4 <= nseg; sg += 4) {
                        float v4[4];
                        #pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const float w = wts[(sg + q) * group + r];
                            const int64_t pi = (int64_t)u + c_first + sg + q;
                            v4[q] = w != 0.f ? __ldcg(&p.part_o[(pi * group + r) * D + col]) * w : 0.f;
                        }
                        #pragma unroll
                        for (int q = 0; q < 4; ++q) acc[q] += v4[q];
                    }
                    for (; sg < nseg; ++sg) {
                        const float w = wts[sg * group + r];
                        const int64_t pi = (int64_t)u + c_first + sg;
                        if (w != 0.f) acc[0] += w * __ldcg(&p.part_o[(pi * group + r) * D + col]);
                    }
                    const float ost = (acc[0] + acc[1]) + (acc[2] + acc[3]);
                    const float lst = mstar[2 * r + 1];
                    const int64_t orow = (int64_t)b * g.hq + h * group + r;
                    p.out[orow * D + col] = __float2bfloat16(ost / lst);
                    if (col == 0 && p.lse) p.lse[orow] = (mstar[2 * r] + __log2f(lst)) * 0.69314718055994531f;
                }
                if (ctid == 0) p.counters[u] = 0;
            }
        }
        asm volatile("bar.sync 1, %0;" ::"n"(CT));
    }
}

template <int NH, bool CAP>
cudaError_t launch_decode4_t(const sp_cache* c, DecodeParams& p, int grid, cudaStream_t s) {
    // merge buffer: the warps' [group][D] partials, or two [grid][group] arrays
    // for the merge across CTAs, whichever is larger (a multiple of 4)
    constexpr int kCap = NH == 1 ? 113 * 1024 : 227 * 1024;
    const int group = c->geo.group;
    const int mo = std::max(kD4Warps * group * kD4Dim, 2 * grid * group);
    p.merge_floats = (mo + 3) & ~3;
    const int merge_bytes = (p.merge_floats + kD4Warps * group * 2) * 4;
    constexpr int kMaxStages4 = 32;
    constexpr int kMisc = kMaxStages4 * 24 + 16 + 32 * 32 + 16 + 128;   // barriers, descriptions, flags, batch, alignment
    // a multiple of the warps, so a stage always belongs to the same one
    p.nst = std::min(kMaxStages4, (kCap - merge_bytes - kMisc) / kD4StageBytes) / kD4Warps * kD4Warps;
    p.owners = kD4Warps;
    if (p.nst < kD4Warps) return cudaErrorInvalidConfiguration;
    const int smem = p.nst * kD4StageBytes + merge_bytes + kMisc;
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
