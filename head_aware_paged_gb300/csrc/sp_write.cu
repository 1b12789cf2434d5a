// sp_write.cu -- new queries and keys rotated to their positions, and the
// rotated keys and the values written into their heads' pages, in one launch.
//
// Mathematics: with a = p w_i (p the token's position, w_i the pair's
// frequency, i < d/2, the "rotate half" pairing of element i with i + d/2)
//     x'[i]       = x[i] cos a - x[i + d/2] sin a
//     x'[i + d/2] = x[i + d/2] cos a + x[i] sin a
// in fp32, rounded once: to bf16 (queries, bf16 pages) or to the page's codes.
// Far positions: the host gives w_i as a fraction of a turn in 64-bit fixed
// point, so p * w_i modulo 2^64 is the angle modulo a turn, reduced by the
// multiplication's own overflow.  An angle is off by the frequency's rounding in
// double, about p w_i 2^-54 turns (2^-34 at a million radians), by 2^-33 turns
// for the last bit of p w_i and as much where it is cut to 32 bits, and, the
// largest part, by 2^-26 turns (1e-7 radians) where it becomes an fp32 number of
// half turns; sincospif adds its own rounding.  One (cos, sin) per token and pair
// serves every head.
//
// Bound by memory: 4 bytes a q element, 2 + the page type's size a stored
// k / v element; a token that a head does not keep is not read.  Measured,
// 8,192 rows of 32 query and 8 KV heads: 31.8 us for every head GLOBAL (201 MB,
// 6.3 TB/s, 93 % of the copy rate), 24.8 us for one of eight (150 MB); FP8 and
// 4-bit pages 30.5 and 33.7 us.  64 rows of 64 sequences: 3.8 us.  A thread
// rotates one chunk of 8 dimensions and its partner chunk (16-byte loads and
// stores; a whole block of 16 for 4-bit pages, whose scale needs its maximum).
//
// Page allocation rides along: the host mirror knows every unit's demand, so
// unit u's new pages are the free-stack entries below top - off[u] and no
// block waits for another.  A block that writes a row reads old pages from the
// table and new ones from the stack, which this launch does not change; the
// last blocks of the grid put the new pages into the table.
//
// A captured call is replayed when the stack, and perhaps the sequence, have
// moved on: one that needs new pages is refused, and a captured launch asks the
// device what each sequence holds by then, before it writes a row or a length
// (an instance of its own: 28.5 instead of 26.9 us replaying the 8,192 rows).
#include <cmath>
#include <cstring>
#include <memory>

#include "sp_device.cuh"
#include "sp_internal.h"

namespace sp {

namespace {

constexpr int kWriteThreads = 256;
constexpr int kMaxTok = 4;                  // tokens of a block, at most

// MAXS sequences and MAXU (sequence, KV head) units: a call's parameters are
// copied at launch, so a small call uses the small record.
template <int MAXS, int MAXU>
struct WriteParams {
    Meta meta;
    Geo geo;
    int32_t layer, n_seqs, rows, top;      // top: free-stack height before the call
    int32_t row_blocks, tok, new_pages;    // blocks that write rows, tokens of each; any new page or length?
    int32_t scaled;                        // channel scales other than 1 may be set
    int64_t q_stride, k_stride, v_stride;  // elements between tokens
    const __nv_bfloat16 *q, *k, *v;
    __nv_bfloat16* q_out;
    void *kpool, *vpool;
    uint64_t turn[64];                     // frequency, in 2^-64 turns a position
    int32_t seq[MAXS], n_old[MAXS], n_new[MAXS], pos[MAXS], row0[MAXS + 1];
    int32_t off[MAXU + 1];                 // prefix of the units' new pages
};

// Eight elements of each half, rotated; fp32.  cs: this chunk's first (cos,
// sin, cos, sin) of two frequencies, the next two nc further.
__device__ __forceinline__ void rotate8(const uint4& xa, const uint4& yb, const float4* cs, int nc,
                                        float* x, float* y) {
    const uint32_t xw[4] = {xa.x, xa.y, xa.z, xa.w}, yw[4] = {yb.x, yb.y, yb.z, yb.w};
    #pragma unroll
    for (int e = 0; e < 4; ++e) {
        const __nv_bfloat162 u = *reinterpret_cast<const __nv_bfloat162*>(&xw[e]);
        const __nv_bfloat162 v = *reinterpret_cast<const __nv_bfloat162*>(&yw[e]);
        const float x0 = __low2float(u), x1 = __high2float(u), y0 = __low2float(v), y1 = __high2float(v);
        const float4 c = cs[e * nc];
        x[2 * e] = x0 * c.x - y0 * c.y;
        y[2 * e] = y0 * c.x + x0 * c.y;
        x[2 * e + 1] = x1 * c.z - y1 * c.w;
        y[2 * e + 1] = y1 * c.z + x1 * c.w;
    }
}
__device__ __forceinline__ void plain8(const uint4& a, float* x) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
    #pragma unroll
    for (int e = 0; e < 4; ++e) {
        const __nv_bfloat162 u = *reinterpret_cast<const __nv_bfloat162*>(&w[e]);
        x[2 * e] = __low2float(u);
        x[2 * e + 1] = __high2float(u);
    }
}
__device__ __forceinline__ uint4 bf16x8(const float* x) {
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}
// N elements times their channels' reciprocal scales.
template <int N>
__device__ __forceinline__ void times(float* x, const float* inv) {
    #pragma unroll
    for (int i = 0; i < N; i += 4) {
        const float4 f = __ldg(reinterpret_cast<const float4*>(inv + i));
        x[i] *= f.x; x[i + 1] *= f.y; x[i + 2] *= f.z; x[i + 3] *= f.w;
    }
}
// e4m3 of eight elements (nearest even, saturating).
__device__ __forceinline__ uint2 e4m3x8(const float* x) {
    uint32_t o[2] = {0u, 0u};
    #pragma unroll
    for (int e = 0; e < 4; ++e) {
        uint16_t code;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(code) : "f"(x[2 * e + 1]), "f"(x[2 * e]));
        o[e >> 1] |= (uint32_t)code << (16 * (e & 1));
    }
    return make_uint2(o[0], o[1]);
}

enum { kBf16, kFp8, kFp4 };

// Pages a unit of n tokens owns (unit_pages of sp_rules.h in 32 bits, P = 2^lp).
__device__ __forceinline__ int32_t pages32(const UnitPol& u, const int32_t* idx, int32_t n, int lp) {
    const int32_t up = (1 << lp) - 1;
    if (u.kind == kGlobal) return (n + up) >> lp;
    if (u.kind == kLocal)
        return ((min(n, u.sink) + up) >> lp) + min(u.ring, (max(0, n - u.sink) + up) >> lp);
    return ((int32_t)count_below(idx, u.n_idx, n) + up) >> lp;
}

// Where a token's row of one KV head goes: false if the head does not keep it.
// n: what the sequence holds after the call.
struct RowAt { int32_t page; int32_t slot; };
template <bool GRAPH, typename PR>
__device__ __forceinline__ bool row_at(const PR& p, int b, int h, int32_t t, int32_t n, RowAt& at) {
    const Geo& g = p.geo;
    const int lp = 31 - __clz(g.page);
    const int64_t row = g.unit_row(p.seq[b], p.layer, h);
    const UnitPol pol = p.meta.pol[row];
    const int32_t* idx = p.meta.idx + (int64_t)p.seq[b] * g.max_idx_per_seq + pol.idx_off;
    int32_t us = t;                                     // unit slot (unit_slot of sp_rules.h)
    if (pol.kind == kLocal && t >= pol.sink) {
        const int32_t ring = pol.ring << lp;
        if (t < n - ring) return false;                 // a newer token takes its slot
        us = (pol.sink_pages << lp) + (int32_t)((uint32_t)(t - pol.sink) % (uint32_t)ring);
    } else if (pol.kind == kRetrieval) {
        us = (int32_t)count_below(idx, pol.n_idx, t);
        if (us >= pol.n_idx || idx[us] != t) return false;
    }
    const int32_t pg = us >> lp;
    // old pages are in the table; new ones come from the stack
    const int32_t have = GRAPH ? p.meta.npages[row] : p.new_pages ? pages32(pol, idx, p.n_old[b], lp) : pg + 1;
    at.page = pg < have ? p.meta.ptab[row * g.max_pages_unit + pg]
              : GRAPH ? -1                              // (released, and filled under another policy)
                      : p.meta.fstack[p.top - 1 - (p.off[b * g.hkv + h] + pg - have)];
    at.slot = us & (g.page - 1);
    if (at.page < 0 || at.page >= g.num_pages) {
        atomicOr(p.meta.status, kStatusBadPage);
        return false;
    }
    return true;
}

// (Five blocks an SM, four for 4-bit pages: with more registers and fewer blocks
// 28.5 instead of 24.8 us, and 40.2 instead of 31.7 us.)
// GRAPH: the instance for captured calls.
template <int KV, bool GRAPH, typename PR>
__global__ void __launch_bounds__(kWriteThreads, KV == kFp4 ? 4 : 5)
k_write_rope(const __grid_constant__ PR p) {
    const Geo& g = p.geo;
    const int tid = threadIdx.x;
    if ((int)blockIdx.x >= p.row_blocks) {
        // page tables: a warp per unit puts its new pages in, and the lengths
        const int warp = tid >> 5, lane = tid & 31;
        if (blockIdx.y != 0) return;
        const int u = ((int)blockIdx.x - p.row_blocks) * (kWriteThreads / 32) + warp;
        if (u < p.n_seqs * g.hkv) {
            const int b = u / g.hkv, h = u % g.hkv;
            const int64_t row = g.unit_row(p.seq[b], p.layer, h);
            if constexpr (GRAPH) {                         // no pages; a length only grows
                int32_t* len = p.meta.seqlen + (int64_t)p.seq[b] * g.layers + p.layer;
                if (lane == 0 && h == 0 && *len >= p.n_old[b] && *len < p.n_new[b]) *len = p.n_new[b];
                return;
            }
            const UnitPol pol = p.meta.pol[row];
            const int32_t* idx = p.meta.idx + (int64_t)p.seq[b] * g.max_idx_per_seq + pol.idx_off;
            const int32_t have = pages32(pol, idx, p.n_old[b], 31 - __clz(g.page));
            const int32_t off = p.off[u], cnt = p.off[u + 1] - off;
            if (have + cnt > g.max_pages_unit || off + cnt > p.top) {      // the host checked; never expected
                if (lane == 0) atomicOr(p.meta.status, kStatusBadState);
            } else {
                int32_t* tab = p.meta.ptab + row * g.max_pages_unit + have;
                for (int j = lane; j < cnt; j += 32) tab[j] = p.meta.fstack[p.top - 1 - (off + j)];
                if (lane == 0) p.meta.npages[row] = have + cnt;
            }
            if (lane == 0 && h == 0) p.meta.seqlen[(int64_t)p.seq[b] * g.layers + p.layer] = p.n_new[b];
            if (lane == 0 && u == 0) p.meta.status[1] = p.top - p.off[p.n_seqs * g.hkv];
        }
        return;
    }
    constexpr int CH = KV == kFp4 ? 16 : 8;              // k / v dimensions of a chunk
    // angles, [token][pair of a chunk][chunk]: lanes read neighbouring chunks
    __shared__ float4 cs[kMaxTok * 32];
    __shared__ int32_t tok_b[kMaxTok], tok_t[kMaxTok], tok_n[kMaxTok];
    const int D = g.d, half = D / 2;
    const int r0 = (int)blockIdx.x * p.tok, nt = min(p.tok, p.rows - r0);
    // queries: two chunk pairs a pass (four 16-byte loads in flight a thread),
    // the first pass's loads ahead of the angles
    const int stride = kWriteThreads * gridDim.y, first = blockIdx.y * kWriteThreads + tid;
    const int nc = half / 8;                             // chunks of a head's half
    const int lq = 28 - __clz(half), q_row = g.hq << lq, q_all = p.q ? nt * q_row : 0;   // nc = 2^lq
    uint4 qa[2], qb[2];
    int qt[2], qat[2];                                   // token, element inside its row
    auto fetch = [&](int e0) {
        #pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int e = e0 + k * stride;
            if (e >= q_all) break;
            qt[k] = e / q_row;
            const int w = e - qt[k] * q_row;
            qat[k] = (w >> lq) * D + (w & ((1 << lq) - 1)) * 8;
            const __nv_bfloat16* src = p.q + (int64_t)(r0 + qt[k]) * p.q_stride + qat[k];
            qa[k] = *reinterpret_cast<const uint4*>(src);
            qb[k] = *reinterpret_cast<const uint4*>(src + half);
        }
    };
    fetch(first);
    if (tid < nt) {
        int a = 0, z = p.n_seqs - 1;                     // sequence with row0[b] <= row < row0[b + 1]
        while (a < z) {
            const int mid = (a + z + 1) >> 1;
            if (p.row0[mid] <= r0 + tid) a = mid; else z = mid - 1;
        }
        tok_b[tid] = a;
        tok_t[tid] = p.pos[a] + (r0 + tid - p.row0[a]);
        if constexpr (GRAPH) {                           // what it holds now: n_old, or what came since
            const int32_t held = p.meta.seqlen[(int64_t)p.seq[a] * g.layers + p.layer];
            tok_n[tid] = max(p.n_new[a], held);
            if (held < p.n_old[a]) {                     // released since: write no row of it
                tok_b[tid] = -1;
                atomicOr(p.meta.status, kStatusBadState);
            }
        }
    }
    __syncthreads();
    for (int e = tid; e < nt * half; e += kWriteThreads) {
        const int t = e / half, f = e % half;
        const uint64_t turns = (uint64_t)(uint32_t)tok_t[t] * p.turn[f];
        // nearest 2^-32 turn, as a signed number of half turns
        const float x = (float)(int32_t)(uint32_t)((turns + 0x80000000ull) >> 32) * 4.6566128730773926e-10f;
        float2* c = reinterpret_cast<float2*>(cs + (t * 4 + ((f & 7) >> 1)) * nc + (f >> 3)) + (f & 1);
        sincospif(x, &c->y, &c->x);
    }
    __syncthreads();
    for (int e0 = first; e0 < q_all; e0 += 2 * stride) {
        if (e0 != first) fetch(e0);
        #pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (e0 + k * stride >= q_all) break;
            float x[8], y[8];
            rotate8(qa[k], qb[k], cs + qt[k] * half / 2 + ((qat[k] & (D - 1)) >> 3), nc, x, y);
            __nv_bfloat16* dst = p.q_out + (int64_t)(r0 + qt[k]) * g.hq * D + qat[k];
            *reinterpret_cast<uint4*>(dst) = bf16x8(x);
            *reinterpret_cast<uint4*>(dst + half) = bf16x8(y);
        }
    }
    const int kc = half / CH, per = g.hkv * kc;
    for (int e = first; e < nt * per; e += stride) {
        const int t = e / per, h = (e - t * per) / kc, c = (e - t * per) % kc;
        RowAt at;
        const int b = tok_b[t];
        if (GRAPH && b < 0) continue;
        if (!row_at<GRAPH>(p, b, h, tok_t[t], GRAPH ? tok_n[t] : p.n_new[b], at)) continue;
        const __nv_bfloat16* ks = p.k + (int64_t)(r0 + t) * p.k_stride + h * D + c * CH;
        const __nv_bfloat16* vs = p.v + (int64_t)(r0 + t) * p.v_stride + h * D + c * CH;
        const float4* ang = cs + t * half / 2 + c * (CH / 8);
        const int64_t so = ((int64_t)p.layer * g.hkv + h) * D + c * CH;
        if constexpr (KV == kFp4) {
            const uint4* k4 = reinterpret_cast<const uint4*>(ks);
            const uint4* k4b = reinterpret_cast<const uint4*>(ks + half);
            const uint4 ka[2] = {k4[0], k4[1]}, kb[2] = {k4b[0], k4b[1]};
            const int64_t go = fp4_group_off(at.page, at.slot, g.page);
            uint8_t* kg = static_cast<uint8_t*>(p.kpool) + go;
            uint8_t* vg = static_cast<uint8_t*>(p.vpool) + go;
            const int s = at.slot & 15;
            float x[16], y[16];
            uint32_t sc;
            rotate8(ka[0], kb[0], ang, nc, x, y);
            rotate8(ka[1], kb[1], ang + 1, nc, x + 8, y + 8);
            if (p.scaled) {
                times<16>(x, p.meta.kinv + so);
                times<16>(y, p.meta.kinv + so + half);
            }
            *reinterpret_cast<uint2*>(kg + fp4_k_code(s, c)) = fp4_quant16(x, sc);
            kg[fp4_k_scale(s, c)] = (uint8_t)sc;
            *reinterpret_cast<uint2*>(kg + fp4_k_code(s, c + 4)) = fp4_quant16(y, sc);
            kg[fp4_k_scale(s, c + 4)] = (uint8_t)sc;
            const uint4* v4 = reinterpret_cast<const uint4*>(vs);
            const uint4* v4b = reinterpret_cast<const uint4*>(vs + half);
            plain8(v4[0], x);
            plain8(v4[1], x + 8);
            plain8(v4b[0], y);
            plain8(v4b[1], y + 8);
            if (p.scaled) {
                times<16>(x, p.meta.vinv + so);
                times<16>(y, p.meta.vinv + so + half);
            }
            *reinterpret_cast<uint2*>(vg + fp4_v_code(s, c)) = fp4_quant16(x, sc);
            vg[fp4_v_scale(s, c)] = (uint8_t)sc;
            *reinterpret_cast<uint2*>(vg + fp4_v_code(s, c + 4)) = fp4_quant16(y, sc);
            vg[fp4_v_scale(s, c + 4)] = (uint8_t)sc;
        } else {
            const uint4 ka = *reinterpret_cast<const uint4*>(ks);
            const uint4 kb = *reinterpret_cast<const uint4*>(ks + half);
            const uint4 va = *reinterpret_cast<const uint4*>(vs);
            const uint4 vb = *reinterpret_cast<const uint4*>(vs + half);
            const int64_t dst = ((int64_t)at.page * g.page + at.slot) * D + c * 8;
            float x[8], y[8];
            rotate8(ka, kb, ang, nc, x, y);
            if constexpr (KV == kFp8) {
                uint8_t* kp = static_cast<uint8_t*>(p.kpool) + dst;
                uint8_t* vp = static_cast<uint8_t*>(p.vpool) + dst;
                if (p.scaled) {
                    times<8>(x, p.meta.kinv + so);
                    times<8>(y, p.meta.kinv + so + half);
                }
                *reinterpret_cast<uint2*>(kp) = e4m3x8(x);
                *reinterpret_cast<uint2*>(kp + half) = e4m3x8(y);
                plain8(va, x);
                plain8(vb, y);
                if (p.scaled) {
                    times<8>(x, p.meta.vinv + so);
                    times<8>(y, p.meta.vinv + so + half);
                }
                *reinterpret_cast<uint2*>(vp) = e4m3x8(x);
                *reinterpret_cast<uint2*>(vp + half) = e4m3x8(y);
            } else {
                __nv_bfloat16* kp = static_cast<__nv_bfloat16*>(p.kpool) + dst;
                __nv_bfloat16* vp = static_cast<__nv_bfloat16*>(p.vpool) + dst;
                *reinterpret_cast<uint4*>(kp) = bf16x8(x);
                *reinterpret_cast<uint4*>(kp + half) = bf16x8(y);
                *reinterpret_cast<uint4*>(vp) = va;
                *reinterpret_cast<uint4*>(vp + half) = vb;
            }
        }
    }
}

constexpr int kSmallSeqs = 32, kSmallUnits = 256;
typedef WriteParams<kSmallSeqs, kSmallUnits> SmallWrite;
typedef WriteParams<kMaxCallSeqs, kMaxDecodeUnits> LargeWrite;
static_assert(sizeof(LargeWrite) <= 32764, "write parameters exceed the kernel parameter space");

template <bool GRAPH, typename PR>
void launch_write(const Geo& g, const PR& p, dim3 grid, cudaStream_t stream) {
    if (g.fp4) k_write_rope<kFp4, GRAPH><<<grid, kWriteThreads, 0, stream>>>(p);
    else if (g.fp8) k_write_rope<kFp8, GRAPH><<<grid, kWriteThreads, 0, stream>>>(p);
    else k_write_rope<kBf16, GRAPH><<<grid, kWriteThreads, 0, stream>>>(p);
}

template <typename PR>
sp_status write_rope(sp_cache* c, int32_t layer, const int32_t* seqs, int32_t n_seqs,
                     const int32_t* cu, const int64_t* pos, const __nv_bfloat16* q, int64_t q_stride,
                     const __nv_bfloat16* k, int64_t k_stride, const __nv_bfloat16* v,
                     int64_t v_stride, __nv_bfloat16* q_out, const uint64_t* turn, cudaStream_t stream) {
    std::unique_ptr<PR> pp(new PR());
    PR& p = *pp;
    const int H = c->cfg.num_kv_heads, L = c->cfg.num_layers, P = c->cfg.page_size;
    int32_t demand = 0;
    p.off[0] = 0;
    for (int b = 0; b < n_seqs; ++b) {
        const int seq = seqs[b];
        const int64_t n = c->h_seqlen[(size_t)seq * L + layer], cnt = (int64_t)cu[b + 1] - cu[b];
        const int64_t at = pos ? pos[b] : n;
        if (at < 0 || at > n)
            return fail(SP_ERR_INVALID_ARG, "pos outside [0, tokens held] for sequence " + std::to_string(seq));
        const int64_t n_new = std::max(n, at + cnt);
        if (n_new > c->cfg.max_seq_len)
            return fail(SP_ERR_INVALID_ARG, "sequence " + std::to_string(seq) + " would exceed max_seq_len");
        p.seq[b] = seq;
        p.n_old[b] = (int32_t)n;
        p.n_new[b] = (int32_t)n_new;
        p.pos[b] = (int32_t)at;
        p.row0[b] = cu[b];
        if (n_new != n) p.new_pages = 1;
        for (int h = 0; h < H; ++h) {
            const UnitPol& u = c->h_pol[((size_t)seq * L + layer) * H + h];
            const int32_t* idx = c->h_idx[seq].data() + u.idx_off;
            if (n_new != n) demand += (int32_t)(unit_pages(u, idx, n_new, P) - unit_pages(u, idx, n, P));
            p.off[b * H + h + 1] = demand;
        }
    }
    if (demand > c->h_free)
        return fail(SP_ERR_OUT_OF_PAGES, "call needs " + std::to_string(demand) + " pages, " +
                                             std::to_string(c->h_free) + " free");
    const int rows = cu[n_seqs];
    if (rows == 0) return SP_OK;
    cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
    const cudaError_t ce = cudaStreamIsCapturing(stream, &capture);
    if (ce != cudaSuccess) return cuda_fail(ce, "stream query");
    const bool graph = capture != cudaStreamCaptureStatusNone;
    if (graph && demand > 0)
        return fail(SP_ERR_UNSUPPORTED, "a captured call may not need new pages (" + std::to_string(demand) +
                                            "): replays would take them from the free stack again");
    p.row0[n_seqs] = rows;
    p.meta = c->meta;
    p.geo = c->geo;
    p.layer = layer;
    p.n_seqs = n_seqs;
    p.rows = rows;
    p.top = (int32_t)c->h_free;
    p.scaled = c->h_scaled[layer];
    p.q_stride = q_stride; p.k_stride = k_stride; p.v_stride = v_stride;
    p.q = q; p.k = k; p.v = v; p.q_out = q_out;
    p.kpool = c->kpool; p.vpool = c->vpool;
    std::memcpy(p.turn, turn, sizeof(p.turn));
    // Four tokens a block share its set-up once that still fills the GPU (8,192
    // rows, one head of eight GLOBAL, launches included: 27.0 us with four, 28.9
    // with two, 32.9 with eight, for which the arrays of four do not do); a short
    // call spreads one token's heads over two blocks instead.
    p.tok = rows >= 4 * c->num_sms ? kMaxTok : 1;
    p.row_blocks = (rows + p.tok - 1) / p.tok;
    const int items = (q ? c->cfg.num_q_heads : H) * c->cfg.head_dim / 16;
    const int split = p.tok == 1 && rows < 2 * c->num_sms && items > kWriteThreads ? 2 : 1;
    const int table = p.new_pages ? (n_seqs * H + kWriteThreads / 32 - 1) / (kWriteThreads / 32) : 0;
    const dim3 grid((unsigned)(p.row_blocks + table), (unsigned)split);
    if (graph) launch_write<true>(c->geo, p, grid, stream);
    else launch_write<false>(c->geo, p, grid, stream);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "write launch");
    c->h_free -= demand;
    for (int b = 0; b < n_seqs; ++b) {
        c->h_seqlen[(size_t)seqs[b] * L + layer] = p.n_new[b];
        for (int h = 0; h < H; ++h)
            c->h_npages[((size_t)seqs[b] * L + layer) * H + h] += p.off[b * H + h + 1] - p.off[b * H + h];
    }
    return SP_OK;
}

// Does one of `rows` rows of `len` bytes, `stride` bytes apart from `base` on,
// meet [lo, hi)?
bool rows_meet(const void* base, int64_t stride, int64_t len, int64_t rows, uintptr_t lo, uintptr_t hi) {
    const uintptr_t b = reinterpret_cast<uintptr_t>(base);
    const int64_t d = (int64_t)(lo - b) - len;          // the first row that ends behind lo
    const int64_t r = d < 0 ? 0 : d / stride + 1;
    return r < rows && b + (uintptr_t)(r * stride) < hi;
}

}  // namespace

}  // namespace sp

using namespace sp;

extern "C" sp_status sp_append_kv_rope(sp_cache* c, int32_t layer, const int32_t* seq_ids, int32_t n_seqs,
                                       const int32_t* cu_new, const int64_t* pos, const void* q,
                                       int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                       int64_t v_stride, void* q_out, double rope_theta,
                                       const double* inv_freq, void* stream) {
    if (!c || !cu_new) return fail(SP_ERR_INVALID_ARG, "null argument");
    if (!valid_layer(c, layer)) return fail(SP_ERR_INVALID_ARG, "layer out of range");
    sp_status s = check_seq_list(c, seq_ids, n_seqs);
    if (s != SP_OK) return s;
    if (cu_new[0] != 0) return fail(SP_ERR_INVALID_ARG, "cu_new[0] must be 0");
    for (int b = 0; b < n_seqs; ++b)
        if (cu_new[b + 1] < cu_new[b]) return fail(SP_ERR_INVALID_ARG, "cu_new must be non-decreasing");
    if (cu_new[n_seqs] > c->cfg.max_tokens) return fail(SP_ERR_INVALID_ARG, "more new tokens than max_tokens");
    if (cu_new[n_seqs] > 0) {                    // (without rows there may be no tensors)
        if (!k || !v) return fail(SP_ERR_INVALID_ARG, "null argument");
        if ((q == nullptr) != (q_out == nullptr))
            return fail(SP_ERR_INVALID_ARG, "give both q and q_out or neither");
    }
    const int d = c->cfg.head_dim;
    const int64_t kv = (int64_t)c->cfg.num_kv_heads * d;
    if (k_stride < kv || v_stride < kv || (q && q_stride < (int64_t)c->cfg.num_q_heads * d) ||
        ((k_stride | v_stride | (q ? q_stride : 0)) & 7))
        return fail(SP_ERR_INVALID_ARG, "strides must be >= heads * head_dim and multiples of 8");
    if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) |
         reinterpret_cast<uintptr_t>(q_out)) & 15)
        return fail(SP_ERR_INVALID_ARG, "q, k, v and q_out must be 16-byte aligned");
    if (q && cu_new[n_seqs] > 0) {
        // a block reads its rows while others write theirs: no overlap but a row with itself
        const int64_t rows = cu_new[n_seqs], row = (int64_t)c->cfg.num_q_heads * d;
        const uintptr_t lo = reinterpret_cast<uintptr_t>(q_out), hi = lo + (uintptr_t)(rows * row * 2);
        const bool in_place = q == q_out && (q_stride == row || rows == 1);
        if ((!in_place && rows_meet(q, q_stride * 2, row * 2, rows, lo, hi)) ||
            rows_meet(k, k_stride * 2, kv * 2, rows, lo, hi) || rows_meet(v, v_stride * 2, kv * 2, rows, lo, hi))
            return fail(SP_ERR_INVALID_ARG, "q_out overlaps q, k or v (it may be q itself if q is contiguous)");
    }
    if (!inv_freq && (!(rope_theta > 0.0) || !std::isfinite(rope_theta)))
        return fail(SP_ERR_INVALID_ARG, "rope_theta must be positive and finite");
    // frequencies as fractions of a turn, modulo one turn (whole turns a
    // position rotate nothing), in 2^-64 turns
    uint64_t turn[64] = {};
    const double two_pi = 6.283185307179586476925286766559;
    for (int i = 0; i < d / 2; ++i) {
        const double w = inv_freq ? inv_freq[i] : std::pow(rope_theta, -2.0 * i / d);
        if (!(std::fabs(w) <= 65536.0)) return fail(SP_ERR_INVALID_ARG, "frequencies must be finite, at most 2^16");
        const double f = w / two_pi, frac = f - std::floor(f);      // [0, 1]
        turn[i] = frac < 1.0 ? (uint64_t)(frac * 18446744073709551616.0) : 0;
    }
    s = check_device(c);
    if (s != SP_OK) return s;
    auto* qp = static_cast<const __nv_bfloat16*>(q);
    auto* kp = static_cast<const __nv_bfloat16*>(k);
    auto* vp = static_cast<const __nv_bfloat16*>(v);
    auto* qo = static_cast<__nv_bfloat16*>(q_out);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return no_throw([&] {
        if (n_seqs <= kSmallSeqs && n_seqs * c->cfg.num_kv_heads <= kSmallUnits)
            return write_rope<SmallWrite>(c, layer, seq_ids, n_seqs, cu_new, pos, qp, q_stride, kp, k_stride, vp,
                                          v_stride, qo, turn, st);
        return write_rope<LargeWrite>(c, layer, seq_ids, n_seqs, cu_new, pos, qp, q_stride, kp, k_stride, vp,
                                      v_stride, qo, turn, st);
    });
}
