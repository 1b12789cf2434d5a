// sp_prefill.cu -- prefill calls: the work list (items, their order, their
// CTAs, pieces of long ones), the launch of k_prefill (sp_prefill.cuh), and
// the merge of split items.
#include <algorithm>
#include <climits>
#include <cmath>
#include <memory>
#include <functional>
#include <utility>
#include <vector>

#include "sp_prefill.cuh"

namespace sp {

namespace {

// |V(i)| as the tile plan and the mask see it (one thread per position).
__global__ void k_prefill_counts(Meta meta, Geo g, int seq, int layer, int h,
                                 const int64_t* pos, int npos, int32_t* out) {
    const int64_t urow = g.unit_row(seq, layer, h);
    const UnitPol pol = meta.pol[urow];
    const int32_t* idx = meta.idx + (int64_t)seq * g.max_idx_per_seq + pol.idx_off;
    const int64_t held = meta.seqlen[(int64_t)seq * g.layers + layer];
    for (int k = blockIdx.x * blockDim.x + threadIdx.x; k < npos; k += gridDim.x * blockDim.x) {
        const int64_t i = pos[k];
        if (i < held) continue;
        const int64_t i_lo = held + (i - held) / 128 * 128;
        const int64_t i_hi = i_lo + 127;
        const Plan pl = make_plan(pol, idx, held, i_lo, i_hi, g.page);
        int64_t cnt = 0;
        for (int64_t t = 0; t < pl.ntiles; ++t) {
            const KvTile kt = plan_tile(pl, pol, t, i_lo, i_hi);
            for (int c = 0; c < kt.nkeys; ++c) {
                const int64_t tp = kt.table ? tile_key_position(kt, pol, idx, held, c, g.page) : 0;
                cnt += key_visible<int64_t>(kt, pol, i, c, tp) ? 1 : 0;
            }
        }
        out[k] = (int32_t)cnt;
    }
}

// Pieces of split items -> final rows: per (item, query tile, 32 columns)
// block, one thread per row combines the pieces' (O, m, l): m* = max m, each piece
// weighted by 2^(m - m*), O = sum w O / sum w l, LSE = m* + log2(sum w l) in
// natural-log units.  A row no piece saw gives O = 0, LSE = -inf.
constexpr int kMaxMergeGroups = 1024;
constexpr int kMaxPieces = 8;
struct MergeParams {
    int32_t n_groups, hq;
    const float4* split_o;
    const float2* split_ml;
    __nv_bfloat16* out;
    float* lse;
    int4 groups[kMaxMergeGroups];   // {row_base, first query head, rows, first slot | pieces << 16}
};

template <int D>
__global__ void __launch_bounds__(128) k_prefill_merge(const __grid_constant__ MergeParams p) {
    // block (group, query tile, 32-column slice); thread = row
    const int4 gr = p.groups[blockIdx.x];
    const int t = blockIdx.y, c0 = blockIdx.z * 32, r = threadIdx.x;
    if (r >= gr.z) return;
    const int slot0 = gr.w & 0xFFFF, np = gr.w >> 16;
    float ms[kMaxPieces], wq[kMaxPieces], mx = -INFINITY;
    #pragma unroll
    for (int q = 0; q < kMaxPieces; ++q) {
        ms[q] = -INFINITY;
        wq[q] = 0.f;
        if (q < np) {
            const float2 ml = p.split_ml[((int64_t)(slot0 + q) * 2 + t) * 128 + r];
            ms[q] = ml.x;
            wq[q] = ml.y;
            mx = fmaxf(mx, ml.x);
        }
    }
    float L = 0.f;
    #pragma unroll
    for (int q = 0; q < kMaxPieces; ++q) {
        const float w = ms[q] != -INFINITY ? exp2f(ms[q] - mx) : 0.f;
        L += w * wq[q];
        wq[q] = w;
    }
    const float inv = L > 0.f ? 1.f / L : 0.f;
    float a[32];
    #pragma unroll
    for (int e = 0; e < 32; ++e) a[e] = 0.f;
    #pragma unroll
    for (int q = 0; q < kMaxPieces; ++q) {
        if (q < np) {
            const float4* po = p.split_o + ((int64_t)(slot0 + q) * 2 + t) * (D / 4) * 128 + r;
            #pragma unroll
            for (int e4 = 0; e4 < 8; ++e4) {
                const float4 x = po[(c0 / 4 + e4) * 128];
                a[4 * e4] += wq[q] * x.x; a[4 * e4 + 1] += wq[q] * x.y;
                a[4 * e4 + 2] += wq[q] * x.z; a[4 * e4 + 3] += wq[q] * x.w;
            }
        }
    }
    __nv_bfloat16* orow = p.out + ((int64_t)(gr.x + r) * p.hq + gr.y + t) * D + c0;
    #pragma unroll
    for (int e = 0; e < 32; e += 8)
        *reinterpret_cast<uint4*>(orow + e) =
            make_uint4(pack_bf16(a[e] * inv, a[e + 1] * inv), pack_bf16(a[e + 2] * inv, a[e + 3] * inv),
                       pack_bf16(a[e + 4] * inv, a[e + 5] * inv), pack_bf16(a[e + 6] * inv, a[e + 7] * inv));
    if (p.lse && blockIdx.z == 0)
        p.lse[(int64_t)(gr.x + r) * p.hq + gr.y + t] =
            L == 0.f ? -INFINITY : (mx + __log2f(L)) * 0.69314718055994531f;   // NaN rows: NaN
}

static_assert(sizeof(MergeParams) <= 32764, "merge parameters exceed the kernel parameter space");

}  // namespace

int64_t prefill_max_tiles(const sp_config* c) {
    // work items plus room for the per-CTA offsets behind them
    return ((int64_t)c->max_tokens / 128 + c->max_batch + 1) * c->num_q_heads + 512;
}

// An item counts its key tiles in 20 bits.  Checked before the call's first
// launch: a refused call has launched nothing.
static sp_status check_tiles(const sp_cache* c, int32_t layer, const int32_t* seq_ids, int32_t n_seqs,
                             const int32_t* cu_q) {
    constexpr int64_t kMaxTiles = int64_t(1) << 20;
    for (int b = 0; b < n_seqs; ++b) {
        const int64_t n_b = c->h_seqlen[(size_t)seq_ids[b] * c->cfg.num_layers + layer];
        const int64_t cb = cu_q[b + 1] - cu_q[b];
        if (cb == 0 || plan_tiles_bound(n_b + cb) < kMaxTiles) continue;
        for (int h = 0; h < c->cfg.num_kv_heads; ++h) {
            const UnitPol& u = c->h_pol[((size_t)seq_ids[b] * c->cfg.num_layers + layer) * c->cfg.num_kv_heads + h];
            const int32_t* idx = c->h_idx[seq_ids[b]].data() + u.idx_off;
            for (int64_t r = 0; r < cb; r += 128)
                if (make_plan(u, idx, n_b, n_b + r, n_b + std::min(cb, r + 128) - 1, c->cfg.page_size).ntiles >= kMaxTiles)
                    return fail(SP_ERR_UNSUPPORTED, "more than 2^20 key tiles for one row block");
        }
    }
    return SP_OK;
}

// The call's units [unit0, unit1) (call sequence * hkv + KV head); `first` and
// `last` of the call's launches carry its launch events.
static sp_status prefill_units(sp_cache* c, int32_t layer, const int32_t* seq_ids, int32_t n_seqs,
                               const int32_t* cu_q, const __nv_bfloat16* q, const __nv_bfloat16* k,
                               const __nv_bfloat16* v, __nv_bfloat16* out, float* lse, const Cap& cap,
                               int unit0, int unit1, bool first, bool last, cudaStream_t stream) {
    const int T = cu_q[n_seqs];
    std::unique_ptr<PrefillParams> pp(new PrefillParams());
    PrefillParams& p = *pp;
    p.meta = c->meta;
    p.geo = c->geo;
    p.layer = layer;
    const int group = c->geo.group;
    p.nq = (group % 2 == 0) ? 2 : 1;
    const int pairs = group / p.nq;
    p.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)c->cfg.head_dim));
    p.out = out;
    p.lse = lse;
    p.cap = cap;
    p.hist_row = c->ws.deq_row;
    p.split_o = reinterpret_cast<float4*>(c->ws.split_o);
    p.split_ml = reinterpret_cast<float2*>(c->ws.split_ml);
    struct Cand { int64_t cost; int32_t unit; int4 item; };   // unit: call sequence * Hkv + KV head
    std::vector<Cand> whole;
    {
        size_t n_rb = 0;
        for (int b = 0; b < n_seqs; ++b) n_rb += (size_t)(cu_q[b + 1] - cu_q[b] + 127) / 128;
        whole.reserve(n_rb * c->cfg.num_kv_heads * pairs);
    }
    const int P = c->cfg.page_size;
    for (int b = 0; b < n_seqs; ++b) {
        const int seq = seq_ids[b];
        const int64_t n_b = c->h_seqlen[(size_t)seq * c->cfg.num_layers + layer];
        const int cb = cu_q[b + 1] - cu_q[b];
        p.seq[b] = seq;
        p.n_b[b] = (int32_t)n_b;
        p.cnt[b] = cb;
        p.row0[b] = cu_q[b];
        for (int h = 0; h < c->cfg.num_kv_heads; ++h) {
            const int cu = b * c->cfg.num_kv_heads + h;
            if (cu < unit0 || cu >= unit1) continue;
            const size_t ui = ((size_t)seq * c->cfg.num_layers + layer) * c->cfg.num_kv_heads + h;
            const UnitPol& u = c->h_pol[ui];
            const int32_t* idx = c->h_idx[seq].data() + u.idx_off;
            for (int rb = 0; rb * 128 < cb; ++rb) {
                const int64_t i_lo = n_b + rb * 128;
                const int64_t i_hi = n_b + std::min(cb, rb * 128 + 128) - 1;
                const Plan pl = make_plan(u, idx, n_b, i_lo, i_hi, P);
                // Time model for the assignment, measured per CTA with clock64
                // traces: every K/V tile costs about the same whatever its
                // width (the softmax treats a whole tile), and an item adds the
                // pipeline fill, the epilogue and the hand-over to the next
                // item, about three tiles' worth.
                const int64_t cost = kTileCost * pl.ntiles + kItemCost;
                for (int pr = 0; pr < pairs; ++pr)
                    whole.push_back({cost, b * c->cfg.num_kv_heads + h,
                                     make_int4(b, h, pr | (rb << 8), (int)pl.ntiles)});
            }
        }
    }
    // An item much longer than a CTA's fair share of the call would set the
    // launch's end on its own (a GLOBAL head's row blocks over a long
    // history, next to short LOCAL ones).  Such items are split along their
    // key tiles into pieces of about half a share; each piece leaves its
    // unnormalised O and (m, l) in a workspace slot and k_prefill_merge
    // combines them.
    int64_t total = 0;
    for (const Cand& cd : whole) total += cd.cost;
    const double share = (double)total / std::max(1, c->num_sms);
    std::vector<Cand> cands;
    cands.reserve(whole.size() + kPrefillSplitSlots);
    std::vector<int4> groups;                  // merge: {row_base, first head, rows, slot | pieces << 16}
    int slots = 0;
    for (const Cand& cd : whole) {
        const int nt = cd.item.w;
        int np = 1;
        if ((double)cd.cost > 0.8 * share && nt >= 2 * kMinPieceTiles) {
            np = (int)std::ceil((double)cd.cost / (0.5 * share));
            np = std::min(std::min(np, kMaxPieces), nt / kMinPieceTiles);
            if (slots + np > kPrefillSplitSlots || (int)groups.size() >= kMaxMergeGroups) np = 1;
        }
        if (np <= 1) {
            cands.push_back(cd);
            continue;
        }
        const int b = cd.item.x, h = cd.item.y, pr = cd.item.z & 255, rb = cd.item.z >> 8;
        const int cb = cu_q[b + 1] - cu_q[b];
        groups.push_back(make_int4(cu_q[b] + rb * 128, h * group + pr * p.nq,
                                   std::min(128, cb - rb * 128), slots | (np << 16)));
        for (int q = 0; q < np; ++q) {
            const int t0 = (int)((int64_t)nt * q / np), t1 = (int)((int64_t)nt * (q + 1) / np);
            const int4 it = make_int4(b | (t0 << 10), h, cd.item.z, (t1 - t0) | ((slots + q + 1) << 20));
            cands.push_back({kTileCost * (t1 - t0) + kItemCost, cd.unit, it});
        }
        slots += np;
    }
    // (prefill_max_tiles has room for every call that the entry points let pass)
    if ((int64_t)cands.size() + (c->num_sms + 4) / 4 > c->ws.max_tiles)
        return fail(SP_ERR_UNSUPPORTED, "prefill work list larger than the workspace");
    // Order.  When the call's K/V is larger than about half of L2: unit by
    // unit (units with the most work first), each unit's items longest
    // first, so all CTAs work through one unit's K/V at a time (a GLOBAL
    // head of a 128K sequence holds 67 MB of K and V) instead of every unit
    // whose items have similar lengths at once, which overflows L2 and reads
    // K/V tiles from HBM several times (measured: a 128K layer with two
    // GLOBAL heads reads 8.6 GB instead of 16.5 GB, in the same time).
    // Otherwise longest first over all items, which balances the CTAs'
    // end times a little better (3-9 % faster on 8K-token calls).
    const int n_units = n_seqs * c->cfg.num_kv_heads;
    std::vector<int32_t> rank(n_units, 0);
    int64_t kv_bytes = 0;
    for (int b = 0; b < n_seqs; ++b)
        kv_bytes += (int64_t)(p.n_b[b] + p.cnt[b]) * c->cfg.num_kv_heads * 2 * c->cfg.head_dim *
                    (c->geo.fp8 ? 1 : 2);
    if (kv_bytes > kL2UnitOrderBytes) {
        std::vector<int64_t> unit_cost(n_units, 0);
        for (const Cand& cd : cands) unit_cost[cd.unit] += cd.cost;
        std::vector<int32_t> by_cost(n_units);
        for (int u = 0; u < n_units; ++u) by_cost[u] = u;
        std::stable_sort(by_cost.begin(), by_cost.end(),
                         [&](int32_t a, int32_t b2) { return unit_cost[a] > unit_cost[b2]; });
        for (int r = 0; r < n_units; ++r) rank[by_cost[r]] = r;
    }
    // One sort of packed keys (unit rank, cost descending, candidate index:
    // a stable order); a comparison sort of the records when a field would
    // not fit its bits.
    const size_t n_items = cands.size();
    std::vector<uint32_t> order(n_items);
    if (n_units < (1 << 16) && n_items < (size_t(1) << 20)) {
        // cost = kTileCost * tiles + kItemCost < 2^28 for tiles < 2^20
        std::vector<uint64_t> key(n_items);
        for (size_t i = 0; i < n_items; ++i)
            key[i] = ((uint64_t)rank[cands[i].unit] << 48) |
                     ((uint64_t)((int64_t(1) << 28) - 1 - cands[i].cost) << 20) | (uint64_t)i;
        std::sort(key.begin(), key.end());
        for (size_t i = 0; i < n_items; ++i) order[i] = (uint32_t)(key[i] & 0xFFFFFu);
    } else {
        for (size_t i = 0; i < n_items; ++i) order[i] = (uint32_t)i;
        std::stable_sort(order.begin(), order.end(), [&](uint32_t a, uint32_t b2) {
            const Cand &x = cands[a], &y = cands[b2];
            return rank[x.unit] != rank[y.unit] ? rank[x.unit] < rank[y.unit] : x.cost > y.cost;
        });
    }
    // Greedy assignment in that order: each item goes to the CTA with the
    // least work so far (longest-processing-time rule within a unit; ties to
    // the lower CTA).
    const int grid = (int)std::min<int64_t>(c->num_sms, (int64_t)n_items);
    std::vector<int32_t> owner(n_items);
    std::vector<int32_t> fill(grid + 1, 0);
    {
        typedef std::pair<int64_t, int> LoadCta;
        std::vector<LoadCta> heap(grid);
        for (int g2 = 0; g2 < grid; ++g2) heap[g2] = LoadCta(0, g2);   // a valid min-heap
        const auto later = std::greater<LoadCta>();
        for (size_t k2 = 0; k2 < n_items; ++k2) {
            const uint32_t i = order[k2];
            std::pop_heap(heap.begin(), heap.end(), later);
            LoadCta& top = heap.back();
            owner[i] = top.second;
            ++fill[top.second + 1];
            top.first += cands[i].cost;
            std::push_heap(heap.begin(), heap.end(), later);
        }
    }
    if (n_items == 0) {                        // no rows in these units
        if (last) launch_mark_end(c, stream);
        return SP_OK;
    }
    // The items grouped by CTA (each CTA's in the sorted order), then the CTA
    // offsets: inside the kernel parameters when they fit, else one upload
    // through the next pinned staging buffer (asynchronous; waits only if
    // that buffer's previous copy has not run yet)
    const size_t words = n_items + (grid + 1 + 3) / 4;
    const bool inl = words <= (size_t)kInlineWords;
    int si = -1;
    int4* buf = inl ? p.inl : static_cast<int4*>(stage_acquire(c, words * sizeof(int4), &si));
    if (!buf) return fail(SP_ERR_CUDA, "prefill staging buffer");
    int32_t* off = reinterpret_cast<int32_t*>(buf + n_items);
    for (int g2 = 0; g2 < grid; ++g2) fill[g2 + 1] += fill[g2];
    for (int g2 = 0; g2 <= grid; ++g2) off[g2] = fill[g2];
    for (size_t k2 = 0; k2 < n_items; ++k2) {
        const uint32_t i = order[k2];
        buf[fill[owner[i]]++] = cands[i].item;
    }
    p.n_items = (int32_t)n_items;
    p.inline_words = inl ? (int32_t)words : 0;
    // One MMA issuer per query tile wherever the kernel has that instance:
    // bf16 K/V, head_dim 128, two query tiles per item (the single issuer
    // sits behind its own commits and waits while the other tile's P is
    // ready: 0.67 vs 0.73 of peak on 128K calls, 0.46 vs 0.50 on 8K).
    const bool two = !c->geo.fp8 && p.nq == 2 && c->cfg.head_dim == 128;
    // speculative exponentials (SPEC) for calls whose items average more
    // than kSpecTilesPerItem tiles
    bool spec = false;
    if (two) {
        int64_t tiles_total = 0;
        for (const Cand& cd : cands) tiles_total += cd.item.w & 0xFFFFF;
        spec = tiles_total > kSpecTilesPerItem * (int64_t)n_items;
    }
    cudaError_t e = cudaSuccess;
    if (!inl) {
        p.items = c->ws.tiles;
        p.cta_off = reinterpret_cast<const int32_t*>(c->ws.tiles + n_items);
        e = stage_copy(c, si, c->ws.tiles, words * sizeof(int4), stream);
        if (e != cudaSuccess) return cuda_fail(e, "prefill work list upload");
    }
    CUtensorMap tq, tk, tv;
    std::string err;
    const int D = c->cfg.head_dim;
    if (!encode_tmap_2d(&tq, q, (uint64_t)c->cfg.num_q_heads * D, T,
                        (uint64_t)c->cfg.num_q_heads * D * 2, 64, 128, true, &err) ||
        !encode_tmap_2d(&tk, k, (uint64_t)c->cfg.num_kv_heads * D, T,
                        (uint64_t)c->cfg.num_kv_heads * D * 2, 64, 128, true, &err) ||
        !encode_tmap_2d(&tv, v, (uint64_t)c->cfg.num_kv_heads * D, T,
                        (uint64_t)c->cfg.num_kv_heads * D * 2, 64, 128, true, &err))
        return fail(SP_ERR_CUDA, err);
    if (first && !c->geo.fp4) launch_mark_start(c, stream);
#define SP_PF(DD, PP) \
    if (D == DD && P == PP) e = launch_prefill_t<DD, PP>(c, p, grid, tq, tk, tv, stream); else
#define SP_PF2(PP) \
    if (P == PP) e = spec ? launch_prefill_t<128, PP, false, true, true>(c, p, grid, tq, tk, tv, stream) \
                          : launch_prefill_t<128, PP, false, true>(c, p, grid, tq, tk, tv, stream); else
#define SP_PF8(PP) \
    if (D == 128 && P == PP) e = launch_prefill_t<128, PP, true>(c, p, grid, tq, tk, tv, stream); else
    if (cap.on) {
        e = launch_prefill_capped(c, p, grid, two, tq, tk, tv, stream);
    } else if (c->geo.fp4) {
        e = launch_prefill_rows(c, p, grid, two, spec, tq, tk, tv, stream);
    } else if (c->geo.fp8) {   // FP8 pages (head_dim 128, checked at create)
        SP_PF8(16) SP_PF8(32) SP_PF8(64) SP_PF8(128)
        e = cudaErrorInvalidValue;
    } else if (two) {   // head_dim 128, two query tiles
        SP_PF2(16) SP_PF2(32) SP_PF2(64) SP_PF2(128)
        e = cudaErrorInvalidValue;
    } else {
        SP_PF(64, 16) SP_PF(64, 32) SP_PF(64, 64) SP_PF(64, 128)
        SP_PF(128, 16) SP_PF(128, 32) SP_PF(128, 64) SP_PF(128, 128)
        e = cudaErrorInvalidValue;
    }
#undef SP_PF
#undef SP_PF2
#undef SP_PF8
    if (e != cudaSuccess) return cuda_fail(e, "prefill launch");
    if (!groups.empty()) {
        std::unique_ptr<MergeParams> mp(new MergeParams());
        mp->n_groups = (int32_t)groups.size();
        mp->hq = c->cfg.num_q_heads;
        mp->split_o = p.split_o;
        mp->split_ml = p.split_ml;
        mp->out = out;
        mp->lse = lse;
        std::copy(groups.begin(), groups.end(), mp->groups);
        const dim3 mg((unsigned)groups.size(), (unsigned)p.nq, (unsigned)(D / 32));
        if (D == 128) k_prefill_merge<128><<<mg, 128, 0, stream>>>(*mp);
        else k_prefill_merge<64><<<mg, 128, 0, stream>>>(*mp);
        e = cudaGetLastError();
        if (e != cudaSuccess) return cuda_fail(e, "prefill merge launch");
    }
    if (last) launch_mark_end(c, stream);
    return SP_OK;
}

sp_status prefill_impl(sp_cache* c, int32_t layer, const int32_t* seq_ids, int32_t n_seqs,
                       const int32_t* cu_q, const __nv_bfloat16* q, const __nv_bfloat16* k,
                       const __nv_bfloat16* v, __nv_bfloat16* out, float* lse,
                       const Cap& cap, cudaStream_t stream) {
    if (cu_q[n_seqs] == 0) return SP_OK;
    const sp_status checked = check_tiles(c, layer, seq_ids, n_seqs, cu_q);
    if (checked != SP_OK) return checked;
    const int H = c->cfg.num_kv_heads, units = n_seqs * H;
    if (!c->geo.fp4)
        return prefill_units(c, layer, seq_ids, n_seqs, cu_q, q, k, v, out, lse, cap, 0, units, true, true, stream);
    // 4-bit pages: the units' history becomes bf16 rows in the workspace, as
    // many units at a time as fit, and the bf16 kernel reads those
    // (sp_dequant.cu says why).
    std::unique_ptr<DequantParams> dp(new DequantParams());
    dp->meta = c->meta;
    dp->geo = c->geo;
    dp->layer = layer;
    dp->scaled = c->h_scaled[layer];
    dp->kpool = reinterpret_cast<const uint8_t*>(c->kpool);
    dp->vpool = reinterpret_cast<const uint8_t*>(c->vpool);
    dp->k = c->ws.deq_k;
    dp->v = c->ws.deq_v;
    dp->row0 = c->ws.deq_row;
    std::copy(seq_ids, seq_ids + n_seqs, dp->seq);
    launch_mark_start(c, stream);
    for (int u0 = 0; u0 < units;) {
        int64_t pages = 0;
        int u1 = u0;
        dp->unit0 = u0;
        dp->page_off[0] = 0;
        for (; u1 < units; ++u1) {
            const int b = u1 / H;
            const int64_t n = cu_q[b + 1] > cu_q[b]
                                  ? c->h_npages[((size_t)seq_ids[b] * c->cfg.num_layers + layer) * H + u1 % H] : 0;
            if (pages + n > c->ws.deq_pages) break;   // (one unit always fits)
            pages += n;
            dp->page_off[u1 - u0 + 1] = (int32_t)pages;
        }
        dp->n_units = u1 - u0;
        const cudaError_t e = launch_dequant4(c, *dp, stream);
        if (e != cudaSuccess) return cuda_fail(e, "history conversion launch");
        const sp_status s = prefill_units(c, layer, seq_ids, n_seqs, cu_q, q, k, v, out, lse, cap, u0, u1, u0 == 0,
                                          u1 == units, stream);
        if (s != SP_OK) return s;
        u0 = u1;
    }
    return SP_OK;
}

cudaError_t launch_prefill_counts(const sp_cache* c, int seq, int layer, int h,
                                  const int64_t* pos, int n, int32_t* out, cudaStream_t s) {
    k_prefill_counts<<<(n + 127) / 128, 128, 0, s>>>(c->meta, c->geo, seq, layer, h, pos, n, out);
    return cudaGetLastError();
}

}  // namespace sp
