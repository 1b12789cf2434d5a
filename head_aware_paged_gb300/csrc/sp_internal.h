// sp_internal.h -- handle, device-memory layout and launcher declarations
// shared by the host API (sp_api.cu) and the kernel files.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include <string>
#include <vector>

#include "segpaged.h"
#include "sp_fp4.cuh"
#include "sp_rules.h"

namespace sp {

constexpr int kMaxCallSeqs = 512;     // sequences in one call (kernel parameters)
constexpr int kMaxDecodeUnits = 4096; // (sequence, KV head) units in one decode call
constexpr int kMaxPolicyUnits = 8192; // layers * kv heads

// Device pointers into the caller's meta buffer.
struct Meta {
    UnitPol* pol;        // [max_seqs][layers][hkv]
    int32_t* npages;     // [max_seqs][layers][hkv]
    int32_t* seqlen;     // [max_seqs][layers]
    int32_t* ptab;       // [max_seqs][layers][hkv][max_pages_unit]
    int32_t* idx;        // [max_seqs][max_idx_per_seq]
    int32_t* fstack;     // [num_pages] free-page stack
    int32_t* status;     // [8]: 0 = status word, 1 = stack top (debug mirror)
    float* kscale;       // FP8 pages: [layers][hkv][d] per-channel scales of K
    float* vscale;       //            ... of V
    float* kinv;         //            fp32 reciprocals used to quantise
    float* vinv;
};

// Geometry every kernel needs.
struct Geo {
    int32_t layers, hq, hkv, group, d, page, max_seqs, max_pages_unit,
            max_idx_per_seq, num_pages;
    int32_t fp8;         // pages hold e4m3 codes (1 byte) instead of bf16
    int32_t fp4;         // pages hold e2m1 codes and block scales (sp_fp4.cuh)
    // bytes of one stored K or V row
    __host__ __device__ int32_t row_bytes() const { return fp4 ? kFp4RowBytes : d * (fp8 ? 1 : 2); }
    __host__ __device__ int64_t unit_row(int seq, int layer, int h) const {
        return ((int64_t)seq * layers + layer) * hkv + h;
    }
};

// Per-call list of sequences (kernel parameter).
struct CallSeqs {
    int32_t n;
    int32_t seq[kMaxCallSeqs];   // sequence slot
    int32_t n_old[kMaxCallSeqs]; // tokens held before the call
    int32_t cnt[kMaxCallSeqs];   // new tokens / query rows
    int32_t row0[kMaxCallSeqs];  // first row in the call's packed tensors
};

// Scores capped by a tanh, s' = cap * tanh(s / cap), in log2 units of the raw
// product x = q . k:  tanh(y) = 1 - 2 / (1 + e^2y), so
//     s' log2(e) = a - b / (1 + 2^(k1 x)),
// a = cap log2(e), b = 2 a, k1 = 2 log2(e) / (cap sqrt(d)).  2^(k1 x) may
// overflow to infinity or underflow to 0: the quotient is then 0 or b, the
// limits of tanh.
struct Cap {
    int32_t on;
    float k1, a, b;
    // prefill: the exponentials' fixed reference; a tanh(y) as odd polynomials
    // of the raw product x, of 2, 3 and 4 terms for |x| <= limit[0 .. 2]
    float ref, limit[3], poly[3][4];
};
Cap make_cap(float score_cap, int head_dim);
constexpr float kMinScoreCap = 1.f / 64.f, kMaxScoreCap = 64.f;

// Slots of one decode work item: a page, or for 4-bit pages a run of 64 slots
// whatever the page size.
constexpr int kFp4ItemSlots = 64;
inline int decode_item_slots(const Geo& g) { return g.fp4 ? kFp4ItemSlots : g.page; }

struct DecodeParams {
    Meta meta;
    Geo geo;
    int32_t layer;
    int32_t n_seqs;
    int32_t n_units;             // n_seqs * hkv
    int64_t total_items;         // pages streamed, all units
    int32_t seq[kMaxCallSeqs];
    int32_t tq[kMaxCallSeqs];    // query position per sequence
    int32_t item_off[kMaxDecodeUnits + 1];
    const __nv_bfloat16* q;
    __nv_bfloat16* out;
    float* lse;
    float* part_o;               // [(n_units + grid)][group][d]
    float* part_ml;              // [(n_units + grid)][group][2]
    int32_t* counters;           // [n_units], zero between calls
    float scale_log2;            // log2(e) / sqrt(d)
    Cap cap;                     // capped scores (cap.on = 0: as they are)
    int32_t scaled;              // 4-bit pages: channel scales other than 1 may be set
    int32_t per, rem;            // 4-bit pages: items of a CTA, CTAs that take one more (launcher)
    // Pages chosen for the call (null: none): unit u's GLOBAL head reads the physical
    // pages kept[u * max_pages_unit ..], at most kept_cap, as if they were all.
    const int32_t* kept;
    int32_t kept_cap;
    int32_t nst;                 // pipeline stages (set by the launcher)
    int32_t owners;              // consumer warps that own stages (divides nst)
    int32_t merge_floats;        // merge buffer floats (set by the launcher)
};

// RoPE realignment of stored K rows (sp_rope.cu), one launch per call.
constexpr int kMaxRopeUnits = 2048;   // (sequence, KV head) units in one rope launch
struct RopeParams {
    Meta meta;
    Geo geo;
    int32_t layer;
    int32_t n_units;
    int64_t pos_lo, pos_hi;       // rotate rows whose position is in [pos_lo, pos_hi)
    float cs[64], sn[64];         // cos / sin of delta * theta^(-2i/d), i < d/2
    int32_t unit_seq[kMaxRopeUnits];
    int16_t unit_head[kMaxRopeUnits];
    int32_t unit_n[kMaxRopeUnits];         // tokens the unit's (sequence, layer) holds
    int32_t page_off[kMaxRopeUnits + 1];   // prefix of the units' page counts
};

// Packed-sequence layout (sp_pack_seq / sp_unpack_seq).  The buffer starts
// with PackHeader, then int64 n[layers] (tokens per layer), then
// PackUnit[layers * hkv] in (layer, KV head) order, then the int32 retrieval
// indices of every unit in the same order, then (at payload_off, 256-byte
// aligned) the payload: for each unit its retained K rows then its V rows,
// [rows][head_dim] elements of the page type (bf16, or e4m3 bytes), in
// position order.
constexpr int64_t kPackMagic = 0x3156504B50535053LL;   // "SPSPKPV1" little-endian
constexpr int kTransferRows = 32;                        // rows per copy block
struct PackHeader {
    int64_t magic, version, layers, hkv, head_dim, page_size, n_units, idx_total,
            payload_off, payload_bytes, total_bytes, kv_dtype;
};
struct PackUnit {
    int64_t kind, sink, window, n_idx, rows, row_off, blk_off;
};
struct TransferParams {
    Meta meta;
    Geo geo;
    int32_t seq;
    int32_t unpack;               // 0: pool -> payload, 1: payload -> pool
    int32_t n_units;
    int64_t total_blocks;
    const int64_t* n_layer;       // device: tokens per layer (in the packed buffer)
    const PackUnit* units;        // device: per-unit layout (in the packed buffer)
    uint8_t* payload;             // device
};

struct Workspace {
    void* base;
    size_t bytes;
    // regions
    int4* tiles;          int64_t max_tiles;
    int32_t* tile_ctr;
    float* part_o;        float* part_ml;  int64_t max_parts;
    int32_t* counters;    int64_t max_counter_units;
    float* split_o;       float* split_ml;        // prefill pieces of split items
    int32_t* scratch;     int64_t scratch_ints;   // export / visible-count staging
    // 4-bit pages: a prefill's history as bf16 rows (deq_pages pages of them),
    // and each unit's first row
    __nv_bfloat16* deq_k; __nv_bfloat16* deq_v;  int64_t deq_pages;
    int32_t* deq_row;
};

// Page bounds (sp_bounds.cuh) and the scratch of the choice of pages, in the
// buffer of sp_attach_page_bounds; codes is null while there is none.
struct PageBounds {
    int8_t* codes = nullptr;        // [num_pages][upper, lower][d]
    float* step = nullptr;          // [num_pages]
    uint32_t* score = nullptr;      // [max_batch][hkv][max_pages_unit] order-preserving keys
    int32_t* kept = nullptr;        // the same: physical pages kept, in order
    int32_t* tickets = nullptr;     // [max_batch][hkv], zero between calls
};

}  // namespace sp

struct sp_cache {
    sp_config cfg;
    sp::Geo geo;
    int device = 0;
    int num_sms = 0;
    int decode_ctas = 0;
    __nv_bfloat16* kpool = nullptr;
    __nv_bfloat16* vpool = nullptr;
    sp::Meta meta;
    sp::Workspace ws;
    sp::PageBounds bounds;
    CUtensorMap tm_kpool;   // [num_pages*P rows][d], box {64 or d, P}, 128B swizzle
    CUtensorMap tm_vpool;
    CUtensorMap tm_kpool_half;   // FP8 pages of P >= 64: the same with box {d, P / 2}
    CUtensorMap tm_vpool_half;   // (the decode streams such pages in halves)
    // host mirror (authoritative for lengths, page counts and policies)
    std::vector<sp::UnitPol> h_pol;              // [max_seqs][layers][hkv]
    std::vector<std::vector<int32_t>> h_idx;     // per sequence, CSR by unit
    std::vector<uint8_t> h_policy_set;           // per sequence
    std::vector<int32_t> h_seqlen;               // [max_seqs][layers]
    std::vector<int32_t> h_npages;               // [max_seqs][layers][hkv]
    std::vector<uint8_t> h_scaled;               // [layers]: sp_set_kv_scales was called
    int64_t h_free = 0;
    // Pinned host staging for the per-call prefill work list, so its upload is
    // an asynchronous copy and the host never waits for the device.  A ring:
    // a buffer is refilled only after the copy that last read it has run.
    static constexpr int kStaging = 4;
    int4* stage_buf[kStaging] = {};
    const int4* stage_dev[kStaging] = {};        // the same buffers as device addresses (mapped)
    cudaEvent_t stage_ev[kStaging] = {};
    size_t stage_bytes = 0;                       // size of each buffer
    int stage_next = 0;
    // [capped ? 5 : 0 + (speculative ? 4 : two issuers ? 3 : FP8 ? 2 : D == 128)][log2(P) - 4, or 0]: attributes set
    bool prefill_checked[10][5] = {};
    // Caller's event pair armed by sp_set_launch_events for the next
    // attention call (both null when not armed).
    cudaEvent_t launch_ev[2] = {};
    ~sp_cache();
};

namespace sp {

// Pinned staging ring (sp_api.cu): stage_acquire returns the next buffer once
// the copy that last read it has run (nullptr if `bytes` does not fit);
// stage_copy issues its asynchronous upload to `dst` and records its event.
void* stage_acquire(sp_cache* c, size_t bytes, int* slot);
cudaError_t stage_copy(sp_cache* c, int slot, void* dst, size_t bytes, cudaStream_t s);

// Argument checks shared by the entry points (sp_api.cu); they allocate
// nothing.  check_seq_list: 1..max_batch ids, each in range, with a policy,
// none listed twice.
bool valid_layer(const sp_cache* c, int32_t layer);
bool valid_cap(float score_cap);
int32_t max_unit_pages(const sp_config* c);      // entries of a unit's page table
sp_status check_seq_list(const sp_cache* c, const int32_t* seq_ids, int32_t n_seqs);

// Armed launch events (sp_set_launch_events): the start is recorded right
// before an attention call's first kernel, the end right after its last,
// which also disarms the pair.
inline void launch_mark_start(sp_cache* c, cudaStream_t s) {
    if (c->launch_ev[0]) cudaEventRecord(c->launch_ev[0], s);
}
inline void launch_mark_end(sp_cache* c, cudaStream_t s) {
    if (c->launch_ev[1]) cudaEventRecord(c->launch_ev[1], s);
    c->launch_ev[0] = c->launch_ev[1] = nullptr;
}

// Error plumbing (sp_api.cu).
sp_status fail(sp_status s, const std::string& msg);
sp_status cuda_fail(cudaError_t e, const char* what);
// SP_ERR_INVALID_ARG unless the cache's device is the current one.
sp_status check_device(const sp_cache* c);
// Runs a C entry point's body: no C++ exception (host memory) leaves it.
template <typename F>
sp_status no_throw(F&& body) {
    try {
        return body();
    } catch (...) {
        return fail(SP_ERR_UNSUPPORTED, "no host memory");
    }
}
bool encode_tmap_2d(CUtensorMap* map, const void* base, uint64_t inner, uint64_t rows,
                    uint64_t row_bytes, uint32_t box_inner, uint32_t box_rows,
                    bool swizzle128, std::string* err, bool bytes = false);

// Launchers (return the launch's cudaError_t).
cudaError_t launch_init_meta(const sp_cache* c, cudaStream_t s);
cudaError_t launch_alloc(const sp_cache* c, const CallSeqs& cs, int layer, int32_t top,
                         cudaStream_t s);
cudaError_t launch_scatter(const sp_cache* c, const CallSeqs& cs, int layer,
                           const __nv_bfloat16* k, const __nv_bfloat16* v,
                           int64_t row_stride, int64_t max_items, cudaStream_t s);
cudaError_t launch_release(const sp_cache* c, int seq, int32_t top, cudaStream_t s);
cudaError_t launch_export(const sp_cache* c, int seq, int layer, int h, int32_t* out_ids,
                          int32_t* out_pos, cudaStream_t s);
cudaError_t launch_decode_counts(const sp_cache* c, int seq, int layer, int h,
                                 const int64_t* pos, int n, int32_t* out, cudaStream_t s);
cudaError_t launch_decode(const sp_cache* c, DecodeParams& p, cudaStream_t s);
// Instances for capped scores (sp_decode_capped.cu) and for 4-bit pages
// (sp_decode4.cu, sp_decode4_capped.cu); launch_decode chooses.
cudaError_t launch_decode_capped(const sp_cache* c, DecodeParams& p, int grid, cudaStream_t s);
cudaError_t launch_decode4(const sp_cache* c, DecodeParams& p, int grid, cudaStream_t s);
cudaError_t launch_decode4_capped(const sp_cache* c, DecodeParams& p, int grid, cudaStream_t s);
// One prefill's units whose 4-bit pages become bf16 pages in the workspace
// (sp_dequant.cu): unit (b, h) of the call takes the workspace pages from
// page_off[b * hkv + h - unit0] on.
struct DequantParams {
    Meta meta;
    Geo geo;
    int32_t layer, unit0, n_units;
    int32_t scaled;              // channel scales other than 1 may be set
    const uint8_t *kpool, *vpool;
    __nv_bfloat16 *k, *v;
    int32_t* row0;               // [max_batch][hkv] first row of a unit's copies
    int32_t seq[kMaxCallSeqs];
    int32_t page_off[kMaxDecodeUnits + 1];
};
cudaError_t launch_dequant4(const sp_cache* c, const DequantParams& p, cudaStream_t s);
cudaError_t launch_rope(const sp_cache* c, const RopeParams& p, cudaStream_t s);
// The choice of a decode's pages (sp_choose.cu).
struct ChooseParams {
    Meta meta;
    Geo geo;
    int32_t layer, n_seqs;
    int32_t first, newest, top, cap;   // pages always kept, chosen ones; cap is their sum
    int32_t chunk;                     // candidates of a block (launcher)
    const __nv_bfloat16* q;
    const int8_t* codes;
    const float* step;
    uint32_t* score;
    int32_t* kept;
    int32_t* tickets;
    int32_t* pages;                    // [n_seqs][hkv][cap] page numbers, or null
    int32_t seq[kMaxCallSeqs], n[kMaxCallSeqs];
};
cudaError_t launch_choose(const sp_cache* c, ChooseParams& p, cudaStream_t s);
// A decode over chosen pages in one launch (sp_kept.cuh): units of at most kKeptPages
// kept pages out of kKeptCandidates.
constexpr int kKeptPages = 2048, kKeptCandidates = 4096;
struct KeptParams {
    Meta meta;
    Geo geo;
    int32_t layer, n_seqs;
    int32_t first, newest, top, cap;   // pages always kept, chosen ones; cap is their sum
    int32_t scaled;                    // channel scales other than 1 may be set
    int32_t log_ranks;                 // blocks a unit (launcher)
    const __nv_bfloat16* q;
    __nv_bfloat16* out;
    float* lse;
    int32_t* pages;                    // [n_seqs][hkv][cap] page numbers, or null
    const int8_t* codes;
    const float* step;
    const uint8_t *kpool, *vpool;
    float scale_log2;                  // log2(e) / sqrt(d)
    Cap score_cap;
    int32_t seq[kMaxCallSeqs], n[kMaxCallSeqs];
};
// What the call's units have to do: groups of 16 slots that they read (about), and
// for a small call (n units, else n = 0) those of each and whether its pages are
// chosen.
constexpr int kKeptLoads = 16;
struct KeptLoad {
    int64_t total, longest;
    int32_t n;
    int32_t groups[kKeptLoads];
    bool chosen[kKeptLoads];
};
// bf16 pages (sp_kept.cu, sp_kept_capped.cu), FP8 and 4-bit pages (sp_kept_coded.cu,
// sp_kept_coded_capped.cu).  `serves` is cleared, and nothing launched, where a
// choice in a launch of its own is the better way.
cudaError_t launch_kept_bf16_plain(KeptParams& p, const KeptLoad& load, bool& serves, cudaStream_t s);
cudaError_t launch_kept_bf16_capped(KeptParams& p, const KeptLoad& load, bool& serves, cudaStream_t s);
cudaError_t launch_kept_coded_plain(KeptParams& p, const KeptLoad& load, bool& serves, cudaStream_t s);
cudaError_t launch_kept_coded_capped(KeptParams& p, const KeptLoad& load, bool& serves, cudaStream_t s);
inline cudaError_t launch_kept(KeptParams& p, const KeptLoad& load, bool& serves, cudaStream_t s) {
    if (p.geo.fp8 || p.geo.fp4)
        return p.score_cap.on ? launch_kept_coded_capped(p, load, serves, s) : launch_kept_coded_plain(p, load, serves, s);
    return p.score_cap.on ? launch_kept_bf16_capped(p, load, serves, s) : launch_kept_bf16_plain(p, load, serves, s);
}
// Bounds of the pages that a write of positions [lo[b], hi[b]) of sequence seqs[b]
// touched, where the cache has them (sp_bounds.cu); the lengths are those after
// the write.
sp_status update_bounds(const sp_cache* c, int32_t layer, const int32_t* seqs, int32_t n_seqs,
                        const int64_t* lo, const int64_t* hi, cudaStream_t stream);
cudaError_t launch_transfer(const sp_cache* c, const TransferParams& p, cudaStream_t s);

}  // namespace sp
