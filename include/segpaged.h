/*
 * segpaged.h -- C ABI of libsegpaged.so, a head-aware paged KV cache with
 * mask-free attention for one GB300 GPU (sm_103a).
 *
 * Method: RedKnot SegPagedAttention, as described in the runtime article
 * "How different attention heads see different context" (section 1: why heads
 * may see different context; section 2: the per-(layer, KV head) head
 * classes; section 3: per-head page tables over one physical page pool, local
 * heads trimmed at KV-write time; section 4: one mask-free fused varlen
 * attention over every (query head, KV head) pair's own visible tokens; section
 * 5: the page layout must be built at write time and reused, never rebuilt per
 * attention call) and in the RedKnot news summary (head-class sparsification:
 * globals about 12-15 % of heads; the BUILDSTATE / SELECTVISIBLESTATE /
 * EXECUTE split of the runtime).
 *
 * Conventions for every call
 *   - Every function returns an sp_status; nothing else crosses the ABI.  On
 *     any status other than SP_OK, sp_last_error() holds a one-line message
 *     (thread-local) and, for argument or capacity errors, nothing was
 *     modified and nothing was launched.
 *   - Device memory belongs to the caller.  The library never allocates
 *     device memory: the caller allocates the pool, metadata and workspace
 *     buffers sized by sp_required_bytes() and keeps them alive until
 *     sp_cache_destroy().  Tensor arguments are borrowed until the
 *     stream-ordered work of the call has completed.
 *   - `stream` is a cudaStream_t (0 = legacy default stream).  Calls are
 *     asynchronous unless marked "synchronous".  All calls that touch one
 *     cache must be issued in stream order (one stream, or with events).
 *   - One cache handle must not be used from two host threads at once.
 *   - A call that launches work on a cache wants the cache's device (the
 *     current one at its creation) to be current (SP_ERR_INVALID_ARG otherwise).
 *   - A call captured into a CUDA graph takes its lists, lengths, policies and
 *     whether channel scales were set from the moment of its capture; sequences
 *     that it names must not be released between then and its last replay
 *     (sp_append_kv_rope says what a replayed write does otherwise).
 *   - Tensors are bf16 (2-byte elements), row-major and contiguous unless a
 *     stride is given:  q / out [tokens][num_q_heads][head_dim];
 *     k / v [tokens][num_kv_heads][head_dim]; lse [tokens][num_q_heads] fp32
 *     (natural logarithm of the softmax denominator incl. the max shift;
 *     -inf for a query with no visible token, whose output row is 0).
 *   - Query head h belongs to KV head h / (num_q_heads / num_kv_heads)
 *     (grouped-query attention, KV-cache tutorial section 5.3, 0-indexed).
 *   - Per call order for one layer and chunk: sp_attention_prefill (history
 *     pages + the chunk itself) then sp_append_kv (the chunk); for decode:
 *     sp_append_kv (the new token) then sp_attention_decode.
 */
#ifndef SEGPAGED_H
#define SEGPAGED_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum sp_status {
    SP_OK = 0,
    SP_ERR_INVALID_ARG = 1,    /* bad argument; nothing modified            */
    SP_ERR_OUT_OF_PAGES = 2,   /* pool too small for this call; nothing modified */
    SP_ERR_UNSUPPORTED = 3,    /* shape or size this build does not handle  */
    SP_ERR_CUDA = 4,           /* a CUDA runtime/driver call failed          */
    SP_ERR_DEVICE_STATUS = 5,  /* a kernel flagged an impossible state       */
    SP_ERR_TIMEOUT = 6         /* a bounded device wait gave up              */
} sp_status;

/* Head classes (runtime article section 2).  DENSE attends like GLOBAL; its
 * difference (full re-prefill on reuse) lies outside attention. */
typedef enum sp_kind { SP_GLOBAL = 0, SP_LOCAL = 1, SP_RETRIEVAL = 2 } sp_kind;

/* One (layer, KV head) policy.
 *   GLOBAL:        query i sees positions 0..i.
 *   LOCAL:         query i sees [0, min(sink, i+1)) and [max(0, i-window+1), i];
 *                  sink >= 0, window >= 1.
 *   RETRIEVAL:     query i sees idx[k] <= i; idx strictly ascending, >= 0,
 *                  n_idx >= 0; idx is a host pointer read during the call. */
typedef struct sp_head_policy {
    int32_t kind;
    int32_t sink;
    int32_t window;
    int32_t n_idx;
    const int32_t* idx;
} sp_head_policy;

typedef struct sp_config {
    int32_t num_layers;
    int32_t num_q_heads;
    int32_t num_kv_heads;      /* num_q_heads % num_kv_heads == 0, group <= 16 */
    int32_t head_dim;          /* 64 or 128 */
    int32_t page_size;         /* tokens per page: 16, 32, 64 or 128 */
    int32_t max_seqs;          /* sequence slots 0 .. max_seqs-1 */
    int32_t max_seq_len;       /* longest context a sequence may reach */
    int32_t num_pages;         /* physical pages in the pool (all units share it) */
    int32_t max_idx_per_seq;   /* RETRIEVAL index capacity per sequence (all its units) */
    int32_t max_tokens;        /* most query rows in one prefill / append call */
    int32_t max_batch;         /* most sequences in one call */
    int32_t kv_dtype;          /* sp_kv_dtype of the pages (0 = bf16) */
} sp_config;

/* Element type of the K/V pages.  SP_KV_FP8_E4M3 stores one byte per element
 * (the KV-cache tutorial's quantisation section: FP8 halves the KV cache,
 * per-channel scales keep outlier channels from dominating the range): code =
 * e4m3(x * inv_scale), rounded to nearest even and saturated at +-448, with a
 * scale per (layer, KV head, dimension) for K and for V set by
 * sp_set_kv_scales (1.0 until set); the stored value is code * scale.
 * FP8 pages need head_dim 128.  Decode and prefill read them: decode with
 * f16 MMAs (see sp_set_kv_scales), prefill by turning each history tile into
 * bf16(code * scale) rows in shared memory before its bf16 MMAs (a chunk's
 * own rows enter its attention as the caller's bf16 values).
 * sp_rope_realign on FP8 pages dequantises each key with its channel
 * scales, rotates in fp32 (every product and sum rounded once) and writes
 * the codes again as a write would.
 *
 * SP_KV_FP4_E2M1 stores 72 bytes a row instead of 256 (head_dim 128 only):
 * every 16 neighbouring dimensions share one scale, an unsigned float of 5
 * exponent and 3 mantissa bits (0, 2^-17 .. 10240), the value nearest
 * amax / 6; an element is the e2m1 value (0, .5, 1, 1.5, 2, 3, 4, 6, signed)
 * nearest x / scale.  Both round to nearest, ties to even, and saturate; an
 * element that is NaN is stored as 6 * scale and does not count in amax.  The
 * channel scales of sp_set_kv_scales (1.0 until set) apply first, as for FP8:
 * x * (1 / channel scale) is what the block quantises, and the stored value is
 * code * scale * channel scale.  Every call that takes a cache takes such a
 * one: decode multiplies code * scale (exact in f16) with q * channel scale
 * in f16 (times a power of two per head that keeps it in range), prefill reads bf16(code * scale * channel scale) from copies that it
 * makes in the workspace, sp_rope_realign
 * dequantises, rotates and quantises again with new block scales, and a packed
 * row is its 64 code bytes (two dimensions a byte, the even one low), then its
 * 8 scales. */
typedef enum { SP_KV_BF16 = 0, SP_KV_FP8_E4M3 = 1, SP_KV_FP4_E2M1 = 4 } sp_kv_dtype;

typedef struct sp_cache sp_cache;  /* opaque host handle */

/* Bytes of the three caller-owned device buffers for cfg (host only, no GPU).
 *   pool: K pages then V pages, each [num_pages][page_size][head_dim] elements
 *         of kv_dtype (bf16, or one byte for FP8); FP4: [num_pages]
 *         [page_size / 16][1152] bytes, 16 rows' codes and their scales.
 *   meta: page tables, policies, retrieval lists, free-page stack, status.
 *   ws:   per-call scratch (prefill work list, decode split partials; FP4:
 *         also bf16 copies of a prefill's history: what max_batch sequences of
 *         max_seq_len hold in one layer, the whole pool's rows or 2 GiB,
 *         whichever is least, and at least one unit's). */
sp_status sp_required_bytes(const sp_config* cfg, size_t* pool_bytes,
                            size_t* meta_bytes, size_t* ws_bytes);

/* Create a handle over caller-owned buffers (each 1024-byte aligned, at least
 * the sizes above, on the current CUDA device).  Initialises meta (all units
 * empty, every page free) and waits for that to finish: synchronous.  The
 * handle owns a few small pinned HOST buffers (4 x the prefill work list, at
 * most a few MB) so that sp_attention_prefill uploads its work list without
 * blocking the host; sp_cache_destroy waits for their last copies and frees
 * them.  No device memory is allocated. */
sp_status sp_cache_create(const sp_config* cfg, void* pool, void* meta, void* ws,
                          sp_cache** out);

/* Free the host handle only; the caller frees its device buffers. */
sp_status sp_cache_destroy(sp_cache* cache);

/* BUILDSTATE, step 1 (runtime article section 2): set the policy of every
 * (layer, KV head) of sequence `seq`; p has num_layers * num_kv_heads entries,
 * layer-major.  The sequence must hold no tokens (fresh or released).  Copies
 * the retrieval lists to the device on `stream`. */
sp_status sp_set_policy(sp_cache* cache, int32_t seq, const sp_head_policy* p,
                        void* stream);

/* BUILDSTATE, step 2 (runtime article section 3, build from dense K/V, trimming
 * local heads to their visible tokens): write positions 0 .. n_tokens-1 of
 * (seq, layer) from dense k, v laid out [n_tokens][num_kv_heads][head_dim]
 * with `row_stride` elements between consecutive tokens (>= kv_heads*head_dim,
 * multiple of 8).  The (seq, layer) must be empty.  Pages are allocated in
 * this call; only retained rows are copied. */
sp_status sp_build_cache(sp_cache* cache, int32_t seq, int32_t layer,
                         const void* k, const void* v, int64_t n_tokens,
                         int64_t row_stride, void* stream);

/* Append cu_new[b+1] - cu_new[b] new tokens to (seq_ids[b], layer) for
 * b < n_seqs; k, v [cu_new[n_seqs]][num_kv_heads][head_dim] contiguous.
 * GLOBAL heads store every token, LOCAL heads write sink slots or overwrite the
 * oldest ring slot, RETRIEVAL heads store only listed positions.  seq_ids and
 * cu_new are host arrays; sequences must be distinct. */
sp_status sp_append_kv(sp_cache* cache, int32_t layer, const int32_t* seq_ids,
                       int32_t n_seqs, const int32_t* cu_new, const void* k,
                       const void* v, void* stream);

/* Append with the rotary embedding applied on the way: new queries and keys
 * arrive unrotated, as a fused projection leaves them.  For the c_b =
 * cu_new[b+1] - cu_new[b] tokens of sequence seq_ids[b], whose positions are
 * pos[b], pos[b] + 1, ...:
 *   - q_out[row] = q[row] rotated to its position (bf16);
 *   - k[row] rotated and v[row] go into the pages as sp_append_kv would write
 *     them (the rotated key enters the page type with one rounding: no bf16
 *     in between for FP8 and FP4 pages).
 * The rotation is that of sp_rope_realign with delta = position: pair
 * (i, i + head_dim/2) turns by position * w_i, w_i = rope_theta^(-2i/head_dim),
 * or inv_freq[i] where inv_freq (host, [head_dim / 2], |w| <= 2^16) is given
 * (rope_theta is then not read).  Frequencies are double, angles are reduced
 * in 64-bit fixed point, cos, sin and the rotation are fp32.
 *   pos: host array of first positions, 0 <= pos[b] <= tokens held, or null =
 *     append at the end.  Positions below what the sequence holds are
 *     overwritten in place wherever the head keeps them (recomputed tokens of
 *     a reused segment), the rest is appended; no token is dropped, and the
 *     length becomes max(held, pos[b] + c_b).
 *   q [cu_new[n_seqs]] rows of num_q_heads * head_dim elements q_stride apart,
 *     k and v likewise with num_kv_heads (strides in elements, multiples of 8,
 *     at least a row); all 16-byte aligned.  q and q_out may both be null: keys
 *     and values only.  q_out is contiguous; it may be q itself if q is, and
 *     overlaps the inputs in no other way.
 * A prompt chunk attends before it is stored (sp_attention_prefill wants its
 * keys rotated already); afterwards this call stores the unrotated rows, q null.
 * One launch, pages included; works for every page type and head class.
 * Captured into a graph: a call that needs new pages is refused
 * (SP_ERR_UNSUPPORTED; replays would take them from the free stack again).
 * Another counts once, when it is captured, and keeps its positions and whether
 * channel scales were set.  A replay writes them again wherever the head still
 * keeps them, whatever else was appended or released in between, and no length
 * shrinks; while a listed sequence holds fewer tokens than at the capture
 * (released), nothing of it is written and the status word is set. */
sp_status sp_append_kv_rope(sp_cache* cache, int32_t layer, const int32_t* seq_ids,
                            int32_t n_seqs, const int32_t* cu_new, const int64_t* pos,
                            const void* q, int64_t q_stride, const void* k,
                            int64_t k_stride, const void* v, int64_t v_stride,
                            void* q_out, double rope_theta, const double* inv_freq,
                            void* stream);

/* The same with angles of positions on several axes (time, height and width of a
 * video's patches, for one): pair (i, i + head_dim/2) turns by P(axis_of[i], row) *
 * w_i, w_i as above.  Where the tokens are stored (pos) and where they stand for
 * the rotation are then two things: pos still counts tokens.
 *   axis_pos: DEVICE array of int64 positions, element (axis, row) at axis *
 *     axis_stride + row * row_stride (strides in elements, >= 0; 8-byte aligned;
 *     rows are those of q, k and v).  Any int64 is a position: p * w is reduced
 *     modulo a turn in 64-bit fixed point, off by |p| (2^-65 + |w| 2^-53) turns at
 *     most (inv_freq: 2^-55 for 2^-53), and the angle is rounded to 2^-32 turns.
 *   n_axes: 1 .. 4; axis_of: host array [head_dim / 2] of axes in [0, n_axes).
 * q_out may not overlap the positions.  A call captured into a graph reads the
 * positions when it is replayed. */
sp_status sp_append_kv_rope_axes(sp_cache* cache, int32_t layer, const int32_t* seq_ids,
                                 int32_t n_seqs, const int32_t* cu_new, const int64_t* pos,
                                 const void* q, int64_t q_stride, const void* k,
                                 int64_t k_stride, const void* v, int64_t v_stride,
                                 void* q_out, const int64_t* axis_pos, int64_t axis_stride,
                                 int64_t row_stride, int32_t n_axes, const int32_t* axis_of,
                                 double rope_theta, const double* inv_freq, void* stream);

/* The rotation alone, rows to rows: q_out and k_out get q and k rotated to their
 * positions on the axes (as in sp_append_kv_rope_axes, the same roundings).  No cache
 * is involved: a prompt's chunk is rotated by this call, attends
 * (sp_attention_prefill) and is stored (sp_append_kv).  q [rows] of num_q_heads *
 * head_dim elements q_stride apart, k likewise (strides in elements, multiples of
 * 8, at least a row); q_out and k_out contiguous; all 16-byte aligned.  A side with
 * 0 heads is left out.  An output may be its own input if that is contiguous and
 * overlaps nothing else.  head_dim 64 or 128 (SP_ERR_UNSUPPORTED otherwise), at
 * most 1024 heads a side, rows below 2^31.  Runs on the current device. */
sp_status sp_rope_axes(const void* q, int64_t q_stride, int32_t num_q_heads, const void* k,
                       int64_t k_stride, int32_t num_kv_heads, int32_t head_dim, int64_t rows,
                       const int64_t* axis_pos, int64_t axis_stride, int64_t row_stride,
                       int32_t n_axes, const int32_t* axis_of, double rope_theta,
                       const double* inv_freq, void* q_out, void* k_out, void* stream);

/* EXECUTE, prefill (runtime article section 4): causal attention of a chunk.
 * Rows cu_q[b] .. cu_q[b+1]-1 of q belong to sequence seq_ids[b] and sit at
 * absolute positions n_b .. n_b + c_b - 1, where n_b is what (seq, layer)
 * already holds; keys below n_b come from the cache pages, the rest from the
 * chunk's own k, v (same row layout as q's rows, num_kv_heads heads).  Each
 * query head attends over exactly its KV head's visible set; no mask tensor.
 * out [cu_q[n_seqs]][num_q_heads][head_dim] bf16; lse nullable.  q, k and v
 * must be 16-byte aligned and out 32-byte aligned (SP_ERR_INVALID_ARG
 * otherwise).  Does not modify the cache: call sp_append_kv with the same
 * k, v afterwards. */
sp_status sp_attention_prefill(sp_cache* cache, int32_t layer,
                               const int32_t* seq_ids, int32_t n_seqs,
                               const int32_t* cu_q, const void* q,
                               const void* k, const void* v, void* out,
                               float* lse, void* stream);

/* EXECUTE, decode: one query per sequence at position t = n - 1, where n is
 * what (seq_ids[b], layer) holds (its own token was appended first).
 * q, out [n_seqs][num_q_heads][head_dim]; lse [n_seqs][num_q_heads] nullable.
 * Split-KV: the visible pages of all units are streamed by persistent CTAs;
 * partial results are merged in the same launch. */
sp_status sp_attention_decode(sp_cache* cache, int32_t layer,
                              const int32_t* seq_ids, int32_t n_seqs,
                              const void* q, void* out, float* lse, void* stream);

/* The two attention calls with scores capped by a tanh: the softmax is taken
 * of score_cap * tanh(s / score_cap), s = q . k / sqrt(head_dim), over each
 * head's visible keys.  score_cap in [1/64, 64] (SP_ERR_INVALID_ARG
 * otherwise); everything else is as for sp_attention_prefill and
 * sp_attention_decode (lse is that of the capped scores).  Prefill's sums are
 * exact to fp32 for values of 2^-28 <= |v| <= 2^20 at every cap (a row whose
 * scores all lie near -64 weighs smaller ones in fp32's subnormals).  In all four calls a
 * key that a row does not see, and a row of another sequence, may enter its
 * sums with the weight 0: k and v must be finite (a NaN in q stays in its row,
 * whose output and lse are NaN). */
sp_status sp_attention_prefill_capped(sp_cache* cache, int32_t layer,
                                      const int32_t* seq_ids, int32_t n_seqs,
                                      const int32_t* cu_q, const void* q,
                                      const void* k, const void* v, float score_cap,
                                      void* out, float* lse, void* stream);
sp_status sp_attention_decode_capped(sp_cache* cache, int32_t layer,
                                     const int32_t* seq_ids, int32_t n_seqs,
                                     const void* q, float score_cap, void* out,
                                     float* lse, void* stream);

/* Decode over chosen pages: a GLOBAL head reads, of the pages that hold what it
 * sees, the first sink_pages, the newest recent_pages and the top_pages others with
 * the highest scores for this query (ties: the lower page); all of them while there
 * are no more than sink_pages + recent_pages + top_pages.  LOCAL and RETRIEVAL heads
 * read what sp_attention_decode reads.  Everything else is as there; score_cap as
 * for sp_attention_decode_capped, 0 for scores as they are.
 *
 * A page's score comes from bounds of its keys, kept for every full page of a
 * GLOBAL head: in each dimension c the largest and smallest of its stored keys
 * (code * scales, rounded to fp32), on the grid of s = 2^e, the least e in [-50, 50]
 * with max |key| <= 127 * 2^e: hi_c = ceil(max / s), lo_c = floor(min / s), at most
 * +-127.  A query head's elements are rounded to a grid t = 2^f chosen the same way,
 * x_c = round(q_c / t), ties to even.  The head's score is
 * s t sum_c max(x_c hi_c, x_c lo_c), an upper bound of the rounded query's products
 * with the page's keys; the page's is the largest of the KV head's query heads.
 * Scores are exact (whole numbers times powers of two): which pages are kept does
 * not depend on the order of sums.  A NaN key does not count; with a NaN in q the
 * pages kept are any, and the row's output is NaN.
 *   pages: DEVICE array [n_seqs][num_kv_heads][sink_pages + recent_pages + top_pages]
 *     of the kept pages' numbers (page j holds the tokens from j * page_size on) in
 *     ascending order, -1 behind the last and for LOCAL and RETRIEVAL heads; nullable.
 *   recent_pages >= 1 (the newest page has no bounds until it is full), the others
 *   >= 0; each at most 2^20.
 *
 * The bounds live in a caller-owned device buffer (256-byte aligned, at least
 * sp_page_bounds_bytes bytes: 2 * head_dim + 4 per page, and as scratch of the choice
 * 8 bytes for every page that max_batch sequences of max_seq_len tokens have in one
 * layer), attached while no sequence holds tokens (SP_ERR_INVALID_ARG otherwise; null
 * detaches).  Both want the cache's device to be current and wait for it first, so that
 * no earlier call still uses a buffer that is detached or replaced; keep it alive until
 * then, or until the cache is destroyed, and replay no graph captured with it afterwards.  While it is attached,
 * every call that writes keys (sp_build_cache, sp_append_kv, the rope forms,
 * sp_rope_realign, sp_unpack_seq) also computes the bounds of the full pages that it
 * touched, in one more launch a layer; attach the buffer before capturing such calls.
 * Two decodes of one cache share the scratch, as they share the workspace: stream
 * order. */
sp_status sp_page_bounds_bytes(const sp_config* cfg, size_t* bytes);
sp_status sp_attach_page_bounds(sp_cache* cache, void* buffer);
sp_status sp_attention_decode_select(sp_cache* cache, int32_t layer, const int32_t* seq_ids,
                                     int32_t n_seqs, const void* q, int32_t top_pages,
                                     int32_t sink_pages, int32_t recent_pages,
                                     float score_cap, void* out, float* lse, int32_t* pages,
                                     void* stream);

/* Decode without any device allocation by the caller for scratch: the same
 * computation as sp_attention_decode, but the split-KV scratch (partial
 * outputs, their max / sum and the merge tickets) lives in a fixed 4 MiB
 * device array compiled into this library instead of the cache's workspace.
 * (The method's sources have no counterpart; this entry point is for
 * callers that cannot allocate device memory when they decode: a plain C host
 * without a device allocator, or a serving loop that must not call cudaMalloc
 * mid-step because it can synchronise the device or is forbidden after
 * start-up.)
 *   - The caller still passes the cache, q, out and lse, as for
 *     sp_attention_decode.
 *   - Limit: (n_seqs * num_kv_heads + SM count) * group * (head_dim + 2) * 4
 *     bytes plus the tickets must fit in 4 MiB; larger calls return
 *     SP_ERR_UNSUPPORTED before any launch (use sp_attention_decode).
 *   - The first call on each device looks up the array's device address
 *     (cudaGetSymbolAddress, with that device current); make that first call
 *     before any stream capture.
 *   - Every call shares the one array; the tickets are cleared at the start of
 *     each call.  Calls that overlap on the GPU (other streams, other caches)
 *     race on the array and must not be issued concurrently.
 *   - Every GPU that loads the library holds the array until the process
 *     exits. */
sp_status sp_attention_decode_static_scratch(sp_cache* cache, int32_t layer,
                                             const int32_t* seq_ids, int32_t n_seqs,
                                             const void* q, void* out, float* lse,
                                             void* stream);

/* FP8 and FP4 pages: the per-channel scales of `layer`.  k_scale, v_scale are host
 * arrays [num_kv_heads][head_dim] of floats in [2^-14, 128]; the pages store
 * e4m3(x * (1 / scale)) with the reciprocal taken in fp32 (FP4: the block
 * format of x * (1 / scale), see sp_kv_dtype).  Decode rebuilds
 * each element as code * scale in f16 (the scale rounded to f16 first), so the
 * range keeps scales normal in f16 and 448 * scale below the f16 maximum;
 * q and P enter the decode MMAs as f16 as well.  Only while no sequence holds
 * tokens in `layer` (SP_ERR_INVALID_ARG otherwise); for a bf16 cache or a
 * scale outside the range SP_ERR_INVALID_ARG.  Synchronous. */
sp_status sp_set_kv_scales(sp_cache* cache, int32_t layer, const float* k_scale,
                           const float* v_scale, void* stream);

/* RoPE realignment of reused keys (news summary, "Elastic Sparsity": the
 * first recovery step is RoPE position alignment).  For every listed sequence
 * and KV head kv_head (-1 = all KV heads) of `layer`, rotates in place every
 * STORED K row whose token position p satisfies pos_lo <= p < pos_hi by
 * `delta` positions of rotary embedding: with a_i = delta * rope_theta^(-2i/d)
 * for i < d/2 (the "rotate half" pairing of element i with element i + d/2),
 *     k'[i]       = k[i] cos a_i - k[i + d/2] sin a_i
 *     k'[i + d/2] = k[i + d/2] cos a_i + k[i] sin a_i.
 * The angles are formed and reduced modulo 2 pi in double precision on the
 * host; the rotation runs in fp32 and rounds to bf16 (at most one bf16 ulp
 * from the exact rotation of the stored value).  FP8 pages: each code is
 * dequantised with its channel's K scale, the pair rotated in fp32 with
 * every product and sum rounded once, and the results written as new codes
 * like a write (e4m3(v * fp32(1 / scale)), saturating); FP4 pages likewise,
 * with new block scales.  V and the recorded positions
 * are not changed: a caller reusing KV computed at other positions stores it
 * at its new positions and calls this with delta = new - old.  Rows outside
 * [pos_lo, pos_hi), rows a policy does not store, and other heads are left
 * untouched.  SP_ERR_INVALID_ARG for a bad list or head, pos_lo > pos_hi,
 * rope_theta <= 0 or |delta| > 2^40.  The news summary names no such entry
 * point; this is its RoPE-alignment step applied to the paged layout. */
sp_status sp_rope_realign(sp_cache* cache, int32_t layer, const int32_t* seq_ids,
                          int32_t n_seqs, int32_t kv_head, int64_t pos_lo,
                          int64_t pos_hi, int64_t delta, double rope_theta,
                          void* stream);

/* On-device retrieval selection, heavy hitters (runtime article section 2:
 * retrieval heads see "the top-p important tokens"; section 5 measures an
 * H2O heavy-hitter decode scenario).  No cache is involved: run it on the
 * prompt's dense q / k before setting a RETRIEVAL(I) policy.
 *   q_obs [n_obs][num_q_heads][head_dim] bf16: the observation rows, the last
 *         n_obs query rows of the prompt (positions n - n_obs .. n - 1);
 *   k     [n][num_kv_heads][head_dim] bf16: the prompt's keys (positions 0..n-1).
 * For KV head h the score of key j is the causal softmax probability
 * (scale 1/sqrt(head_dim), visible keys j <= position of the row) summed over
 * h's query heads (grouped-query attention, query head q belongs to KV head
 * q / (num_q_heads / num_kv_heads)) and over the observation rows.  The
 * selection of head h is the topk highest scores among keys j < n - recent
 * (ties: lower j first), then the recent window n - recent .. n - 1, all in
 * ascending order.
 * Outputs (device): idx [num_kv_heads][topk + recent] int32, row h holding
 * min(topk, n - recent) + min(recent, n) indices followed by -1; counts
 * [num_kv_heads] int32 (nullable); scores [num_kv_heads][n] fp32 (nullable).
 * workspace: device scratch of sp_select_workspace_bytes(...) bytes, 256-byte
 * aligned.  Asynchronous on `stream`.  The runtime article names no such
 * entry point; it is the selection step its retrieval heads assume. */
sp_status sp_select_workspace_bytes(int32_t n_obs, int32_t n, int32_t num_q_heads,
                                    int32_t num_kv_heads, size_t* bytes);
sp_status sp_select_heavy_hitters(const void* q_obs, int32_t n_obs, const void* k, int32_t n,
                                  int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                  int32_t topk, int32_t recent, int32_t* idx, int32_t* counts,
                                  float* scores, void* workspace, size_t workspace_bytes,
                                  void* stream);

/* The "top-p" form of the same selection (runtime article section 2, "the
 * top-p important tokens"), with the same scores, outputs and workspace:
 * for head h the candidates j < n - recent are ranked by score (descending;
 * ties: lower j first) and the shortest prefix whose summed score reaches
 * top_p times the candidates' total score is kept, at most max_keys keys
 * (the page budget the caller sizes the RETRIEVAL pages for; none when the
 * total is 0), then the recent window.  idx rows are max_keys + recent wide.
 * The sums are taken in float64, so a count whose exact prefix mass lies
 * within a few float64 roundings of the boundary may come out one higher or
 * lower than exact arithmetic would give.  SP_ERR_INVALID_ARG unless
 * 0 < top_p <= 1, as well as for the arguments sp_select_heavy_hitters
 * refuses. */
sp_status sp_select_heavy_hitters_top_p(const void* q_obs, int32_t n_obs, const void* k, int32_t n,
                                        int32_t num_q_heads, int32_t num_kv_heads,
                                        int32_t head_dim, float top_p, int32_t max_keys,
                                        int32_t recent, int32_t* idx, int32_t* counts,
                                        float* scores, void* workspace, size_t workspace_bytes,
                                        void* stream);

/* Pack / unpack one sequence for a prefill/decode-disaggregated transfer (news
 * summary, "system gains": in the PD-separated setting only the tokens each
 * head keeps travel, up to 6.3x fewer KV bytes).  The summary names no such
 * entry points; these carry its trimmed per-head layout across.
 *
 * sp_pack_seq writes into the device buffer dst (256-byte aligned) a header
 * (layer count, KV heads, head_dim, page_size, tokens per layer, every unit's
 * policy and retrieval list, per-unit row offsets) followed by the payload:
 * for each (layer, KV head) unit in order, its retained K rows then its
 * retained V rows, [rows][head_dim] elements of the page type each (bf16, or
 * e4m3 bytes for FP8 pages), in position order (GLOBAL
 * every token, LOCAL the sink then the newest ring's worth, RETRIEVAL its
 * listed positions).  *packed_bytes receives the total size; with dst NULL the
 * call only returns that size (no GPU work).  SP_ERR_INVALID_ARG if
 * dst_bytes is smaller.  The header upload is synchronous; the copy runs on
 * `stream`.
 *
 * sp_unpack_seq restores such a buffer into sequence slot `seq` of this cache,
 * which must hold no tokens and have the same layer count, KV heads, head_dim,
 * page_size and page type (FP8 scales are the receiver's own: set them equal
 * before unpacking): it sets the packed policy, allocates pages for every layer
 * and copies the rows into their slots, so the tables, visible sets and
 * attention results equal the source's.  It reads the header (synchronous),
 * checks it against its own size and policies, and checks page capacity
 * before changing anything (SP_ERR_INVALID_ARG / SP_ERR_OUT_OF_PAGES). */
sp_status sp_pack_seq(sp_cache* cache, int32_t seq, void* dst, size_t dst_bytes,
                      size_t* packed_bytes, void* stream);
sp_status sp_unpack_seq(sp_cache* cache, int32_t seq, const void* src, size_t src_bytes,
                        void* stream);

/* Return every page of `seq` (all layers) to the free stack and empty it; the
 * policy stays set. */
sp_status sp_release_seq(sp_cache* cache, int32_t seq, void* stream);

/* SELECTVISIBLESTATE, for tests: the device page table of one unit.
 * Synchronous.  Writes *npages, page_ids[npages] (physical page ids) and
 * slot_pos[npages * page_size] (token position held by each slot, -1 if
 * empty), as the device-side slot rules see them.  cap bounds both arrays
 * (in pages); SP_ERR_INVALID_ARG if the unit holds more. */
sp_status sp_export_table(sp_cache* cache, int32_t seq, int32_t layer,
                          int32_t kv_head, int32_t* npages, int32_t* page_ids,
                          int32_t* slot_pos, int32_t cap, void* stream);

/* For tests: |V(i)| of one unit for n host positions, computed on the device
 * by the same visible-range functions the attention kernels use.  A position
 * must be below what the unit holds plus max_tokens.  Synchronous. */
sp_status sp_visible_count(sp_cache* cache, int32_t seq, int32_t layer,
                           int32_t kv_head, const int64_t* positions, int32_t n,
                           int32_t* counts, void* stream);

/* Host-side mirrors, no GPU work: tokens held by (seq, layer); free pages. */
sp_status sp_seq_len(const sp_cache* cache, int32_t seq, int32_t layer, int32_t* n);
sp_status sp_free_pages(const sp_cache* cache, int32_t* n);

/* Work accounting from the host policy mirror (no GPU work):
 *   visible (query, key) pairs of a prefill of rows n0 .. n0+c-1 of (seq, layer),
 *   summed over query heads (FLOP = 4 * head_dim * pairs);
 *   visible K+V bytes one decode query at position t of each listed sequence
 *   reads in `layer` (head_dim elements of the page type per row). */
sp_status sp_count_prefill_pairs(const sp_cache* cache, int32_t seq, int32_t layer,
                                 int64_t n0, int64_t c, int64_t* pairs);
sp_status sp_count_decode_bytes(const sp_cache* cache, int32_t layer,
                                const int32_t* seq_ids, int32_t n_seqs,
                                const int64_t* t, int64_t* bytes);

/* Synchronise `stream` and read the device status word: SP_OK, or
 * SP_ERR_DEVICE_STATUS / SP_ERR_TIMEOUT if a kernel flagged a problem (the
 * word is then cleared).  *word (nullable) receives the raw flags. */
sp_status sp_get_status(sp_cache* cache, void* stream, int32_t* word);

/* Check of the bounded waits every kernel uses (no fault, no hang): one
 * warp waits on a shared-memory mbarrier for at most limit_cycles
 * ([1000, 2e9] clock cycles).  mode 0: nothing arrives, the wait gives up and
 * raises the timeout flag of the cache's status word, so the next
 * sp_get_status returns SP_ERR_TIMEOUT (and clears it); mode 1: a second
 * warp arrives after limit_cycles / 8 and the status stays clear; mode 2:
 * two warps that must leave together (the pattern of the prefill's FP8
 * converter pair) each wait on their own barrier, one completes and one
 * never does; both leave after the limit (SP_ERR_TIMEOUT as in mode 0) and
 * neither is left at a named barrier.
 * Asynchronous on `stream`; SP_ERR_INVALID_ARG for other arguments. */
sp_status sp_selftest_bounded_wait(sp_cache* cache, int64_t limit_cycles, int32_t mode,
                                   void* stream);

/* Instrumentation for profilers and benchmarks (the pages have no
 * counterpart).  Arms one pair of caller-created CUDA events (cudaEvent_t
 * handles passed as void*) for the next attention call on this cache
 * (sp_attention_prefill, sp_attention_decode, their capped forms,
 * sp_attention_decode_select or sp_attention_decode_static_scratch): that call records start_event on its
 * stream immediately before its first kernel launch and end_event
 * immediately after its last one (the prefill's merge included), so the
 * interval between them is the device time of the call's kernels without
 * the host's planning, which otherwise shows in events recorded around the
 * call whenever the device is idle while the host plans.  The pair is used
 * by one call and then disarmed (a call that fails may leave it armed).
 * Both null disarms.  The events stay owned by the caller and
 * must stay alive until that call has been made.
 * SP_ERR_INVALID_ARG for a null cache or exactly one null event. */
sp_status sp_set_launch_events(sp_cache* cache, void* start_event, void* end_event);

/* Message of the last failing call on this thread ("" if none). */
const char* sp_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* SEGPAGED_H */
