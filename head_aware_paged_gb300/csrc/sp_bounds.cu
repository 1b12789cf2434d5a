// sp_bounds.cu -- page bounds (sp_bounds.cuh) of the pages that a write has
// touched, from the keys as the pages hold them.
//
// A page's bounds are a function of its contents, taken when the page is full:
// a query keeps its newest page whatever it holds.  Every write computes them
// for the full pages that it touched, after its rows are in place (the keys come
// from L2 then), so nothing else has to remember which bounds are stale.  The
// device's own length, page table and head class decide whether a page is
// there and full, so a replayed write leaves them right whatever was appended
// or released in between.
//
// Bound by latency: 2 P d bytes of keys a page come from L2, and a block looks up one
// page.  An 8,192-token prompt of 8 GLOBAL heads (1,024 pages, 17 MB) 7.3 us; launched
// while the write's last blocks run, the write and its bounds together end 2.2 us
// earlier than one after the other.
#include "sp_bounds.cuh"
#include "sp_device.cuh"
#include "sp_internal.h"

namespace sp {

namespace {

constexpr int kBoundThreads = 256;

struct BoundsParams {
    Meta meta;
    Geo geo;
    int32_t layer, n_seqs;
    int8_t* codes;
    float* step;
    const void* kpool;
    int32_t seq[kMaxCallSeqs], page0[kMaxCallSeqs];   // sequence, its first touched page
    int32_t off[kMaxCallSeqs + 1];                    // prefix of the touched pages
};

enum { kBf16, kFp8, kFp4 };

__device__ __forceinline__ void widen(float& lo, float& hi, float x) {
    lo = fminf(lo, x);
    hi = fmaxf(hi, x);
}

// A block per (touched page, KV head).  A thread takes N neighbouring dimensions
// of every R-th row; the block's rows meet in shared memory.
template <int KV, int D>
__global__ void __launch_bounds__(kBoundThreads) k_bounds(const __grid_constant__ BoundsParams p) {
    constexpr int N = KV == kBf16 ? 8 : 16;
    constexpr int T = D / N;                          // threads of a row
    constexpr int R = kBoundThreads / T;              // rows of a pass
    constexpr int W = kBoundThreads / 32;
    __shared__ float part[2][W][D];
    __shared__ float top[W];
    const Geo& g = p.geo;
    int a = 0, z = p.n_seqs - 1;                      // sequence with off[a] <= blockIdx.x < off[a + 1]
    while (a < z) {
        const int mid = (a + z + 1) >> 1;
        if (p.off[mid] <= (int)blockIdx.x) a = mid; else z = mid - 1;
    }
    const int seq = p.seq[a], h = blockIdx.y;
    const int32_t pg = p.page0[a] + ((int)blockIdx.x - p.off[a]);
    const int64_t row = g.unit_row(seq, p.layer, h);
    asm volatile("griddepcontrol.wait;" ::: "memory");       // the write is done
    if (p.meta.pol[row].kind != kGlobal || pg >= p.meta.npages[row] ||
        (int64_t)(pg + 1) * g.page > p.meta.seqlen[(int64_t)seq * g.layers + p.layer])
        return;
    const int32_t page = p.meta.ptab[row * g.max_pages_unit + pg];
    if (page < 0 || page >= g.num_pages) {
        if (threadIdx.x == 0) atomicOr(p.meta.status, kStatusBadPage);
        return;
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, c0 = (tid % T) * N;
    float lo[N], hi[N];
    #pragma unroll
    for (int i = 0; i < N; ++i) { lo[i] = INFINITY; hi[i] = -INFINITY; }
    for (int r = tid / T; r < g.page; r += R) {
        if constexpr (KV == kFp4) {
            const uint8_t* grp = static_cast<const uint8_t*>(p.kpool) + fp4_group_off(page, r, g.page);
            float x[16];
            fp4_value16(*reinterpret_cast<const uint2*>(grp + fp4_k_code(r & 15, c0 / 16)),
                        grp[fp4_k_scale(r & 15, c0 / 16)], x);
            #pragma unroll
            for (int i = 0; i < N; ++i) widen(lo[i], hi[i], x[i]);
        } else {
            const int64_t at = ((int64_t)page * g.page + r) * D + c0;
            const uint4 v = KV == kFp8
                ? *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.kpool) + at)
                : *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.kpool) + at);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            #pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (KV == kFp8) {
                    uint32_t h2[2];
                    f16x2x2_of_e4m3x4(w[i], h2[0], h2[1]);
                    #pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2[e]));
                        widen(lo[4 * i + 2 * e], hi[4 * i + 2 * e], f.x);
                        widen(lo[4 * i + 2 * e + 1], hi[4 * i + 2 * e + 1], f.y);
                    }
                } else {
                    const __nv_bfloat162 b = *reinterpret_cast<const __nv_bfloat162*>(&w[i]);
                    widen(lo[2 * i], hi[2 * i], __low2float(b));
                    widen(lo[2 * i + 1], hi[2 * i + 1], __high2float(b));
                }
            }
        }
    }
    // rows of a warp, then of the block
    #pragma unroll
    for (int i = 0; i < N; ++i) {
        #pragma unroll
        for (int o = T; o < 32; o <<= 1) {
            lo[i] = fminf(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], o));
            hi[i] = fmaxf(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], o));
        }
        if (lane < T) {
            part[0][warp][c0 + i] = lo[i];
            part[1][warp][c0 + i] = hi[i];
        }
    }
    __syncthreads();
    float m = INFINITY, M = -INFINITY;
    if (tid < D) {
        #pragma unroll
        for (int w = 0; w < W; ++w) {
            m = fminf(m, part[0][w][tid]);
            M = fmaxf(M, part[1][w][tid]);
        }
        if (M < m) m = M = 0.f;                       // NaN in every row
        if constexpr (KV != kBf16) {                  // (positive, so it keeps the order)
            const float s = p.meta.kscale[((int64_t)p.layer * g.hkv + h) * D + tid];
            m *= s;
            M *= s;
        }
    }
    float A = tid < D ? fmaxf(fabsf(m), fabsf(M)) : 0.f;
    #pragma unroll
    for (int o = 16; o > 0; o >>= 1) A = fmaxf(A, __shfl_xor_sync(0xffffffffu, A, o));
    if (lane == 0) top[warp] = A;
    __syncthreads();
    #pragma unroll
    for (int w = 0; w < W; ++w) A = fmaxf(A, top[w]);
    const int e = grid_exponent(A);
    if (tid < D) {
        const float up = grid_step(-e);               // exact
        int8_t* out = p.codes + (int64_t)page * 2 * D + tid;
        out[0] = (int8_t)fminf(fmaxf(ceilf(M * up), -127.f), 127.f);
        out[D] = (int8_t)fminf(fmaxf(floorf(m * up), -127.f), 127.f);
    }
    if (tid == 0) p.step[page] = grid_step(e);
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// Places in the caller's buffer; the whole size.
size_t place(const sp_config& cfg, int max_pages_unit, uint8_t* base, PageBounds* b) {
    const size_t pages = cfg.num_pages, units = (size_t)cfg.max_batch * cfg.num_kv_heads;
    size_t o = 0;
    auto take = [&](size_t bytes) { const size_t at = o; o = up256(o + bytes); return base + at; };
    uint8_t* codes = take(pages * 2 * cfg.head_dim);
    uint8_t* step = take(pages * 4);
    uint8_t* score = take(units * max_pages_unit * 4);
    uint8_t* kept = take(units * max_pages_unit * 4);
    uint8_t* tickets = take(units * 4);
    if (b) {
        b->codes = reinterpret_cast<int8_t*>(codes);
        b->step = reinterpret_cast<float*>(step);
        b->score = reinterpret_cast<uint32_t*>(score);
        b->kept = reinterpret_cast<int32_t*>(kept);
        b->tickets = reinterpret_cast<int32_t*>(tickets);
    }
    return o;
}

}  // namespace

sp_status update_bounds(const sp_cache* c, int32_t layer, const int32_t* seqs, int32_t n_seqs,
                        const int64_t* lo, const int64_t* hi, cudaStream_t stream) {
    if (!c->bounds.codes) return SP_OK;
    const int H = c->cfg.num_kv_heads, L = c->cfg.num_layers, P = c->cfg.page_size;
    cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
    cudaError_t e = cudaStreamIsCapturing(stream, &capture);
    if (e != cudaSuccess) return cuda_fail(e, "stream query");
    const bool graph = capture != cudaStreamCaptureStatusNone;
    BoundsParams p;                                           // (its lists are filled as far as they are used)
    p.n_seqs = p.off[0] = 0;
    for (int b = 0; b < n_seqs; ++b) {
        if (hi[b] <= lo[b]) continue;
        const UnitPol* pol = &c->h_pol[((size_t)seqs[b] * L + layer) * H];
        bool global = false;
        for (int h = 0; h < H; ++h) global = global || pol[h].kind == kGlobal;
        // Full pages of sequences with GLOBAL heads.  A replay may meet other heads and
        // lengths than the capture (the kernel asks the device what is there by then):
        // in a graph every page that the write touches.
        const int64_t first = lo[b] / P, n = c->h_seqlen[(size_t)seqs[b] * L + layer];
        const int64_t end = graph ? cdiv64(hi[b], P) : min64(cdiv64(hi[b], P), n / P);
        if (!(global || graph) || end <= first) continue;
        p.seq[p.n_seqs] = seqs[b];
        p.page0[p.n_seqs] = (int32_t)first;
        p.off[p.n_seqs + 1] = p.off[p.n_seqs] + (int32_t)(end - first);
        ++p.n_seqs;
    }
    if (p.n_seqs == 0) return SP_OK;
    p.meta = c->meta;
    p.geo = c->geo;
    p.layer = layer;
    p.codes = c->bounds.codes;
    p.step = c->bounds.step;
    p.kpool = c->kpool;
    // launched while the write's last blocks run
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)p.off[p.n_seqs], (unsigned)H);
    cfg.blockDim = dim3(kBoundThreads);
    cfg.stream = stream;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    const BoundsParams& q = p;
    if (c->geo.fp4) e = cudaLaunchKernelEx(&cfg, k_bounds<kFp4, 128>, q);
    else if (c->geo.fp8) e = cudaLaunchKernelEx(&cfg, k_bounds<kFp8, 128>, q);
    else if (c->geo.d == 128) e = cudaLaunchKernelEx(&cfg, k_bounds<kBf16, 128>, q);
    else e = cudaLaunchKernelEx(&cfg, k_bounds<kBf16, 64>, q);
    return e == cudaSuccess ? SP_OK : cuda_fail(e, "page bounds launch");
}

}  // namespace sp

using namespace sp;

extern "C" sp_status sp_page_bounds_bytes(const sp_config* cfg, size_t* bytes) {
    size_t pool, meta, ws;
    const sp_status s = sp_required_bytes(cfg, &pool, &meta, &ws);      // (checks the configuration)
    if (s != SP_OK) return s;
    if (!bytes) return fail(SP_ERR_INVALID_ARG, "null output");
    *bytes = place(*cfg, max_unit_pages(cfg), nullptr, nullptr);
    return SP_OK;
}

extern "C" sp_status sp_attach_page_bounds(sp_cache* c, void* buffer) {
    if (!c) return fail(SP_ERR_INVALID_ARG, "null handle");
    if (reinterpret_cast<uintptr_t>(buffer) & 255) return fail(SP_ERR_INVALID_ARG, "buffer must be 256-byte aligned");
    for (const int32_t n : c->h_seqlen)
        if (n != 0) return fail(SP_ERR_INVALID_ARG, "the cache holds tokens; release them first");
    const sp_status s = check_device(c);
    if (s != SP_OK) return s;
    // Released sequences may still have writes and decodes on their way: they end before
    // a buffer is let go or cleared.
    cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return cuda_fail(e, "waiting for the device");
    if (!buffer) {
        c->bounds = PageBounds{};
        return SP_OK;
    }
    PageBounds b;
    const size_t bytes = place(c->cfg, c->geo.max_pages_unit, static_cast<uint8_t*>(buffer), &b);
    e = cudaMemset(buffer, 0, bytes);
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return cuda_fail(e, "page bounds initialisation");
    c->bounds = b;
    return SP_OK;
}
