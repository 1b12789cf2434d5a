// sp_rope_axes.cu -- queries and keys of a prompt's chunk rotated to positions on
// several axes, rows to rows, in one launch (no cache involved).
//
// Mathematics: pair (i, i + d/2) of a row turns by p[axis_of[i]] w_i:
//     x'[i]       = x[i] cos a - x[i + d/2] sin a
//     x'[i + d/2] = x[i + d/2] cos a + x[i] sin a
// in fp32, rounded once to bf16.  Angles as for the writes into the pages
// (sp_rotate.cuh): one (cos, sin) per row and pair serves every head of q and k.
//
// Bound by memory: 2 bytes an element read and as much written.  32,768 rows of 32
// query and 8 KV heads (671 MB) 103 us, 6.5 TB/s, 0.96 of the copy rate; 777 rows of
// 28 and 4 heads 4.0 us, launch and two dependent loads.  Four rows a block share its
// start from 2,048 rows on; fewer rows take a block each, for more of them.
#include "sp_rotate.cuh"

namespace sp {

namespace {

constexpr int kRotThreads = 256;
constexpr int kRotRows = 4;                  // rows of a block, at most

struct RotateParams {
    const __nv_bfloat16 *q, *k;
    __nv_bfloat16 *q_out, *k_out;
    int64_t q_stride, k_stride, rows;
    int32_t hq, hkv, d, per;                 // heads (0: no such tensor), head_dim, rows a block
    uint64_t turn[64];
    Axes axes;
};

__global__ void __launch_bounds__(kRotThreads) k_rope_axes(const __grid_constant__ RotateParams p) {
    __shared__ float4 cs[kRotRows * 32];     // [row][pair of a chunk][chunk]
    const int tid = threadIdx.x, half = p.d / 2, nc = half / 8, lc = 31 - __clz(nc);
    const int64_t r0 = (int64_t)blockIdx.x * p.per;
    const int n = (int)min64(p.per, p.rows - r0);
    for (int e = tid; e < n * half; e += kRotThreads) {
        const int t = e / half, f = e % half;
        const uint64_t at = (uint64_t)__ldg(p.axes.pos + p.axes.of[f] * p.axes.axis_stride + (r0 + t) * p.axes.row_stride);
        reinterpret_cast<float2*>(cs + (t * 4 + ((f & 7) >> 1)) * nc + (f >> 3))[f & 1] = cos_sin(at * p.turn[f]);
    }
    __syncthreads();
    const int heads = p.hq + p.hkv, all = (n * heads) << lc;
    for (int e = tid; e < all; e += kRotThreads) {
        const int c = e & (nc - 1), th = e >> lc, t = th / heads, h = th - t * heads;
        const bool is_q = h < p.hq;
        const int hh = is_q ? h : h - p.hq;
        const __nv_bfloat16* src = (is_q ? p.q : p.k) + (r0 + t) * (is_q ? p.q_stride : p.k_stride) + hh * p.d + c * 8;
        __nv_bfloat16* dst = (is_q ? p.q_out : p.k_out) + ((r0 + t) * (is_q ? p.hq : p.hkv) + hh) * p.d + c * 8;
        const uint4 a = *reinterpret_cast<const uint4*>(src), b = *reinterpret_cast<const uint4*>(src + half);
        float x[8], y[8];
        rotate8(a, b, cs + t * half / 2 + c, nc, x, y);
        *reinterpret_cast<uint4*>(dst) = bf16x8(x);
        *reinterpret_cast<uint4*>(dst + half) = bf16x8(y);
    }
}

}  // namespace

}  // namespace sp

using namespace sp;

extern "C" sp_status sp_rope_axes(const void* q, int64_t q_stride, int32_t num_q_heads, const void* k,
                                  int64_t k_stride, int32_t num_kv_heads, int32_t head_dim, int64_t rows,
                                  const int64_t* axis_pos, int64_t axis_stride, int64_t row_stride,
                                  int32_t n_axes, const int32_t* axis_of, double rope_theta,
                                  const double* inv_freq, void* q_out, void* k_out, void* stream) {
    if (head_dim != 64 && head_dim != 128) return fail(SP_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
    if (num_q_heads < 0 || num_q_heads > 1024 || num_kv_heads < 0 || num_kv_heads > 1024)
        return fail(SP_ERR_INVALID_ARG, "head counts must lie in [0, 1024]");
    if (rows < 0 || rows >= (int64_t(1) << 31)) return fail(SP_ERR_INVALID_ARG, "rows outside [0, 2^31)");
    RotateParams p{};
    sp_status s = axes_of(axis_pos, axis_stride, row_stride, n_axes, axis_of, head_dim, p.axes);
    if (s != SP_OK) return s;
    s = turns_of(rope_theta, inv_freq, head_dim, p.turn);
    if (s != SP_OK) return s;
    struct Side { const void* in; void* out; int64_t stride, len; } sides[2] = {
        {q, q_out, q_stride, (int64_t)num_q_heads * head_dim}, {k, k_out, k_stride, (int64_t)num_kv_heads * head_dim}};
    if (rows == 0 || num_q_heads + num_kv_heads == 0) return SP_OK;
    if (!axis_pos) return fail(SP_ERR_INVALID_ARG, "null argument");
    for (const Side& x : sides) {
        if (x.len == 0) continue;
        if (!x.in || !x.out) return fail(SP_ERR_INVALID_ARG, "null argument");
        if (x.stride < x.len || (x.stride & 7))
            return fail(SP_ERR_INVALID_ARG, "strides must be >= heads * head_dim and multiples of 8");
        if ((reinterpret_cast<uintptr_t>(x.in) | reinterpret_cast<uintptr_t>(x.out)) & 15)
            return fail(SP_ERR_INVALID_ARG, "q, k, q_out and k_out must be 16-byte aligned");
    }
    // blocks read some rows while others are written: no overlap but a row with itself
    for (int o = 0; o < 2; ++o) {
        if (sides[o].len == 0) continue;
        const uintptr_t lo = reinterpret_cast<uintptr_t>(sides[o].out), hi = lo + (uintptr_t)(rows * sides[o].len * 2);
        bool meet = axes_meet(p.axes, rows, lo, hi);
        for (int i = 0; i < 2; ++i) {
            const Side& x = sides[i];
            if (x.len == 0) continue;
            const bool in_place = i == o && x.in == x.out && (x.stride == x.len || rows == 1);
            meet = meet || (!in_place && rows_meet(x.in, x.stride * 2, x.len * 2, rows, lo, hi));
        }
        const Side& other = sides[1 - o];
        if (other.len != 0)
            meet = meet || rows_meet(other.out, other.len * 2, other.len * 2, rows, lo, hi);
        if (meet)
            return fail(SP_ERR_INVALID_ARG, "an output overlaps another tensor (it may be its own input if that is contiguous)");
    }
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.k = static_cast<const __nv_bfloat16*>(k);
    p.q_out = static_cast<__nv_bfloat16*>(q_out);
    p.k_out = static_cast<__nv_bfloat16*>(k_out);
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.rows = rows;
    p.hq = num_q_heads;
    p.hkv = num_kv_heads;
    p.d = head_dim;
    p.per = rows >= 2048 ? kRotRows : 1;
    const unsigned blocks = (unsigned)((rows + p.per - 1) / p.per);
    k_rope_axes<<<blocks, kRotThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? SP_OK : cuda_fail(e, "rotation launch");
}
