// sp_rotate.cuh -- the rotary embedding's angles and rotations, shared by the
// writes into the pages (sp_write.cu) and the rotation of plain rows
// (sp_rope_axes.cu).
//
// A frequency is a 64-bit fraction of a turn (sp_turns.h), so position * frequency
// modulo 2^64 is the angle modulo a turn, whatever the position's size or sign: off
// by |position| times the fraction's own error.
#pragma once
#include <cmath>

#include "sp_device.cuh"
#include "sp_internal.h"
#include "sp_turns.h"

namespace sp {

// Host: the d / 2 frequencies (rope_theta^(-2i/d), or inv_freq where given) in
// 2^-64 turns a position, modulo one turn (whole turns a position rotate nothing).
inline sp_status turns_of(double rope_theta, const double* inv_freq, int d, uint64_t (&turn)[64]) {
    if (!inv_freq && (!(rope_theta > 0.0) || !std::isfinite(rope_theta)))
        return fail(SP_ERR_INVALID_ARG, "rope_theta must be positive and finite");
    for (int i = 0; i < d / 2; ++i) {
        const double w = inv_freq ? inv_freq[i] : std::pow(rope_theta, -2.0 * i / d);
        if (!(std::fabs(w) <= 65536.0)) return fail(SP_ERR_INVALID_ARG, "frequencies must be finite, at most 2^16");
        turn[i] = turn_of(w);
    }
    return SP_OK;
}

// Positions on several axes: device array, element (axis, row) at axis *
// axis_stride + row * row_stride; pair i of the dimensions turns by the position
// on axis of[i].
constexpr int kMaxAxes = 4;
struct Axes {
    const int64_t* pos;
    int64_t axis_stride, row_stride;
    int32_t n;
    uint8_t of[64];
};

// Host: checks an axis map and the positions' array (which may be null: a call
// without rows); fills ax.
inline sp_status axes_of(const int64_t* pos, int64_t axis_stride, int64_t row_stride, int32_t n_axes,
                         const int32_t* axis_of, int d, Axes& ax) {
    if (!axis_of) return fail(SP_ERR_INVALID_ARG, "null argument");
    if (n_axes < 1 || n_axes > kMaxAxes) return fail(SP_ERR_INVALID_ARG, "between 1 and 4 axes");
    if (reinterpret_cast<uintptr_t>(pos) & 7) return fail(SP_ERR_INVALID_ARG, "positions must be 8-byte aligned");
    if (axis_stride < 0 || row_stride < 0) return fail(SP_ERR_INVALID_ARG, "position strides must not be negative");
    for (int i = 0; i < d / 2; ++i) {
        if (axis_of[i] < 0 || axis_of[i] >= n_axes) return fail(SP_ERR_INVALID_ARG, "axis_of names an axis that is not there");
        ax.of[i] = (uint8_t)axis_of[i];
    }
    ax.pos = pos;
    ax.axis_stride = axis_stride;
    ax.row_stride = row_stride;
    ax.n = n_axes;
    return SP_OK;
}

// Host: does one of `rows` rows of `len` bytes, `stride` bytes apart from `base`
// on, meet [lo, hi)?
inline bool rows_meet(const void* base, int64_t stride, int64_t len, int64_t rows, uintptr_t lo, uintptr_t hi) {
    const uintptr_t b = reinterpret_cast<uintptr_t>(base);
    if (stride == 0) rows = rows < 1 ? rows : 1;         // (positions that every row shares)
    const int64_t d = (int64_t)(lo - b) - len;          // the first row that ends behind lo
    const int64_t r = d < 0 ? 0 : stride ? d / stride + 1 : 1;
    return r < rows && b + (uintptr_t)(r * stride) < hi;
}

// Host: do the positions of `rows` rows meet [lo, hi)?
inline bool axes_meet(const Axes& ax, int64_t rows, uintptr_t lo, uintptr_t hi) {
    for (int a = 0; a < ax.n; ++a)
        if (rows_meet(ax.pos + a * ax.axis_stride, ax.row_stride * 8, 8, rows, lo, hi)) return true;
    return false;
}

// Cosine and sine of an angle in 2^-64 turns: the nearest 2^-32 turn, as a signed
// number of half turns.
__device__ __forceinline__ float2 cos_sin(uint64_t turns) {
    const float x = (float)(int32_t)(uint32_t)((turns + 0x80000000ull) >> 32) * 4.6566128730773926e-10f;
    float2 r;
    sincospif(x, &r.y, &r.x);
    return r;
}

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
__device__ __forceinline__ uint4 bf16x8(const float* x) {
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

}  // namespace sp
