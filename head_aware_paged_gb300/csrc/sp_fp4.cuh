// sp_fp4.cuh -- 4-bit K/V pages: the number formats and where a row's codes
// and scales lie in a page.
//
// A row (head_dim 128) is 8 blocks of 16 neighbouring dimensions.  Block b
// has one scale s_b, an unsigned float of 5 exponent and 3 mantissa bits (the
// f16 number whose bits are code << 7: 2^-17 .. 10240 and 0), the value
// nearest amax_b / 6; element x is the e2m1 value (0, .5, 1, 1.5, 2, 3, 4, 6,
// signed) nearest x / s_b.  Both roundings are to nearest, ties to even, and
// saturate (a scale at 10240, an element at 6).  A scale of 10240 at most
// keeps every code * scale finite and exact in f16 (2 + 4 significant bits),
// which is what the attention kernels multiply.
//
// 72 bytes a row instead of bf16's 256.  Rows lie in groups of 16 slots, 1152
// contiguous bytes each: 1024 of codes, then 128 of scales, so any run of
// groups of a page is one untiled bulk copy.  Inside a group the order is the
// one the decode kernel's fragments want (bank-conflict-free 16-, 8- and
// 4-byte reads, sp_decode4.cuh):
//   K codes   row position kpos(s) of slot s, dimensions in order;
//   K scales  one 32-bit word per (row position mod 8, block pair): the two
//             blocks of position g, then of position g + 8;
//   V codes   slots in order, the 8-byte block units of slots 2, 3 mod 4
//             with their halves swapped;
//   V scales  one 32-bit word per (block, slot mod 4): slots j, j+4, j+8, j+12.
#pragma once
#if defined(__CUDACC__)
#include <cuda_fp16.h>
#endif
#include <stdint.h>

#include "sp_rules.h"

namespace sp {

constexpr int kFp4Group = 16;                 // slots in a group
constexpr int kFp4RowBytes = 72;              // 64 code bytes and 8 scales
constexpr int kFp4GroupBytes = kFp4Group * kFp4RowBytes;
constexpr int kFp4ScaleOff = kFp4Group * 64;  // scales behind the group's codes
constexpr float kFp4MaxScale = 10240.f;

// Byte offset of the group that holds `slot` (0 .. P-1) of physical page `page`.
SP_HD int64_t fp4_group_off(int64_t page, int slot, int P) {
    return (page * P + (slot & ~15)) * kFp4RowBytes;
}
// K row position of slot s (0..15): the product's row i = 2j, 2j+1, 2j+8, 2j+9
// holds slot j, j+4, j+8, j+12.
SP_HD int fp4_kpos(int s) { return 2 * (s & 3) + ((s >> 2) & 1) + (s & 8); }
// Offsets inside a group of block b's 8 code bytes and of its scale.
SP_HD int fp4_k_code(int s, int b) { return fp4_kpos(s) * 64 + b * 8; }
SP_HD int fp4_v_code(int s, int b) { return s * 64 + (b ^ (((s >> 1) & 1) << 2)) * 8; }
SP_HD int fp4_k_scale(int s, int b) {
    const int i = fp4_kpos(s);
    return kFp4ScaleOff + (((i & 7) * 4 + (b >> 1)) << 2) + ((i >> 3) << 1) + (b & 1);
}
SP_HD int fp4_v_scale(int s, int b) { return kFp4ScaleOff + b * 16 + (s & 3) * 4 + (s >> 2); }

#if defined(__CUDACC__)

// Scale code of a block whose largest magnitude is amax.  amax / 6 is amax times
// the rounded sixth, corrected once by its residual: then it is a tie between
// two scales only where amax is 6 times that tie.  (Any other amax is a step of
// its own off, two thirds of the quotient's step at least; the product alone,
// a quarter of a step too large, reached the tie 19/16 from just below.)
__device__ __forceinline__ uint32_t fp4_scale_code(float amax) {
    constexpr float kSixth = 0.16666667163372039794921875f;
    const float a = fminf(amax, 6.f * kFp4MaxScale), q = a * kSixth;
    const float f = __fmaf_rn(__fmaf_rn(-q, 6.f, a), kSixth, q);
    if (f < 6.103515625e-05f) return (uint32_t)__float2int_rn(f * 131072.f);   // below 2^-14: steps of 2^-17
    const uint32_t u = __float_as_uint(f);
    return ((u + 0x7FFFFu + ((u >> 20) & 1u)) >> 20) - (112u << 3);            // 3 mantissa bits, ties to even
}
__device__ __forceinline__ float fp4_scale_value(uint32_t code) {
    return __half2float(__ushort_as_half((unsigned short)(code << 7)));
}
// Two elements, already divided by their scale, as one byte of codes.
__device__ __forceinline__ uint32_t fp4_pair_code(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b8 c;\n\tcvt.rn.satfinite.e2m1x2.f32 c, %2, %1;\n\tcvt.u32.u8 %0, c;\n\t}"
        : "=r"(r) : "f"(lo), "f"(hi));
    return r;
}
// The four code bytes of a word as f16 pairs (the even dimension low).
__device__ __forceinline__ void fp4_word_f16(uint32_t w, uint32_t& p0, uint32_t& p1, uint32_t& p2,
                                             uint32_t& p3) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(p0), "=r"(p1), "=r"(p2), "=r"(p3) : "r"(w));
}

// A block of 16 values: its 8 code bytes and its scale code.  x / s is x times
// the rounded reciprocal, corrected once by its residual x - y s (iterative
// refinement): the uncorrected product misses ties between two e2m1 values (a
// scale mantissa of 13/8 at 1.75, for one), the corrected one is exact there.
__device__ __forceinline__ uint2 fp4_quant16(float (&x)[16], uint32_t& scale_code) {
    float amax = 0.f;
    #pragma unroll
    for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(x[i]));
    scale_code = fp4_scale_code(amax);
    if (scale_code == 0) return make_uint2(0u, 0u);   // largest value below half the least scale
    if (amax > 1e30f) {                               // an infinity has no residual: far past 6 s will do
        #pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = fabsf(x[i]) > 1e30f ? copysignf(1e30f, x[i]) : x[i];
    }
    const float s = fp4_scale_value(scale_code), inv = __frcp_rn(s);
    float y[16];
    #pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float q = x[i] * inv;
        y[i] = __fmaf_rn(__fmaf_rn(-q, s, x[i]), inv, q);
    }
    uint32_t w[2] = {0u, 0u};
    #pragma unroll
    for (int i = 0; i < 8; ++i) w[i >> 2] |= fp4_pair_code(y[2 * i], y[2 * i + 1]) << (8 * (i & 3));
    return make_uint2(w[0], w[1]);
}
// ... and back: code * scale of the 16 elements.
__device__ __forceinline__ void fp4_value16(uint2 codes, uint32_t scale_code, float (&x)[16]) {
    const float s = fp4_scale_value(scale_code);
    #pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t p[4];
        fp4_word_f16(h ? codes.y : codes.x, p[0], p[1], p[2], p[3]);
        #pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __half2 v = *reinterpret_cast<const __half2*>(&p[e]);
            x[8 * h + 2 * e] = __low2float(v) * s;
            x[8 * h + 2 * e + 1] = __high2float(v) * s;
        }
    }
}

#endif

}  // namespace sp
