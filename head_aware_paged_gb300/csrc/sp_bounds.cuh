// sp_bounds.cuh -- page bounds: what the choice of pages for a query reads of
// every page instead of its keys.
//
// For a full page of a GLOBAL head with stored keys k_j, in every dimension c
//     M_c = max_j k_j[c],  m_c = min_j k_j[c];
// with A the largest |M_c|, |m_c| and s = 2^e, the least -50 <= e <= 50 with
// A <= 127 s,
//     hi_c = ceil(M_c / s),  lo_c = floor(m_c / s)      (8 bits, at most +-127)
// so s hi_c and s lo_c bound the page's keys from both sides.  A query head q is
// put on such a grid too (t = 2^f, x_c = q_c / t to the nearest, ties to even), and
//     score = s t sum_c max(x_c hi_c, x_c lo_c)
// bounds the products of the rounded query with the page's keys from above.  The
// sum is a whole number below 2^21 and s and t are powers of two: the score is
// exact in fp32 in whatever order it is summed, and so is every comparison.
//
// 2 d + 4 bytes a page: 1/128 of the K and V of 64 bf16 rows.  Bounds in 8 bits
// cost at most a step of the page's largest magnitude over 127 in each dimension,
// outwards; the query's rounding half a step of its own.
#pragma once
#include <stdint.h>

#include "sp_rules.h"

namespace sp {

constexpr int kGridLow = -50, kGridHigh = 50;

// Exponent of the least power of two with a <= 127 * 2^e, clamped; a >= 0 (not NaN).
SP_HD int grid_exponent(float a) {
#if defined(__CUDA_ARCH__)
    const uint32_t u = __float_as_uint(a);
#else
    uint32_t u;
    __builtin_memcpy(&u, &a, 4);
#endif
    // a = 1.m 2^E: 127 2^(E - 6) = 1.984375 2^E
    const int e = (int)(u >> 23) - 127 - 6 + ((u & 0x7FFFFFu) > 0x7E0000u ? 1 : 0);
    return e < kGridLow ? kGridLow : e > kGridHigh ? kGridHigh : e;
}
// 2^e, |e| <= 126.
SP_HD float grid_step(int e) {
    const uint32_t u = (uint32_t)(e + 127) << 23;
#if defined(__CUDA_ARCH__)
    return __uint_as_float(u);
#else
    float f;
    __builtin_memcpy(&f, &u, 4);
    return f;
#endif
}

// The pages that a query over n tokens keeps of a GLOBAL head: all, or `cap` of
// them.  Laid end to end their slots are [0, this): all are full but the newest.
SP_HD int64_t kept_slots(int64_t n, int P, int64_t cap) {
    const int64_t nb = cdiv64(n, P);
    return nb > cap ? n - (nb - cap) * P : n;
}

}  // namespace sp
