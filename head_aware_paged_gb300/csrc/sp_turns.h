// sp_turns.h -- rotary frequencies as fractions of a turn, in 2^-64 turns a position:
// position * fraction modulo 2^64 is then the angle modulo a turn.
#pragma once
#include <stdint.h>

#include <cmath>

namespace sp {

// w radians a position, |w| <= 2^16.  The fraction is off by 2^-65 turns (rounded to
// the nearest) and, from the double's own roundings of w / (2 pi), by |w| 2^-55.  It is
// taken of |w|, where subtracting the whole turns is exact and small fractions keep
// their bits; -w turns back by exactly as much as w turns.
inline uint64_t turn_of(double w) {
    const double two_pi = 6.283185307179586476925286766559;
    const double f = std::fabs(w) / two_pi;
    // (below 2^64: the largest double under 1, times 2^64, is whole)
    const uint64_t t = (uint64_t)std::rint((f - std::floor(f)) * 18446744073709551616.0);
    return w < 0.0 ? 0 - t : t;
}

}  // namespace sp
