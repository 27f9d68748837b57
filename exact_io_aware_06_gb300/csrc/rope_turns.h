// rope_turns.h -- a rotation frequency, radians per position, as the kernels hold it: turns per
// position with the whole ones dropped, a 64-bit fraction.  Host code.
//
// f / (2 pi) as a double is off by up to 2^-53 of its value and more: at position 2^31 by 2^-21 turns for
// f = 10 and 2^-18 for f = 100.  Here 1 / (2 pi) is the sum of three doubles (off by 2^-164), the first
// two products are taken exactly, as product and remainder (fma), and whole turns leave each piece by
// integer arithmetic: the fraction is off by under 2^-62 for |f| up to 2^64.
#pragma once

#include <cmath>
#include <cstdint>
#include <cstring>

namespace fa {

constexpr double kMaxRopeFreq = 0x1p64;

// x less whole numbers, times 2^64, rounded to the nearest.  (From the double's bits: frexp and ldexp
// took 2.5 us of host time for 64 frequencies.)
inline uint64_t fraction64(double x) {
    uint64_t bits;
    std::memcpy(&bits, &x, sizeof bits);
    const int exponent = static_cast<int>(bits >> 52 & 0x7ff);
    const uint64_t m = (bits & ((uint64_t{1} << 52) - 1)) | uint64_t{1} << 52;  // |x| = m 2^(exponent - 1075)
    const int down = 1011 - exponent;
    if (down > 54 || down <= -64) return 0;  // below 2^-66, subnormal or zero; or a whole number
    const uint64_t r = down > 0 ? (m + (uint64_t{1} << (down - 1))) >> down : m << -down;
    return bits >> 63 ? 0 - r : r;
}

// |f| <= kMaxRopeFreq.
inline uint64_t rope_turns(double f) {
    constexpr double kHi = 0x1.45f306dc9c883p-3, kMid = -0x1.6b01ec5417056p-57, kLo = -0x1.6447e493ad4cep-111;
    const double hi = f * kHi, mid = f * kMid;
    return fraction64(hi) + fraction64(std::fma(f, kHi, -hi)) + fraction64(mid) + fraction64(std::fma(f, kMid, -mid)) +
           fraction64(f * kLo);
}

}  // namespace fa
