// Host code: a frequency in radians per position step as a 64-bit fraction of a turn.
//
// Fixed point throughout: |f| = m 2^e with a 53-bit integer m, times 1 / (2 pi) held to 192 bits,
// whole turns dropped (they do not show at integer positions) and rounded to 64 bits. Below 2^64
// radians the product is off by less than 2^-128 of a turn before that rounding, so the fraction is
// off by 2^-65 of a turn, and its product with any 32-bit position by 2^-34. (A quotient in double
// precision, however it is reduced, has 53 good bits, fewer for every bit of whole turns: at a
// position near 2^31 that is 2^-22 of a turn for 7 radians a step, 2^-12 for 10^4.)
#pragma once
#include <cstdint>
#include <cstring>

namespace xs {

// Whether turns_per_step holds: finite and below 2^64 in magnitude.
inline bool turns_fit(double f) { return f > -0x1p64 && f < 0x1p64; }

inline unsigned long long turns_per_step(double f) {
  // 2^192 / (2 pi), least significant word first.
  static const uint64_t inverse[3] = {0x36d8a5664f10e410ull, 0x7f09d5f47d4d3770ull,
                                      0x28be60db9391054aull};
  uint64_t bits;
  std::memcpy(&bits, &f, 8);
  const int exponent = static_cast<int>(bits >> 52 & 0x7ff);
  uint64_t m = bits & 0xfffffffffffffull;
  if (exponent != 0) m |= 1ull << 52;
  const int e = (exponent != 0 ? exponent : 1) - 1075;   // |f| = m 2^e, e <= 11
  uint64_t p[6] = {0, 0, 0, 0, 0, 0};                    // m 2^192 / (2 pi), below 2^243
  uint64_t carry = 0;
  for (int i = 0; i < 3; ++i) {
    const unsigned __int128 t = static_cast<unsigned __int128>(m) * inverse[i] + carry;
    p[i] = static_cast<uint64_t>(t);
    carry = static_cast<uint64_t>(t >> 64);
  }
  p[3] = carry;
  // The 64 bits of weights 2^-1 to 2^-64: p 2^(e - 128), rounded by the bit below them.
  const int down = 128 - e;   // 117 at least
  if (down > 255) return 0;
  const int word = down / 64, shift = down % 64;
  const uint64_t value = shift == 0 ? p[word] : p[word] >> shift | p[word + 1] << (64 - shift);
  const uint64_t half = p[(down - 1) / 64] >> ((down - 1) % 64) & 1;
  const uint64_t turn = value + half;   // past the last unit: a whole turn, which is none
  return bits >> 63 ? 0 - turn : turn;
}

}  // namespace xs
