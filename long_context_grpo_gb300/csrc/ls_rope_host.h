// Host side of the rotary angles: inverse frequencies to fixed-point turns.
#pragma once

#include <cmath>

#include "ls_ops.h"

namespace ls {

// Fills a->turns, a->rot and a->factor; false if the factor is not finite or a
// frequency is not within +-2^20 a token.
// inv_freq / 2 pi is formed as a product of two doubles with its rounding error (fma), so the
// fraction is right to about 2^-64 and position * fraction to 2^-33 turns at position 2^31.
inline bool rope_turns(const double* inv_freq, int rot_dim, double factor, RopeArgs* a) {
  // 1 / 2 pi as an unevaluated sum of two doubles
  constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;
  if (!std::isfinite(factor)) return false;
  for (int i = 0; i < rot_dim / 2; ++i) {
    const double f = std::fabs(inv_freq[i]);
    if (!(f <= 1048576.0)) return false;
    const double p = f * kHi;
    const double e = std::fma(f, kHi, -p) + f * kLo;
    // p modulo 1 is exact (p >= 0: a negative frequency turns the other way); then both parts in units of 2^-64 modulo 2^64
    const double fp = p - std::floor(p);
    // fp < 1 has at most 53 significant bits: top 32 bits, then the rest
    const double top = std::floor(std::ldexp(fp, 32));
    const double rest = std::ldexp(fp, 32) - top;
    uint64_t u = (static_cast<uint64_t>(top) << 32) + static_cast<uint64_t>(std::ldexp(rest, 32));
    u += static_cast<uint64_t>(static_cast<int64_t>(std::nearbyint(std::ldexp(e, 64))));
    a->turns[i] = inv_freq[i] < 0.0 ? 0u - u : u;
  }
  a->rot = rot_dim;
  a->factor = static_cast<float>(factor);
  return true;
}

}  // namespace ls
