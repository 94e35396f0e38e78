#pragma once

#include <stdint.h>

namespace muon {

// Division of 31-bit numbers by a number of [1, 2^31) fixed per launch (a multiplication and a
// shift): with s = ceil(log2 d) and m = floor(2^32 (2^s - d) / d) + 1, n / d is
// (umulhi(m, n) + n) >> s for every n < 2^31 (Granlund and Montgomery, "Division by invariant
// integers using multiplication", 1994).
struct Div {
  uint32_t d, m, s;
  explicit Div(uint32_t d_) : d(d_), m(0), s(0) {
    while (s < 31 && (1u << s) < d) ++s;
    m = (uint32_t)(((1ull << 32) * ((1ull << s) - d)) / d + 1);
  }
  __device__ __forceinline__ uint32_t quot(uint32_t n) const { return (__umulhi(m, n) + n) >> s; }
};

}  // namespace muon
