// fixed_div.h -- division by a number that the host knows (prefill and paged cache).
#pragma once

#include <cstdint>

namespace chs {

// Exact division of a non-negative int n < 2^31 by a fixed divisor d >= 1:
// n / d == (n * m) >> (31 + l) with l = ceil(log2 d) and m = ceil(2^(31+l) / d)
// (the rounding error n*(m*d - 2^(31+l)) / (d * 2^(31+l)) stays below 1/d).
// The multiplier is made on the host; the device pays one wide multiply
// instead of a division sequence.
struct FixedDiv {
  uint32_t m, shift, d;
  __device__ __forceinline__ int div(int n) const {
    return (int)(((uint64_t)(uint32_t)n * m) >> shift);
  }
  __device__ __forceinline__ int mod(int n) const { return n - div(n) * (int)d; }
};

// Multiplier and shift for FixedDiv (exact for dividends below 2^31).
inline FixedDiv make_fixed_div(uint32_t d) {
  uint32_t l = 0;
  while ((1ull << l) < d) ++l;
  const unsigned __int128 one = 1;
  const uint64_t m = (uint64_t)(((one << (31 + l)) + d - 1) / d);
  return FixedDiv{(uint32_t)m, 31 + l, d};
}

}  // namespace chs
