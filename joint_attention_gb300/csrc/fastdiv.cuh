// fastdiv.cuh — division by a number that a launch fixes.
#pragma once
#include <cstdint>

namespace jattn {

// Division of n < 2^31 by a fixed d >= 1 through a multiply-high: with
// l = ceil(log2 d) and m = floor(2^32 (2^l - d) / d) + 1, n / d =
// (mulhi(n, m) + n) >> l (the round-up method for invariant divisors, as in
// Hacker's Delight, ch. 10); mulhi(n, m) + n < 2^32 for n < 2^31.
struct DivU31 {
  uint32_t m, l;
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return (__umulhi(n, m) + n) >> l; }
};
inline DivU31 make_div_u31(uint32_t d) {
  uint32_t l = 0;
  while ((uint64_t{1} << l) < d) ++l;
  DivU31 r;
  r.l = l;
  r.m = static_cast<uint32_t>(((uint64_t{1} << 32) * ((uint64_t{1} << l) - d)) / d + 1);
  return r;
}

}  // namespace jattn
