// divide.h -- divisions by numbers that are the same for a whole launch, as a
// multiplication by what the host works out once.  (It includes nothing of HIP's, so
// that a host program can check it: include it after seq.h.)
#pragma once

#include <cstdint>

namespace recis {

// x / d for x * d < 2^32.
struct Div {
  unsigned d, mul;
};
inline Div div_by(int64_t d) { return Div{(unsigned)d, d > 1 ? (unsigned)(((1ull << 32) + d - 1) / d) : 0}; }
__device__ __forceinline__ unsigned divided(unsigned x, Div v) { return v.d == 1 ? x : __umulhi(x, v.mul); }

// x / d for 0 <= x < 2^31, without a division: the compiler's takes some 30 dependent
// instructions, and a block of few tiles does a dozen before its first load.
struct Quick {
  int d, shift;
  unsigned mul, one;
  Quick() = default;
  explicit Quick(int64_t by) : d((int)by), shift(0), mul(0), one(~0u) {
    if (by <= 1) return;
    int bits = 0;
    while ((1ll << bits) < by) ++bits;
    mul = (unsigned)((1ull << (31 + bits)) / by + 1);
    shift = bits - 1;
    one = 0;
  }
};
__device__ __forceinline__ int divided(int x, const Quick& q) {
  return (int)((__umulhi((unsigned)x, q.mul) + ((unsigned)x & q.one)) >> q.shift);
}

}  // namespace recis
