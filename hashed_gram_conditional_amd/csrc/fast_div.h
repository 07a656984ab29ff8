// Division of a 64-bit index by a fixed divisor with one high multiply: with
// M = floor((2^64 - 1) / d) + 1 = (2^64 + e) / d and 0 <= e < d, hi64(g M) is
// floor(g / d) for every g with g d < 2^64, which the callers' size limits keep.
// d = 1 has no such M and returns g.
#pragma once

#include <stdint.h>

#include <hip/hip_runtime.h>

struct EngramFastDiv {
  int64_t d;
  uint64_t magic;
  explicit EngramFastDiv(int64_t divisor)
      : d(divisor), magic(divisor > 1 ? UINT64_MAX / (uint64_t)divisor + 1 : 0) {}
  __device__ __forceinline__ int64_t div(int64_t g) const {
    return d == 1 ? g : (int64_t)__umul64hi((uint64_t)g, magic);
  }
};
