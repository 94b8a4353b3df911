// The key interval of the histogram selects, in plain integer arithmetic: a round lays
// kTkBins bins of 2^shift keys over [lo, hi] and goes on inside one of them.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define RKV_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define RKV_HOST_DEVICE inline
#endif

namespace rkv {

constexpr int kTkBins = 1024;

// The smallest shift with (range >> shift) < kTkBins, or one more.
RKV_HOST_DEVICE int tk_shift(uint32_t range) {
#ifdef __CUDA_ARCH__
  const int zeros = __clz((int)range);
#else
  const int zeros = range ? __builtin_clz(range) : 32;
#endif
  return range < (uint32_t)kTkBins ? 0 : (32 - zeros) - 10;
}

// The last key of the bin that starts at nlo, inside [nlo, hi].  The bin's end may lie
// past 2^32 (a NaN's key is the largest there is), so the width is cut, not the end.
RKV_HOST_DEVICE uint32_t tk_upper(uint32_t nlo, uint32_t hi, int shift) {
  const uint32_t width = (1u << shift) - 1u, left = hi - nlo;
  return nlo + (left < width ? left : width);
}

}  // namespace rkv
