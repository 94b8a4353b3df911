// What the dense attention kernels share: a row's results from its softmax state, and where
// the parts of a unit lie that several CTAs worked on.
#pragma once

#include "rkv_flat.cuh"

namespace rkv {

// Running maximum of a row that saw nothing: no logit lies below it, and differences with
// it are never inf - inf.
constexpr float kNoMax = -3.402823466e+38f;
constexpr float kLn2 = 0.6931471805599453f;

// A row's results from its maximum m and sum l.  l = 0: it saw nothing, and nothing is what it
// weighs; a NaN among its logits has left l a NaN, which stays one.
__device__ __forceinline__ float inverse_of(float l) { return l == 0.f ? 0.f : 1.f / l; }
__device__ __forceinline__ float lse_of(float m, float l) { return l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2; }

// Where the parts of a split unit lie: CTA c's at slot 2 c, but the first CTA's at 2 c + 1
// when its share began before the unit.
struct PartSlots {
  int c0, c1, late;
  __device__ __forceinline__ PartSlots(long long ux, int per, int pad, long long total, int N)
      : c0(flat_cta(ux + pad, total, N)), c1(flat_cta(ux + per - 1, total, N)), late(flat_first(total, c0, N) < ux) {}
  __device__ __forceinline__ size_t operator[](int c) const { return 2 * (size_t)c + (c == c0 ? late : 0); }
};

}  // namespace rkv
