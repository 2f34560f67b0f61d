// How the two phases of attention over a shared prefix meet.
#pragma once

#include <cuda_runtime.h>

namespace jfa {

// How a row of phase 2 of a shared prefix joins what phase 1 left of it: its own unnormalised sums
// times `own`, and the prior result times `prior`; lse is the natural log of the whole sum.
struct PagedJoin {
  float own, prior, lse;
};
// m: maximum in log2 units, l: sum of exp2(x - m); prior: log2 of phase 1's sum
__device__ __forceinline__ PagedJoin paged_join_prior(float m, float l, float prior) {
  const float top = fmaxf(m, prior), ref = top == -INFINITY ? 0.f : top;
  const float f = exp2f(m - ref), g = exp2f(prior - ref);
  const float s = fmaf(l, f, g), inv = s > 0.f ? 1.f / s : (s == 0.f ? 0.f : s);  // no key: 0; NaN stays NaN
  return PagedJoin{f * inv, g * inv, s == 0.f ? -INFINITY : (ref + log2f(s)) * 0.6931471805599453f};
}

}  // namespace jfa
