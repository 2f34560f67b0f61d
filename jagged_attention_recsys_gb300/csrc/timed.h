// Event timing of one kernel launch (jfa_profile_*), shared by the files that hold C entry
// points.
#pragma once

#include <cuda_runtime.h>

namespace jfa {

// Records events around the launches of its scope when profiling is on.
struct Timed {
  int kind;
  cudaStream_t s;
  cudaEvent_t a = nullptr, b = nullptr;
  Timed(int k, cudaStream_t st);
  ~Timed();
  Timed(const Timed&) = delete;
  Timed& operator=(const Timed&) = delete;
};

}  // namespace jfa
