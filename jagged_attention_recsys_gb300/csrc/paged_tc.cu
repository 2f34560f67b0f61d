// Attention over a paged cache for many query rows, over all keys (paged_tc.cuh).
#include "paged_tc.cuh"

namespace jfa {

cudaError_t launch_paged_tc(const Paged& p, const TileShape& t, int ctas, const PagedWs& w, cudaStream_t s) {
  return launch_tc<kAll>(p, t, ctas, w, s);
}

}  // namespace jfa
