// Attention over a paged cache for many query rows, over a window of keys and the sinks (paged_tc.cuh).
#include "paged_tc.cuh"

namespace jfa {

cudaError_t launch_paged_tc_window(const Paged& p, const TileShape& t, int ctas, const PagedWs& w, cudaStream_t s) {
  return launch_tc<kWindow>(p, t, ctas, w, s);
}

}  // namespace jfa
