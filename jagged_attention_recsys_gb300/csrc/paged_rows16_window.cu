// Attention over a paged cache for few query rows, over a window of keys and the sinks (paged_rows16.cuh).
#include "paged_rows16.cuh"

namespace jfa {

cudaError_t launch_paged_rows16_window(const Paged& p, const TileShape& t, int ctas, const PagedWs& w, cudaStream_t s) {
  return launch_rows16<kWindow>(p, t, ctas, w, s);
}

}  // namespace jfa
