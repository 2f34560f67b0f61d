// Attention over a paged cache for few query rows, over a shared prefix: both phases (paged_rows16.cuh).
#include "paged_rows16.cuh"

namespace jfa {

cudaError_t launch_paged_rows16_shared(const Paged& p, const TileShape& t, int ctas, const PagedWs& w, cudaStream_t s) {
  return launch_rows16<kShared>(p, t, ctas, w, s);
}

}  // namespace jfa
