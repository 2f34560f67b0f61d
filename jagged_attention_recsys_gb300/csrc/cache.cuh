// Device parts of the calls that write to or read from a paged cache: where a token's rows lie.
#pragma once

#include "paged.cuh"

namespace jfa {

// The sequence of new token t: the guess serves batches of equal lengths (one token each in
// a serving step) with one look, otherwise a binary search.  Any contents of offs end it,
// with b inside the batch.
__device__ __forceinline__ int find_sequence(const Paged& p, int64_t t) {
  const int64_t g = t * p.batch / p.total_q;
  if (__ldg(p.offs + g) <= t && t < __ldg(p.offs + g + 1)) return (int)g;
  int64_t lo = 0, hi = p.batch - 1;
  while (lo < hi) {  // the first b with offs[b + 1] > t
    const int64_t m = (lo + hi) >> 1;
    if (__ldg(p.offs + m + 1) > t) hi = m;
    else lo = m + 1;
  }
  return (int)lo;
}

// Cache position of new token t of sequence b; -1: it has none (before the cache's start, or
// the arrays do not describe a batch, which is recorded).
__device__ __forceinline__ int token_position(const Paged& p, int64_t t, int b, int* status) {
  const int64_t lo = __ldg(p.offs + b), hi = __ldg(p.offs + b + 1), len = __ldg(p.lens + b);
  if (t < lo || t >= hi || hi > p.total_q || len < 0 || len > ((int64_t)p.width << p.page_shift)) {
    atomicExch(status, (int)JFA_ERR_BAD_OFFSETS);
    return -1;
  }
  const int64_t pos = len - (hi - t);
  return pos < 0 ? -1 : (int)pos;
}

// The whole batch's description, once per call without a plan, cut over the grid.
__device__ __forceinline__ void check_batch(const Paged& p, PagedHeader* hdr) {
  const int64_t most = (int64_t)p.width << p.page_shift;
  for (int64_t b = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; b < p.batch; b += (int64_t)gridDim.x * blockDim.x) {
    const int64_t lo = __ldg(p.offs + b), hi = __ldg(p.offs + b + 1), len = __ldg(p.lens + b);
    if (hi < lo || (b == 0 && lo != 0) || (b == p.batch - 1 && hi != p.total_q) || len < 0 || len > most)
      atomicExch(&hdr->status, (int)JFA_ERR_BAD_OFFSETS);
  }
}

}  // namespace jfa
