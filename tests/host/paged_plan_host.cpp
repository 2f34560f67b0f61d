// The paged attention's work plan (csrc/paged.cuh) on the host: cuts, walks over shares and joins of
// cut tiles, as the kernels run them, with every index they would use checked against the arrays.
#include <algorithm>
#include <cstdint>

// what the device code names and this file does not call
struct HostDim3 { int x, y, z; };
static HostDim3 threadIdx, blockIdx;
template <typename T> static T __ldg(const T* x) { return *x; }
template <typename T> static T __shfl_up_sync(unsigned, T x, int) { return x; }
template <typename T> static T atomicExch(T*, T x) { return x; }
template <typename T> static T atomicCAS(T* at, T, T) { return *at; }
static void __syncthreads() {}
static int __syncthreads_or(int x) { return x; }
static uint32_t __float_as_uint(float) { return 0; }
static float __uint_as_float(uint32_t) { return 0; }
using std::max;
using std::min;

#include "paged.cuh"

using namespace jfa;

namespace {
Paged request(const int64_t* x, const int64_t* offs, const int64_t* lens) {
  Paged p{};
  p.offs = offs;
  p.lens = lens;
  p.batch = x[0];
  p.total_q = x[1];
  p.width = (int)x[2];
  p.page_shift = (int)x[3];
  p.heads_q = (int)x[4];
  p.heads_k = (int)x[5];
  p.group = p.heads_q / p.heads_k;
  p.causal = (int)x[6];
  return p;
}
TileShape shape(const int64_t* x) {
  TileShape t{};
  t.rows = (int)x[7];
  t.tokens = (int)x[8];
  t.gsub = (int)x[9];
  t.nsub = (int)x[10];
  t.keys = (int)x[11];
  t.overhead = (int)x[12];
  t.share = (int)x[13];
  return t;
}
}  // namespace

extern "C" {

// The plan of a request, [ctas + 1] places of four ints; false: no batch.
int plan(const int64_t* x, const int64_t* offs, const int64_t* lens, int ctas, int64_t* cum, int* pos) {
  const Paged p = request(x, offs, lens);
  const TileShape t = shape(x);
  bool bad = false;
  cum[0] = 0;
  for (int64_t b = 0; b < p.batch; ++b) {
    const int64_t c = checked_cost(p, t, b);
    bad |= c < 0;
    cum[b + 1] = cum[b] + (c < 0 ? 0 : c);
  }
  for (int c = 0; c <= ctas; ++c) ((PagedPos*)pos)[c] = paged_cut(p, t, ctas, c, cum, cum[p.batch], bad);
  return !bad;
}

// All CTAs of a request on the plan in pos.  seen [T * heads_q] counts the times that a row is
// computed: blocks of keys as they are walked, and once where the row's result is written (whole
// tiles in the walk, others by the join); returns the number of indexes outside the arrays.
int64_t run(const int64_t* x, const int64_t* offs, const int64_t* lens, int ctas, const int* pos, int64_t* blocks,
            int64_t* written) {
  const Paged p = request(x, offs, lens);
  const TileShape t = shape(x);
  PagedWs w{};
  w.pos = (PagedPos*)const_cast<int*>(pos);
  int64_t outside = 0;
  auto row = [&](int q0, int tok, int head, int64_t n, int64_t* count) {
    if (q0 < 0 || tok < 0 || (int64_t)q0 + tok >= p.total_q || head < 0 || head >= p.heads_q) ++outside;
    else count[((int64_t)q0 + tok) * p.heads_q + head] += n;
  };
  for (int c = 0; c < ctas; ++c) {
    const PagedPos share[2] = {paged_pos(p, t, w, c), paged_pos(p, t, w, c + 1)};
    PagedWalk walk;
    walk.init(share);
    PagedSegment g;
    while (walk.next(p, t, g)) {
      if (g.b < 0 || g.b >= p.batch) ++outside;
      if (g.blk0 < 0 || g.blk1 < g.blk0 || (int64_t)g.blk1 * t.keys >= (int64_t)g.seq.lk + t.keys) ++outside;
      if (g.seq.lk > ((int64_t)p.width << p.page_shift)) ++outside;
      for (int r = 0; r < t.rows; ++r) {
        const int tok = g.tile * t.tokens + r / t.gsub, gh = g.unit % t.nsub * t.gsub + r % t.gsub;
        if (tok >= g.seq.lq || gh >= p.group) continue;
        const int head = g.unit / t.nsub * p.group + gh;
        row(g.seq.q0, tok, head, g.blk1 - g.blk0, blocks);
        if (g.slot < 0) row(g.seq.q0, tok, head, 1, written);
      }
    }
    PagedCutTile cut;
    if (!cut.find(p, t, w, ctas, c)) continue;
    if (cut.last >= ctas) ++outside;
    for (int r = 0; r < t.rows; ++r) {
      int tok, head;
      if (cut.row(p, t, r, tok, head)) row(cut.seq.q0, tok, head, 1, written);
    }
  }
  return outside;
}

}  // extern "C"
