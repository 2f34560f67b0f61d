// The parts of a cut tile (csrc/paged.cuh) on the host: what the join looks up, a warp's 32 lanes at a time, against the
// parts that the walks over the CTAs' shares leave.
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

// x: batch, total_q, width, page_shift, heads_q, heads_k, causal, window, sinks, then the seven numbers of a
// tile's shape.  spread: parts that cut tiles may have, counts [spread + 1] how many have each number.
// Returns the number of mistakes.
extern "C" int64_t parts(const int64_t* x, const int64_t* offs, const int64_t* lens, int ctas, int spread, int64_t* counts) {
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
  p.window = (int)x[7];
  p.sinks = (int)x[8];
  TileShape t{};
  t.rows = (int)x[9];
  t.tokens = (int)x[10];
  t.gsub = (int)x[11];
  t.nsub = (int)x[12];
  t.keys = (int)x[13];
  t.overhead = (int)x[14];
  t.share = (int)x[15];
  int64_t* cum = new int64_t[p.batch + 1];
  PagedPos* pos = new PagedPos[ctas + 1];
  cum[0] = 0;
  for (int64_t b = 0; b < p.batch; ++b) cum[b + 1] = cum[b] + checked_cost(p, t, b);
  for (int c = 0; c <= ctas; ++c) pos[c] = paged_cut(p, t, ctas, c, cum, cum[p.batch], false);
  PagedWs w{};
  w.pos = pos;
  // what the walks leave: of every CTA, its segments that are parts of tiles
  struct Part { int b, unit, tile, blocks, slot; };
  Part* left = new Part[2 * ctas]();
  int64_t wrong = 0, found = 0, joined = 0;
  for (int c = 0; c < ctas; ++c) {
    const PagedPos share[2] = {paged_pos(p, t, w, c), paged_pos(p, t, w, c + 1)};
    PagedWalk walk;
    walk.init(share);
    PagedSegment g;
    while (walk.next(p, t, g)) {
      if (g.slot < 0) continue;
      wrong += left[2 * c + g.slot].blocks != 0;  // a slot holds one part
      left[2 * c + g.slot] = Part{g.b, g.unit, g.tile, g.blk1 - g.blk0, g.slot};
      found += g.blk1 > g.blk0;
    }
  }
  for (int c = 0; c < ctas; ++c) {
    PagedCutTile warp, thread;
    // a warp's lanes all look, whatever the first of them find
    auto lanes = [](auto f) {
      unsigned on = 0;
      for (int i = 0; i < 32; ++i) on |= (unsigned)(f(i) ? 1 : 0) << i;
      int n = 0;
      while (n < 32 && (on >> n & 1)) ++n;
      return n;
    };
    const bool is = warp.find(p, t, w, ctas, c, lanes);
    wrong += is != thread.find(p, t, w, ctas, c);
    if (!is) continue;
    wrong += warp.last != thread.last || warp.last >= ctas;
    int n = 0;
    for (int i0 = c; i0 <= warp.last; i0 += 32)
      for (int i = i0; i < i0 + 32; ++i) {
        if (!warp.part(p, t, w, c, i)) continue;
        const Part& at = left[2 * i + (i == c ? 1 : 0)];
        wrong += i >= ctas || at.blocks == 0 || at.b != warp.end.b || at.unit != warp.end.unit || at.tile != warp.end.tile;
        ++n;
      }
    joined += n;
    if (n > spread) ++wrong;
    else ++counts[n];
  }
  wrong += joined != found;  // every part is a tile's, once
  delete[] cum;
  delete[] pos;
  delete[] left;
  return wrong;
}
