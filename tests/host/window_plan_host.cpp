// The paged attention's work plan under a window with sinks, and over groups of sequences
// (csrc/paged.cuh), on the host: which keys every query row meets, and which it looks up.
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

// x: batch, total_q, width, page_shift, heads_q, heads_k, causal, window, sinks, seqs, then the seven
// numbers of a tile's shape; groups may be null.  Plans the request and walks every CTA's share.
// met [T][keys]: how often a row of a token's first head met a key that it sees; written [T * heads_q].
// Returns the number of mistakes: indexes outside the arrays, blocks out of order, keys that a row sees
// in a box that is not looked up.
extern "C" int64_t walk(const int64_t* x, const int64_t* offs, const int64_t* lens, const int64_t* groups, int ctas,
                        int64_t keys, int32_t* met, int64_t* written, int64_t* blocks) {
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
  p.seqs = x[9];
  p.groups = groups;
  TileShape t{};
  t.rows = (int)x[10];
  t.tokens = (int)x[11];
  t.gsub = (int)x[12];
  t.nsub = (int)x[13];
  t.keys = (int)x[14];
  t.overhead = (int)x[15];
  t.share = (int)x[16];
  int64_t* cum = new int64_t[p.batch + 1];
  PagedPos* pos = new PagedPos[ctas + 1];
  bool bad = false;
  cum[0] = 0;
  for (int64_t b = 0; b < p.batch; ++b) {
    const int64_t c = checked_cost(p, t, b);
    bad |= c < 0;
    cum[b + 1] = cum[b] + (c < 0 ? 0 : c);
  }
  for (int c = 0; c <= ctas; ++c) pos[c] = paged_cut(p, t, ctas, c, cum, cum[p.batch], bad);
  PagedWs w{};
  w.pos = pos;
  int64_t wrong = 0, most = 0;
  const int box = min(1 << p.page_shift, t.keys);
  for (int c = 0; c < ctas; ++c) {
    const PagedPos share[2] = {paged_pos(p, t, w, c), paged_pos(p, t, w, c + 1)};
    PagedWalk walk;
    walk.init(share);
    PagedSegment g;
    int64_t mine = 0;
    while (walk.next(p, t, g)) {
      mine += g.blk1 - g.blk0;
      int before = -1;
      for (int i = g.blk0; i < g.blk1; ++i) {
        const int real = g.span.block(i), k0 = real * t.keys;
        wrong += real <= before || k0 >= g.seq.lk || (i >= g.span.ns && real < g.span.first);
        before = real;
        for (int r = 0; r < t.rows; r += t.gsub) {
          const int tok = g.tile * t.tokens + r / t.gsub;
          if (tok >= g.seq.lq || g.unit != 0) continue;
          const int64_t at = g.seq.off + tok;
          for (int k = k0; k < min(k0 + t.keys, g.seq.lk); ++k) {
            const bool sees = !p.causal || (k <= at && (p.window == 0 || at - k < p.window || k < p.sinks));
            if (!sees) continue;
            ++met[((int64_t)g.seq.q0 + tok) * keys + k];
            const int b0 = k / box * box;  // the box that the key is loaded with
            wrong += p.window > 0 && !(paged_sees(p, g.span.low, b0) || b0 + box > g.span.low);
            wrong += p.window > 0 && !paged_sees(p, g.span.low, k);
          }
        }
      }
      for (int r = 0; r < t.rows; ++r) {
        const int tok = g.tile * t.tokens + r / t.gsub, gh = g.unit % t.nsub * t.gsub + r % t.gsub;
        if (tok >= g.seq.lq || gh >= p.group || g.slot >= 0) continue;
        ++written[((int64_t)g.seq.q0 + tok) * p.heads_q + g.unit / t.nsub * p.group + gh];
      }
    }
    most = max(most, mine);
    PagedCutTile cut;
    if (!cut.find(p, t, w, ctas, c)) continue;
    for (int r = 0; r < t.rows; ++r) {
      int tok, head;
      if (cut.row(p, t, r, tok, head)) ++written[((int64_t)cut.seq.q0 + tok) * p.heads_q + head];
    }
  }
  *blocks = most;  // of the busiest CTA
  delete[] cum;
  delete[] pos;
  return bad ? -1 : wrong;
}
