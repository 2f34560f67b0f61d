// Device parts that the kernels over a paged cache share: the walk over a CTA's share of the
// work, page addresses, MXFP8 conversions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "internal.h"
#include "serve.h"

namespace jfa {

// One sequence of a request.
struct PagedSeq {
  int q0, lq, lk, tiles;
  int64_t off;  // position of its first new token: lk - lq (negative: tokens before the cache)
};
// The new tokens [x, y) of sequence b; [-1, -1): its group is not one of the batch's.
struct PagedBounds {
  int64_t x, y;
};
template <int MODE = kAny>
__device__ __forceinline__ PagedBounds paged_bounds(const Paged& p, int64_t b) {
  if (!serves_shared(MODE) || !p.groups) return PagedBounds{__ldg(p.offs + b), __ldg(p.offs + b + 1)};
  const int64_t s = __ldg(p.groups + b), n = __ldg(p.groups + b + 1);
  if (s < 0 || n < s || n > p.seqs || (b == 0 && s != 0) || (b == p.batch - 1 && n != p.seqs)) return PagedBounds{-1, -1};
  return PagedBounds{__ldg(p.offs + s), __ldg(p.offs + n)};
}
// Whether a sequence of so many own keys is the short kernel's.
template <int MODE = kAny>
__device__ __forceinline__ bool is_few(const Paged& p, int64_t keys) {
  return serves_shared(MODE) && p.few > 0 && keys <= p.few;
}
template <int MODE = kAny>
__device__ __forceinline__ PagedSeq paged_seq(const Paged& p, const TileShape& t, int b) {
  PagedSeq s;
  const PagedBounds n = paged_bounds<MODE>(p, b);
  const int64_t a = n.x, e = n.y, l = __ldg(p.lens + b);
  // (what a plan was not made for and is no batch either has no tokens)
  const bool ok = a >= 0 && e >= a && e <= p.total_q && l >= 0 && l <= ((int64_t)p.width << p.page_shift);
  s.q0 = (int)a;
  s.lq = ok && !is_few<MODE>(p, l) ? (int)(e - a) : 0;
  s.lk = (int)l;
  s.off = l - (e - a);
  s.tiles = (s.lq + t.tokens - 1) / t.tokens;
  return s;
}
// Keys the last row of a tile sees, and the blocks that hold them.
__device__ __forceinline__ int tile_keys(const Paged& p, const TileShape& t, const PagedSeq& s, int tile) {
  if (!p.causal) return s.lk;
  const int64_t last = s.off + min((int64_t)(tile + 1) * t.tokens, (int64_t)s.lq);
  return last < 0 ? 0 : (int)last;
}

// The blocks of keys that a tile meets, by number: `nb` of them, the first `ns` from the cache's
// start (they hold the sinks), the others from block `first` on.  Without a window ns = first = 0.
struct PagedSpan {
  int nb, ns, first;
  int low;  // position of the first key of the window of the tile's first row
  __device__ __forceinline__ int block(int i) const { return i < ns ? i : i - ns + first; }
};
// off: position of the sequence's first new token, end: keys that the tile's last row sees
template <int MODE = kAny>
__device__ __forceinline__ PagedSpan paged_span(const Paged& p, const TileShape& t, int64_t off, int end, int tile) {
  PagedSpan s;
  s.nb = (end + t.keys - 1) / t.keys;
  s.ns = s.first = s.low = 0;
  if (serves_windows(MODE) && p.window > 0) {
    const int64_t low = off + (int64_t)tile * t.tokens - p.window + 1;
    s.low = (int)min(max((int64_t)0, low), (int64_t)end);
    s.first = min(s.low / t.keys, max(s.nb - 1, 0));
    s.ns = min(p.sinks / t.keys + (p.sinks % t.keys != 0), s.first);
    s.nb -= s.first - s.ns;
  }
  return s;
}
// Whether any row of the tile may see the key at position x (that its last row sees)
__device__ __forceinline__ bool paged_sees(const Paged& p, int low, int x) { return x >= low || x < p.sinks; }

// ------------------------------------------------------------------- cutting the work
template <int MODE = kAny>
struct SeqCost {
  int64_t off, lk, tiles, s, over;
  int64_t most;  // a window: keys that a tile meets at most, with its sinks and part of a block
  int causal;
  // cost of the tiles in front of tile t, t <= tiles - 1
  __device__ int64_t before(int64_t t) const {
    if (!causal) return t * (over + lk);
    // tile u sees max(0, off + (u + 1) s) keys, and meets at most `most`
    int64_t u0 = off < 0 ? (-off) / s : 0;  // tiles that see nothing
    if (u0 > t) u0 = t;
    int64_t u1 = t;  // tiles that meet all that they see
    if constexpr (serves_windows(MODE)) {
      if (most < (int64_t)1 << 40) u1 = most > off ? (most - off) / s : 0;
      if (u1 > t) u1 = t;
      if (u1 < u0) u1 = u0;
    }
    const int64_t c = t * over + (u1 - u0) * off + s * ((u1 * (u1 + 1) - u0 * (u0 + 1)) / 2);
    return serves_windows(MODE) && u1 < t ? c + (t - u1) * most : c;
  }
  __device__ int64_t total() const {
    return tiles == 0 ? 0 : before(tiles - 1) + over + (serves_windows(MODE) ? min(lk, most) : lk);
  }
};
template <int MODE = kAny>
__device__ __forceinline__ SeqCost<MODE> seq_cost(const Paged& p, const TileShape& t, int64_t lq, int64_t lk) {
  SeqCost<MODE> c;
  c.off = lk - lq;
  c.lk = lk;
  c.s = t.tokens;
  c.tiles = (lq + t.tokens - 1) / t.tokens;
  c.over = t.overhead;
  c.most = (int64_t)1 << 40;
  if (serves_windows(MODE) && p.window > 0)
    c.most = (int64_t)p.window + t.tokens + t.keys + ((int64_t)p.sinks + t.keys - 1) / t.keys * t.keys;
  c.causal = p.causal;
  return c;
}

// Cost of sequence b in all its units, or -1: the arrays do not describe a batch.
template <int MODE = kAny>
__device__ __forceinline__ int64_t checked_cost(const Paged& p, const TileShape& t, int64_t b) {
  const PagedBounds n = paged_bounds<MODE>(p, b);
  const int64_t a = n.x, e = n.y, lk = __ldg(p.lens + b);
  if (a < 0 || e < a || e > p.total_q || lk < 0 || lk > ((int64_t)p.width << p.page_shift) || (b == 0 && a != 0) ||
      (b == p.batch - 1 && e != p.total_q))
    return -1;
  if (is_few<MODE>(p, lk)) return 0;
  return (int64_t)p.heads_k * t.nsub * seq_cost<MODE>(p, t, e - a, lk).total();
}

// Where CTA c of `ctas` begins (c = ctas: the end); cum[b]: cost of the sequences before b, in all
// W = cum[B].  Little work goes to fewer CTAs, so that a share is worth its tile's fixed cost.
template <int MODE = kAny>
__device__ __forceinline__ PagedPos paged_cut(const Paged& p, const TileShape& t, int ctas, int c, const int64_t* cum,
                                              int64_t W, bool bad) {
  const int64_t n = max((int64_t)1, min((int64_t)ctas, W / t.share));
  PagedPos r{(int)p.batch, 0, 0, 0};  // the end; a bad batch begins there
  const int64_t x = W / n * c + W % n * c / n;
  if (bad || c >= n || x >= W) return r;
  int64_t lo = 0, hi = p.batch - 1;
  while (lo < hi) {  // the first b with cum[b + 1] > x
    const int64_t m = (lo + hi) >> 1;
    if (cum[m + 1] > x) hi = m;
    else lo = m + 1;
  }
  const PagedBounds bounds = paged_bounds<MODE>(p, lo);
  const SeqCost<MODE> sc = seq_cost<MODE>(p, t, bounds.y - bounds.x, __ldg(p.lens + lo));
  const int64_t S = sc.total(), y = x - cum[lo];
  const int64_t unit = y / S, z = y - unit * S;
  int64_t tl = 0, th = sc.tiles - 1;
  while (tl < th) {  // the last tile with before(tile) <= z
    const int64_t m = (tl + th + 1) >> 1;
    if (sc.before(m) <= z) tl = m;
    else th = m - 1;
  }
  const int64_t vis = tl == sc.tiles - 1 || !sc.causal ? sc.lk : max((int64_t)0, sc.off + (tl + 1) * sc.s);
  const int64_t nb = paged_span<MODE>(p, t, sc.off, (int)vis, (int)tl).nb;
  const int64_t d = z - sc.before(tl) - sc.over;
  const int64_t blk = d <= 0 ? 0 : (d + t.keys / 2) / t.keys;
  r.b = (int)lo;
  r.unit = (int)unit;
  r.tile = (int)tl;
  r.blk = (int)blk;
  if (blk > 0 && blk >= nb) {  // the cut falls on the tile's end
    r.tile = (int)tl + 1;
    r.blk = 0;
  }
  return r;
}

// Where CTA c's share begins in the workspace's plan.  A plan of another request may name what this one
// does not have; such a place is the end, so that whatever the plan, only this request's arrays are met.
__device__ __forceinline__ PagedPos paged_pos(const Paged& p, const TileShape& t, const PagedWs& w, int c) {
  const PagedPos x = w.pos[c];
  if ((x.b | x.unit | x.tile | x.blk) < 0 || x.b >= p.batch || x.unit >= p.heads_k * t.nsub)
    return PagedPos{(int)p.batch, 0, 0, 0};
  return x;
}

// Whether the first phase found the batch invalid: the second then computes nothing either.
__device__ __forceinline__ bool prior_failed(const Paged& p) {
  return *(const volatile int*)p.prior_status == (int)JFA_ERR_BAD_OFFSETS;
}

// A CTA's share, [pos[0], pos[1]), in shared memory.  With w.ctas > 0 there is no plan (a batch of
// at most kPlanInCta sequences): every CTA scans the batch by itself, in `scratch` (at least
// kPlanScratch bytes), and leaves its cut and its status in the workspace for the join.  All
// threads of the CTA call it (at least 128), ahead of any other use of scratch.  Returns
// where the CTA records errors.
template <int MODE = kAny>
__device__ __forceinline__ int* paged_share(const Paged& p, const TileShape& t, const PagedWs& w, PagedPos* pos,
                                            void* scratch) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = blockIdx.x;
  if (w.ctas == 0) {
    if (tid < 2) pos[tid] = paged_pos(p, t, w, c + tid);
    __syncthreads();
    return &w.hdr->status;
  }
  constexpr int kThreads = 128, kEach = kPlanInCta / kThreads;  // threads that scan, sequences of each
  int64_t* cum = (int64_t*)scratch;      // [kPlanInCta + 1]
  int64_t* sums = cum + kPlanInCta + 1;  // [kThreads / 32]
  int64_t cost[kEach], x = 0;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int b = tid * kEach + i;
    cost[i] = tid < kThreads && b < p.batch ? checked_cost<MODE>(p, t, b) : 0;
    bad |= cost[i] < 0;
    x += cost[i];
  }
  if (serves_shared(MODE) && p.phase == 2 && tid == 0) bad |= prior_failed(p);
  bad = __syncthreads_or(bad) != 0;
  int64_t before = x;
  if (tid < kThreads) {
    for (int m = 1; m < 32; m <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, before, m);
      if (lane >= m) before += y;
    }
    if (lane == 31) sums[warp] = before;
    before -= x;
  }
  __syncthreads();
  if (tid < kThreads) {
    for (int i = 0; i < warp; ++i) before += sums[i];
    if (tid == 0) cum[0] = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) cum[tid * kEach + i + 1] = before += cost[i];
  }
  __syncthreads();
  if (tid < 2) {
    pos[tid] = paged_cut<MODE>(p, t, w.ctas, c + tid, cum, cum[p.batch], bad);
    if (tid == 0 || c == w.ctas - 1) w.pos[c + tid] = pos[tid];
    if (tid == 0) w.cta_status[c] = bad ? JFA_ERR_BAD_OFFSETS : JFA_OK;
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // scratch may be TMA's from here on
  __syncthreads();
  return w.cta_status + c;
}

// Walks the segments of a CTA's share: [blk0, blk1) of the nb key blocks that a tile meets.
struct PagedSegment {
  int b, unit, tile, blk0, blk1, nb;
  PagedSpan span;
  PagedSeq seq;
  int slot;  // partial slot (0 or 1) of the CTA, or -1: the tile is whole
};
struct PagedWalk {
  PagedPos at, end;
  PagedSeq seq;
  bool fresh;
  __device__ __forceinline__ void init(const PagedPos* share) {  // [begin, end)
    at = share[0];
    end = share[1];
    fresh = true;
  }
  template <int MODE = kAny>
  __device__ __forceinline__ bool next(const Paged& p, const TileShape& t, PagedSegment& s) {
    const int units = p.heads_k * t.nsub;
    for (;;) {
      if (at.b > end.b || at.b >= p.batch) return false;
      if (fresh) {
        seq = paged_seq<MODE>(p, t, at.b);
        fresh = false;
      }
      if (at.tile >= seq.tiles) {
        at.tile = 0;
        at.blk = 0;
        if (seq.tiles == 0 || ++at.unit >= units) {
          at.unit = 0;
          ++at.b;
          fresh = true;
        }
        continue;
      }
      const bool same = at.b == end.b && at.unit == end.unit && at.tile == end.tile;
      if (same ? at.blk >= end.blk
               : at.b == end.b && (at.unit > end.unit || (at.unit == end.unit && at.tile > end.tile)))
        return false;
      s.b = at.b;
      s.unit = at.unit;
      s.tile = at.tile;
      s.seq = seq;
      s.span = paged_span<MODE>(p, t, seq.off, tile_keys(p, t, seq, at.tile), at.tile);
      s.nb = s.span.nb;
      s.blk0 = min(at.blk, s.nb);
      s.blk1 = same ? min(end.blk, s.nb) : s.nb;
      s.slot = s.blk0 > 0 ? 0 : s.blk1 < s.nb ? 1 : -1;
      ++at.tile;
      at.blk = 0;
      return true;
    }
  }
};

// How many of 32 lanes, from the first on and without a gap, `f` holds for: one thread in a warp's place.
struct OneThread {
  template <class F>
  __device__ __forceinline__ int operator()(F f) const {
    int n = 0;
    while (n < 32 && f(n)) ++n;
    return n;
  }
};

// The tile that the cut at CTA c's end falls into, where its parts begin with CTA c's last one; they
// go to CTA `last`.
struct PagedCutTile {
  PagedPos end;
  PagedSeq seq;
  int last;
  __device__ __forceinline__ bool same(const PagedPos& x) const {
    return x.b == end.b && x.unit == end.unit && x.tile == end.tile;
  }
  // False: no tile is cut here, or it begins in an earlier CTA's share, or the plan is another request's.
  template <int MODE = kAny>
  __device__ __forceinline__ bool begins(const Paged& p, const TileShape& t, const PagedWs& w, int ctas, int c) {
    end = paged_pos(p, t, w, c + 1);
    if (end.blk == 0 || end.b >= p.batch || c + 1 == ctas) return false;
    const PagedPos at = paged_pos(p, t, w, c);
    if (same(at) && at.blk > 0) return false;
    seq = paged_seq<MODE>(p, t, end.b);
    return end.tile < seq.tiles;
  }
  // Whether CTA i, whose parts would follow CTA i - 1's, has work of the tile (or a share that is empty).
  __device__ __forceinline__ bool goes_on(const Paged& p, const TileShape& t, const PagedWs& w, int ctas, int i) const {
    return i < ctas && same(paged_pos(p, t, w, i));
  }
  // lanes: looks at 32 CTAs at a time.
  template <int MODE = kAny, class Lanes = OneThread>
  __device__ __forceinline__ bool find(const Paged& p, const TileShape& t, const PagedWs& w, int ctas, int c,
                                       Lanes lanes = Lanes{}) {
    if (!begins<MODE>(p, t, w, ctas, c)) return false;
    last = c + 1;
    for (int n = 32; n == 32; last += n) n = lanes([&](int i) { return goes_on(p, t, w, ctas, last + 1 + i); });
    return true;
  }
  // Whether CTA i, of those from c on, has a part: not one without work inside the tile.
  __device__ __forceinline__ bool part(const Paged& p, const TileShape& t, const PagedWs& w, int c, int i) const {
    if (i > last) return false;
    const PagedPos a = paged_pos(p, t, w, i), e = paged_pos(p, t, w, i + 1);
    return i == c || !(same(e) && a.blk >= e.blk);
  }
  // Token and head of row r; false: it has none.
  __device__ __forceinline__ bool row(const Paged& p, const TileShape& t, int r, int& tok, int& head) const {
    const int gh = (end.unit % t.nsub) * t.gsub + r % t.gsub;
    tok = end.tile * t.tokens + r / t.gsub;
    head = end.unit / t.nsub * p.group + gh;
    return tok < seq.lq && gh < p.group;
  }
};

// Page of a position, or -1 for an index outside the cache (recorded in the status word, where a
// timeout or an invalid batch stays).
__device__ __forceinline__ int paged_page(const Paged& p, int b, int pos, int* status) {
  const int page = __ldg(p.table + (int64_t)b * p.width + (pos >> p.page_shift));
  if ((uint32_t)page >= (uint64_t)p.pages) {
    atomicCAS(status, (int)JFA_OK, (int)JFA_ERR_BAD_PAGES);
    return -1;
  }
  return page;
}
// Row (in units of a head's row) of a position inside the cache arrays.
__device__ __forceinline__ int64_t paged_row(const Paged& p, int page, int head, int pos) {
  return (((int64_t)page * p.heads_k + head) << p.page_shift) + (pos & ((1 << p.page_shift) - 1));
}

// ------------------------------------------------------------------------------- MXFP8
// Scales are E8M0 with exponents kept in [-100, 119]: codes times scale then stay finite and
// normal in fp32 and bf16 (448 * 2^119 = 1.75 * 2^127; larger values saturate there, and blocks
// below 2^-100 lose at most 2^-110 of absolute value).
constexpr int kMxMinExp = -100, kMxMaxExp = 119;

// The smallest e with amax <= 448 * 2^e = 1.75 * 2^(e + 8), from amax's bits.
__device__ __forceinline__ int mx_scale_exp(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, kMxMinExp), kMxMaxExp);
}
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Two values as e4m3 codes (round to nearest even, saturating): lo in the low byte.
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// The values of two e4m3 codes (exact in fp16 and fp32).
__device__ __forceinline__ float2 e4m3_values(uint32_t pair) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)pair));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

}  // namespace jfa
