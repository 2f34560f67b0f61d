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
__device__ __forceinline__ PagedSeq paged_seq(const Paged& p, const TileShape& t, int b) {
  PagedSeq s;
  const int64_t a = __ldg(p.offs + b), e = __ldg(p.offs + b + 1), l = __ldg(p.lens + b);
  s.q0 = (int)a;
  s.lq = (int)(e - a);
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

// Walks the segments of a CTA's share: [blk0, blk1) of a tile's nb key blocks.
struct PagedSegment {
  int b, unit, tile, blk0, blk1, nb;
  PagedSeq seq;
  int slot;  // partial slot (0 or 1) of the CTA, or -1: the tile is whole
};
struct PagedWalk {
  PagedPos at, end;
  PagedSeq seq;
  bool fresh;
  __device__ __forceinline__ void init(const PagedPos* pos, int cta) {
    const int4* q = reinterpret_cast<const int4*>(pos + cta);
    const int4 a = __ldg(q), e = __ldg(q + 1);
    at = PagedPos{a.x, a.y, a.z, a.w};
    end = PagedPos{e.x, e.y, e.z, e.w};
    fresh = true;
  }
  __device__ __forceinline__ bool next(const Paged& p, const TileShape& t, PagedSegment& s) {
    const int units = p.heads_k * t.nsub;
    for (;;) {
      if (at.b > end.b || at.b >= p.batch) return false;
      if (fresh) {
        seq = paged_seq(p, t, at.b);
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
      s.nb = (tile_keys(p, t, seq, at.tile) + t.keys - 1) / t.keys;
      s.blk0 = at.blk;
      s.blk1 = same ? end.blk : s.nb;
      s.slot = s.blk0 > 0 ? 0 : s.blk1 < s.nb ? 1 : -1;
      ++at.tile;
      at.blk = 0;
      return true;
    }
  }
};

// Page of a position, or -1 for an index outside the cache (recorded in the status word).
__device__ __forceinline__ int paged_page(const Paged& p, int b, int pos, int* status) {
  const int page = __ldg(p.table + (int64_t)b * p.width + (pos >> p.page_shift));
  if ((uint32_t)page >= (uint64_t)p.pages) {
    atomicExch(status, (int)JFA_ERR_BAD_PAGES);
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
