// Internal declarations of the operators around attention over a paged cache (norms with
// rotary positions, the cache, the attention).  The public ABI is include/jfa.h.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "jfa.h"

namespace jfa {

// ------------------------------------------------------------- norms and rotary positions
constexpr int kMaxNormDim = 256;

// One of the two tensors (queries, keys) of a norm_rope call; strides in elements.
struct NormRopeSide {
  const void* x;
  const void* dy;  // backward only
  const float* w;  // norm weight [dim], or nullptr: ones
  void* out;       // forward: y; backward: dx
  float* dw;       // backward: weight gradient [dim], or nullptr
  int64_t sx, sdy, sout;
  int heads;
};
struct NormRopeArgs {
  NormRopeSide side[2];
  const int64_t* pos;
  int64_t tokens;
  int dim, rot, layout;
  int norm;
  float eps, inv_dim, amp;
  // Rotation of pair i per position, in turns, as a 64-bit binary fraction: position times
  // turn, modulo one turn, is the low 64 bits of an integer product.
  unsigned long long turn[kMaxNormDim / 2];
};
// part: workspace of the weight gradients' partial sums, norm_rope_parts() * 2 * dim floats.
cudaError_t launch_norm_rope_fwd(const NormRopeArgs& a, int dtype, cudaStream_t s);
cudaError_t launch_norm_rope_bwd(const NormRopeArgs& a, int dtype, float* part, cudaStream_t s);
constexpr int kNormRopeParts = 1024;  // most partial sums a backward writes

// ------------------------------------------------------------- paged cache and attention
enum : int { kCacheF32 = 0, kCacheBf16 = 1, kCacheMx = 2 };

// One request on a paged cache.
struct Paged {
  const int64_t* offs;   // [B+1] new tokens
  const int64_t* lens;   // [B] cached tokens, the new ones among them
  const int32_t* table;  // [B, width] page of every page_size positions
  int64_t batch, total_q, pages;
  int width, page_shift;
  int heads_q, heads_k, group;  // group = heads_q / heads_k
  int dim_qk, dim_v, kind;      // kind: kCache*
  float scale;
  int causal;
  void *kc, *vc;      // [pages, heads_k, page, dim]
  uint8_t *ks, *vs;   // [pages, heads_k, page, dim / 32] E8M0 scales (kCacheMx)
  const void *q, *k, *v;
  int64_t sq, sk, sv;  // elements between tokens
  void* o;             // [T, heads_q, dim_v]
  float* lse;          // [T, heads_q]
};

// Where a CTA's share of the attention begins: block `blk` of keys of tile `tile` of unit
// `unit` (a key head, or a part of its queries) of sequence b.
struct __align__(16) PagedPos {
  int b, unit, tile, blk;
};

// Header of the workspace (offset 0); the first word is the status, as in every workspace.
struct PagedHeader {
  int status;
  int pad[63];
};
static_assert(sizeof(PagedHeader) == 256, "workspace header");

// How a kernel tiles the queries of a sequence that share a key head: a tile is `tokens`
// consecutive tokens by `gsub` of the group's heads, at most `rows` rows, row = token * gsub
// + head; a group larger than a tile is cut into nsub parts.  Keys go in blocks of `keys`.
struct TileShape {
  int rows, tokens, gsub, nsub, keys;
  int overhead;  // cost of a tile beside its keys, in keys
  int share;     // least cost of a CTA's share
};

constexpr int kMaxPagedCtas = 640, kMaxTcCtas = 160;
// Keys of a block of the 16-row kernel.
constexpr int paged_rows16_keys(int dim_qk, int dim_v, int kind) {
  return kind == kCacheBf16 && dim_qk + dim_v > 128 ? 32 : 64;
}

// Batches that every CTA of the attention scans by itself, so that an unplanned call needs no plan
// launch (4 us of the 15 that a step of four users takes); and the scratch it takes.
constexpr int kPlanInCta = 512;
constexpr int kPlanScratch = 8 * (kPlanInCta + 1 + 4);

struct PagedWs {
  int ctas;         // 0: pos holds a plan; else the number of CTAs, which cut the work themselves
  int hold;         // test hook (jfa_test_hold): one role of CTA 0 waits for what never comes
  int* cta_status;  // [n_ctas] errors of CTAs without a plan, for the join
  PagedHeader* hdr;
  PagedPos* pos;   // [n_ctas + 1]
  int64_t* cum;    // [B + 1] cost of the sequences before b
  float* part_ml;  // [2 n_ctas][rows][2] (running max in log2 units, row sum)
  float* part_o;   // [2 n_ctas][rows][dim_v] unnormalised
};

enum : int { kPagedSimt = 0, kPagedRows16 = 1, kPagedTc = 2 };
// The kernel that serves a request, its tiles and its number of CTAs.
int paged_kernel(const Paged& p, int dtype);
TileShape paged_shape(const Paged& p, int kernel);
int paged_ctas(const Paged& p, int kernel);
size_t paged_layout(const Paged& p, void* base, PagedWs* out);

// Whether later attention launches are held (jfa_test_hold).
void paged_set_test_hold(int on);

cudaError_t launch_cache_write(const Paged& p, int dtype, PagedHeader* hdr, int planned, cudaStream_t s);
cudaError_t launch_cache_read(const Paged& p, int dtype, void* k, void* v, PagedHeader* hdr, int planned,
                              cudaStream_t s);
cudaError_t launch_paged_plan(const Paged& p, const TileShape& t, int ctas, const PagedWs& w, cudaStream_t s);
cudaError_t launch_paged_simt(const Paged& p, const TileShape& t, int ctas, int dtype, const PagedWs& w,
                              cudaStream_t s);
cudaError_t launch_paged_rows16(const Paged& p, const TileShape& t, int ctas, const PagedWs& w, cudaStream_t s);
cudaError_t launch_paged_tc(const Paged& p, const TileShape& t, int ctas, const PagedWs& w, cudaStream_t s);
cudaError_t launch_paged_combine(const Paged& p, const TileShape& t, int ctas, int dtype, const PagedWs& w,
                                 cudaStream_t s);

}  // namespace jfa
