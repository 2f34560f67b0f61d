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

// What a kernel over a paged cache is compiled for: attention of all keys, of a window with sinks, one
// of the two phases of a shared prefix, or any of these as the request says.
enum : int { kAll = 0, kWindow = 1, kShared = 2, kAny = 3 };
constexpr bool serves_windows(int mode) { return mode == kWindow || mode == kAny; }
constexpr bool serves_shared(int mode) { return mode == kShared || mode == kAny; }

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
  // Window: a query at position x sees the keys y <= x with x - y < window, and the first `sinks`.
  // window = 0: all up to x.
  int window, sinks;
  // Shared prefix.  Phase 1: the "sequences" of the request are groups, sequence b the tokens of the
  // sequences groups[b] .. groups[b + 1] - 1 of `seqs`, and its results are left in prior_o and
  // prior_lse (log2 units) in fp32.  Phase 2 adds them to its own.
  int phase;
  const int64_t* groups;
  int64_t seqs;
  float *prior_o, *prior_lse;  // [T, heads_q, dim_v], [T, heads_q]
  const int* prior_status;     // phase 2: how phase 1 ended
  int few;                     // phase 2: sequences of at most so many own keys are the short kernel's
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
// The workspace of attention over a shared prefix: phase 2's, then phase 1's header and plan (its
// parts lie in phase 2's place, which begins behind it) and its results.  Where phase 2 is the short
// kernel's alone, both have the first header.
size_t shared_layout(const Paged& prefix, const Paged& own, void* base, PagedWs* first, PagedWs* second, float** prior_o,
                     float** prior_lse);

// Whether later attention launches are held (jfa_test_hold).
void paged_set_test_hold(int on);

cudaError_t launch_cache_write(const Paged& p, int dtype, PagedHeader* hdr, int planned, cudaStream_t s);
cudaError_t launch_cache_read(const Paged& p, int dtype, void* k, void* v, PagedHeader* hdr, int planned,
                              cudaStream_t s);
// The batch of a call without tokens, checked.
cudaError_t launch_cache_check(const Paged& p, PagedHeader* hdr, cudaStream_t s);
// a.side: queries (heads 0: none) and keys; p.v, p.sv: values.
cudaError_t launch_append(const Paged& p, const NormRopeArgs& a, int dtype, PagedHeader* hdr, int planned, cudaStream_t s);
// (Calls without windows and prefixes have instances of their own: carried along, those cost a step of four
// users 4 us and the MXFP8 step 25.)
cudaError_t launch_paged_plan(const Paged& p, const TileShape& t, int ctas, const PagedWs& w, cudaStream_t s);
cudaError_t launch_paged_simt(const Paged& p, const TileShape& t, int ctas, int dtype, const PagedWs& w,
                              cudaStream_t s);
// One translation unit for each of kAll, kWindow, kShared.
cudaError_t launch_paged_rows16(const Paged& p, const TileShape& t, int ctas, const PagedWs& w, cudaStream_t s);
cudaError_t launch_paged_rows16_window(const Paged& p, const TileShape& t, int ctas, const PagedWs& w, cudaStream_t s);
cudaError_t launch_paged_rows16_shared(const Paged& p, const TileShape& t, int ctas, const PagedWs& w, cudaStream_t s);
cudaError_t launch_paged_tc(const Paged& p, const TileShape& t, int ctas, const PagedWs& w, cudaStream_t s);
cudaError_t launch_paged_tc_window(const Paged& p, const TileShape& t, int ctas, const PagedWs& w, cudaStream_t s);
cudaError_t launch_paged_tc_shared(const Paged& p, const TileShape& t, int ctas, const PagedWs& w, cudaStream_t s);
// Phase 2 of a shared prefix for the sequences of at most p.few own keys; hdr is the call's header, whose
// status it goes on with.  paged_few: p.few for a request, 0 where the tiled kernels take all; paged_short:
// no sequence can have more.
int paged_few(const Paged& p);
bool paged_short(const Paged& p);
cudaError_t launch_paged_short(const Paged& p, int dtype, PagedHeader* hdr, cudaStream_t s);
cudaError_t launch_paged_combine(const Paged& p, const TileShape& t, int ctas, int dtype, const PagedWs& w,
                                 cudaStream_t s);

}  // namespace jfa
