// C entry points of the operators around attention over a paged cache (include/jfa.h):
// argument checks, workspaces and dispatch.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "internal.h"
#include "serve.h"
#include "timed.h"

namespace jfa {
namespace {

jfa_status cu(cudaError_t e) { return e == cudaSuccess ? JFA_OK : JFA_ERR_CUDA; }
bool finite_at_least(double x, double low) { return x >= low && x <= 1.7976931348623157e308; }

// ------------------------------------------------------------- norms and rotary positions
jfa_status check_rope(const jfa_rope& r, int dim) {
  if (r.dim < 0 || r.dim > dim || (r.dim & 1)) return JFA_ERR_INVALID_ARG;
  if (r.dim == 0) return JFA_OK;
  if (r.layout != JFA_ROPE_HALVES && r.layout != JFA_ROPE_PAIRS) return JFA_ERR_INVALID_ARG;
  if (r.scaling < JFA_ROPE_PLAIN || r.scaling > JFA_ROPE_YARN) return JFA_ERR_INVALID_ARG;
  if (!finite_at_least(r.base, 1.0) || !isfinite(r.amp)) return JFA_ERR_INVALID_ARG;
  if (r.scaling != JFA_ROPE_PLAIN && !finite_at_least(r.factor, 1.0)) return JFA_ERR_INVALID_ARG;
  if (r.scaling == JFA_ROPE_NTK && r.dim < 4) return JFA_ERR_INVALID_ARG;
  if (r.scaling == JFA_ROPE_YARN &&
      (!(r.orig_len > 0) || !isfinite(r.orig_len) || !finite_at_least(r.turns_slow, 0.0) ||
       !(r.turns_fast > r.turns_slow) || !isfinite(r.turns_fast)))
    return JFA_ERR_INVALID_ARG;
  return JFA_OK;
}

// theta_i / 2 pi as a 64-bit fraction of a turn
unsigned long long rope_turn(const jfa_rope& r, int i) {
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  double base = r.base;
  if (r.scaling == JFA_ROPE_NTK) base *= pow(r.factor, r.dim / (double)(r.dim - 2));
  double theta = pow(base, -2.0 * i / r.dim);
  if (r.scaling == JFA_ROPE_LINEAR) theta /= r.factor;
  if (r.scaling == JFA_ROPE_YARN) {
    double keep = (r.orig_len * theta / kTwoPi - r.turns_slow) / (r.turns_fast - r.turns_slow);
    keep = keep < 0 ? 0 : keep > 1 ? 1 : keep;
    theta *= keep + (1 - keep) / r.factor;
  }
  return (unsigned long long)ldexp(theta / kTwoPi, 64);  // theta <= 1: below 2^62
}

jfa_status check_norm_rope(const jfa_norm_rope_params* p) {
  if (!p) return JFA_ERR_INVALID_ARG;
  if (p->tokens < 0 || p->heads_q < 0 || p->heads_k < 0 || (int64_t)p->heads_q + p->heads_k < 1 || p->dim < 1)
    return JFA_ERR_INVALID_ARG;
  if (p->dtype != JFA_F32 && p->dtype != JFA_BF16) return JFA_ERR_INVALID_ARG;
  if (p->norm != 0 && p->norm != 1) return JFA_ERR_INVALID_ARG;
  if (p->norm && !(p->eps >= 0.f && isfinite(p->eps))) return JFA_ERR_INVALID_ARG;
  if (p->dim > kMaxNormDim || p->tokens > INT32_MAX || (int64_t)p->heads_q + p->heads_k > 65536)
    return JFA_ERR_UNSUPPORTED;
  return check_rope(p->rope, p->dim);
}

// One tensor: every pointer that a call with tokens and heads needs, and its stride.
jfa_status norm_rope_side(const jfa_norm_rope_params* p, int heads, const void* x, int64_t sx, const void* dy,
                          int64_t sdy, bool bwd, const float* w, void* out, int64_t sout, float* dw, NormRopeSide* s) {
  const int64_t row = (int64_t)heads * p->dim;
  const uintptr_t align = p->dtype == JFA_BF16 ? 1 : 3;
  if (!p->norm && (w || dw)) return JFA_ERR_INVALID_ARG;
  if (heads > 0 && p->tokens > 0) {
    const bool need_x = !bwd || p->norm;
    if ((need_x && !x) || !out || (bwd && !dy)) return JFA_ERR_INVALID_ARG;
    if (((uintptr_t)x | (uintptr_t)out | (uintptr_t)dy) & align) return JFA_ERR_INVALID_ARG;
    if (p->tokens > 1 && ((need_x && sx < row) || sout < row || (bwd && sdy < row))) return JFA_ERR_INVALID_ARG;
  }
  if (((uintptr_t)w | (uintptr_t)dw) & 3) return JFA_ERR_INVALID_ARG;
  *s = NormRopeSide{x, dy, w, out, heads > 0 ? dw : nullptr, sx, sdy, sout, heads};
  return JFA_OK;
}

void norm_rope_common(const jfa_norm_rope_params* p, const int64_t* pos, NormRopeArgs* a) {
  a->pos = pos;
  a->tokens = p->tokens;
  a->dim = p->dim;
  a->rot = p->rope.dim;
  a->layout = p->rope.layout;
  a->norm = p->norm;
  a->eps = p->eps;
  a->inv_dim = 1.f / p->dim;
  a->amp = p->rope.amp;
  for (int i = 0; i < kMaxNormDim / 2; ++i) a->turn[i] = i < p->rope.dim / 2 ? rope_turn(p->rope, i) : 0;
}

size_t norm_rope_ws(const jfa_norm_rope_params* p) { return sizeof(float) * 2 * (size_t)kNormRopeParts * p->dim; }

// ------------------------------------------------------------------------- paged cache
jfa_status check_paged(const jfa_paged_params* p) {
  if (!p) return JFA_ERR_INVALID_ARG;
  if (p->batch < 0 || p->total_q < 0 || p->pages < 0 || p->heads_q < 1 || p->heads_k < 1 || p->dim_qk < 1 ||
      p->dim_v < 1 || p->max_pages < 0)
    return JFA_ERR_INVALID_ARG;
  if (p->batch == 0 && p->total_q != 0) return JFA_ERR_INVALID_ARG;
  if (p->dtype != JFA_F32 && p->dtype != JFA_BF16) return JFA_ERR_INVALID_ARG;
  if (p->cache_dtype != JFA_F32 && p->cache_dtype != JFA_BF16 && p->cache_dtype != JFA_MXFP8) return JFA_ERR_INVALID_ARG;
  if ((p->flags & ~JFA_PLANNED) != 0) return JFA_ERR_INVALID_ARG;
  if (p->page_size < 1) return JFA_ERR_INVALID_ARG;
  if (p->cache_dtype != JFA_MXFP8 && p->cache_dtype != p->dtype) return JFA_ERR_UNSUPPORTED;
  if (p->page_size < 16 || p->page_size > 256 || (p->page_size & (p->page_size - 1)) != 0) return JFA_ERR_UNSUPPORTED;
  const int unit = p->cache_dtype == JFA_MXFP8 ? 32 : 8;
  if (p->dim_qk % unit || p->dim_v % unit || p->dim_qk > 256 || p->dim_v > 256) return JFA_ERR_UNSUPPORTED;
  // the kernels round positions and tokens up to whole tiles in 32 bits
  constexpr int64_t kMost = (int64_t)INT32_MAX - 255;
  if (p->total_q > kMost || p->batch > INT32_MAX || p->pages > INT32_MAX ||
      (int64_t)p->max_pages * p->page_size > kMost || p->heads_q > 65536 || p->heads_k > 65536)
    return JFA_ERR_UNSUPPORTED;
  return JFA_OK;
}

jfa_status check_paged_attention(const jfa_paged_params* p) {
  jfa_status st = check_paged(p);
  if (st != JFA_OK) return st;
  if (p->heads_q % p->heads_k != 0) return JFA_ERR_INVALID_ARG;
  if (p->causal != 0 && p->causal != 1) return JFA_ERR_INVALID_ARG;
  if (!(p->scale > 0.f) || !isfinite(p->scale)) return JFA_ERR_INVALID_ARG;
  if (p->dim_qk > 128 || p->dim_v > 128) return JFA_ERR_UNSUPPORTED;
  // the plan's costs are 64-bit: tiles (at most a query row each) times the keys they may see
  const double cost = (double)p->heads_q * (double)p->total_q * ((double)p->max_pages * p->page_size + 1024.0);
  if (cost > 4.0e18) return JFA_ERR_UNSUPPORTED;
  return JFA_OK;
}

bool aligned(const void* x, uintptr_t a) { return x && ((uintptr_t)x & (a - 1)) == 0; }

jfa_status check_index(const jfa_paged_params* p, const int64_t* offs, const int64_t* lens, const int32_t* table) {
  if (!aligned(offs, 8)) return JFA_ERR_INVALID_ARG;
  if (p->batch > 0 && (!aligned(lens, 8) || (p->max_pages > 0 && !aligned(table, 4)))) return JFA_ERR_INVALID_ARG;
  return JFA_OK;
}

// the cache's arrays; heads' rows are loaded 16 bytes at a time
jfa_status check_cache(const jfa_paged_params* p, const void* kc, const void* vc, const uint8_t* ks, const uint8_t* vs) {
  if (p->pages == 0) return JFA_OK;
  if (!aligned(kc, 16) || !aligned(vc, 16)) return JFA_ERR_INVALID_ARG;
  if (p->cache_dtype == JFA_MXFP8 && (!aligned(ks, 16) || !aligned(vs, 16))) return JFA_ERR_INVALID_ARG;
  return JFA_OK;
}

// rows of T tokens: 16-byte aligned, a stride of whole 16 bytes that holds a token's heads
jfa_status check_rows(const jfa_paged_params* p, const void* x, int64_t stride, int64_t row) {
  if (p->total_q == 0) return JFA_OK;
  const int64_t unit = p->dtype == JFA_BF16 ? 8 : 4;
  if (!aligned(x, 16)) return JFA_ERR_INVALID_ARG;
  if (p->total_q > 1 && (stride < row || stride % unit != 0)) return JFA_ERR_INVALID_ARG;
  return JFA_OK;
}

Paged make_paged(const jfa_paged_params* p, const int64_t* offs, const int64_t* lens, const int32_t* table,
                 const void* kc, const void* vc, const uint8_t* ks, const uint8_t* vs) {
  Paged r{};
  r.offs = offs;
  r.lens = lens;
  r.table = table;
  r.batch = p->batch;
  r.total_q = p->total_q;
  r.pages = p->pages;
  r.width = p->max_pages;
  while ((1 << r.page_shift) < p->page_size) ++r.page_shift;
  r.heads_q = p->heads_q;
  r.heads_k = p->heads_k;
  r.group = p->heads_q / p->heads_k;
  r.dim_qk = p->dim_qk;
  r.dim_v = p->dim_v;
  r.kind = p->cache_dtype == JFA_MXFP8 ? kCacheMx : p->cache_dtype == JFA_BF16 ? kCacheBf16 : kCacheF32;
  r.scale = p->scale;
  r.causal = p->causal;
  r.kc = const_cast<void*>(kc);
  r.vc = const_cast<void*>(vc);
  r.ks = const_cast<uint8_t*>(ks);
  r.vs = const_cast<uint8_t*>(vs);
  r.sq = p->stride_q;
  r.sk = p->stride_k;
  r.sv = p->stride_v;
  return r;
}

std::atomic<int> g_paged_hold{0};

jfa_status check_ws(const Paged& p, void* ws, size_t bytes, PagedWs* w) {
  if (!ws || ((uintptr_t)ws & 255u) != 0) return JFA_ERR_WORKSPACE;
  if (bytes < paged_layout(p, ws, w)) return JFA_ERR_WORKSPACE;
  w->hold = g_paged_hold.load(std::memory_order_relaxed);
  return JFA_OK;
}

// The cache calls have no plan of their own: a call without JFA_PLANNED resets the header, and
// the kernel records what it finds wrong.
jfa_status cache_status(const jfa_paged_params* p, const PagedWs& w, cudaStream_t s) {
  if (p->flags & JFA_PLANNED) return JFA_OK;
  return cu(cudaMemsetAsync(w.hdr, 0, sizeof(PagedHeader), s));
}

jfa_status plan_paged(const Paged& r, int kernel, const PagedWs& w, cudaStream_t s) {
  Timed t(JFA_KERNEL_SCHEDULE, s);
  return cu(launch_paged_plan(r, paged_shape(r, kernel), paged_ctas(r, kernel), w, s));
}

// One pass of the attention over its plan, or the cuts that its CTAs make.
jfa_status run_paged(const Paged& r, int dtype, int mode, bool planned, PagedWs w, cudaStream_t s) {
  const int kernel = paged_kernel(r, dtype);
  const int ctas = paged_ctas(r, kernel);
  jfa_status st;
  if (!planned) {
    if (r.total_q > 0 && r.batch <= kPlanInCta) w.ctas = ctas;
    else if ((st = plan_paged(r, kernel, w, s)) != JFA_OK) return st;
  }
  if (r.total_q == 0) return JFA_OK;
  const TileShape shape = paged_shape(r, kernel);
  constexpr decltype(&launch_paged_tc) tc[] = {launch_paged_tc, launch_paged_tc_window, launch_paged_tc_shared};
  constexpr decltype(&launch_paged_rows16) few[] = {launch_paged_rows16, launch_paged_rows16_window,
                                                    launch_paged_rows16_shared};
  Timed t(JFA_KERNEL_PAGED, s);
  st = cu(kernel == kPagedTc       ? tc[mode](r, shape, ctas, w, s)
          : kernel == kPagedRows16 ? few[mode](r, shape, ctas, w, s)
                                   : launch_paged_simt(r, shape, ctas, dtype, w, s));
  if (st != JFA_OK) return st;
  return cu(launch_paged_combine(r, shape, ctas, dtype, w, s));
}

jfa_status check_window(const jfa_paged_params* p, int32_t window, int32_t sinks) {
  jfa_status st = check_paged_attention(p);
  if (st != JFA_OK) return st;
  if (window < 1 || sinks < 0) return JFA_ERR_INVALID_ARG;
  return p->causal ? JFA_OK : JFA_ERR_UNSUPPORTED;
}
// All positions there are need no more than that.
void set_window(const jfa_paged_params* p, int32_t window, int32_t sinks, Paged* r) {
  const int most = p->max_pages > 0 ? p->max_pages * p->page_size : 1;
  r->window = window < most ? window : most;
  r->sinks = sinks < most ? sinks : most;
}

// What the calls over a paged cache check of their arguments, and the request they make of them.
jfa_status paged_request(const jfa_paged_params* p, const void* q, const void* k_cache, const void* v_cache,
                         const uint8_t* k_scale, const uint8_t* v_scale, const int64_t* offs, const int64_t* lens,
                         const int32_t* table, void* o, float* lse, Paged* r) {
  jfa_status st;
  if ((st = check_index(p, offs, lens, table)) != JFA_OK ||
      (st = check_cache(p, k_cache, v_cache, k_scale, v_scale)) != JFA_OK ||
      (st = check_rows(p, q, p->stride_q, (int64_t)p->heads_q * p->dim_qk)) != JFA_OK)
    return st;
  if (p->total_q > 0 && (!aligned(o, 16) || !aligned(lse, 16))) return JFA_ERR_INVALID_ARG;
  *r = make_paged(p, offs, lens, table, k_cache, v_cache, k_scale, v_scale);
  r->q = q;
  r->o = o;
  r->lse = lse;
  return JFA_OK;
}

// The prefixes' side of a call: groups in the place of sequences, and no mask.
jfa_status check_shared(const jfa_paged_params* p, int64_t groups, int32_t prefix_pages) {
  jfa_status st = check_paged_attention(p);
  if (st != JFA_OK) return st;
  if (groups < 0 || prefix_pages < 0 || (groups == 0 && p->batch > 0)) return JFA_ERR_INVALID_ARG;
  jfa_paged_params g = *p;
  g.batch = groups;
  g.max_pages = prefix_pages;
  if (groups == 0) g.total_q = 0;
  return check_paged_attention(&g);
}
void prefix_request(int64_t groups, int32_t prefix_pages, Paged* r) {
  r->seqs = r->batch;
  r->batch = groups;
  r->width = prefix_pages;
  r->causal = 0;
}

}  // namespace

void paged_set_test_hold(int on) { g_paged_hold.store(on != 0, std::memory_order_relaxed); }
}  // namespace jfa

using namespace jfa;

extern "C" {

size_t jfa_norm_rope_workspace_size(const jfa_norm_rope_params* p) {
  return check_norm_rope(p) == JFA_OK ? norm_rope_ws(p) : 0;
}

jfa_status jfa_norm_rope_fwd(const jfa_norm_rope_params* p, const void* q, const void* k, const int64_t* pos,
                             const float* wq, const float* wk, void* yq, void* yk, jfa_stream_t stream) {
  jfa_status st = check_norm_rope(p);
  if (st != JFA_OK) return st;
  NormRopeArgs a;
  if ((st = norm_rope_side(p, p->heads_q, q, p->stride_q, nullptr, 0, false, wq, yq, p->stride_yq, nullptr,
                           &a.side[0])) != JFA_OK ||
      (st = norm_rope_side(p, p->heads_k, k, p->stride_k, nullptr, 0, false, wk, yk, p->stride_yk, nullptr,
                           &a.side[1])) != JFA_OK)
    return st;
  if (p->tokens > 0 && p->rope.dim > 0 && !aligned(pos, 8)) return JFA_ERR_INVALID_ARG;
  if (p->tokens == 0) return JFA_OK;
  norm_rope_common(p, pos, &a);
  Timed t(JFA_KERNEL_NORM_ROPE, (cudaStream_t)stream);
  return cu(launch_norm_rope_fwd(a, p->dtype, (cudaStream_t)stream));
}

jfa_status jfa_norm_rope_bwd(const jfa_norm_rope_params* p, const void* q, const void* k, const int64_t* pos,
                             const float* wq, const float* wk, const void* dyq, const void* dyk, void* dq, void* dk,
                             float* dwq, float* dwk, void* ws, size_t ws_bytes, jfa_stream_t stream) {
  jfa_status st = check_norm_rope(p);
  if (st != JFA_OK) return st;
  NormRopeArgs a;
  if ((st = norm_rope_side(p, p->heads_q, q, p->stride_q, dyq, p->stride_yq, true, wq, dq, p->stride_dq, dwq,
                           &a.side[0])) != JFA_OK ||
      (st = norm_rope_side(p, p->heads_k, k, p->stride_k, dyk, p->stride_yk, true, wk, dk, p->stride_dk, dwk,
                           &a.side[1])) != JFA_OK)
    return st;
  if (p->tokens > 0 && p->rope.dim > 0 && !aligned(pos, 8)) return JFA_ERR_INVALID_ARG;
  if (!ws || ((uintptr_t)ws & 255u) != 0 || ws_bytes < norm_rope_ws(p)) return JFA_ERR_WORKSPACE;
  cudaStream_t s = (cudaStream_t)stream;
  // no row: the weights' gradients are zero
  const size_t bytes = sizeof(float) * p->dim;
  if (dwq && (p->tokens == 0 || p->heads_q == 0) && (st = cu(cudaMemsetAsync(dwq, 0, bytes, s))) != JFA_OK) return st;
  if (dwk && (p->tokens == 0 || p->heads_k == 0) && (st = cu(cudaMemsetAsync(dwk, 0, bytes, s))) != JFA_OK) return st;
  if (p->tokens == 0) return JFA_OK;
  norm_rope_common(p, pos, &a);
  Timed t(JFA_KERNEL_NORM_ROPE, s);
  return cu(launch_norm_rope_bwd(a, p->dtype, (float*)ws, s));
}

size_t jfa_paged_workspace_size(const jfa_paged_params* p) {
  if (check_paged(p) != JFA_OK) return 0;
  return paged_layout(make_paged(p, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr), nullptr, nullptr);
}

jfa_status jfa_cache_write(const jfa_paged_params* p, const void* k, const void* v, const int64_t* offs,
                           const int64_t* lens, const int32_t* table, void* k_cache, void* v_cache, uint8_t* k_scale,
                           uint8_t* v_scale, void* ws, size_t ws_bytes, jfa_stream_t stream) {
  jfa_status st = check_paged(p);
  if (st != JFA_OK) return st;
  if ((st = check_index(p, offs, lens, table)) != JFA_OK ||
      (st = check_cache(p, k_cache, v_cache, k_scale, v_scale)) != JFA_OK ||
      (st = check_rows(p, k, p->stride_k, (int64_t)p->heads_k * p->dim_qk)) != JFA_OK ||
      (st = check_rows(p, v, p->stride_v, (int64_t)p->heads_k * p->dim_v)) != JFA_OK)
    return st;
  Paged r = make_paged(p, offs, lens, table, k_cache, v_cache, k_scale, v_scale);
  PagedWs w;
  if ((st = check_ws(r, ws, ws_bytes, &w)) != JFA_OK) return st;
  r.k = k;
  r.v = v;
  cudaStream_t s = (cudaStream_t)stream;
  Timed t(JFA_KERNEL_CACHE, s);
  if ((st = cache_status(p, w, s)) != JFA_OK) return st;
  return cu(launch_cache_write(r, p->dtype, w.hdr, p->flags & JFA_PLANNED, s));
}

jfa_status jfa_rope_append(const jfa_paged_params* p, const jfa_rope* rope, int32_t norm, float eps, const void* q,
                           const void* k, const void* v, const int64_t* pos, const float* wq, const float* wk,
                           const int64_t* offs, const int64_t* lens, const int32_t* table, void* yq, int64_t stride_yq,
                           void* k_cache, void* v_cache, uint8_t* k_scale, uint8_t* v_scale, void* ws, size_t ws_bytes,
                           jfa_stream_t stream) {
  jfa_status st = check_paged(p);
  if (st != JFA_OK) return st;
  // norm and rotation of the queries and keys, as in jfa_norm_rope_fwd
  jfa_norm_rope_params n{};
  n.tokens = p->total_q;
  n.heads_q = q ? p->heads_q : 0;
  n.heads_k = p->heads_k;
  n.dim = p->dim_qk;
  n.dtype = p->dtype;
  n.norm = norm;
  n.eps = eps;
  if (rope) n.rope = *rope;
  if ((st = check_norm_rope(&n)) != JFA_OK) return st;
  if (!q && yq) return JFA_ERR_INVALID_ARG;
  if ((st = check_index(p, offs, lens, table)) != JFA_OK ||
      (st = check_cache(p, k_cache, v_cache, k_scale, v_scale)) != JFA_OK ||
      (st = check_rows(p, k, p->stride_k, (int64_t)p->heads_k * p->dim_qk)) != JFA_OK ||
      (st = check_rows(p, v, p->stride_v, (int64_t)p->heads_k * p->dim_v)) != JFA_OK)
    return st;
  const int64_t row = (int64_t)p->heads_q * p->dim_qk;
  if (q && ((st = check_rows(p, q, p->stride_q, row)) != JFA_OK || (st = check_rows(p, yq, stride_yq, row)) != JFA_OK))
    return st;
  NormRopeArgs a;
  if ((st = norm_rope_side(&n, n.heads_q, q, p->stride_q, nullptr, 0, false, wq, yq, stride_yq, nullptr, &a.side[0])) !=
          JFA_OK ||
      (st = norm_rope_side(&n, n.heads_k, k, p->stride_k, nullptr, 0, false, wk, const_cast<void*>(k), p->stride_k,
                           nullptr, &a.side[1])) != JFA_OK)  // (their output is the cache)
    return st;
  if (pos && !aligned(pos, 8)) return JFA_ERR_INVALID_ARG;
  norm_rope_common(&n, pos, &a);
  Paged r = make_paged(p, offs, lens, table, k_cache, v_cache, k_scale, v_scale);
  PagedWs w;
  if ((st = check_ws(r, ws, ws_bytes, &w)) != JFA_OK) return st;
  r.v = v;
  cudaStream_t s = (cudaStream_t)stream;
  Timed t(JFA_KERNEL_CACHE, s);
  if ((st = cache_status(p, w, s)) != JFA_OK) return st;
  const int planned = p->flags & JFA_PLANNED;
  if (p->total_q == 0) return planned ? JFA_OK : cu(launch_cache_check(r, w.hdr, s));
  return cu(launch_append(r, a, p->dtype, w.hdr, planned, s));
}

jfa_status jfa_cache_read(const jfa_paged_params* p, const void* k_cache, const void* v_cache, const uint8_t* k_scale,
                          const uint8_t* v_scale, const int64_t* offs, const int64_t* lens, const int32_t* table,
                          void* k, void* v, void* ws, size_t ws_bytes, jfa_stream_t stream) {
  jfa_status st = check_paged(p);
  if (st != JFA_OK) return st;
  if ((st = check_index(p, offs, lens, table)) != JFA_OK ||
      (st = check_cache(p, k_cache, v_cache, k_scale, v_scale)) != JFA_OK)
    return st;
  if (p->total_q > 0 && (!aligned(k, 16) || !aligned(v, 16))) return JFA_ERR_INVALID_ARG;
  const Paged r = make_paged(p, offs, lens, table, k_cache, v_cache, k_scale, v_scale);
  PagedWs w;
  if ((st = check_ws(r, ws, ws_bytes, &w)) != JFA_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  Timed t(JFA_KERNEL_CACHE, s);
  if ((st = cache_status(p, w, s)) != JFA_OK) return st;
  return cu(launch_cache_read(r, p->dtype, k, v, w.hdr, p->flags & JFA_PLANNED, s));
}

jfa_status jfa_paged_plan(const jfa_paged_params* p, const int64_t* offs, const int64_t* lens, void* ws,
                          size_t ws_bytes, jfa_stream_t stream) {
  jfa_status st = check_paged_attention(p);
  if (st != JFA_OK) return st;
  if (!aligned(offs, 8) || (p->batch > 0 && !aligned(lens, 8))) return JFA_ERR_INVALID_ARG;
  const Paged r = make_paged(p, offs, lens, nullptr, nullptr, nullptr, nullptr, nullptr);
  PagedWs w;
  if ((st = check_ws(r, ws, ws_bytes, &w)) != JFA_OK) return st;
  return plan_paged(r, paged_kernel(r, p->dtype), w, (cudaStream_t)stream);
}

jfa_status jfa_paged_fwd(const jfa_paged_params* p, const void* q, const void* k_cache, const void* v_cache,
                         const uint8_t* k_scale, const uint8_t* v_scale, const int64_t* offs, const int64_t* lens,
                         const int32_t* table, void* o, float* lse, void* ws, size_t ws_bytes, jfa_stream_t stream) {
  jfa_status st = check_paged_attention(p);
  if (st != JFA_OK) return st;
  Paged r;
  if ((st = paged_request(p, q, k_cache, v_cache, k_scale, v_scale, offs, lens, table, o, lse, &r)) != JFA_OK) return st;
  PagedWs w;
  if ((st = check_ws(r, ws, ws_bytes, &w)) != JFA_OK) return st;
  return run_paged(r, p->dtype, kAll, (p->flags & JFA_PLANNED) != 0, w, (cudaStream_t)stream);
}

jfa_status jfa_paged_window_plan(const jfa_paged_params* p, int32_t window, int32_t sinks, const int64_t* offs,
                                 const int64_t* lens, void* ws, size_t ws_bytes, jfa_stream_t stream) {
  jfa_status st = check_window(p, window, sinks);
  if (st != JFA_OK) return st;
  if (!aligned(offs, 8) || (p->batch > 0 && !aligned(lens, 8))) return JFA_ERR_INVALID_ARG;
  Paged r = make_paged(p, offs, lens, nullptr, nullptr, nullptr, nullptr, nullptr);
  set_window(p, window, sinks, &r);
  PagedWs w;
  if ((st = check_ws(r, ws, ws_bytes, &w)) != JFA_OK) return st;
  return plan_paged(r, paged_kernel(r, p->dtype), w, (cudaStream_t)stream);
}

jfa_status jfa_paged_window_fwd(const jfa_paged_params* p, int32_t window, int32_t sinks, const void* q,
                                const void* k_cache, const void* v_cache, const uint8_t* k_scale,
                                const uint8_t* v_scale, const int64_t* offs, const int64_t* lens, const int32_t* table,
                                void* o, float* lse, void* ws, size_t ws_bytes, jfa_stream_t stream) {
  jfa_status st = check_window(p, window, sinks);
  if (st != JFA_OK) return st;
  Paged r;
  if ((st = paged_request(p, q, k_cache, v_cache, k_scale, v_scale, offs, lens, table, o, lse, &r)) != JFA_OK) return st;
  set_window(p, window, sinks, &r);
  PagedWs w;
  if ((st = check_ws(r, ws, ws_bytes, &w)) != JFA_OK) return st;
  return run_paged(r, p->dtype, kWindow, (p->flags & JFA_PLANNED) != 0, w, (cudaStream_t)stream);
}

size_t jfa_shared_workspace_size(const jfa_paged_params* p, int64_t groups, int32_t prefix_pages) {
  if (check_shared(p, groups, prefix_pages) != JFA_OK) return 0;
  const Paged own = make_paged(p, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr);
  Paged prefix = own;
  prefix_request(groups, prefix_pages, &prefix);
  PagedWs a, b;
  float *o, *l;
  return shared_layout(prefix, own, nullptr, &a, &b, &o, &l);
}

jfa_status jfa_shared_fwd(const jfa_paged_params* p, int64_t groups, int32_t prefix_pages, const void* q,
                          const void* k_cache, const void* v_cache, const uint8_t* k_scale, const uint8_t* v_scale,
                          const int64_t* offs, const int64_t* lens, const int32_t* table, const int64_t* group_offs,
                          const int64_t* prefix_lens, const int32_t* prefix_table, void* o, float* lse, void* ws,
                          size_t ws_bytes, jfa_stream_t stream) {
  jfa_status st = check_shared(p, groups, prefix_pages);
  if (st != JFA_OK) return st;
  if (p->flags & JFA_PLANNED) return JFA_ERR_UNSUPPORTED;
  Paged own;
  if ((st = paged_request(p, q, k_cache, v_cache, k_scale, v_scale, offs, lens, table, o, lse, &own)) != JFA_OK) return st;
  if (groups > 0 && (!aligned(group_offs, 8) || !aligned(prefix_lens, 8) || (prefix_pages > 0 && !aligned(prefix_table, 4))))
    return JFA_ERR_INVALID_ARG;
  Paged prefix = own;
  prefix_request(groups, prefix_pages, &prefix);
  prefix.groups = group_offs;
  prefix.lens = prefix_lens;
  prefix.table = prefix_table;
  if (!ws || ((uintptr_t)ws & 255u) != 0) return JFA_ERR_WORKSPACE;
  PagedWs first, second;
  float *prior_o, *prior_lse;
  if (ws_bytes < shared_layout(prefix, own, ws, &first, &second, &prior_o, &prior_lse)) return JFA_ERR_WORKSPACE;
  first.hold = second.hold = g_paged_hold.load(std::memory_order_relaxed);
  prefix.phase = 1;
  own.phase = 2;
  prefix.prior_o = own.prior_o = prior_o;
  prefix.prior_lse = own.prior_lse = prior_lse;
  own.prior_status = &first.hdr->status;
  cudaStream_t s = (cudaStream_t)stream;
  // (no group, no sequence: nothing to find wrong in the prefixes)
  if ((st = groups > 0 ? run_paged(prefix, p->dtype, kShared, false, first, s)
                       : cu(cudaMemsetAsync(first.hdr, 0, sizeof(PagedHeader), s))) != JFA_OK)
    return st;
  own.few = paged_few(own);
  if (!paged_short(own) && (st = run_paged(own, p->dtype, kShared, false, second, s)) != JFA_OK) return st;
  if (own.few == 0) return JFA_OK;
  Timed t(JFA_KERNEL_PAGED, s);
  return cu(launch_paged_short(own, p->dtype, second.hdr, s));
}

}  // extern "C"
