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
  if ((st = check_index(p, offs, lens, table)) != JFA_OK ||
      (st = check_cache(p, k_cache, v_cache, k_scale, v_scale)) != JFA_OK ||
      (st = check_rows(p, q, p->stride_q, (int64_t)p->heads_q * p->dim_qk)) != JFA_OK)
    return st;
  if (p->total_q > 0 && (!aligned(o, 16) || !aligned(lse, 16))) return JFA_ERR_INVALID_ARG;
  Paged r = make_paged(p, offs, lens, table, k_cache, v_cache, k_scale, v_scale);
  PagedWs w;
  if ((st = check_ws(r, ws, ws_bytes, &w)) != JFA_OK) return st;
  r.q = q;
  r.o = o;
  r.lse = lse;
  cudaStream_t s = (cudaStream_t)stream;
  const int kernel = paged_kernel(r, p->dtype);
  const int ctas = paged_ctas(r, kernel);
  if (!(p->flags & JFA_PLANNED)) {
    if (p->total_q > 0 && p->batch <= kPlanInCta) w.ctas = ctas;
    else if ((st = plan_paged(r, kernel, w, s)) != JFA_OK) return st;
  }
  if (p->total_q == 0) return JFA_OK;
  const TileShape shape = paged_shape(r, kernel);
  Timed t(JFA_KERNEL_PAGED, s);
  st = cu(kernel == kPagedTc       ? launch_paged_tc(r, shape, ctas, w, s)
          : kernel == kPagedRows16 ? launch_paged_rows16(r, shape, ctas, w, s)
                                   : launch_paged_simt(r, shape, ctas, p->dtype, w, s));
  if (st != JFA_OK) return st;
  return cu(launch_paged_combine(r, shape, ctas, p->dtype, w, s));
}

}  // extern "C"
