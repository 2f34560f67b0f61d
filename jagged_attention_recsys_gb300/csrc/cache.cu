// The paged cache: new keys and values written into their pages, as they are or in MXFP8,
// and read back.
//
// MXFP8: the columns of a row go in blocks of 32; a block has one power-of-two scale 2^e,
// e the smallest with max|x| <= 448 * 2^e, and e4m3 codes of x * 2^-e (exact product, one
// rounding to nearest even: at most 2^-4 of a normal code's value).  A page holds each key
// head's rows together, [page, head, position, column], so that the attention finds the
// positions of a page and head in one stretch.
//
// Bound: HBM (bytes in plus bytes out; nothing to compute).  A warp takes a token, or part of
// one where there are fewer tokens than warps; a lane takes eight columns, so a row of 128
// is half a warp, loads are 16 (bf16) or 32 bytes a lane and consecutive over the token's
// heads, and four lanes share a block's maximum by two shuffles.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "paged.cuh"

namespace jfa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ void load8(float (&v)[8], const __nv_bfloat16* x) {
  const uint4 a = __ldcs(reinterpret_cast<const uint4*>(x));
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(float (&v)[8], const float* x) {
  const float4 a = __ldcs(reinterpret_cast<const float4*>(x)), b = __ldcs(reinterpret_cast<const float4*>(x) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* y, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // the result's type: one rounding
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
  }
  *reinterpret_cast<uint4*>(y) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* y, const float (&v)[8]) {
  reinterpret_cast<float4*>(y)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(y)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

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

// Eight columns of a row into the cache.  All lanes call it; `ok` says which have a row.
template <typename T, int KIND>
__device__ __forceinline__ void write8(const Paged& p, void* codes, uint8_t* scales, int64_t row, int chunk, int dim,
                                       const float (&v)[8], bool ok) {
  if constexpr (KIND == kCacheMx) {
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(v[i]));  // a NaN is passed over, and stays one in its code
    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
    const int e = mx_scale_exp(a);
    const float f = exp2i(-e);
    if (ok) {
      uint2 c;
      c.x = e4m3_pair(v[0] * f, v[1] * f) | e4m3_pair(v[2] * f, v[3] * f) << 16;
      c.y = e4m3_pair(v[4] * f, v[5] * f) | e4m3_pair(v[6] * f, v[7] * f) << 16;
      *reinterpret_cast<uint2*>((uint8_t*)codes + row * dim + chunk * 8) = c;
      if ((chunk & 3) == 0) scales[row * (dim >> 5) + (chunk >> 2)] = (uint8_t)(e + 127);
    }
  } else {
    if (ok) store8((T*)codes + row * dim + chunk * 8, v);
  }
}
template <typename T, int KIND>
__device__ __forceinline__ void read8(float (&v)[8], const void* codes, const uint8_t* scales, int64_t row, int chunk,
                                      int dim) {
  if constexpr (KIND == kCacheMx) {
    const uint2 c = __ldcs(reinterpret_cast<const uint2*>((const uint8_t*)codes + row * dim + chunk * 8));
    const float f = __uint_as_float((uint32_t)__ldg(scales + row * (dim >> 5) + (chunk >> 2)) << 23);
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = e4m3_values((w[i >> 1] >> (16 * (i & 1))) & 0xffffu);
      v[2 * i] = x.x * f;
      v[2 * i + 1] = x.y * f;
    }
  } else {
    load8(v, (const T*)codes + row * dim + chunk * 8);
  }
}

// One tensor of a token: chunks [c0, c1) of its heads * dim / 8.
template <typename T, int KIND, bool WRITE>
__device__ __forceinline__ void token_rows(const Paged& p, int64_t t, int pos, int page, int c0, int c1, int dim,
                                           const T* in, int64_t stride, T* out, void* codes, uint8_t* scales) {
  const int lane = threadIdx.x & 31, per = dim / 8;
  constexpr int U = 4;  // chunks a lane has in flight
  for (int base = c0; base < c1; base += 32 * U) {
    float v[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = base + 32 * u + lane;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] = 0.f;
      if (c < c1) {
        if (WRITE) load8(v[u], in + t * stride + (int64_t)c * 8);
        else if (page >= 0) read8<T, KIND>(v[u], codes, scales, paged_row(p, page, c / per, pos), c % per, dim);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = base + 32 * u + lane;
      if (WRITE) {
        const int h = c / per;
        write8<T, KIND>(p, codes, scales, paged_row(p, page, h, pos), c - h * per, dim, v[u], c < c1);
      } else if (c < c1) {
        store8(out + (t * p.heads_k * (int64_t)dim + (int64_t)c * 8), v[u]);
      }
    }
  }
}

template <typename T, int KIND, bool WRITE>
__global__ void __launch_bounds__(kThreads)
cache_kernel(const __grid_constant__ Paged p, T* k_out, T* v_out, PagedHeader* hdr, int parts, int planned) {
  // a plan that found the batch invalid: nothing is computed (page errors do not stop the call,
  // so the check does not depend on what other CTAs have met so far)
  if (planned && *(volatile int*)&hdr->status == (int)JFA_ERR_BAD_OFFSETS) return;
  if (!planned) {  // the whole batch's description, once per call
    const int64_t most = (int64_t)p.width << p.page_shift;
    for (int64_t b = (int64_t)blockIdx.x * kThreads + threadIdx.x; b < p.batch; b += (int64_t)gridDim.x * kThreads) {
      const int64_t lo = __ldg(p.offs + b), hi = __ldg(p.offs + b + 1), len = __ldg(p.lens + b);
      if (hi < lo || (b == 0 && lo != 0) || (b == p.batch - 1 && hi != p.total_q) || len < 0 || len > most)
        atomicExch(&hdr->status, (int)JFA_ERR_BAD_OFFSETS);
    }
  }
  const int64_t tasks = p.total_q * parts, nw = (int64_t)gridDim.x * kWarps;
  const int ck = p.heads_k * (p.dim_qk / 8), cv = p.heads_k * (p.dim_v / 8);
  for (int64_t task = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); task < tasks; task += nw) {
    const int64_t t = task / parts;
    const int part = (int)(task - t * parts);
    const int b = find_sequence(p, t);
    const int pos = token_position(p, t, b, &hdr->status);
    const int page = pos >= 0 ? paged_page(p, b, pos, &hdr->status) : -1;
    if (WRITE && page < 0) continue;
    // a part is a stretch of whole groups of 32 chunks
    auto cut = [&](int n, int i) { return min(n, (int)(((int64_t)((n + 31) / 32) * i / parts) * 32)); };
    token_rows<T, KIND, WRITE>(p, t, max(pos, 0), page, cut(ck, part), cut(ck, part + 1), p.dim_qk, (const T*)p.k,
                               p.sk, k_out, p.kc, p.ks);
    token_rows<T, KIND, WRITE>(p, t, max(pos, 0), page, cut(cv, part), cut(cv, part + 1), p.dim_v, (const T*)p.v,
                               p.sv, v_out, p.vc, p.vs);
  }
}

template <typename T, int KIND, bool WRITE>
cudaError_t launch_t(const Paged& p, void* k, void* v, PagedHeader* hdr, int planned, cudaStream_t s) {
  // warps a token: one, more where the tokens alone do not fill the GPU
  const int64_t warps = (int64_t)num_sms() * kWarps * 4;
  const int most = (p.heads_k * ((p.dim_qk > p.dim_v ? p.dim_qk : p.dim_v) / 8) + 31) / 32;
  int64_t parts = (warps + p.total_q - 1) / p.total_q;
  if (parts > most) parts = most;
  int64_t grid = (p.total_q * parts + kWarps - 1) / kWarps;
  const int64_t cap = (int64_t)num_sms() * 8;
  if (grid > cap) grid = cap;
  cache_kernel<T, KIND, WRITE><<<(unsigned)grid, kThreads, 0, s>>>(p, (T*)k, (T*)v, hdr, (int)parts, planned);
  return cudaGetLastError();
}
template <bool WRITE>
cudaError_t launch_kind(const Paged& p, int dtype, void* k, void* v, PagedHeader* hdr, int planned, cudaStream_t s) {
  if (p.total_q == 0) return cudaSuccess;
  if (dtype == JFA_BF16)
    return p.kind == kCacheMx ? launch_t<__nv_bfloat16, kCacheMx, WRITE>(p, k, v, hdr, planned, s)
                              : launch_t<__nv_bfloat16, kCacheBf16, WRITE>(p, k, v, hdr, planned, s);
  return p.kind == kCacheMx ? launch_t<float, kCacheMx, WRITE>(p, k, v, hdr, planned, s)
                            : launch_t<float, kCacheF32, WRITE>(p, k, v, hdr, planned, s);
}

}  // namespace

cudaError_t launch_cache_write(const Paged& p, int dtype, PagedHeader* hdr, int planned, cudaStream_t s) {
  return launch_kind<true>(p, dtype, nullptr, nullptr, hdr, planned, s);
}
cudaError_t launch_cache_read(const Paged& p, int dtype, void* k, void* v, PagedHeader* hdr, int planned, cudaStream_t s) {
  return launch_kind<false>(p, dtype, k, v, hdr, planned, s);
}

}  // namespace jfa
