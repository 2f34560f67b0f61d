// The second phase of attention behind shared prefixes for sequences with few keys of their own:
// candidates of a token or a few, scored against a long prefix.
//
// Bound: latency.  The tiled kernels take 7 us a tile here, of which the keys are nothing: the walk's
// look-ups, the loads' round trip through the ring and the join of four warps, one after the other (16
// users' 64 candidates of 1 to 4 tokens, 8,192 tiles: 191 us).  So a warp takes a token and a key head by
// itself, four query heads at a time: a lane has four columns, keys are looked up 32 at a time and
// loaded four at once, a score is the warp's sum.  fp32 throughout.  What phase 1 left of the rows is
// asked for first and used last.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cache.cuh"
#include "internal.h"
#include "paged_join.cuh"
#include "serve.h"

namespace jfa {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kScan = 4 * kThreads;  // sequences that a CTA checks by itself
// Query heads and keys at a time, and CTAs an SM, for the figure above: four keys at a time in three
// CTAs 53 us, in four 49; two keys in five 50; one key in six 56.
constexpr int H = 4, K = 2, kCtas = 4;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float4 four(const __nv_bfloat16* x) {
  const uint2 w = __ldg(reinterpret_cast<const uint2*>(x));
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xffff0000u));
}
__device__ __forceinline__ float4 four(const float* x) { return __ldg(reinterpret_cast<const float4*>(x)); }
__device__ __forceinline__ void put(__nv_bfloat16* y, const float4& v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(y) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ void put(float* y, const float4& v) { *reinterpret_cast<float4*>(y) = v; }

// Columns c .. c + 3 of a cache row
template <int KIND>
__device__ __forceinline__ float4 cached(const void* values, const uint8_t* scales, int64_t row, int dim, int c) {
  if constexpr (KIND == kCacheF32) return four((const float*)values + row * dim + c);
  if constexpr (KIND == kCacheBf16) return four((const __nv_bfloat16*)values + row * dim + c);
  const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>((const uint8_t*)values + row * dim + c));
  const float f = __uint_as_float((uint32_t)__ldg(scales + row * (dim >> 5) + (c >> 5)) << 23);
  const float2 a = e4m3_values(w & 0xffffu), b = e4m3_values(w >> 16);
  return make_float4(a.x * f, a.y * f, b.x * f, b.y * f);
}
__device__ __forceinline__ float dot4(const float4& a, const float4& b) {
  return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, a.w * b.w)));
}

// A batch that is none becomes the call's status, unless a wait of phase 1 ran out.
__device__ __forceinline__ void record_bad(PagedHeader* hdr) {
  if (atomicCAS(&hdr->status, (int)JFA_OK, (int)JFA_ERR_BAD_OFFSETS) == (int)JFA_ERR_BAD_PAGES)
    atomicCAS(&hdr->status, (int)JFA_ERR_BAD_PAGES, (int)JFA_ERR_BAD_OFFSETS);
}
__device__ __forceinline__ bool is_bad(const Paged& p, int64_t b) {
  const int64_t lo = __ldg(p.offs + b), hi = __ldg(p.offs + b + 1), len = __ldg(p.lens + b);
  return lo < 0 || hi < lo || hi > p.total_q || (b == 0 && lo != 0) || (b == p.batch - 1 && hi != p.total_q) || len < 0 ||
         len > ((int64_t)p.width << p.page_shift);
}
__global__ void __launch_bounds__(kThreads)
paged_short_check_kernel(const __grid_constant__ Paged p, PagedHeader* hdr) {
  if (p.batch == 0 && blockIdx.x == 0 && threadIdx.x == 0 && __ldg(p.offs) != 0) record_bad(hdr);
  for (int64_t b = (int64_t)blockIdx.x * kThreads + threadIdx.x; b < p.batch; b += (int64_t)gridDim.x * kThreads)
    if (is_bad(p, b)) record_bad(hdr);
}

template <typename T, int KIND>
__global__ void __launch_bounds__(kThreads, kCtas)
paged_short_kernel(const __grid_constant__ Paged p, PagedHeader* hdr) {
  if (p.batch <= kScan) {
    bool bad = *(volatile int*)&hdr->status == (int)JFA_ERR_BAD_OFFSETS;
#pragma unroll
    for (int i = 0; i < kScan / kThreads; ++i) {
      const int64_t b = threadIdx.x + i * kThreads;
      if (b < p.batch) bad |= is_bad(p, b);
    }
    if (__syncthreads_or(bad)) {
      if (blockIdx.x == 0 && threadIdx.x == 0) record_bad(hdr);
      return;
    }
  } else if (*(volatile int*)&hdr->status == (int)JFA_ERR_BAD_OFFSETS) {
    return;  // phase 1 or the check in front found it
  }
  const int lane = threadIdx.x & 31, c = 4 * lane;
  const bool in_k = c < p.dim_qk, in_v = c < p.dim_v;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  const float to_log2 = p.scale * kLog2e;
  const int parts = (p.group + H - 1) / H;  // of a key head's query heads
  const int64_t tasks = p.total_q * p.heads_k * parts, nw = (int64_t)gridDim.x * kWarps;
  for (int64_t task = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); task < tasks; task += nw) {
    const int64_t t = task / (p.heads_k * parts);
    const int rest = (int)(task % (p.heads_k * parts)), head_k = rest / parts;
    const int h0 = head_k * p.group + rest % parts * H, hn = min(H, p.group - rest % parts * H);
    const int64_t row0 = t * p.heads_q + h0;
    float4 q[H];
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const bool on = h < hn;
      q[h] = on && in_k ? four((const T*)p.q + t * p.sq + (int64_t)(h0 + h) * p.dim_qk + c) : zero;
    }
    const int b = find_sequence(p, t);
    const int64_t len = __ldg(p.lens + b), pos = len - (__ldg(p.offs + b + 1) - t);
    const int n = (int)max((int64_t)0, p.causal ? min(len, pos + 1) : len);  // keys the rows see
    float m[H], l[H];
    float4 o[H];
#pragma unroll
    for (int h = 0; h < H; ++h) {
      m[h] = -INFINITY;
      l[h] = 0.f;
      o[h] = zero;
    }
    for (int j0 = 0; j0 < n; j0 += 32) {
      int64_t mine = -1;  // this lane's key
      if (j0 + lane < n) {
        const int page = paged_page(p, b, j0 + lane, &hdr->status);
        if (page >= 0) mine = paged_row(p, page, head_k, j0 + lane);
      }
      const int most = min(32, n - j0);
      for (int i = 0; i < most; i += K) {
        float4 k[K], v[K];
#pragma unroll
        for (int u = 0; u < K; ++u) {
          const int64_t row = __shfl_sync(0xffffffffu, mine, (i + u) & 31);
          const bool there = i + u < most && row >= 0;  // behind a bad page: zeros
          k[u] = there && in_k ? cached<KIND>(p.kc, p.ks, row, p.dim_qk, c) : zero;
          v[u] = there && in_v ? cached<KIND>(p.vc, p.vs, row, p.dim_v, c) : zero;
        }
        float s[H][K];
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
          for (int u = 0; u < K; ++u) s[h][u] = dot4(q[h], k[u]);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1)
#pragma unroll
          for (int h = 0; h < H; ++h)
#pragma unroll
            for (int u = 0; u < K; ++u) s[h][u] += __shfl_xor_sync(0xffffffffu, s[h][u], x);
#pragma unroll
        for (int h = 0; h < H; ++h) {
          float top = m[h];
#pragma unroll
          for (int u = 0; u < K; ++u) {
            s[h][u] = i + u < most ? s[h][u] * to_log2 : -INFINITY;
            top = fmaxf(top, s[h][u]);
          }
          const float ref = top == -INFINITY ? 0.f : top, a = exp2f(m[h] - ref);
          m[h] = top;
          l[h] *= a;
          o[h] = make_float4(o[h].x * a, o[h].y * a, o[h].z * a, o[h].w * a);
#pragma unroll
          for (int u = 0; u < K; ++u) {
            const float e = exp2f(s[h][u] - ref);
            l[h] += e;
            o[h] = make_float4(fmaf(e, v[u].x, o[h].x), fmaf(e, v[u].y, o[h].y), fmaf(e, v[u].z, o[h].z),
                               fmaf(e, v[u].w, o[h].w));
          }
        }
      }
    }
    // phase 1's share of the rows; asked for ahead of the keys it would cost registers and so warps (51 us)
    float4 prior[H];
    float prior_lse[H];
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const bool on = h < hn;
      prior[h] = on && in_v ? *reinterpret_cast<const float4*>(p.prior_o + (row0 + h) * p.dim_v + c) : zero;
      prior_lse[h] = on ? p.prior_lse[row0 + h] : 0.f;
    }
#pragma unroll
    for (int h = 0; h < H; ++h) {
      if (h >= hn) break;
      const PagedJoin j = paged_join_prior(m[h], l[h], prior_lse[h]);
      if (in_v)
        put((T*)p.o + (row0 + h) * p.dim_v + c,
            make_float4(fmaf(prior[h].x, j.prior, o[h].x * j.own), fmaf(prior[h].y, j.prior, o[h].y * j.own),
                        fmaf(prior[h].z, j.prior, o[h].z * j.own), fmaf(prior[h].w, j.prior, o[h].w * j.own)));
      if (lane == 0) p.lse[row0 + h] = j.lse;
    }
  }
}

template <typename T, int KIND>
cudaError_t short_t(const Paged& p, PagedHeader* hdr, cudaStream_t s) {
  const int64_t warps = p.total_q * p.heads_k * ((p.group + H - 1) / H), most = (int64_t)num_sms() * 8;
  int64_t grid = (warps + kWarps - 1) / kWarps;
  if (grid > most) grid = most;
  paged_short_kernel<T, KIND><<<(unsigned)grid, kThreads, 0, s>>>(p, hdr);
  return cudaGetLastError();
}

}  // namespace

bool paged_short(const Paged& p) { return ((int64_t)p.width << p.page_shift) <= kShortKeys; }

cudaError_t launch_paged_short(const Paged& p, int dtype, PagedHeader* hdr, cudaStream_t s) {
  if (p.batch > kScan || p.total_q == 0) {
    const int64_t need = (p.batch + kThreads - 1) / kThreads, most = num_sms();
    paged_short_check_kernel<<<(unsigned)(need < 1 ? 1 : need < most ? need : most), kThreads, 0, s>>>(p, hdr);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || p.total_q == 0) return e;
  }
  if (dtype == JFA_BF16)
    return p.kind == kCacheMx ? short_t<__nv_bfloat16, kCacheMx>(p, hdr, s) : short_t<__nv_bfloat16, kCacheBf16>(p, hdr, s);
  return p.kind == kCacheMx ? short_t<float, kCacheMx>(p, hdr, s) : short_t<float, kCacheF32>(p, hdr, s);
}

}  // namespace jfa
