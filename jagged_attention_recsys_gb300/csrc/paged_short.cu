// The second phase of attention behind shared prefixes for sequences with few keys of their own:
// candidates of a token or a few, scored against a long prefix.
//
// Bound: latency.  The tiled kernels take 7 us a tile here, of which the keys are nothing: the walk's
// look-ups, the loads' round trip through the ring and the join of four warps, one after the other (16
// users' 64 candidates of 1 to 4 tokens, 8,192 tiles: 191 us).  So a warp takes a token and a key head by
// itself, four query heads at a time.  For the scores two lanes have a key, half of its columns each,
// against queries in shared memory; for the output a lane has four columns of every key.  fp32
// throughout.  Those candidates take 50 us.  (A score as the warp's sum, two keys at a time: 44 us, but
// 27 where a few sequences of 16 keys are among 128 of more, which this takes 16 for.)
//
// The lengths are on the device, so that the tiled kernels are launched too unless the pages decide
// it, and pass over these sequences as this kernel does over the others (12 us where none has few keys).  The
// whole call with 2, 8, 12 and 16 own keys, and with the tiled kernels alone, us:
//   groups, heads, prefix                              pages of 16 keys     wider pages          tiled kernels
//   16 of 64 x 2 tokens, 32 on 8, 256 keys, bf16       97 115 124 136       111 128 142 150      142
//   64 of 16 x 1 token, 8 on 8, 500 keys, bf16         83 93 99 107         97 107 115 122       130
//   8 of 64 x 1 token, 32 on 8, 256 keys, bf16         68 72 76 81          78 83 87 91          92
//   4 of 32 x 4 tokens, 32 on 4, 1,000 keys, bf16      70 74 79 83          83 87 91 95          95
//   16 of 64 x 2 tokens, 32 on 8, 4,096 keys, bf16     228 244 255 265      242 259 267 279      271
//   the first, MXFP8                                   101 117 130 142      115 132 146 156      165
//   the last, MXFP8                                    257 271 285 296      271 283 298 310      320
//   8 of 64 x 1 token, 32 on 8 of 80, 64 keys, bf16    158 - 163 165        167 - 173 174        363-385 (CUDA cores)
//   the same, heads of 128, fp32                       232 - 243 248        244 - 255 259        451-583 (CUDA cores)
// So it takes up to 16 keys, but beside the tensor-core kernels over bf16 pages that may hold more, where those are
// launched anyway, up to 12.  With more than 16 tokens a sequence on average hardly one has so few, and the tiled
// kernels take all.
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
constexpr int H = 4, K = 4;  // query heads, and values, at a time
constexpr int kFew = 16;     // own keys at most: half a warp's lanes
constexpr int kFewWide = 12;  // and beside tensor-core kernels over bf16 pages that may hold more
constexpr int kMaxDim = 128;
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
__device__ __forceinline__ void add4(float4& s, float k, const float4& q) {
  s = make_float4(fmaf(k, q.x, s.x), fmaf(k, q.y, s.y), fmaf(k, q.z, s.z), fmaf(k, q.w, s.w));
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
__global__ void __launch_bounds__(kThreads, 4)
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
  // the queries' four heads of a column side by side, so that a lane reads them at once
  __shared__ float4 queries[kWarps][kMaxDim];
  float4* qs = queries[threadIdx.x >> 5];
  const int lane = threadIdx.x & 31, c = 4 * lane;
  const bool in_v = c < p.dim_v;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  const float to_log2 = p.scale * kLog2e;
  const int key = lane & (kFew - 1), half = p.dim_qk / 2, c0 = lane / kFew * half;
  const int parts = (p.group + H - 1) / H;  // of a key head's query heads
  const int64_t tasks = p.total_q * p.heads_k * parts, nw = (int64_t)gridDim.x * kWarps;
  for (int64_t task = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); task < tasks; task += nw) {
    const int64_t t = task / (p.heads_k * parts);
    const int rest = (int)(task % (p.heads_k * parts)), head_k = rest / parts;
    const int h0 = head_k * p.group + rest % parts * H, hn = min(H, p.group - rest % parts * H);
    const int64_t row0 = t * p.heads_q + h0;
    const int b = find_sequence(p, t);
    const int64_t len = __ldg(p.lens + b), pos = len - (__ldg(p.offs + b + 1) - t);
    if (len > p.few) continue;  // the tiled kernels'
    const int n = (int)max((int64_t)0, p.causal ? min(len, pos + 1) : len);  // keys the rows see
    int64_t mine = -1;  // the row of this lane's key
    if (key < n) {
      const int page = paged_page(p, b, key, &hdr->status);
      if (page >= 0) mine = paged_row(p, page, head_k, key);
    }
    float4 q[H];
#pragma unroll
    for (int h = 0; h < H; ++h)
      q[h] = h < hn && c < p.dim_qk ? four((const T*)p.q + t * p.sq + (int64_t)(h0 + h) * p.dim_qk + c) : zero;
    __syncwarp();  // the last row's have been read
    if (c < p.dim_qk) {
      qs[c] = make_float4(q[0].x, q[1].x, q[2].x, q[3].x);
      qs[c + 1] = make_float4(q[0].y, q[1].y, q[2].y, q[3].y);
      qs[c + 2] = make_float4(q[0].z, q[1].z, q[2].z, q[3].z);
      qs[c + 3] = make_float4(q[0].w, q[1].w, q[2].w, q[3].w);
    }
    __syncwarp();
    // scores of this lane's key, over its half of the columns
    float4 s4 = zero;
    if (mine >= 0) {
#pragma unroll 8
      for (int i = 0; i < half; i += 4) {
        const float4 k = cached<KIND>(p.kc, p.ks, mine, p.dim_qk, c0 + i);
        add4(s4, k.x, qs[c0 + i]);
        add4(s4, k.y, qs[c0 + i + 1]);
        add4(s4, k.z, qs[c0 + i + 2]);
        add4(s4, k.w, qs[c0 + i + 3]);
      }
    }
    float s[H] = {s4.x, s4.y, s4.z, s4.w}, m[H], l[H];
    float4 o[H];
#pragma unroll
    for (int h = 0; h < H; ++h) {
      s[h] += __shfl_xor_sync(0xffffffffu, s[h], kFew);
      s[h] = key < n ? s[h] * to_log2 : -INFINITY;  // behind a bad page: a key of zeros
      m[h] = s[h];
#pragma unroll
      for (int x = kFew / 2; x > 0; x >>= 1) m[h] = fmaxf(m[h], __shfl_xor_sync(0xffffffffu, m[h], x));
      s[h] = exp2f(s[h] - (m[h] == -INFINITY ? 0.f : m[h]));
      l[h] = s[h];
#pragma unroll
      for (int x = kFew / 2; x > 0; x >>= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], x);
      o[h] = zero;
    }
    for (int i = 0; i < n; i += K) {
      float4 v[K];
#pragma unroll
      for (int u = 0; u < K; ++u) {
        const int64_t row = __shfl_sync(0xffffffffu, mine, (i + u) & (kFew - 1));
        v[u] = i + u < n && row >= 0 && in_v ? cached<KIND>(p.vc, p.vs, row, p.dim_v, c) : zero;
      }
#pragma unroll
      for (int u = 0; u < K; ++u)
#pragma unroll
        for (int h = 0; h < H; ++h) {
          const float e = __shfl_sync(0xffffffffu, s[h], (i + u) & (kFew - 1));
          o[h] = make_float4(fmaf(e, v[u].x, o[h].x), fmaf(e, v[u].y, o[h].y), fmaf(e, v[u].z, o[h].z), fmaf(e, v[u].w, o[h].w));
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

int paged_few(const Paged& p) {
  if (p.total_q > kFew * p.batch) return 0;
  if (p.kind != kCacheBf16 || ((int64_t)p.width << p.page_shift) <= kFew) return kFew;
  return paged_kernel(p, JFA_BF16) == kPagedSimt ? kFew : kFewWide;
}
bool paged_short(const Paged& p) { return paged_few(p) > 0 && ((int64_t)p.width << p.page_shift) <= kFew; }

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
