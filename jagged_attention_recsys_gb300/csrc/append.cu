// New tokens appended to a paged cache in one pass: RMS norm and rotary positions of queries and keys
// (norm_rope.cu has the formulas), the queries to their place, the keys and the values to their pages,
// as they are or in MXFP8 (cache.cu has the format).
//
// Keys are coded from their fp32 values: no rounding to the queries' type comes between.
//
// Bound: HBM; each value is read once and written once, where three calls read and write the
// keys twice and launch four kernels.  A warp takes a run of up to 32 tokens, or part of a token's heads
// where there are fewer tokens than warps; its lanes first look up a token each (sequence, position,
// page: a chain of dependent loads that would otherwise be paid token by token).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cache.cuh"
#include "internal.h"
#include "norm_rope.cuh"
#include "serve.h"

namespace jfa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// The row of the cache for head 0 and the position for the rotation of new token t; row -1: none.
struct Place {
  int64_t row, pos;
};
__device__ __forceinline__ Place place_of(const Paged& p, const int64_t* pos, int64_t t, PagedHeader* hdr) {
  const int b = find_sequence(p, t);
  const int at = token_position(p, t, b, &hdr->status);
  const int page = at >= 0 ? paged_page(p, b, at, &hdr->status) : -1;
  Place r{-1, pos ? __ldg(pos + t) : __ldg(p.lens + b) - (__ldg(p.offs + b + 1) - t)};
  if (page >= 0) r.row = paged_row(p, page, 0, at);
  return r;
}

// ------------------------------------------------------------------ rows of any shape
// A warp a row, a lane a column of 32 at a time: a block of MXFP8 is the warp's.
template <typename T, int KIND>
__device__ __forceinline__ void put_block(T* cache, uint8_t* codes, uint8_t* scales, int64_t row, int dim, int c, float x) {
  if constexpr (KIND == kCacheMx) {
    float a = fabsf(x);  // a NaN is passed over, and stays one in its code
    for (int m = 16; m > 0; m >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, m));
    const int e = mx_scale_exp(a);
    codes[row * dim + c] = (uint8_t)e4m3_pair(x * exp2i(-e), 0.f);
    if ((c & 31) == 0) scales[row * (dim >> 5) + (c >> 5)] = (uint8_t)(e + 127);
  } else if (c < dim) {
    cache[row * dim + c] = from_f<T>(x);
  }
}

template <typename T, int KIND>
__global__ void __launch_bounds__(kThreads)
append_any_kernel(const __grid_constant__ Paged p, const __grid_constant__ NormRopeArgs a, PagedHeader* hdr, int planned) {
  __shared__ float rows[kWarps][kMaxNormDim];
  if (planned && *(volatile int*)&hdr->status == (int)JFA_ERR_BAD_OFFSETS) return;
  if (!planned) check_batch(p, hdr);
  const int lane = threadIdx.x & 31;
  float* y = rows[threadIdx.x >> 5];
  const int hq = a.side[0].heads, hk = p.heads_k, H = hq + 2 * hk;
  const int64_t n = p.total_q * H, nw = (int64_t)gridDim.x * kWarps;
  for (int64_t i = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); i < n; i += nw) {
    const int64_t t = i / H;
    const int h = (int)(i - t * H);
    Place at{-1, 0};
    if (lane == 0) at = place_of(p, a.pos, t, hdr);
    at.row = __shfl_sync(0xffffffffu, at.row, 0);
    at.pos = __shfl_sync(0xffffffffu, at.pos, 0);
    if (h >= hq + hk) {  // a row of values, as it is
      if (at.row < 0) continue;
      const int64_t row = at.row + ((int64_t)(h - hq - hk) << p.page_shift);
      const T* x = (const T*)p.v + t * p.sv + (int64_t)(h - hq - hk) * p.dim_v;
      for (int c0 = 0; c0 < p.dim_v; c0 += 32) {
        const int c = c0 + lane;
        put_block<T, KIND>((T*)p.vc, (uint8_t*)p.vc, p.vs, row, p.dim_v, c, c < p.dim_v ? to_f(x[c]) : 0.f);
      }
      continue;
    }
    const int side = h >= hq, head = side ? h - hq : h;
    const NormRopeSide& sd = a.side[side];
    const T* x = (const T*)sd.x + t * sd.sx + (int64_t)head * a.dim;
    float r = 1.f;
    if (a.norm) {
      float ss = 0.f;
      for (int c = lane; c < a.dim; c += 32) {
        const float v = to_f(x[c]);
        ss = fmaf(v, v, ss);
      }
      r = rsqrtf(fmaf(group_sum(ss, 32), a.inv_dim, a.eps));
    }
    auto norm = [&](int c) { return a.norm ? to_f(x[c]) * (r * (sd.w ? __ldg(sd.w + c) : 1.f)) : to_f(x[c]); };
    __syncwarp();  // the last row has left
    for (int k = lane; k < a.rot / 2; k += 32) {
      const float2 cs = rotation(at.pos, a.turn[k], a.amp);
      const int2 c = pair_cols(k, a.rot, a.layout);
      const float u = norm(c.x), w = norm(c.y);
      y[c.x] = fmaf(u, cs.x, -w * cs.y);
      y[c.y] = fmaf(u, cs.y, w * cs.x);
    }
    for (int c = a.rot + lane; c < a.dim; c += 32) y[c] = norm(c);
    __syncwarp();
    if (!side) {
      T* out = (T*)sd.out + t * sd.sout + (int64_t)head * a.dim;
      for (int c = lane; c < a.dim; c += 32) out[c] = from_f<T>(y[c]);
    } else if (at.row >= 0) {
      const int64_t row = at.row + ((int64_t)head << p.page_shift);
      for (int c0 = 0; c0 < a.dim; c0 += 32) {
        const int c = c0 + lane;
        put_block<T, KIND>((T*)p.kc, (uint8_t*)p.kc, p.ks, row, a.dim, c, c < a.dim ? y[c] : 0.f);
      }
    }
  }
}

template <typename T, int KIND>
cudaError_t append_t(const Paged& p, const NormRopeArgs& a, PagedHeader* hdr, int planned, cudaStream_t s) {
  const int64_t warps = p.total_q * (a.side[0].heads + 2 * p.heads_k), most = (int64_t)num_sms() * 8;
  int64_t grid = (warps + kWarps - 1) / kWarps;
  if (grid > most) grid = most;
  append_any_kernel<T, KIND><<<(unsigned)grid, kThreads, 0, s>>>(p, a, hdr, planned);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append(const Paged& p, const NormRopeArgs& a, int dtype, PagedHeader* hdr, int planned, cudaStream_t s) {
  if (dtype == JFA_BF16)
    return p.kind == kCacheMx ? append_t<__nv_bfloat16, kCacheMx>(p, a, hdr, planned, s)
                              : append_t<__nv_bfloat16, kCacheBf16>(p, a, hdr, planned, s);
  return p.kind == kCacheMx ? append_t<float, kCacheMx>(p, a, hdr, planned, s)
                            : append_t<float, kCacheF32>(p, a, hdr, planned, s);
}

}  // namespace jfa
