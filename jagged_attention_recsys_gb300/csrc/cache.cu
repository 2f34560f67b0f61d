// The paged cache: new keys and values written into their pages, as they are or in MXFP8,
// and read back.
//
// MXFP8: the columns of a row go in blocks of 32; a block has one power-of-two scale 2^e,
// e the smallest with max|x| <= 448 * 2^e, and e4m3 codes of x * 2^-e (exact product, one
// rounding to nearest even: at most 2^-4 of a normal code's value).  A page holds each key
// head's rows together, [page, head, position, column], so that the attention finds the
// positions of a page and head in one stretch.
//
// Bound: HBM (bytes in plus bytes out; nothing to compute).  A warp takes a run of up to 32
// consecutive tokens, or part of a token's heads where there are fewer tokens than warps: its
// lanes first look up a token each (sequence, position, page: a chain of dependent loads that
// would otherwise be paid token by token).  A lane then takes a piece of 16 columns of all heads'
// through all the run's tokens (two lanes share a block's maximum by one shuffle): its place in a
// token's rows is worked out once a run, not once a token, which took two thirds of the
// instructions (145 us and 63 us for the two figures below).
// In flight: four tokens of a lane in 24 warps for a write, two in 32 for a read.
// Measured, bf16 and MXFP8: 118 K tokens of 8 heads of 128 written in 132 us, 5.6 TB/s; 61 users
// of 8 heads of 128 and 64 read back in 54 us, 5.2 TB/s; 83% and 77% of the copy rate.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cache.cuh"

namespace jfa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// CTAs of an SM: a write with two (143 us) or a read with three (59 us) has less in flight, a read
// with five (61 us) too few registers
template <bool WRITE>
constexpr int kCtas = WRITE ? 3 : 4;

// W columns of a row as they lie in memory
template <typename T, int W>
struct Raw {
  static constexpr int N = W * sizeof(T) / 16;
  uint4 q[N];
  __device__ __forceinline__ void load(const T* x) {
#pragma unroll
    for (int i = 0; i < N; ++i) q[i] = __ldcs(reinterpret_cast<const uint4*>(x) + i);
  }
  __device__ __forceinline__ void store(T* y) const {
#pragma unroll
    for (int i = 0; i < N; ++i) reinterpret_cast<uint4*>(y)[i] = q[i];
  }
  __device__ __forceinline__ void store_past(T* y) const {  // past the L2: rows read back are read once
#pragma unroll
    for (int i = 0; i < N; ++i) __stcs(reinterpret_cast<uint4*>(y) + i, q[i]);
  }
  __device__ __forceinline__ void get(float (&v)[W]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 2) {
          v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
          v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        } else {
          v[4 * i + j] = __uint_as_float(w[j]);
        }
      }
    }
  }
  __device__ __forceinline__ void set(const float (&v)[W]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 2)  // the result's type: one rounding
          asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[j]) : "f"(v[8 * i + 2 * j + 1]), "f"(v[8 * i + 2 * j]));
        else
          w[j] = __float_as_uint(v[4 * i + j]);
      }
      q[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < N; ++i) q[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  // 16 codes times their scale
  __device__ __forceinline__ void set_mx(const uint4& c, float f) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    float x[W];
#pragma unroll
    for (int j = 0; j < W / 2; ++j) {
      const float2 y = e4m3_values((w[j >> 1] >> (16 * (j & 1))) & 0xffffu);
      x[2 * j] = y.x * f;
      x[2 * j + 1] = y.y * f;
    }
    set(x);
  }
};

// 16 columns as MXFP8.  All lanes call it (a block is two lanes'); `ok` says which have a row.
template <typename T>
__device__ __forceinline__ void write_mx(const Raw<T, 16>& raw, uint8_t* codes, uint8_t* scale, int col, bool ok) {
  float v[16], a = 0.f;
  raw.get(v);
#pragma unroll
  for (int i = 0; i < 16; ++i) a = fmaxf(a, fabsf(v[i]));  // a NaN is passed over, and stays one in its code
  a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
  const int e = mx_scale_exp(a);
  const float f = exp2i(-e);
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = e4m3_pair(v[4 * i] * f, v[4 * i + 1] * f) | e4m3_pair(v[4 * i + 2] * f, v[4 * i + 3] * f) << 16;
  if (ok) {
    *reinterpret_cast<uint4*>(codes) = make_uint4(c[0], c[1], c[2], c[3]);
    if ((col & 1) == 0) *scale = (uint8_t)(e + 127);
  }
}

// One of a token's tensors in the cache: n tokens from the one at `x` on, `stride` apart, whose
// rows of head 0 the warp's lanes hold.  A lane takes a piece of W columns, c of all heads', through
// all the tokens, U of them in flight: where a piece lies in a token's rows is worked out once.
template <typename T, int KIND, bool WRITE>
__device__ __forceinline__ void move_rows(T* x, int64_t stride, uint8_t* cache, uint8_t* scales, int dim,
                                          int page_shift, int c0, int c1, int64_t row, int n, int lane) {
  constexpr bool MX = KIND == kCacheMx;
  constexpr int W = MX ? 16 : 8, E = MX ? 1 : (int)sizeof(T), U = !WRITE || (MX && sizeof(T) == 4) ? 2 : 4;
  const int per = dim / W;
  const uint32_t row_bytes = (uint32_t)dim * E, row_scales = (uint32_t)dim >> 5;
  for (int c = c0 + lane; c - lane < c1; c += 32) {
    const bool ok = c < c1;
    const int head = c / per, col = c - head * per;
    uint8_t* at0 = cache + ((uint64_t)(row_bytes * (uint32_t)head) << page_shift) + col * W * E;
    uint8_t* sc0 = scales + ((uint64_t)(row_scales * (uint32_t)head) << page_shift) + (col >> 1);
    T* y = x + (int64_t)c * W;
    for (int i = 0; i < n; i += U) {
      int64_t r[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        r[u] = __shfl_sync(0xffffffffu, row, (i + u) & 31);
        if (i + u >= n) r[u] = -1;
      }
      if constexpr (WRITE) {
        Raw<T, W> raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (ok && r[u] >= 0) raw[u].load(y + (i + u) * stride);
          else raw[u].zero();
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const bool live = ok && r[u] >= 0;
          if constexpr (MX)
            write_mx<T>(raw[u], at0 + r[u] * row_bytes, sc0 + r[u] * row_scales, col, live);
          else if (live)
            raw[u].store((T*)(at0 + r[u] * row_bytes));
        }
      } else if constexpr (MX) {
        uint4 code[U];
        float f[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          code[u] = make_uint4(0u, 0u, 0u, 0u);
          f[u] = 0.f;
          if (ok && r[u] >= 0) {
            code[u] = __ldcs(reinterpret_cast<const uint4*>(at0 + r[u] * row_bytes));
            f[u] = __uint_as_float((uint32_t)__ldg(sc0 + r[u] * row_scales) << 23);
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          Raw<T, W> raw;
          raw.set_mx(code[u], f[u]);
          if (ok && i + u < n) raw.store_past(y + (i + u) * stride);
        }
      } else {
        Raw<T, W> raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          raw[u].zero();
          if (ok && r[u] >= 0) raw[u].load((const T*)(at0 + r[u] * row_bytes));
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (ok && i + u < n) raw[u].store_past(y + (i + u) * stride);
      }
    }
  }
}

// A call without tokens has its batch checked all the same.
__global__ void __launch_bounds__(kThreads)
cache_check_kernel(const __grid_constant__ Paged p, PagedHeader* hdr) {
  if (p.batch == 0 && __ldg(p.offs) != 0) hdr->status = JFA_ERR_BAD_OFFSETS;
  check_batch(p, hdr);
}

template <typename T, int KIND, bool WRITE>
__global__ void __launch_bounds__(kThreads, kCtas<WRITE>)
cache_kernel(const __grid_constant__ Paged p, T* k_out, T* v_out, PagedHeader* hdr, int run, int parts, int planned) {
  constexpr bool MX = KIND == kCacheMx;
  constexpr int W = MX ? 16 : 8;
  // a plan that found the batch invalid: nothing is computed (page errors do not stop the call,
  // so the check does not depend on what other CTAs have met so far)
  if (planned && *(volatile int*)&hdr->status == (int)JFA_ERR_BAD_OFFSETS) return;
  if (!planned) check_batch(p, hdr);
  const int lane = threadIdx.x & 31;
  const int perk = p.dim_qk / W, perv = p.dim_v / W;  // pieces of a head
  const int ck = p.heads_k * perk, cv = p.heads_k * perv;
  const int64_t runs = (p.total_q + run - 1) / run;
  const int64_t tasks = runs * parts, nw = (int64_t)gridDim.x * kWarps;
  for (int64_t task = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); task < tasks; task += nw) {
    const int64_t t0 = task / parts * run;
    const int part = (int)(task % parts);
    // this lane's token: its row of the cache for head 0, or -1
    int64_t row = -1;
    if (lane < run && t0 + lane < p.total_q) {
      const int b = find_sequence(p, t0 + lane);
      const int pos = token_position(p, t0 + lane, b, &hdr->status);
      const int page = pos >= 0 ? paged_page(p, b, pos, &hdr->status) : -1;
      if (page >= 0) row = paged_row(p, page, 0, pos);
    }
    const int n = (int)min((int64_t)run, p.total_q - t0);
    // a part is a stretch of whole groups of 32 pieces
    auto cut = [&](int m, int i) { return min(m, (int)((int64_t)((m + 31) / 32) * i / parts) * 32); };
    const int k0 = cut(ck, part), k1 = cut(ck, part + 1), v0 = cut(cv, part), v1 = cut(cv, part + 1);
    move_rows<T, KIND, WRITE>(WRITE ? (T*)p.k + t0 * p.sk : k_out + t0 * ck * W, WRITE ? p.sk : (int64_t)ck * W,
                              (uint8_t*)p.kc, p.ks, p.dim_qk, p.page_shift, k0, k1, row, n, lane);
    move_rows<T, KIND, WRITE>(WRITE ? (T*)p.v + t0 * p.sv : v_out + t0 * cv * W, WRITE ? p.sv : (int64_t)cv * W,
                              (uint8_t*)p.vc, p.vs, p.dim_v, p.page_shift, v0, v1, row, n, lane);
  }
}

}  // namespace

cudaError_t launch_cache_check(const Paged& p, PagedHeader* hdr, cudaStream_t s) {
  const int64_t need = (p.batch + kThreads - 1) / kThreads, cap = num_sms();
  cache_check_kernel<<<(unsigned)(need < 1 ? 1 : need < cap ? need : cap), kThreads, 0, s>>>(p, hdr);
  return cudaGetLastError();
}

namespace {

template <typename T, int KIND, bool WRITE>
cudaError_t launch_t(const Paged& p, void* k, void* v, PagedHeader* hdr, int planned, cudaStream_t s) {
  // Runs of up to 32 tokens, as long as lets every warp of a full GPU take the same number of them
  // (2.03 runs a warp cost three rounds); with fewer tokens than warps, several warps a token
  // instead (a serving step of 256 tokens would leave most SMs without work).
  constexpr int W = KIND == kCacheMx ? 16 : 8;
  const int64_t warps = (int64_t)num_sms() * kWarps * kCtas<WRITE>;
  const int64_t rounds = (p.total_q + 32 * warps - 1) / (32 * warps);
  const int64_t run = (p.total_q + rounds * warps - 1) / (rounds * warps);
  const int most = (p.heads_k * ((p.dim_qk > p.dim_v ? p.dim_qk : p.dim_v) / W) + 31) / 32;
  int64_t parts = run > 1 ? 1 : (warps + p.total_q - 1) / p.total_q;
  if (parts > most) parts = most;
  int64_t grid = ((p.total_q + run - 1) / run * parts + kWarps - 1) / kWarps;
  const int64_t cap = (int64_t)num_sms() * kCtas<WRITE>;
  if (grid > cap) grid = cap;
  cache_kernel<T, KIND, WRITE><<<(unsigned)grid, kThreads, 0, s>>>(p, (T*)k, (T*)v, hdr, (int)run, (int)parts, planned);
  return cudaGetLastError();
}
template <bool WRITE>
cudaError_t launch_kind(const Paged& p, int dtype, void* k, void* v, PagedHeader* hdr, int planned, cudaStream_t s) {
  if (p.total_q == 0) {
    if (planned) return cudaSuccess;
    return launch_cache_check(p, hdr, s);
  }
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
