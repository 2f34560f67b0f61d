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
// would otherwise be paid token by token), then the warp goes through them.  A lane takes 16
// columns (two lanes share a block's maximum by one shuffle), consecutive over the token's heads,
// with a piece of the keys and one of the values in flight; 24 (write) or 32 warps an SM do the
// rest (two pieces each: 157 us for a write of 118 K tokens of 8 heads of 128, so 145).  Measured
// from bf16 to MXFP8: that write 145 us, 5.1 TB/s; 61 users read back 63 us, 4.4 TB/s.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "paged.cuh"

namespace jfa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// CTAs of an SM: a write's conversion to MXFP8 spills at four (154 us, so 145); a read wants the
// loads in flight (three: 68 us, so 63)
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

// Pieces of W columns of one token's tensor: a lane's next piece is 32 further on.
template <int W>
struct Piece {
  int c, head, col;  // index, head, piece of the head
  __device__ __forceinline__ Piece(int c0, int per) : c(c0), head(c0 / per), col(c0 - c0 / per * per) {}
  __device__ __forceinline__ void next(int per, int dh, int dc) {  // dh, dc: 32 / per and 32 % per
    c += 32;
    head += dh;
    col += dc;
    if (col >= per) {
      col -= per;
      ++head;
    }
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

template <typename T, int KIND, bool WRITE>
__global__ void __launch_bounds__(kThreads, kCtas<WRITE>)
cache_kernel(const __grid_constant__ Paged p, T* k_out, T* v_out, PagedHeader* hdr, int run, int parts, int planned) {
  constexpr bool MX = KIND == kCacheMx;
  constexpr int W = MX ? 16 : 8;
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
  const int lane = threadIdx.x & 31;
  const int perk = p.dim_qk / W, perv = p.dim_v / W;  // pieces of a head
  const int ck = p.heads_k * perk, cv = p.heads_k * perv;
  const int dhk = 32 / perk, dck = 32 - dhk * perk, dhv = 32 / perv, dcv = 32 - dhv * perv;
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
    for (int i = 0; i < n; ++i) {
      const int64_t t = t0 + i, r0 = __shfl_sync(0xffffffffu, row, i);
      const bool has = r0 >= 0;
      if (WRITE && !has) continue;
      // the token's rows of head 0, a head's step from there on, and the token's own rows
      constexpr int E = MX ? 1 : (int)sizeof(T);
      uint8_t *kc = (uint8_t*)p.kc + r0 * p.dim_qk * E, *vc = (uint8_t*)p.vc + r0 * p.dim_v * E;
      uint8_t *ks = p.ks + r0 * (p.dim_qk >> 5), *vs = p.vs + r0 * (p.dim_v >> 5);
      const uint32_t hk = (uint32_t)p.dim_qk * E << p.page_shift, hv = (uint32_t)p.dim_v * E << p.page_shift;
      const uint32_t hks = (uint32_t)(p.dim_qk >> 5) << p.page_shift, hvs = (uint32_t)(p.dim_v >> 5) << p.page_shift;
      const T *kin = (const T*)p.k + t * p.sk, *vin = (const T*)p.v + t * p.sv;
      T *kout = k_out + t * ck * W, *vout = v_out + t * cv * W;
      Piece<W> pk(k0 + lane, perk), pv(v0 + lane, perv);
      for (; pk.c - lane < k1 || pv.c - lane < v1; pk.next(perk, dhk, dck), pv.next(perv, dhv, dcv)) {
        const bool okk = pk.c < k1, okv = pv.c < v1;
        uint8_t *ck_at = kc + (uint64_t)pk.head * hk + pk.col * W * E, *cv_at = vc + (uint64_t)pv.head * hv + pv.col * W * E;
        uint8_t *sk_at = ks + (uint64_t)pk.head * hks + (pk.col >> 1), *sv_at = vs + (uint64_t)pv.head * hvs + (pv.col >> 1);
        Raw<T, W> rk, rv;
        rk.zero();
        rv.zero();
        if constexpr (WRITE) {
          if (okk) rk.load(kin + (uint32_t)pk.c * W);
          if (okv) rv.load(vin + (uint32_t)pv.c * W);
          if constexpr (MX) {
            write_mx<T>(rk, ck_at, sk_at, pk.col, okk);
            write_mx<T>(rv, cv_at, sv_at, pv.col, okv);
          } else {
            if (okk) rk.store((T*)ck_at);
            if (okv) rv.store((T*)cv_at);
          }
        } else {
          if constexpr (MX) {
            uint4 code_k = make_uint4(0u, 0u, 0u, 0u), code_v = code_k;
            float fk = 0.f, fv = 0.f;
            if (okk && has) {
              code_k = __ldcs(reinterpret_cast<const uint4*>(ck_at));
              fk = __uint_as_float((uint32_t)__ldg(sk_at) << 23);
            }
            if (okv && has) {
              code_v = __ldcs(reinterpret_cast<const uint4*>(cv_at));
              fv = __uint_as_float((uint32_t)__ldg(sv_at) << 23);
            }
            rk.set_mx(code_k, fk);
            rv.set_mx(code_v, fv);
          } else {
            if (okk && has) rk.load((const T*)ck_at);
            if (okv && has) rv.load((const T*)cv_at);
          }
          if (okk) rk.store(kout + (uint32_t)pk.c * W);
          if (okv) rv.store(vout + (uint32_t)pv.c * W);
        }
      }
    }
  }
}

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
