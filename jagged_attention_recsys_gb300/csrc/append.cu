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
//
// Measured: 64 prompts of up to 4,096 tokens, 32 + 8 heads of 128, to MXFP8: 590 us, 83% of the copy rate
// (four rows of a lane on their way; six 701, three 600, two 636; three CTAs an SM; two 663, four 603);
// a warp a row instead, 5,476.  Rows that do not divide into slots take that: 64 K tokens of 32 + 8 heads of
// 80, bf16, with 20 columns rotated 1,994 us, with all 80 243; heads of 64 to MXFP8 with 34 rotated 2,045, with all
// 148.  61 sequences of up to 700 tokens in fp32, 8 heads of 80 with 48 columns
// in pairs: 60 us, 77%.  A token each of 256 users: 7.7 us on the GPU; the call on the host takes longer.
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

// ------------------------------------------------------------------ rows of whole lane slots
// Eight columns of a row as they go to the cache.
__device__ __forceinline__ void put_octet(__nv_bfloat16* y, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(y) = make_uint4(tc::pack_bf16(x[0], x[1]), tc::pack_bf16(x[2], x[3]), tc::pack_bf16(x[4], x[5]),
                                            tc::pack_bf16(x[6], x[7]));
}
__device__ __forceinline__ void put_octet(float* y, const float (&x)[8]) {
  const float4 q[2] = {make_float4(x[0], x[1], x[2], x[3]), make_float4(x[4], x[5], x[6], x[7])};
  store32(y, q);
}
__device__ __forceinline__ uint2 octet_codes(const float (&x)[8], float f) {
  return make_uint2(e4m3_pair(x[0] * f, x[1] * f) | e4m3_pair(x[2] * f, x[3] * f) << 16,
                    e4m3_pair(x[4] * f, x[5] * f) | e4m3_pair(x[6] * f, x[7] * f) << 16);
}
__device__ __forceinline__ float octet_max(const float (&x)[8]) {
  float m = fabsf(x[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));  // a NaN is passed over, and stays one in its code
  return m;
}
// A slot's columns [a, a + 8) and [b, b + 8) in order
template <int LAYOUT>
__device__ __forceinline__ void octets(const Slot16& s, float (&a)[8], float (&b)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (LAYOUT == JFA_ROPE_HALVES) {
      a[2 * j] = s.a[j].x;
      a[2 * j + 1] = s.a[j].y;
      b[2 * j] = s.b[j].x;
      b[2 * j + 1] = s.b[j].y;
    } else {
      float(&o)[8] = j < 2 ? a : b;
      const int k = 4 * (j & 1);
      o[k] = s.a[j].x;
      o[k + 1] = s.b[j].x;
      o[k + 2] = s.a[j].y;
      o[k + 3] = s.b[j].y;
    }
  }
}

// A warp's steps over a token: rows of queries, then of keys (32 / group rows of a side a step, a slot a
// lane), then pieces of 16 columns of values, 32 a step.  parts warps share a token's steps.
struct AppendShape {
  int group, slots, run, parts;
};

template <typename T, int LAYOUT, int KIND>
__global__ void __launch_bounds__(kThreads, 3)
append_kernel(const __grid_constant__ Paged p, const __grid_constant__ NormRopeArgs a, const AppendShape g, PagedHeader* hdr,
              int planned) {
  constexpr bool MX = KIND == kCacheMx;
  constexpr int U = Raw16<T>::kBatch;
  __shared__ __align__(16) float tables[kWarps][2 * kMaxPairs];
  __shared__ __align__(16) float weights[2][kMaxNormDim];
  __shared__ __align__(16) float tops[MX ? kWarps : 1][64];  // largest values of the octets of a step's rows
  if (planned && *(volatile int*)&hdr->status == (int)JFA_ERR_BAD_OFFSETS) return;
  if (!planned) check_batch(p, hdr);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < 2 * a.dim; i += kThreads) {
    const float* w = a.side[i >= a.dim].w;
    weights[i >= a.dim][plane_at<LAYOUT == JFA_ROPE_HALVES ? 2 : 4>(i % a.dim, kMaxNormDim)] = w ? w[i % a.dim] : 1.f;
  }
  __syncthreads();
  float* tb = tables[warp];
  const int per = 32 / g.group, sub = lane / g.group, ls = lane % g.group;
  const bool lane_ok = ls < g.slots;
  const Slot sl = slot_of(lane_ok ? ls : 0, a.rot, LAYOUT);
  Turns turns;
  turns.init(a, lane);
  const int steps_q = (a.side[0].heads + per - 1) / per, steps_k = steps_q + (p.heads_k + per - 1) / per;
  const int pieces = p.heads_k * (p.dim_v / V), steps = steps_k + (pieces + 31) / 32;
  const int64_t runs = (p.total_q + g.run - 1) / g.run;
  const int64_t tasks = runs * g.parts, nw = (int64_t)gridDim.x * kWarps;
  for (int64_t task = (int64_t)blockIdx.x * kWarps + warp; task < tasks; task += nw) {
    const int64_t t0 = task / g.parts * g.run;
    const int part = (int)(task % g.parts);
    const int s0 = (int)((int64_t)steps * part / g.parts), s1 = (int)((int64_t)steps * (part + 1) / g.parts);
    const int n = (int)min((int64_t)g.run, p.total_q - t0);
    Place mine{-1, 0};
    if (lane < n) mine = place_of(p, a.pos, t0 + lane, hdr);
    for (int i = 0; i < n; ++i) {
      const int64_t t = t0 + i, row0 = __shfl_sync(0xffffffffu, mine.row, i);
      bool fresh = a.rot > 0;
      for (int sb = s0; sb < s1; sb += U) {
        Raw16<T> raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int st = sb + u;
          raw[u].zero();
          if (st < s1 && st < steps_k) {
            const int side = st >= steps_q, h = (st - (side ? steps_q : 0)) * per + sub;
            const NormRopeSide& sd = a.side[side];
            if (h < sd.heads && lane_ok) {
              const T* x = (const T*)sd.x + t * sd.sx + (int64_t)h * a.dim;
              raw[u].load(x + sl.a, x + sl.b);
            }
          } else if (st < s1) {
            const int c = (st - steps_k) * 32 + lane;
            if (c < pieces) {
              const T* x = (const T*)p.v + t * p.sv + (int64_t)c * V;
              raw[u].load(x, x + 8);
            }
          }
        }
        if (fresh && sb < steps_k) {  // under the first rows' loads
          turns.table(tb, a, __shfl_sync(0xffffffffu, mine.pos, i), lane);
          fresh = false;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int st = sb + u;
          if (st >= s1) break;
          if (st >= steps_k) {
            // ---- values, as they are
            const int c = (st - steps_k) * 32 + lane, head = c / (p.dim_v / V), col = c % (p.dim_v / V) * V;
            const int64_t row = row0 + ((int64_t)head << p.page_shift);
            const bool ok = c < pieces && row0 >= 0;
            Slot16 v;
            raw[u].template get<JFA_ROPE_HALVES>(v);
            float x[8], y[8];
            octets<JFA_ROPE_HALVES>(v, x, y);
            if constexpr (MX) {
              float m = fmaxf(octet_max(x), octet_max(y));
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));  // a block is two lanes'
              const int e = mx_scale_exp(m);
              const uint2 lo = octet_codes(x, exp2i(-e)), hi = octet_codes(y, exp2i(-e));
              if (ok) {
                *reinterpret_cast<uint4*>((uint8_t*)p.vc + row * p.dim_v + col) = make_uint4(lo.x, lo.y, hi.x, hi.y);
                if ((lane & 1) == 0) p.vs[row * (p.dim_v >> 5) + (col >> 5)] = (uint8_t)(e + 127);
              }
            } else if (ok) {
              put_octet((T*)p.vc + row * p.dim_v + col, x);
              put_octet((T*)p.vc + row * p.dim_v + col + 8, y);
            }
            continue;
          }
          const int side = st >= steps_q, h = (st - (side ? steps_q : 0)) * per + sub;
          const NormRopeSide& sd = a.side[side];
          Slot16 v;
          raw[u].template get<LAYOUT>(v);
          if (a.norm) {
            float2 ss = tc::fmul2(v.a[0], v.a[0]);
#pragma unroll
            for (int j = 1; j < 4; ++j) ss = tc::ffma2(v.a[j], v.a[j], ss);
#pragma unroll
            for (int j = 0; j < 4; ++j) ss = tc::ffma2(v.b[j], v.b[j], ss);
            const float r = rsqrtf(fmaf(group_sum(ss.x + ss.y, g.group), a.inv_dim, a.eps));
            const float2 rr = make_float2(r, r);
            Slot16 w;
            weights16<LAYOUT>(w, weights[side], sl);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              v.a[j] = tc::fmul2(v.a[j], tc::fmul2(w.a[j], rr));
              v.b[j] = tc::fmul2(v.b[j], tc::fmul2(w.b[j], rr));
            }
          }
          if (sl.rot) turn16<false>(v, tb, sl.pair0);
          const bool ok = h < sd.heads && lane_ok;
          if (!side) {
            T* y = (T*)sd.out + t * sd.sout + (int64_t)h * a.dim;
            if (ok) Raw16<T>::template store<LAYOUT>(y + sl.a, y + sl.b, v);
            continue;
          }
          // ---- keys, to their page
          const int64_t row = row0 + ((int64_t)h << p.page_shift);
          float x[8], y[8];
          octets<LAYOUT>(v, x, y);
          if constexpr (MX) {
            // a block's four octets may be four lanes' or two: their maxima meet in shared memory
            float* top = tops[warp] + sub * (a.dim >> 3);
            __syncwarp();  // the last step's have been read
            if (lane_ok) {
              top[sl.a >> 3] = octet_max(x);
              top[sl.b >> 3] = octet_max(y);
            }
            __syncwarp();
            if (ok && row0 >= 0) {
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                const int col = half ? sl.b : sl.a;
                const float4 m = *reinterpret_cast<const float4*>(top + (col >> 5) * 4);
                const int e = mx_scale_exp(fmaxf(fmaxf(m.x, m.y), fmaxf(m.z, m.w)));
                *reinterpret_cast<uint2*>((uint8_t*)p.kc + row * a.dim + col) = octet_codes(half ? y : x, exp2i(-e));
                if ((col & 31) == 0) p.ks[row * (a.dim >> 5) + (col >> 5)] = (uint8_t)(e + 127);
              }
            }
          } else if (ok && row0 >= 0) {
            put_octet((T*)p.kc + row * a.dim + sl.a, x);
            put_octet((T*)p.kc + row * a.dim + sl.b, y);
          }
        }
      }
    }
  }
}

bool append_shape(const Paged& p, const NormRopeArgs& a, size_t e, AppendShape* g) {
  const size_t unit = 8 * e;  // bytes of an access
  if (a.dim % V != 0 || a.rot % V != 0 || p.dim_v % V != 0) return false;
  uintptr_t all = (uintptr_t)p.v | (uintptr_t)(p.sv * e);
  if (p.kind != kCacheMx) all |= (uintptr_t)p.kc | (uintptr_t)p.vc;
  for (const NormRopeSide& s : a.side)
    if (s.heads > 0) all |= (uintptr_t)s.x | (uintptr_t)(s.sx * e) | (&s == a.side ? (uintptr_t)s.out | (uintptr_t)(s.sout * e) : 0);
  if (all & (unit - 1)) return false;
  g->slots = a.dim / V;
  g->group = 1;
  while (g->group < g->slots) g->group *= 2;
  // Runs as long as lets every warp of a full GPU take the same number of them; with fewer tokens than
  // warps, several warps share a token's steps.
  const int per = 32 / g->group;
  const int steps = (a.side[0].heads + per - 1) / per + (p.heads_k + per - 1) / per + (p.heads_k * (p.dim_v / V) + 31) / 32;
  const int64_t warps = (int64_t)num_sms() * kWarps * 3;
  const int64_t rounds = (p.total_q + 32 * warps - 1) / (32 * warps);
  g->run = (int)((p.total_q + rounds * warps - 1) / (rounds * warps));
  int64_t parts = g->run > 1 ? 1 : (warps + p.total_q - 1) / p.total_q;
  if (parts > steps) parts = steps;
  g->parts = (int)parts;
  return true;
}

template <typename T, int KIND>
cudaError_t append_t(const Paged& p, const NormRopeArgs& a, PagedHeader* hdr, int planned, cudaStream_t s) {
  AppendShape g;
  if (append_shape(p, a, sizeof(T), &g)) {
    const int64_t tasks = (p.total_q + g.run - 1) / g.run * g.parts, most = (int64_t)num_sms() * 3;
    int64_t grid = (tasks + kWarps - 1) / kWarps;
    if (grid > most) grid = most;
    if (a.layout == JFA_ROPE_HALVES)
      append_kernel<T, JFA_ROPE_HALVES, KIND><<<(unsigned)grid, kThreads, 0, s>>>(p, a, g, hdr, planned);
    else
      append_kernel<T, JFA_ROPE_PAIRS, KIND><<<(unsigned)grid, kThreads, 0, s>>>(p, a, g, hdr, planned);
    return cudaGetLastError();
  }
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
