// RMS norm of every query and key head with the rotary position embedding in one pass, and
// its gradient.
//
// Per row x of D values (one token, one head):
//   n = x r w, r = 1 / sqrt(mean(x^2) + eps); the pairs (a, b) of the first `rot` columns
//   turn by the angle pos theta_i: y_a = amp (n_a c - n_b s), y_b = amp (n_a s + n_b c).
// Backward: g = amp R^T dy; dw += g x r; with u = g w: dx = r (u - x r^2 <u, x> / D).
//
// Bound: HBM.  Each value is read once and written once (the backward reads x and dy and
// recomputes r), about 12 to 21 lane instructions a value against the 21 a value the SMs
// can issue at the copy bandwidth, so the arithmetic has to stay lean:
//  * Angles.  The frequencies come as 64-bit binary fractions of a turn.  pos times such a
//    fraction modulo one turn is the low half of an integer product, exact to |pos| 2^-64
//    turns (position 10^9: 5e-11), with no 64-bit floating point and no range reduction;
//    sincospif of the top 32 bits then gives cos and sin to about 1e-7.
//  * A row is D/16 lane slots of 16 values (two 16-byte loads in bf16).  A slot holds whole
//    pairs in both layouts, so the rotation needs no exchange between lanes, and a lane's
//    slot is the same in every row it touches: its (cos, sin) are computed once a token
//    and serve all the heads of the warp's part, its frequencies once a kernel.
//  * Weight gradients: every lane sums its 16 columns in registers over all its rows, the
//    CTA adds its lanes in a fixed order and writes one partial, a second kernel adds the
//    partials in order: no atomics, the same bits every time on one GPU.
// Rows that do not divide into slots (dim or rotated columns not multiples of 16, pointers
// or strides not multiples of 16 bytes) take the *_any kernels: one warp a row, single
// values.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "serve.h"

namespace jfa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int V = 16;  // values of a lane slot

template <typename T>
struct Row16;
template <>
struct Row16<__nv_bfloat16> {
  uint4 a, b;
  __device__ void load(const __nv_bfloat16* pa, const __nv_bfloat16* pb) {
    a = __ldcs(reinterpret_cast<const uint4*>(pa));
    b = __ldcs(reinterpret_cast<const uint4*>(pb));
  }
  __device__ void get(float (&v)[V]) const {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ uint32_t pack(float lo, float hi) {  // round to nearest even, the result's type
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ void store(__nv_bfloat16* pa, __nv_bfloat16* pb, const float (&v)[V]) {
    __stcs(reinterpret_cast<uint4*>(pa), make_uint4(pack(v[0], v[1]), pack(v[2], v[3]), pack(v[4], v[5]), pack(v[6], v[7])));
    __stcs(reinterpret_cast<uint4*>(pb),
           make_uint4(pack(v[8], v[9]), pack(v[10], v[11]), pack(v[12], v[13]), pack(v[14], v[15])));
  }
};
template <>
struct Row16<float> {
  float4 q[4];
  __device__ void load(const float* pa, const float* pb) {
    q[0] = __ldcs(reinterpret_cast<const float4*>(pa));
    q[1] = __ldcs(reinterpret_cast<const float4*>(pa) + 1);
    q[2] = __ldcs(reinterpret_cast<const float4*>(pb));
    q[3] = __ldcs(reinterpret_cast<const float4*>(pb) + 1);
  }
  __device__ void get(float (&v)[V]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[4 * i] = q[i].x;
      v[4 * i + 1] = q[i].y;
      v[4 * i + 2] = q[i].z;
      v[4 * i + 3] = q[i].w;
    }
  }
  static __device__ void store(float* pa, float* pb, const float (&v)[V]) {
    __stcs(reinterpret_cast<float4*>(pa), make_float4(v[0], v[1], v[2], v[3]));
    __stcs(reinterpret_cast<float4*>(pa) + 1, make_float4(v[4], v[5], v[6], v[7]));
    __stcs(reinterpret_cast<float4*>(pb), make_float4(v[8], v[9], v[10], v[11]));
    __stcs(reinterpret_cast<float4*>(pb) + 1, make_float4(v[12], v[13], v[14], v[15]));
  }
};

// (cos, sin) of pos turns, times amp
__device__ __forceinline__ float2 rotation(int64_t pos, unsigned long long turn, float amp) {
  const unsigned long long phase = (unsigned long long)pos * turn;  // modulo one turn
  float s, c;
  sincospif((float)(int32_t)(phase >> 32) * 4.656612873077392578125e-10f, &s, &c);  // 2^-31: half turns
  return make_float2(amp * c, amp * s);
}

// A lane's place in a row: columns [a, a+8) and [b, b+8).  Halves layout: value i of the
// first eight pairs with value i of the second; pairs layout: neighbours pair up.
struct Slot {
  int a, b, pair0;  // pair0: index of the slot's first pair
  bool rot;
};
__device__ __forceinline__ Slot slot_of(int slot, int rot, int layout) {
  Slot r;
  r.rot = slot * V < rot;
  r.pair0 = slot * 8;
  if (r.rot && layout == JFA_ROPE_HALVES) {
    r.a = 8 * slot;
    r.b = rot / 2 + 8 * slot;
  } else {
    r.a = V * slot;
    r.b = V * slot + 8;
  }
  return r;
}

// v turned by cs (sign = 1) or back (sign = -1)
template <int LAYOUT>
__device__ __forceinline__ void turn16(float (&v)[V], const float2 (&cs)[8], float sign) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int ia = LAYOUT == JFA_ROPE_HALVES ? i : 2 * i, ib = LAYOUT == JFA_ROPE_HALVES ? 8 + i : 2 * i + 1;
    const float a = v[ia], b = v[ib], s = sign * cs[i].y;
    v[ia] = fmaf(a, cs[i].x, -b * s);
    v[ib] = fmaf(a, s, b * cs[i].x);
  }
}

__device__ __forceinline__ float group_sum(float x, int group) {
  for (int m = group >> 1; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}

__device__ __forceinline__ void load_weight(float (&w)[V], const float* p, const Slot& sl, bool lane_ok) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    w[i] = p && lane_ok ? __ldg(p + sl.a + i) : 1.f;
    w[8 + i] = p && lane_ok ? __ldg(p + sl.b + i) : 1.f;
  }
}

// The rows of one token's part, warp by warp.  group lanes (a power of two) serve a row, of
// which slots = D/16 have values; parts warps share a token's heads.
struct FastShape {
  int group, slots, parts;
};

// Visits the part's rows of both tensors: f(side, head, valid).  Every lane of the warp
// calls f the same number of times.
template <class F>
__device__ __forceinline__ void each_row(const NormRopeArgs& p, int side, const FastShape& g, int part, int lane, F f) {
  const int per = 32 / g.group, sub = lane / g.group, H = p.side[side].heads;
  const int steps = (H + per - 1) / per;
  const int s0 = (int)((int64_t)steps * part / g.parts), s1 = (int)((int64_t)steps * (part + 1) / g.parts);
#pragma unroll 2
  for (int s = s0; s < s1; ++s) {
    const int h = s * per + sub;
    f(h, h < H);
  }
}

template <typename T, int LAYOUT>
__global__ void __launch_bounds__(kThreads)
norm_rope_fwd_kernel(const __grid_constant__ NormRopeArgs p, const FastShape g) {
  const int lane = threadIdx.x & 31;
  const int ls = lane % g.group;
  const bool lane_ok = ls < g.slots;
  const Slot sl = slot_of(lane_ok ? ls : 0, p.rot, LAYOUT);
  unsigned long long turn[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) turn[i] = sl.rot ? p.turn[sl.pair0 + i] : 0;
  const int64_t nw = (int64_t)gridDim.x * kWarps, tasks = p.tokens * g.parts;
  for (int64_t task = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); task < tasks; task += nw) {
    const int64_t t = task / g.parts;
    const int part = (int)(task - t * g.parts);
    float2 cs[8];
    if (sl.rot) {
      const int64_t pos = __ldg(p.pos + t);
#pragma unroll
      for (int i = 0; i < 8; ++i) cs[i] = rotation(pos, turn[i], p.amp);
    }
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
      const NormRopeSide& sd = p.side[side];
      if (sd.heads == 0) continue;
      float w[V];
      load_weight(w, sd.w, sl, lane_ok);
      const T* x = (const T*)sd.x + t * sd.sx;
      T* y = (T*)sd.out + t * sd.sout;
      each_row(p, side, g, part, lane, [&](int h, bool ok) {
        ok = ok && lane_ok;
        float v[V];
        if (ok) {
          Row16<T> r;
          r.load(x + (int64_t)h * p.dim + sl.a, x + (int64_t)h * p.dim + sl.b);
          r.get(v);
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i) v[i] = 0.f;
        }
        if (p.norm) {
          float ss = 0.f;
#pragma unroll
          for (int i = 0; i < V; ++i) ss = fmaf(v[i], v[i], ss);
          const float r = rsqrtf(fmaf(group_sum(ss, g.group), p.inv_dim, p.eps));
#pragma unroll
          for (int i = 0; i < V; ++i) v[i] *= r * w[i];
        }
        if (sl.rot) turn16<LAYOUT>(v, cs, 1.f);
        if (ok) Row16<T>::store(y + (int64_t)h * p.dim + sl.a, y + (int64_t)h * p.dim + sl.b, v);
      });
    }
  }
}

// Adds the CTA's per-lane sums of one tensor in a fixed order (lanes of a slot, then warps)
// and writes the CTA's partial.
__device__ __forceinline__ void write_partial(const float (&acc)[V], const Slot& sl, const FastShape& g, int ls,
                                              bool lane_ok, float* red, float* part, int dim) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float x = acc[i];
    for (int m = 16; m >= g.group; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    if (lane < g.group && lane_ok) red[warp * dim + (i < 8 ? sl.a + i : sl.b + i - 8)] = x;
  }
  __syncthreads();
  for (int c = threadIdx.x; c < dim; c += kThreads) {
    float x = 0.f;
    for (int w = 0; w < kWarps; ++w) x += red[w * dim + c];
    part[c] = x;
  }
  __syncthreads();
}

template <typename T, int LAYOUT>
__global__ void __launch_bounds__(kThreads)
norm_rope_bwd_kernel(const __grid_constant__ NormRopeArgs p, const FastShape g, float* part_ws) {
  extern __shared__ float red[];
  const int lane = threadIdx.x & 31;
  const int ls = lane % g.group;
  const bool lane_ok = ls < g.slots;
  const Slot sl = slot_of(lane_ok ? ls : 0, p.rot, LAYOUT);
  const int64_t nw = (int64_t)gridDim.x * kWarps, tasks = p.tokens * g.parts;
  unsigned long long turn[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) turn[i] = sl.rot ? p.turn[sl.pair0 + i] : 0;
#pragma unroll 1
  for (int side = 0; side < 2; ++side) {
    const NormRopeSide& sd = p.side[side];
    if (sd.heads == 0) continue;
    float acc[V], w[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    load_weight(w, sd.w, sl, lane_ok);
    for (int64_t task = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); task < tasks; task += nw) {
      const int64_t t = task / g.parts;
      const int part = (int)(task - t * g.parts);
      float2 cs[8];
      if (sl.rot) {
        const int64_t pos = __ldg(p.pos + t);
#pragma unroll
        for (int i = 0; i < 8; ++i) cs[i] = rotation(pos, turn[i], p.amp);
      }
      const T* x = (const T*)sd.x + t * sd.sx;
      const T* dy = (const T*)sd.dy + t * sd.sdy;
      T* dx = (T*)sd.out + t * sd.sout;
      each_row(p, side, g, part, lane, [&](int h, bool ok) {
        ok = ok && lane_ok;
        float v[V], d[V];
        if (ok) {
          Row16<T> rx, rd;
          const int64_t o = (int64_t)h * p.dim;
          if (p.norm) rx.load(x + o + sl.a, x + o + sl.b);
          rd.load(dy + o + sl.a, dy + o + sl.b);
          if (p.norm) rx.get(v);
          rd.get(d);
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i) v[i] = d[i] = 0.f;
        }
        if (sl.rot) turn16<LAYOUT>(d, cs, -1.f);
        if (p.norm) {
          float ss = 0.f, ux = 0.f;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            ss = fmaf(v[i], v[i], ss);
            ux = fmaf(d[i] * w[i], v[i], ux);
          }
          const float r = rsqrtf(fmaf(group_sum(ss, g.group), p.inv_dim, p.eps));
          const float k = group_sum(ux, g.group) * p.inv_dim * r * r;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            acc[i] = fmaf(d[i], v[i] * r, acc[i]);
            d[i] = r * fmaf(-v[i], k, d[i] * w[i]);
          }
        }
        if (ok) Row16<T>::store(dx + (int64_t)h * p.dim + sl.a, dx + (int64_t)h * p.dim + sl.b, d);
      });
    }
    if (sd.dw) write_partial(acc, sl, g, ls, lane_ok, red, part_ws + ((int64_t)blockIdx.x * 2 + side) * p.dim, p.dim);
  }
}

// ------------------------------------------------------------------ rows of any shape
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x) { return (T)x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float x) { return __float2bfloat16_rn(x); }

// Columns of pair i
__device__ __forceinline__ int2 pair_cols(int i, int rot, int layout) {
  return layout == JFA_ROPE_HALVES ? make_int2(i, rot / 2 + i) : make_int2(2 * i, 2 * i + 1);
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
norm_rope_fwd_any_kernel(const __grid_constant__ NormRopeArgs p) {
  const int lane = threadIdx.x & 31;
  const int H = p.side[0].heads + p.side[1].heads;
  const int64_t rows = p.tokens * H, nw = (int64_t)gridDim.x * kWarps;
  for (int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); row < rows; row += nw) {
    const int64_t t = row / H;
    int h = (int)(row - t * H);
    const NormRopeSide& sd = p.side[h >= p.side[0].heads];
    if (h >= p.side[0].heads) h -= p.side[0].heads;
    const T* x = (const T*)sd.x + t * sd.sx + (int64_t)h * p.dim;
    T* y = (T*)sd.out + t * sd.sout + (int64_t)h * p.dim;
    float r = 1.f;
    if (p.norm) {
      float ss = 0.f;
      for (int c = lane; c < p.dim; c += 32) {
        const float a = to_f(x[c]);
        ss = fmaf(a, a, ss);
      }
      r = rsqrtf(fmaf(group_sum(ss, 32), p.inv_dim, p.eps));
    }
    __syncwarp();  // y may be x: the row has been read for its norm before any value changes
    auto n = [&](int c) { return p.norm ? to_f(x[c]) * (r * (sd.w ? __ldg(sd.w + c) : 1.f)) : to_f(x[c]); };
    for (int i = lane; i < p.rot / 2; i += 32) {
      const float2 cs = rotation(__ldg(p.pos + t), p.turn[i], p.amp);
      const int2 c = pair_cols(i, p.rot, p.layout);
      const float a = n(c.x), b = n(c.y);
      y[c.x] = from_f<T>(fmaf(a, cs.x, -b * cs.y));
      y[c.y] = from_f<T>(fmaf(a, cs.y, b * cs.x));
    }
    for (int c = p.rot + lane; c < p.dim; c += 32) y[c] = from_f<T>(n(c));
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
norm_rope_bwd_any_kernel(const __grid_constant__ NormRopeArgs p, float* part_ws) {
  extern __shared__ float red[];  // [kWarps][2][dim]: a lane adds to its own columns only
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < kWarps * 2 * p.dim; i += kThreads) red[i] = 0.f;
  __syncthreads();
  const int H = p.side[0].heads + p.side[1].heads;
  const int64_t rows = p.tokens * H, nw = (int64_t)gridDim.x * kWarps;
  for (int64_t row = (int64_t)blockIdx.x * kWarps + warp; row < rows; row += nw) {
    const int64_t t = row / H;
    int h = (int)(row - t * H);
    const int side = h >= p.side[0].heads;
    const NormRopeSide& sd = p.side[side];
    if (side) h -= p.side[0].heads;
    const T* x = (const T*)sd.x + t * sd.sx + (int64_t)h * p.dim;
    const T* dy = (const T*)sd.dy + t * sd.sdy + (int64_t)h * p.dim;
    T* dx = (T*)sd.out + t * sd.sout + (int64_t)h * p.dim;
    float* dw = red + (warp * 2 + side) * p.dim;
    auto w = [&](int c) { return sd.w ? __ldg(sd.w + c) : 1.f; };
    float r = 1.f, k = 0.f;
    if (p.norm) {
      float ss = 0.f, ux = 0.f;
      for (int i = lane; i < p.rot / 2; i += 32) {
        const float2 cs = rotation(__ldg(p.pos + t), p.turn[i], p.amp);
        const int2 c = pair_cols(i, p.rot, p.layout);
        const float a = to_f(x[c.x]), b = to_f(x[c.y]), da = to_f(dy[c.x]), db = to_f(dy[c.y]);
        ss = fmaf(a, a, fmaf(b, b, ss));
        ux = fmaf(fmaf(da, cs.x, db * cs.y) * w(c.x), a, fmaf(fmaf(db, cs.x, -da * cs.y) * w(c.y), b, ux));
      }
      for (int c = p.rot + lane; c < p.dim; c += 32) {
        const float a = to_f(x[c]);
        ss = fmaf(a, a, ss);
        ux = fmaf(to_f(dy[c]) * w(c), a, ux);
      }
      r = rsqrtf(fmaf(group_sum(ss, 32), p.inv_dim, p.eps));
      k = group_sum(ux, 32) * p.inv_dim * r * r;
    }
    __syncwarp();  // dx may be dy or x: both have been read whole before any value changes
    auto put = [&](int c, float g, float a) {
      if (p.norm) {
        dw[c] = fmaf(g, a * r, dw[c]);
        g = r * fmaf(-a, k, g * w(c));
      }
      dx[c] = from_f<T>(g);
    };
    for (int i = lane; i < p.rot / 2; i += 32) {
      const float2 cs = rotation(__ldg(p.pos + t), p.turn[i], p.amp);
      const int2 c = pair_cols(i, p.rot, p.layout);
      const float a = p.norm ? to_f(x[c.x]) : 0.f, b = p.norm ? to_f(x[c.y]) : 0.f;
      const float da = to_f(dy[c.x]), db = to_f(dy[c.y]);
      put(c.x, fmaf(da, cs.x, db * cs.y), a);
      put(c.y, fmaf(db, cs.x, -da * cs.y), b);
    }
    for (int c = p.rot + lane; c < p.dim; c += 32) {
      const float a = p.norm ? to_f(x[c]) : 0.f;
      put(c, to_f(dy[c]), a);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * p.dim; i += kThreads) {
    float x = 0.f;
    for (int v = 0; v < kWarps; ++v) x += red[v * 2 * p.dim + i];
    part_ws[(int64_t)blockIdx.x * 2 * p.dim + i] = x;
  }
}

// dw[c] of both tensors: the CTAs' partials added in a fixed order, 32 columns a CTA.
constexpr int kSumWarps = 16;
__global__ void __launch_bounds__(kSumWarps * 32)
norm_rope_dw_kernel(const float* __restrict__ part, int parts, int dim, float* dwq, float* dwk) {
  __shared__ float red[kSumWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float* dw = blockIdx.y == 0 ? dwq : dwk;
  if (!dw) return;
  float acc = 0.f;
  if (c < dim)
    for (int i = warp; i < parts; i += kSumWarps) acc += part[((int64_t)i * 2 + blockIdx.y) * dim + c];
  red[warp][lane] = acc;
  __syncthreads();
  if (warp == 0 && c < dim) {
    float x = 0.f;
    for (int w = 0; w < kSumWarps; ++w) x += red[w][lane];
    dw[c] = x;
  }
}

bool fast_shape(const NormRopeArgs& a, size_t e, FastShape* g) {
  if (a.dim % V != 0 || a.rot % V != 0) return false;
  for (const NormRopeSide& s : a.side) {
    if (s.heads == 0) continue;
    if (((uintptr_t)s.x | (uintptr_t)s.dy | (uintptr_t)s.out) & 15) return false;
    if ((s.sx * e) % 16 || (s.sdy * e) % 16 || (s.sout * e) % 16) return false;
  }
  g->slots = a.dim / V;
  g->group = 1;
  while (g->group < g->slots) g->group *= 2;
  // With fewer tokens than the GPU has warps to give, several warps share a token's heads.
  const int per = 32 / g->group;
  const int hmax = a.side[0].heads > a.side[1].heads ? a.side[0].heads : a.side[1].heads;
  const int steps = (hmax + per - 1) / per;
  const int64_t warps = (int64_t)num_sms() * kWarps * 2;
  int64_t parts = (warps + a.tokens - 1) / a.tokens;
  if (parts > steps) parts = steps;
  g->parts = (int)(parts < 1 ? 1 : parts);
  return true;
}

int grid_for(int64_t warps, int per_sm, int cap) {
  int64_t n = (warps + kWarps - 1) / kWarps;
  const int64_t most = (int64_t)num_sms() * per_sm;
  if (n > most) n = most;
  if (n > cap) n = cap;
  return (int)(n < 1 ? 1 : n);
}

template <typename T>
cudaError_t fwd_t(const NormRopeArgs& a, cudaStream_t s) {
  FastShape g;
  if (fast_shape(a, sizeof(T), &g)) {
    const int grid = grid_for(a.tokens * g.parts, 4, INT32_MAX);
    if (a.layout == JFA_ROPE_HALVES)
      norm_rope_fwd_kernel<T, JFA_ROPE_HALVES><<<grid, kThreads, 0, s>>>(a, g);
    else
      norm_rope_fwd_kernel<T, JFA_ROPE_PAIRS><<<grid, kThreads, 0, s>>>(a, g);
  } else {
    const int grid = grid_for(a.tokens * (a.side[0].heads + a.side[1].heads), 8, INT32_MAX);
    norm_rope_fwd_any_kernel<T><<<grid, kThreads, 0, s>>>(a);
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t bwd_t(const NormRopeArgs& a, float* part, cudaStream_t s) {
  FastShape g;
  int grid;
  if (fast_shape(a, sizeof(T), &g)) {
    grid = grid_for(a.tokens * g.parts, 4, kNormRopeParts);
    const size_t smem = sizeof(float) * kWarps * a.dim;
    if (a.layout == JFA_ROPE_HALVES)
      norm_rope_bwd_kernel<T, JFA_ROPE_HALVES><<<grid, kThreads, smem, s>>>(a, g, part);
    else
      norm_rope_bwd_kernel<T, JFA_ROPE_PAIRS><<<grid, kThreads, smem, s>>>(a, g, part);
  } else {
    grid = grid_for(a.tokens * (a.side[0].heads + a.side[1].heads), 6, kNormRopeParts);
    norm_rope_bwd_any_kernel<T><<<grid, kThreads, sizeof(float) * kWarps * 2 * a.dim, s>>>(a, part);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || (!a.side[0].dw && !a.side[1].dw)) return e;
  norm_rope_dw_kernel<<<dim3((a.dim + 31) / 32, 2), kSumWarps * 32, 0, s>>>(part, grid, a.dim, a.side[0].dw,
                                                                             a.side[1].dw);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope_fwd(const NormRopeArgs& a, int dtype, cudaStream_t s) {
  return dtype == JFA_BF16 ? fwd_t<__nv_bfloat16>(a, s) : fwd_t<float>(a, s);
}
cudaError_t launch_norm_rope_bwd(const NormRopeArgs& a, int dtype, float* part, cudaStream_t s) {
  return dtype == JFA_BF16 ? bwd_t<__nv_bfloat16>(a, part, s) : bwd_t<float>(a, part, s);
}

}  // namespace jfa
