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
//  * Angles.  The frequencies come as 64-bit binary fractions of a turn, made on the host from
//    doubles (within 2^-53 turns).  pos times such a fraction modulo one turn is the low half
//    of an integer product, which loses no more, with no 64-bit floating point and no range
//    reduction; sincospif of what the top 32 bits lie beside the nearest quarter turn then gives cos
//    and sin to about 6e-8.
//  * A row is D/16 lane slots of 16 values (two 16-byte loads in bf16).  A slot holds whole
//    pairs in both layouts, so the rotation needs no exchange between lanes, and a lane's
//    slot is the same in every row it touches: its (cos, sin) are computed once a token
//    and serve all the heads of the warp's part, its frequencies once a kernel.
//  * Weight gradients: every lane sums its 16 columns in registers over all its rows, the
//    CTA adds its lanes in a fixed order and writes one partial, a second kernel adds the
//    partials in order: no atomics, the same bits every time on one GPU.
// Rows that do not divide into slots (dim or rotated columns not multiples of 16, pointers or
// strides not multiples of an access, 16 bytes in bf16 and 32 in fp32) take the *_any kernels:
// one warp a row, single values.
// Measured: 131 K tokens of 32 + 8 heads of 128, bf16: 415 us, 6.5 TB/s, 95% of the copy rate (four
// rows of a lane in flight, three CTAs an SM; four CTAs: 483 us).  20 K tokens of 8 + 8 heads of
// 80 in fp32, where 5 of 8 lanes have values: 43 us, 4.7 TB/s (three rows in flight: 57 us).
// Backward, 66 K tokens of 32 + 8 heads of 128: 389 us, 5.2 TB/s.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "norm_rope.cuh"
#include "serve.h"
#include "tc_ptx.cuh"

namespace jfa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// group lanes (a power of two) serve a row, of which slots = D/16 have values; parts warps share
// a token's heads.  A step is the 32 / group rows of one tensor that a warp takes at once.
struct FastShape {
  int group, slots, parts;
};

template <typename T, int LAYOUT>
__global__ void __launch_bounds__(kThreads, 3)
norm_rope_fwd_kernel(const __grid_constant__ NormRopeArgs p, const FastShape g) {
  __shared__ __align__(16) float tables[kWarps][2 * kMaxPairs];
  __shared__ __align__(16) float weights[2][kMaxNormDim];
  constexpr int U = Raw16<T>::kBatch;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < 2 * p.dim; i += kThreads) {
    const float* w = p.side[i >= p.dim].w;
    weights[i >= p.dim][plane_at<LAYOUT == JFA_ROPE_HALVES ? 2 : 4>(i % p.dim, kMaxNormDim)] = w ? w[i % p.dim] : 1.f;
  }
  __syncthreads();
  float* tb = tables[warp];
  const int per = 32 / g.group, sub = lane / g.group, ls = lane % g.group;
  const bool lane_ok = ls < g.slots;
  const Slot sl = slot_of(lane_ok ? ls : 0, p.rot, LAYOUT);
  Turns turns;
  turns.init(p, lane);
  const int steps_q = (p.side[0].heads + per - 1) / per, steps = steps_q + (p.side[1].heads + per - 1) / per;
  const int64_t nw = (int64_t)gridDim.x * kWarps, tasks = p.tokens * g.parts;
  for (int64_t task = (int64_t)blockIdx.x * kWarps + warp; task < tasks; task += nw) {
    const int64_t t = task / g.parts;
    const int part = (int)(task - t * g.parts);
    const int s0 = (int)((int64_t)steps * part / g.parts), s1 = (int)((int64_t)steps * (part + 1) / g.parts);
    bool fresh = p.rot > 0;
    for (int sb = s0; sb < s1; sb += U) {
      Raw16<T> raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int side = sb + u >= steps_q, h = (sb + u - (side ? steps_q : 0)) * per + sub;
        const NormRopeSide& sd = p.side[side];
        if (sb + u < s1 && h < sd.heads && lane_ok) {
          const T* x = (const T*)sd.x + t * sd.sx + (int64_t)h * p.dim;
          raw[u].load(x + sl.a, x + sl.b);
        } else {
          raw[u].zero();
        }
      }
      if (fresh) {  // under the first rows' loads
        turns.table(tb, p, __ldg(p.pos + t), lane);
        fresh = false;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (sb + u >= s1) break;
        const int side = sb + u >= steps_q, h = (sb + u - (side ? steps_q : 0)) * per + sub;
        const NormRopeSide& sd = p.side[side];
        Slot16 v;
        raw[u].template get<LAYOUT>(v);
        if (p.norm) {
          float2 ss = tc::fmul2(v.a[0], v.a[0]);
#pragma unroll
          for (int j = 1; j < 4; ++j) ss = tc::ffma2(v.a[j], v.a[j], ss);
#pragma unroll
          for (int j = 0; j < 4; ++j) ss = tc::ffma2(v.b[j], v.b[j], ss);
          const float r = rsqrtf(fmaf(group_sum(ss.x + ss.y, g.group), p.inv_dim, p.eps));
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
        if (h < sd.heads && lane_ok) {
          T* y = (T*)sd.out + t * sd.sout + (int64_t)h * p.dim;
          Raw16<T>::template store<LAYOUT>(y + sl.a, y + sl.b, v);
        }
      }
    }
  }
}

// Adds the CTA's per-lane sums of one tensor in a fixed order (lanes of a slot, then warps)
// and writes the CTA's partial.
template <int LAYOUT>
__device__ __forceinline__ void write_partial(const Slot16& acc, const Slot& sl, const FastShape& g, bool lane_ok,
                                              float* red, float* part, int dim) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int j = i & 7;  // values 0 .. 7: a's, 8 .. 15: b's
    const float2 two = i < 8 ? acc.a[j >> 1] : acc.b[j >> 1];
    float x = j & 1 ? two.y : two.x;
    for (int m = 16; m >= g.group; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    const int c = LAYOUT == JFA_ROPE_HALVES ? (i < 8 ? sl.a : sl.b) + j : sl.a + 2 * j + (i >= 8);
    if (lane < g.group && lane_ok) red[warp * dim + c] = x;
  }
  __syncthreads();
  for (int c = threadIdx.x; c < dim; c += kThreads) {
    float x = 0.f;
    for (int w = 0; w < kWarps; ++w) x += red[w * dim + c];
    part[c] = x;
  }
  __syncthreads();
}

// One row of each tensor in flight a lane and three CTAs an SM: more warps hide more here than more
// rows a warp (two rows at two CTAs: 445 us for 65539 tokens of 40 heads of 128, so 389 us).
template <typename T, int LAYOUT>
__global__ void __launch_bounds__(kThreads, 3)
norm_rope_bwd_kernel(const __grid_constant__ NormRopeArgs p, const FastShape g, float* part_ws) {
  extern __shared__ float red[];
  __shared__ __align__(16) float tables[kWarps][2 * kMaxPairs];
  __shared__ __align__(16) float weights[2][kMaxNormDim];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < 2 * p.dim; i += kThreads) {
    const float* w = p.side[i >= p.dim].w;
    weights[i >= p.dim][plane_at<LAYOUT == JFA_ROPE_HALVES ? 2 : 4>(i % p.dim, kMaxNormDim)] = w ? w[i % p.dim] : 1.f;
  }
  __syncthreads();
  float* tb = tables[warp];
  const int per = 32 / g.group, sub = lane / g.group, ls = lane % g.group;
  const bool lane_ok = ls < g.slots;
  const Slot sl = slot_of(lane_ok ? ls : 0, p.rot, LAYOUT);
  Turns turns;
  turns.init(p, lane);
  const int64_t nw = (int64_t)gridDim.x * kWarps, tasks = p.tokens * g.parts;
#pragma unroll 1
  for (int side = 0; side < 2; ++side) {
    const NormRopeSide& sd = p.side[side];
    if (sd.heads == 0) continue;
    const int steps = (sd.heads + per - 1) / per;
    Slot16 acc;
#pragma unroll
    for (int j = 0; j < 4; ++j) acc.a[j] = acc.b[j] = make_float2(0.f, 0.f);
    for (int64_t task = (int64_t)blockIdx.x * kWarps + warp; task < tasks; task += nw) {
      const int64_t t = task / g.parts;
      const int part = (int)(task - t * g.parts);
      const int s0 = (int)((int64_t)steps * part / g.parts), s1 = (int)((int64_t)steps * (part + 1) / g.parts);
      bool fresh = p.rot > 0;
      for (int step = s0; step < s1; ++step) {
        const int h = step * per + sub;
        const bool ok = h < sd.heads && lane_ok;
        Raw16<T> rx, rd;
        rd.zero();
        rx.zero();
        if (ok) {
          const int64_t o = (int64_t)h * p.dim;
          const T* dy = (const T*)sd.dy + t * sd.sdy + o;
          rd.load(dy + sl.a, dy + sl.b);
          if (p.norm) {
            const T* x = (const T*)sd.x + t * sd.sx + o;
            rx.load(x + sl.a, x + sl.b);
          }
        }
        if (fresh) {  // under the first row's loads
          turns.table(tb, p, __ldg(p.pos + t), lane);
          fresh = false;
        }
        Slot16 d;
        rd.template get<LAYOUT>(d);
        if (sl.rot) turn16<true>(d, tb, sl.pair0);
        if (p.norm) {
          Slot16 v, w;
          rx.template get<LAYOUT>(v);
          weights16<LAYOUT>(w, weights[side], sl);
          float2 ss = make_float2(0.f, 0.f), ux = ss;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            ss = tc::ffma2(v.a[j], v.a[j], ss);
            ss = tc::ffma2(v.b[j], v.b[j], ss);
            ux = tc::ffma2(tc::fmul2(d.a[j], w.a[j]), v.a[j], ux);
            ux = tc::ffma2(tc::fmul2(d.b[j], w.b[j]), v.b[j], ux);
          }
          float s2 = ss.x + ss.y, su = ux.x + ux.y;
          for (int m = g.group >> 1; m > 0; m >>= 1) {  // side by side: one latency
            s2 += __shfl_xor_sync(0xffffffffu, s2, m);
            su += __shfl_xor_sync(0xffffffffu, su, m);
          }
          const float r = rsqrtf(fmaf(s2, p.inv_dim, p.eps));
          const float k = su * p.inv_dim * r * r;
          const float2 rr = make_float2(r, r), kn = make_float2(-k, -k);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            acc.a[j] = tc::ffma2(d.a[j], tc::fmul2(v.a[j], rr), acc.a[j]);
            acc.b[j] = tc::ffma2(d.b[j], tc::fmul2(v.b[j], rr), acc.b[j]);
            d.a[j] = tc::fmul2(rr, tc::ffma2(v.a[j], kn, tc::fmul2(d.a[j], w.a[j])));
            d.b[j] = tc::fmul2(rr, tc::ffma2(v.b[j], kn, tc::fmul2(d.b[j], w.b[j])));
          }
        }
        if (ok) {
          T* dx = (T*)sd.out + t * sd.sout + (int64_t)h * p.dim;
          Raw16<T>::template store<LAYOUT>(dx + sl.a, dx + sl.b, d);
        }
      }
    }
    if (sd.dw)
      write_partial<LAYOUT>(acc, sl, g, lane_ok, red, part_ws + ((int64_t)blockIdx.x * 2 + side) * p.dim, p.dim);
  }
}

// ------------------------------------------------------------------ rows of any shape
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
  const size_t unit = 8 * e;  // bytes of an access
  if (a.dim % V != 0 || a.rot % V != 0) return false;
  for (const NormRopeSide& s : a.side) {
    if (s.heads == 0) continue;
    if (((uintptr_t)s.x | (uintptr_t)s.dy | (uintptr_t)s.out) & (unit - 1)) return false;
    if ((s.sx * e) % unit || (s.sdy * e) % unit || (s.sout * e) % unit) return false;
  }
  g->slots = a.dim / V;
  g->group = 1;
  while (g->group < g->slots) g->group *= 2;
  // With fewer tokens than the GPU has warps to give, several warps share a token's heads.
  const int per = 32 / g->group;
  const int steps = (a.side[0].heads + per - 1) / per + (a.side[1].heads + per - 1) / per;
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
    const int grid = grid_for(a.tokens * g.parts, 3, INT32_MAX);
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
    grid = grid_for(a.tokens * g.parts, 3, kNormRopeParts);
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
