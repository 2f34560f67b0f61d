// Device parts of the RMS norm with rotary positions (norm_rope.cu has the method): rows in lane
// slots, rotations, and single columns of rows of any shape.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "serve.h"
#include "tc_ptx.cuh"

namespace jfa {

constexpr int V = 16;  // values of a lane slot

// A slot's values as eight pairs (a_i, b_i), two to a float2: a[j] = (a_2j, a_2j+1).
struct Slot16 {
  float2 a[4], b[4];
};

// A slot as it lies in memory: columns [a, a + 8) and [b, b + 8).
template <typename T>
struct Raw16;
template <>
struct Raw16<__nv_bfloat16> {
  static constexpr int kBatch = 4;  // rows a lane has in flight
  uint4 a, b;
  __device__ void load(const __nv_bfloat16* pa, const __nv_bfloat16* pb) {
    a = __ldcs(reinterpret_cast<const uint4*>(pa));
    b = __ldcs(reinterpret_cast<const uint4*>(pb));
  }
  __device__ void zero() { a = b = make_uint4(0u, 0u, 0u, 0u); }
  static __device__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
  static __device__ float hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
  template <int LAYOUT>
  __device__ void get(Slot16& s) const {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (LAYOUT == JFA_ROPE_HALVES) {
        s.a[j] = make_float2(lo(w[j]), hi(w[j]));
        s.b[j] = make_float2(lo(w[4 + j]), hi(w[4 + j]));
      } else {
        s.a[j] = make_float2(lo(w[2 * j]), lo(w[2 * j + 1]));
        s.b[j] = make_float2(hi(w[2 * j]), hi(w[2 * j + 1]));
      }
    }
  }
  static __device__ uint32_t pack(float x, float y) {  // round to nearest even: the result's type
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
    return r;
  }
  template <int LAYOUT>
  static __device__ void store(__nv_bfloat16* pa, __nv_bfloat16* pb, const Slot16& s) {
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (LAYOUT == JFA_ROPE_HALVES) {
        w[j] = pack(s.a[j].x, s.a[j].y);
        w[4 + j] = pack(s.b[j].x, s.b[j].y);
      } else {
        w[2 * j] = pack(s.a[j].x, s.b[j].x);
        w[2 * j + 1] = pack(s.a[j].y, s.b[j].y);
      }
    }
    __stcs(reinterpret_cast<uint4*>(pa), make_uint4(w[0], w[1], w[2], w[3]));
    __stcs(reinterpret_cast<uint4*>(pb), make_uint4(w[4], w[5], w[6], w[7]));
  }
};
// 32 bytes in one access: a lane's two 16-byte halves would be half a sector each.
__device__ __forceinline__ void load32(float4* q, const float* x) {
  asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(q[0].x), "=f"(q[0].y), "=f"(q[0].z), "=f"(q[0].w), "=f"(q[1].x), "=f"(q[1].y), "=f"(q[1].z),
                 "=f"(q[1].w)
               : "l"(x));
}
__device__ __forceinline__ void store32(float* x, const float4* q) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(x), "f"(q[0].x), "f"(q[0].y),
               "f"(q[0].z), "f"(q[0].w), "f"(q[1].x), "f"(q[1].y), "f"(q[1].z), "f"(q[1].w)
               : "memory");
}
template <>
struct Raw16<float> {
  static constexpr int kBatch = 2;
  float4 q[4];
  __device__ void load(const float* pa, const float* pb) {
    load32(q, pa);
    load32(q + 2, pb);
  }
  __device__ void zero() { q[0] = q[1] = q[2] = q[3] = make_float4(0.f, 0.f, 0.f, 0.f); }
  template <int LAYOUT>
  __device__ void get(Slot16& s) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (LAYOUT == JFA_ROPE_HALVES) {
        const float4 x = q[j >> 1], y = q[2 + (j >> 1)];
        s.a[j] = j & 1 ? make_float2(x.z, x.w) : make_float2(x.x, x.y);
        s.b[j] = j & 1 ? make_float2(y.z, y.w) : make_float2(y.x, y.y);
      } else {
        s.a[j] = make_float2(q[j].x, q[j].z);
        s.b[j] = make_float2(q[j].y, q[j].w);
      }
    }
  }
  template <int LAYOUT>
  static __device__ void store(float* pa, float* pb, const Slot16& s) {
    float4 w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (LAYOUT == JFA_ROPE_HALVES) {
        const float2* v = j < 2 ? s.a : s.b;
        const int k = 2 * (j & 1);
        w[j] = make_float4(v[k].x, v[k].y, v[k + 1].x, v[k + 1].y);
      } else {
        w[j] = make_float4(s.a[j].x, s.b[j].x, s.a[j].y, s.b[j].y);
      }
    }
    store32(pa, w);
    store32(pb, w + 2);
  }
};

// (cos, sin) of pos turns, times amp.  The quarter turns come off while the angle is an integer: as one float an
// angle near a half turn would be off by 9e-8, what is left of it, at most an eighth of a turn, is by 2e-8.
__device__ __forceinline__ float2 rotation(int64_t pos, unsigned long long turn, float amp) {
  const unsigned long long phase = (unsigned long long)pos * turn;  // modulo one turn
  const uint32_t at = (uint32_t)(phase >> 32) + 0x20000000u;        // the nearest quarter's number, and the rest
  float s, c;
  sincospif((float)((int32_t)(at & 0x3fffffffu) - 0x20000000) * 4.656612873077392578125e-10f, &s, &c);  // 2^-31: half turns
  const float x = at & 0x40000000u ? -s : c, y = at & 0x40000000u ? c : s;
  const float a = at & 0x80000000u ? -amp : amp;
  return make_float2(a * x, a * y);
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

// Where value c of a row lies in shared memory: a lane reads its values by fours, and the fours that
// the lanes of a row read at once lie side by side in one of the planes.  (With a lane's values
// together, two lanes met in every bank: 437 us for the forward's figure in the header.)
template <int PLANES>
__device__ __forceinline__ int plane_at(int c, int size) {
  return (c / 4 % PLANES) * (size / PLANES) + c / (4 * PLANES) * 4 + (c & 3);
}

// The rotations of a token's pairs, computed once by the warp, two to four pairs a lane, into
// its table (cosines, then sines).
constexpr int kMaxPairs = kMaxNormDim / 2;
struct Turns {
  unsigned long long turn[kMaxPairs / 32];
  __device__ __forceinline__ void init(const NormRopeArgs& p, int lane) {
#pragma unroll
    for (int i = 0; i < kMaxPairs / 32; ++i) turn[i] = p.turn[lane + 32 * i];
  }
  __device__ __forceinline__ void table(float* tb, const NormRopeArgs& p, int64_t pos, int lane) const {
    __syncwarp();  // the last token's reads are done
#pragma unroll
    for (int i = 0; i < kMaxPairs / 32; ++i) {
      const int k = lane + 32 * i;
      if (32 * i < p.rot / 2 && k < p.rot / 2) {
        const float2 cs = rotation(pos, turn[i], p.amp);
        const int at = plane_at<2>(k, kMaxPairs);
        tb[at] = cs.x;
        tb[kMaxPairs + at] = cs.y;
      }
    }
    __syncwarp();
  }
};
__device__ __forceinline__ void load4(float2 (&v)[4], const float* x, int size) {  // x: of the first four
  const float4 p = *reinterpret_cast<const float4*>(x), q = *reinterpret_cast<const float4*>(x + size / 2);
  v[0] = make_float2(p.x, p.y);
  v[1] = make_float2(p.z, p.w);
  v[2] = make_float2(q.x, q.y);
  v[3] = make_float2(q.z, q.w);
}
// The slot's pairs turned by the table's angles, backwards with BACK.
template <bool BACK>
__device__ __forceinline__ void turn16(Slot16& v, const float* tb, int pair0) {
  float2 c[4], s[4];
  load4(c, tb + pair0 / 2, kMaxPairs);
  load4(s, tb + kMaxPairs + pair0 / 2, kMaxPairs);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 a = v.a[j], b = v.b[j];
    const float2 sn = make_float2(-s[j].x, -s[j].y);
    v.a[j] = tc::ffma2(a, c[j], tc::fmul2(b, BACK ? s[j] : sn));
    v.b[j] = tc::ffma2(b, c[j], tc::fmul2(a, BACK ? sn : s[j]));
  }
}

__device__ __forceinline__ float group_sum(float x, int group) {
  for (int m = group >> 1; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}

// The slot's weights out of a row of floats in shared memory (planes of the layout), in the slot's order
template <int LAYOUT>
__device__ __forceinline__ void weights16(Slot16& w, const float* row, const Slot& sl) {
  if (LAYOUT == JFA_ROPE_HALVES) {
    load4(w.a, row + sl.a / 2, kMaxNormDim);
    load4(w.b, row + sl.b / 2, kMaxNormDim);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 x = *reinterpret_cast<const float4*>(row + sl.a / 4 + j * (kMaxNormDim / 4));
      w.a[j] = make_float2(x.x, x.z);
      w.b[j] = make_float2(x.y, x.w);
    }
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

}  // namespace jfa
