// Attention over a paged cache for few query rows: up to 16 rows that share a key head (a
// serving step's single tokens with their group of heads, or a few tokens).
//
// Bound: HBM.  A key and its value are read once and meet at most 16 rows, 4 to 32 flops a
// byte, so what counts is that loads never pause.  A CTA has one producer warp, which walks
// the CTA's share of the work ahead of the others and fills a ring of stages (16 or 32
// keys and their values each, by TMA; page table entries are looked up 32 at a time), and four consumer
// warps.  Consecutive stages go to consecutive warps and a warp keeps its own running maximum,
// sum and output, so the warps meet only at a tile's end, where they join through shared
// memory while the producer already fills the ring with the next tile.
//
// The products run on mma.sync (16 x 8 x 16): the 16 rows are its M, where tcgen05's smallest
// tile would be seven eighths empty, and the fragments' operands come straight from the stage
// by ldmatrix (swizzled, no bank conflicts).
//
// MXFP8.  Codes are exact in fp16, and a row of bf16 queries times a power of two that brings
// its largest value to [2^14, 2^15) is exact in fp16 too (values under 2^-31 of the largest lose
// at most 2^-39 of it), so the scores are fp16 products of codes, one block of 32 columns at a
// time, and a block's scale multiplies its fp32 sum.  Values are brought to bf16 (exact: 3-bit
// mantissas times a power of two) in registers.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "paged.cuh"
#include "serve_maps.h"
#include "tc_ptx.cuh"

namespace jfa {
namespace {
using namespace tc;

constexpr int kConsumers = 4;
constexpr int kThreads = 32 * (kConsumers + 1);
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int DQK, int DV, int KIND>
struct Layout {
  static constexpr int E = KIND == kCacheMx ? 1 : 2;  // bytes of an element
  // Keys of a stage: 32, or 16 where twelve stages would not fit otherwise.
  static constexpr int kKeys = paged_rows16_keys(DQK, DV, KIND);
  static constexpr uint32_t KB = kKeys * DQK * E, VB = kKeys * DV * E;
  static constexpr uint32_t KS = KIND == kCacheMx ? kKeys * DQK / 32 : 0, VS = KIND == kCacheMx ? kKeys * DV / 32 : 0;
  static constexpr uint32_t BYTES = KB + VB + KS + VS;  // of a stage's loads
  static constexpr uint32_t STAGE = KB + VB;
  static constexpr uint32_t SCALES = 256;  // a stage's scales (K at 0, V at 128)
  static constexpr uint32_t LIMIT = 113 * 1024;  // two CTAs an SM
  // in front: barriers, abort flag, statistics; then the join's buffer, the scales, the stages
  static constexpr uint32_t ML = 512;  // [warps][16][2] floats
  static constexpr uint32_t JOIN = ML + kConsumers * 16 * 2 * 4;
  static constexpr int JOIN_LD = 36;  // 32 columns a round, padded
  static constexpr uint32_t SCALE0 = JOIN + kConsumers * 16 * JOIN_LD * 4;
  static constexpr int NS_ = (LIMIT - SCALE0 - 1024) / (STAGE + (KS ? SCALES : 0));
  // A multiple of the consumers, so that a stage is always the same warp's: fills land in any
  // order, and a warp that came to a stage before another's previous fill of it had landed
  // would take that fill's parity for its own.
  static constexpr int NS = NS_ >= 16 ? 16 : NS_ / kConsumers * kConsumers;
  static constexpr uint32_t TILES = (SCALE0 + (KS ? NS * SCALES : 0) + 1023) / 1024 * 1024;
  static constexpr uint32_t SMEM = TILES + NS * STAGE + 1024;  // 1 KB to align the base
  static_assert(NS >= 8 && NS % kConsumers == 0 && SMEM <= LIMIT, "stages");
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma_16816_bf16(float (&c)[4], const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
      "%2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_16816_f16(float (&c)[4], const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t e4m3_half2(uint32_t pair) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)pair));
  return h;
}
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// 2^(s - 127); 255 (a scale that is no number) counts as the largest, so that zeros stay zeros
__device__ __forceinline__ float scale_of(uint32_t s) { return __uint_as_float(min(s & 255u, 254u) << 23); }
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void consumers_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kConsumers * 32) : "memory");
}
__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared_f32(uint32_t a, float x) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(x) : "memory");
}
// Byte of 16-byte chunk c of row `row` in a stage's tensor of D columns of E bytes: boxes of 128
// bytes a row (bf16: 64 columns, stacked; MXFP8 at 128), or 64 bytes a row.
template <int D, int E, int kKeys>
__device__ __forceinline__ uint32_t chunk_at(int row, int c) {
  if constexpr (D * E >= 128) return (c >> 3) * (kKeys * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4);
  return row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
}

template <int DQK, int DV, int KIND>
__global__ void __launch_bounds__(kThreads, 2)
paged_rows16_kernel(const __grid_constant__ Paged p, const TileShape t, const PagedWs w,
                    const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v) {
  using L = Layout<DQK, DV, KIND>;
  constexpr int E = L::E, NS = L::NS, kKeys = L::kKeys;
  constexpr bool MX = KIND == kCacheMx;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t sb = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t full = sb, empty = sb + 8 * NS;
  volatile int* abort = (volatile int*)(smem_raw + (sb - smem_u32(smem_raw)) + 16 * NS);
  int* status = &w.hdr->status;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(full + 8 * s, 1);
      mbar_init(empty + 8 * s, 1);
    }
    *abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  PagedWalk walk;
  walk.init(w.pos, blockIdx.x);
  PagedSegment g;
  uint32_t cnt = 0;  // stages so far

  if (warp == kConsumers) {
    // ------------------------------------------------------------------ producer
    if (lane == 0) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    const int box = min(1 << p.page_shift, kKeys), per = kKeys / box;  // rows of a box, boxes of a stage
    const int none = (int)((p.pages * p.heads_k) << p.page_shift);    // behind the last row: read as zeros
    bool ok = true;
    while (ok && walk.next(p, t, g)) {
      const int head = g.unit / t.nsub;
      for (int i0 = g.blk0; ok && i0 < g.blk1; i0 += 32 / per) {
        // this lane's box of the next 32: its first row, or one behind the cache where it has no keys
        const int pos = i0 * kKeys + lane * box;
        int row = none;
        if (pos < g.seq.lk && i0 + lane / per < g.blk1) {
          const int page = paged_page(p, g.b, pos, status);
          if (page >= 0) row = (int)paged_row(p, page, head, pos);
        }
        const int n = min(32 / per, g.blk1 - i0);
        for (int i = 0; i < n; ++i, ++cnt) {
          const uint32_t st = cnt % NS;
          if (!mbar_wait(empty + 8 * st, ((cnt / NS) & 1) ^ 1, abort, status)) {
            ok = false;
            break;
          }
          const uint32_t tile = sb + L::TILES + st * L::STAGE, bar = full + 8 * st;
          if (lane == 0) mbar_expect_tx(bar, L::BYTES);
          for (int s = 0; s < per; ++s) {
            const int r = __shfl_sync(0xffffffffu, row, i * per + s);
            if (lane == 0) {
#pragma unroll
              for (int h = 0; h < (DQK * E + 127) / 128; ++h)
                tma_load_2d(tile + h * kKeys * 128 + s * box * (DQK * E < 128 ? DQK * E : 128), &tm_k, h * (128 / E), r,
                            bar);
#pragma unroll
              for (int h = 0; h < (DV * E + 127) / 128; ++h)
                tma_load_2d(tile + L::KB + h * kKeys * 128 + s * box * (DV * E < 128 ? DV * E : 128), &tm_v,
                            h * (128 / E), r, bar);
              if constexpr (MX) {
                const int64_t rs = r == none ? 0 : r;  // no row: any scales do, its codes are zeros
                const uint32_t sc = sb + L::SCALE0 + st * L::SCALES;
                bulk_load(sc + s * box * (DQK / 32), p.ks + rs * (DQK / 32), box * (DQK / 32), bar);
                bulk_load(sc + 128 + s * box * (DV / 32), p.vs + rs * (DV / 32), box * (DV / 32), bar);
              }
            }
          }
        }
      }
    }
    if (lane == 0) drain_ring(full, NS, cnt, status);  // every load has landed before the CTA leaves
    __syncwarp();
    return;
  }

  // -------------------------------------------------------------------- consumers
  const int rq = lane >> 2, q = lane & 3;  // rows rq and rq + 8 of the tile; column pair q
  constexpr int NT = kKeys / 8;            // score tiles of a stage
  constexpr int OT = DV / 8;               // output tiles
  // a consumer that gave up in a wait walks on without computing, so that its barriers still match
  bool dead = false;
  while (walk.next(p, t, g)) {
    const int head_k = g.unit / t.nsub, gs0 = (g.unit % t.nsub) * t.gsub;
    uint32_t qa[DQK / 16][4];
    int limit[2];  // keys the rows see
    int64_t orow[2];
    float cs[2];   // score units to log2 units
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int r = rq + 8 * x, tok = g.tile * t.tokens + r / t.gsub, gh = gs0 + r % t.gsub;
      const bool row_ok = r < t.rows && tok < g.seq.lq && gh < p.group;
      const int64_t lim = g.seq.off + tok + 1;
      limit[x] = !row_ok ? 0 : p.causal ? (int)max((int64_t)0, lim) : g.seq.lk;
      const int head = head_k * p.group + gh;
      orow[x] = row_ok ? (int64_t)(g.seq.q0 + tok) * p.heads_q + head : -1;
      const __nv_bfloat16* src =
          (const __nv_bfloat16*)p.q + (int64_t)(g.seq.q0 + tok) * p.sq + (int64_t)head * DQK;
      cs[x] = p.scale * kLog2e;
      if constexpr (!MX) {
#pragma unroll
        for (int k = 0; k < DQK / 16; ++k) {
          qa[k][x] = row_ok ? __ldg(reinterpret_cast<const uint32_t*>(src + 16 * k + 2 * q)) : 0u;
          qa[k][2 + x] = row_ok ? __ldg(reinterpret_cast<const uint32_t*>(src + 16 * k + 2 * q + 8)) : 0u;
        }
      } else {
        // columns 16 k + 4 q .. + 3, as the codes of a chunk fall to the lanes
        uint2 v[DQK / 16];
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < DQK / 16; ++k) {
          v[k] = row_ok ? __ldg(reinterpret_cast<const uint2*>(src + 16 * k + 4 * q)) : make_uint2(0u, 0u);
          top = fmaxf(top, fmaxf(fmaxf(fabsf(__uint_as_float(v[k].x << 16)), fabsf(__uint_as_float(v[k].x & 0xffff0000u))),
                                 fmaxf(fabsf(__uint_as_float(v[k].y << 16)), fabsf(__uint_as_float(v[k].y & 0xffff0000u)))));
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = min(max((int)(__float_as_uint(top) >> 23) - 127, -100), 127);  // of the largest
        const float f = exp2i(14 - e);
        cs[x] *= exp2i(e - 14);
#pragma unroll
        for (int k = 0; k < DQK / 16; ++k) {
          qa[k][x] = half2_of(__uint_as_float(v[k].x << 16) * f, __uint_as_float(v[k].x & 0xffff0000u) * f);
          qa[k][2 + x] = half2_of(__uint_as_float(v[k].y << 16) * f, __uint_as_float(v[k].y & 0xffff0000u) * f);
        }
      }
    }
    float o[OT][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < OT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

    for (int blk = g.blk0; blk < g.blk1; ++blk, ++cnt) {
      if ((int)(cnt % kConsumers) != warp) continue;
      const uint32_t st = cnt % NS;
      if (dead || !mbar_wait(full + 8 * st, (cnt / NS) & 1, abort, status)) {
        dead = true;
        continue;
      }
      const uint32_t kt = sb + L::TILES + st * L::STAGE, vt = kt + L::KB, sc = sb + L::SCALE0 + st * L::SCALES;
      const int k0 = blk * kKeys, nk = g.seq.lk - k0;
      if (nk < kKeys) {
        // values behind the sequence's end may be anything: as zeros they meet zero weights
        for (int i = lane; i < kKeys * DV * E / 16; i += 32) {
          const int row = DV * E >= 128 ? (i >> 3) % kKeys : i >> 2;
          if (row >= nk) st_shared_v4(vt + 16 * i, 0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();  // the stage's next loads come through the async proxy
        __syncwarp();
      }
      // ---- scores
      float s[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
        if constexpr (!MX) {
#pragma unroll
          for (int k2 = 0; k2 < DQK / 32; ++k2) {
            uint32_t b[4];
            ldsm4(b, kt + chunk_at<DQK, E, kKeys>(n * 8 + (lane & 7), 4 * k2 + (lane >> 3)));
            mma_16816_bf16(s[n], qa[2 * k2], b[0], b[1]);
            mma_16816_bf16(s[n], qa[2 * k2 + 1], b[2], b[3]);
          }
        } else {
          // scales of this lane's two keys (columns 2 q, 2 q + 1 of the score tile)
          constexpr int NB = DQK / 32;
          uint32_t sk[2];
          if constexpr (NB == 4) {
            sk[0] = ld_shared_u32(sc + (n * 8 + 2 * q) * 4);
            sk[1] = ld_shared_u32(sc + (n * 8 + 2 * q + 1) * 4);
          } else {
            const uint32_t x = ld_shared_u32(sc + (n * 8 + 2 * q) * 2);
            sk[0] = x & 0xffffu;
            sk[1] = x >> 16;
          }
#pragma unroll
          for (int h = 0; h < DQK / 64; ++h) {
            uint32_t b[4];
            ldsm4(b, kt + chunk_at<DQK, E, kKeys>(n * 8 + (lane & 7), 4 * h + (lane >> 3)));
#pragma unroll
            for (int i = 0; i < 2; ++i) {  // a block: two chunks of 16 columns
              float x[4] = {0.f, 0.f, 0.f, 0.f};
              mma_16816_f16(x, qa[4 * h + 2 * i], e4m3_half2(b[2 * i] & 0xffffu), e4m3_half2(b[2 * i] >> 16));
              mma_16816_f16(x, qa[4 * h + 2 * i + 1], e4m3_half2(b[2 * i + 1] & 0xffffu), e4m3_half2(b[2 * i + 1] >> 16));
              const float f0 = scale_of(sk[0] >> (8 * (2 * h + i))), f1 = scale_of(sk[1] >> (8 * (2 * h + i)));
              s[n][0] = fmaf(x[0], f0, s[n][0]);
              s[n][1] = fmaf(x[1], f1, s[n][1]);
              s[n][2] = fmaf(x[2], f0, s[n][2]);
              s[n][3] = fmaf(x[3], f1, s[n][3]);
            }
          }
        }
      }
      // ---- weights
      float mn[2], ref[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int seen = min(limit[x], g.seq.lk) - k0;  // keys of this stage the row sees
        float top = -INFINITY;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float& v = s[n][2 * x + i];
            v = n * 8 + 2 * q + i < seen ? v * cs[x] : -INFINITY;
            top = fmaxf(top, v);
          }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        mn[x] = fmaxf(m[x], top);
        ref[x] = mn[x] == -INFINITY ? 0.f : mn[x];
      }
      if (__any_sync(0xffffffffu, mn[0] != m[0] || mn[1] != m[1])) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float a = ex2(m[x] - ref[x]);
          l[x] *= a;
#pragma unroll
          for (int i = 0; i < OT; ++i) {
            o[i][2 * x] *= a;
            o[i][2 * x + 1] *= a;
          }
          m[x] = mn[x];
        }
      }
      uint32_t pa[NT / 2][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float a = ex2(s[n][2 * x] - ref[x]), b = ex2(s[n][2 * x + 1] - ref[x]);
          l[x] += a + b;
          // the weights' rounding to bf16, as the operand's type (2^-9 on average, signs mixed)
          pa[n >> 1][2 * (n & 1) + x] = pack_bf16(a, b);
        }
      }
      // ---- output
#pragma unroll
      for (int ks = 0; ks < kKeys / 16; ++ks) {
        if constexpr (!MX) {
#pragma unroll
          for (int np = 0; np < DV / 16; ++np) {
            uint32_t b[4];
            ldsm4t(b, vt + chunk_at<DV, E, kKeys>(ks * 16 + ((lane >> 3) & 1) * 8 + (lane & 7), 2 * np + (lane >> 4)));
            mma_16816_bf16(o[2 * np], pa[ks], b[0], b[1]);
            mma_16816_bf16(o[2 * np + 1], pa[ks], b[2], b[3]);
          }
        } else {
          // scales of this lane's four keys of the step
          constexpr int NB = DV / 32;
          uint32_t sv[4];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int key = ks * 16 + 8 * i + 2 * q;
            if constexpr (NB == 4) {
              sv[2 * i] = ld_shared_u32(sc + 128 + key * 4);
              sv[2 * i + 1] = ld_shared_u32(sc + 128 + key * 4 + 4);
            } else {
              const uint32_t x = ld_shared_u32(sc + 128 + key * 2);
              sv[2 * i] = x & 0xffffu;
              sv[2 * i + 1] = x >> 16;
            }
          }
#pragma unroll
          for (int cp = 0; cp < DV / 32; ++cp) {  // two chunks of 16 columns: one block
            uint32_t b[4];
            ldsm4t(b, vt + chunk_at<DV, E, kKeys>(ks * 16 + ((lane >> 3) & 1) * 8 + (lane & 7), 2 * cp + (lane >> 4)));
            float f[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = scale_of(sv[i] >> (8 * cp));
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t ev[2], od[2];  // even and odd columns, as two output tiles
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const uint32_t r = b[2 * c + i];
                const float2 x = fmul2(e4m3_values(r & 0xffffu), make_float2(f[2 * i], f[2 * i]));
                const float2 y = fmul2(e4m3_values(r >> 16), make_float2(f[2 * i + 1], f[2 * i + 1]));
                ev[i] = pack_bf16(x.x, y.x);
                od[i] = pack_bf16(x.y, y.y);
              }
              mma_16816_bf16(o[4 * cp + 2 * c], pa[ks], ev[0], ev[1]);
              mma_16816_bf16(o[4 * cp + 2 * c + 1], pa[ks], od[0], od[1]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + 8 * st);
    }

    // ---- the warps' parts of the tile become one
    const uint32_t ml = sb + L::ML;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
      if (q == 0) {
        st_shared_f32(ml + ((warp * 16 + rq + 8 * x) * 2) * 4, m[x]);
        st_shared_f32(ml + ((warp * 16 + rq + 8 * x) * 2 + 1) * 4, l[x]);
      }
    }
    consumers_sync();
    const float* mls = (const float*)(smem_raw + (ml - smem_u32(smem_raw)));
    auto joined = [&](int r, float& M, float& Ls) {
      M = -INFINITY;
#pragma unroll
      for (int i = 0; i < kConsumers; ++i) M = fmaxf(M, mls[(i * 16 + r) * 2]);
      const float ref = M == -INFINITY ? 0.f : M;
      Ls = 0.f;
#pragma unroll
      for (int i = 0; i < kConsumers; ++i) Ls = fmaf(mls[(i * 16 + r) * 2 + 1], ex2(mls[(i * 16 + r) * 2] - ref), Ls);
    };
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float M, Ls;
      joined(rq + 8 * x, M, Ls);
      const float a = ex2(m[x] - (M == -INFINITY ? 0.f : M));
#pragma unroll
      for (int i = 0; i < OT; ++i) {
        o[i][2 * x] *= a;
        o[i][2 * x + 1] *= a;
      }
    }
    const int tid = threadIdx.x, jr = tid >> 3, jc = (tid & 7) * 4;  // row and columns this thread adds up
    const int tok = g.tile * t.tokens + jr / t.gsub, gh = gs0 + jr % t.gsub;
    const bool jrow_ok = jr < t.rows && tok < g.seq.lq && gh < p.group;
    float M, Ls;
    joined(jr, M, Ls);
    const int64_t out_row = (int64_t)(g.seq.q0 + tok) * p.heads_q + head_k * p.group + gh;
    const int64_t part_row = ((int64_t)blockIdx.x * 2 + g.slot) * t.rows + jr;
    const float inv = Ls > 0.f ? 1.f / Ls : (Ls == 0.f ? 0.f : Ls);
    const float* jb = (const float*)(smem_raw + (sb + L::JOIN - smem_u32(smem_raw)));
#pragma unroll
    for (int rd = 0; rd < DV / 32; ++rd) {
      const uint32_t mine = sb + L::JOIN + warp * 16 * L::JOIN_LD * 4;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = rq + 8 * (e >> 1);
          // MXFP8 output tiles hold even and odd columns of 16
          const int c = MX ? 16 * (i >> 1) + 4 * q + 2 * (e & 1) + (i & 1) : 8 * i + 2 * q + (e & 1);
          st_shared_f32(mine + (r * L::JOIN_LD + c) * 4, o[4 * rd + i][e]);
        }
      consumers_sync();
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int v = 0; v < kConsumers; ++v) {
        const float4 a = *reinterpret_cast<const float4*>(jb + (v * 16 + jr) * L::JOIN_LD + jc);
        x.x += a.x; x.y += a.y; x.z += a.z; x.w += a.w;
      }
      if (g.slot >= 0) {
        if (jr < t.rows) *reinterpret_cast<float4*>(w.part_o + part_row * DV + 32 * rd + jc) = x;
      } else if (jrow_ok) {
        *reinterpret_cast<uint2*>((__nv_bfloat16*)p.o + out_row * DV + 32 * rd + jc) =
            make_uint2(pack_bf16(x.x * inv, x.y * inv), pack_bf16(x.z * inv, x.w * inv));
      }
      consumers_sync();
    }
    if ((tid & 7) == 0) {
      if (g.slot >= 0) {
        if (jr < t.rows) {
          w.part_ml[2 * part_row] = M;
          w.part_ml[2 * part_row + 1] = Ls;
        }
      } else if (jrow_ok) {
        p.lse[out_row] = Ls == 0.f ? -INFINITY : (M + log2f(Ls)) * kLn2;
      }
    }
  }
}

template <int DQK, int DV, int KIND>
cudaError_t launch_t(const Paged& p, const TileShape& t, int ctas, const PagedWs& w, cudaStream_t s) {
  using L = Layout<DQK, DV, KIND>;
  auto kern = paged_rows16_kernel<DQK, DV, KIND>;
  cudaError_t e = kernel_setup((const void*)kern, kThreads, L::SMEM);
  if (e != cudaSuccess) return e;
  const int64_t rows = (p.pages * p.heads_k) << p.page_shift;
  const int box = (1 << p.page_shift) < L::kKeys ? (1 << p.page_shift) : L::kKeys;
  CUtensorMap mk, mv;
  if (!make_rows_map(&mk, p.kc, L::E, rows, DQK, DQK * L::E < 128 ? DQK : 128 / L::E, box) ||
      !make_rows_map(&mv, p.vc, L::E, rows, DV, DV * L::E < 128 ? DV : 128 / L::E, box))
    return cudaErrorInvalidValue;
  kern<<<ctas, kThreads, L::SMEM, s>>>(p, t, w, mk, mv);
  return cudaGetLastError();
}
template <int KIND>
cudaError_t launch_dims(const Paged& p, const TileShape& t, int ctas, const PagedWs& w, cudaStream_t s) {
  if (p.dim_qk == 128)
    return p.dim_v == 128 ? launch_t<128, 128, KIND>(p, t, ctas, w, s) : launch_t<128, 64, KIND>(p, t, ctas, w, s);
  return p.dim_v == 128 ? launch_t<64, 128, KIND>(p, t, ctas, w, s) : launch_t<64, 64, KIND>(p, t, ctas, w, s);
}

}  // namespace

cudaError_t launch_paged_rows16(const Paged& p, const TileShape& t, int ctas, const PagedWs& w, cudaStream_t s) {
  return p.kind == kCacheMx ? launch_dims<kCacheMx>(p, t, ctas, w, s) : launch_dims<kCacheBf16>(p, t, ctas, w, s);
}

}  // namespace jfa
