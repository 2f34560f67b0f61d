// Attention over a paged cache for few query rows: up to 16 rows that share a key head (a
// serving step's single tokens with their group of heads, or a few tokens).
//
// Bound: HBM.  A key and its value are read once and meet at most 16 rows, 4 to 32 flops a
// byte, so what counts is that loads never pause.  A CTA has one producer warp, which walks
// the CTA's share of the work ahead of the others and fills a ring of stages (32 or 64 keys and
// their values each, by TMA; page table entries are looked up 32 at a time), and four consumer
// warps.  Two warps share a stage, half each, and a warp keeps its own running maximum,
// sum and output, so the warps meet only at a tile's end, where they join through shared
// memory while the producer already fills the ring with the next tile.
//
// The products run on mma.sync (16 x 8 x 16) transposed, S^T = K Q^T and O^T = V^T P^T: keys and
// value columns are the 16 of its M and the rows its N, 8 or 16 of them, so that a step with one
// token and up to 8 heads a key head pads little and needs half the registers and MMAs (three
// CTAs an SM instead of two).  tcgen05's smallest tile would be seven eighths empty.  K and V
// come straight from the stage by ldmatrix (swizzled, no bank conflicts), and P turns from S^T's
// layout into an operand's by movmatrix.
//
// MXFP8.  Codes are exact in fp16, and a row of bf16 queries times a power of two that brings
// its largest value to [2^14, 2^15) is exact in fp16 too (values under 2^-31 of the largest lose
// at most 2^-39 of it), so the scores are fp16 products of codes, one block of 32 columns at a
// time, and a block's scale times the row's own power of two multiplies its fp32 sum.  For the
// output the scales go to the weights: a block of columns has a reference scale, the largest it met
// (O is kept in its units), and the weights, rounded to fp16, times scale / reference, at most 1,
// meet fp16 codes.  The largest weight is kept at 2^10 to 2^15, so that one of 2^-25 of it still makes
// a product of 2^-15, which its two roundings to steps of 2^-24 leave within 2^-9.  A stage where a
// weight times a scale may be less takes its values to bf16 instead (exact) and rounds the weights
// alone, to bf16: keys of small weights or values keep their precision beside keys of large ones
// whose values are zero.
//
// Measured: one token for each of 256 users, lengths to 4096, 32 heads on 8 of 128, bf16 pages:
// 317 us, 6.6 TB/s, 97% of the copy rate.  One or two tokens for 96 users, lengths 512 to 16384,
// 32 heads on 4 (16 rows a tile), MXFP8: 183 us, 4.6 TB/s, 68%; the loads alone take 135 us, the
// rest is the consumers' latency: registers allow two CTAs an SM.  With scores of three times the
// spread nearly every stage takes its values to bf16: 228 us (weights scaled in bf16 against codes
// in bf16 instead: 222 us, but 189 us for scores of the usual spread).
//
// Windows and shared prefixes are instances of their own (MODE).  A tile under a window walks the blocks
// that hold its rows' windows and the sinks'; boxes in front of them are not looked up, and what such a
// block holds in front of the window is cleaned, a stage at a time, by the warps that use it.  One token
// for each of 256 users, histories to 8,192, window 1,024 and 4 sinks, 32 heads on 8: 172 to 176 us with the join, 5.7
// to 5.9 TB/s, 85 to 88%.
// Of a shared prefix this is phase 1 where groups have few rows, and phase 2 over the sequences' own
// keys: 128 continuations over up to 1,024 MXFP8 keys each, 32 heads on 4: 42 us; phase 1's results are
// asked for ahead of the join of the four warps.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "paged.cuh"
#include "paged_join.cuh"
#include "serve_maps.h"
#include "tc_ptx.cuh"

namespace jfa {
namespace {
using namespace tc;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// A row's reference is kUp (log2) below the score it was set from and moves when one passes that by
// kRescale.  Over MXFP8 weights stay within 2^15 (a half's largest is 2^16); moved at 2^2 or 2^4 the
// step in the header takes 188 or 183 us.
template <int KIND>
constexpr float kUp = KIND == kCacheMx ? 10.0f : 0.0f;
template <int KIND>
constexpr float kRescale = KIND == kCacheMx ? 5.0f : 8.0f;

template <int DQK, int DV, int KIND, int NT>
struct Layout {
  static constexpr int R = 8 * NT;  // rows of a tile
  static constexpr int kConsumers = 4, kThreads = 32 * (kConsumers + 1);
  static constexpr int E = KIND == kCacheMx ? 1 : 2;  // bytes of an element
  // Keys of a stage, and of each of the two warps that share it.  A stage costs the producer
  // about 850 cycles whatever its size, so at half the size an MXFP8 step ran at its pace.
  static constexpr int kStage = paged_rows16_keys(DQK, DV, KIND), kKeys = kStage / 2;
  static constexpr uint32_t KB = kStage * DQK * E, VB = kStage * DV * E;
  static constexpr uint32_t KS = KIND == kCacheMx ? kStage * DQK / 32 : 0;
  static constexpr uint32_t STAGE = KB + VB;
  static constexpr uint32_t SCALES = 512;  // a stage's scales (K at 0, V at 256)
  static constexpr uint32_t LIMIT = NT == 1 ? 74 * 1024 + 512 : 113 * 1024;
  // in front: barriers, abort flag, statistics; then the join's buffer, the value scales as fp16
  // factors, the scales, the stages
  static constexpr uint32_t ML = 512;  // [warps][R][2] floats
  static constexpr uint32_t JOIN = ML + kConsumers * R * 2 * 4;
  static constexpr int JOIN_LD = 36;  // 32 columns a round, padded
  static constexpr uint32_t FAC = JOIN + kConsumers * R * JOIN_LD * 4;  // [warps][blocks][32 keys] halves
  static constexpr uint32_t SCALE0 = FAC + (KS ? kConsumers * (DV / 32) * 64 : 0);
  static constexpr int NS_ = (LIMIT - SCALE0 - 1024) / (STAGE + (KS ? SCALES : 0));
  // Even, so that a stage is always the same two warps': fills land in any order, and a warp that
  // came to a stage before another's previous fill of it had landed would take that fill's
  // parity for its own.
  static constexpr int NS = (NS_ >= 16 ? 16 : NS_) / 2 * 2;
  static constexpr uint32_t TILES = (SCALE0 + (KS ? NS * SCALES : 0) + 1023) / 1024 * 1024;
  static constexpr uint32_t SMEM = TILES + NS * STAGE + 1024;  // 1 KB to align the base
  static_assert(NS >= 4 && SMEM <= LIMIT, "stages");
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
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
      "%2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_16816_f16(float (&c)[4], const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// c = a b, nothing added
__device__ __forceinline__ void mma_16816_f16_zero(float (&c)[4], const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, "
      "%10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
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
// 2^(s - 127) of byte B of x (0: zero)
template <int B>
__device__ __forceinline__ float scale_byte(uint32_t x) {
  return __uint_as_float((B < 3 ? x << (23 - 8 * B) : x >> 1) & 0x7f800000u);
}
// 16 bytes to shared memory, or zeros; and this thread's arrival once its copies have landed
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
// an 8 x 8 matrix of 16-bit values, transposed
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// The producer warp runs converged and one elected lane issues (from inside a branch of one lane
// an issue costs more).
__device__ __forceinline__ void expect_elected(uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n.reg .pred e;\n.reg .b64 st;\nelect.sync _|e, 0xffffffff;\n"
      "@e mbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n}" ::"r"(bar),
      "r"(bytes)
      : "memory");
}
__device__ __forceinline__ void load_elected(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "{\n.reg .pred e;\nelect.sync _|e, 0xffffffff;\n"
      "@e cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n}" ::"r"(
          dst),
      "l"((uint64_t)map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
template <int THREADS>
__device__ __forceinline__ void consumers_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
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
template <int D, int E, int ROWS>
__device__ __forceinline__ uint32_t chunk_at(int row, int c) {
  if constexpr (D * E >= 128) return (c >> 3) * (ROWS * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4);
  return row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
}

template <int DQK, int DV, int KIND, int NT, int MODE>
__global__ void __launch_bounds__(Layout<DQK, DV, KIND, NT>::kThreads, NT == 1 ? 3 : 2)
paged_rows16_kernel(const __grid_constant__ Paged p, const TileShape t, const PagedWs w,
                    const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v) {
  using L = Layout<DQK, DV, KIND, NT>;
  constexpr int E = L::E, NS = L::NS, kStage = L::kStage, kKeys = L::kKeys, kConsumers = L::kConsumers;
  constexpr bool MX = KIND == kCacheMx, WIN = MODE == kWindow;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t sb = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t full = sb, empty = sb + 8 * NS, hold = sb + 16 * NS + 8;
  volatile int* abort = (volatile int*)(smem_raw + (sb - smem_u32(smem_raw)) + 16 * NS);
  // in the stages' place, before any load
  PagedPos* share = reinterpret_cast<PagedPos*>(smem_raw + (sb - smem_u32(smem_raw)) + L::ML - 32);
  int* status = paged_share<MODE>(p, t, w, share, smem_raw + (sb - smem_u32(smem_raw)) + L::TILES);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(full + 8 * s, MX ? 33 : 1);  // the TMA loads, and every producer lane's scales
      mbar_init(empty + 8 * s, 2);
    }
    mbar_init(hold, 1);  // test hook: nothing arrives on it
    *abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  PagedWalk walk;
  walk.init(share);
  PagedSegment g;
  uint32_t cnt = 0;  // stages so far

  if (warp == kConsumers) {
    // ------------------------------------------------------------------ producer
    if (lane == 0) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    const int box = min(1 << p.page_shift, kStage), per = kStage / box;  // rows of a box, boxes of a stage
    const int none = (int)((p.pages * p.heads_k) << p.page_shift);    // behind the last row: read as zeros
    bool ok = true;
    while (ok && walk.next<MODE>(p, t, g)) {
      const int head = g.unit / t.nsub;
      for (int i0 = g.blk0; ok && i0 < g.blk1; i0 += 32 / per) {
        // this lane's box of the next 32: its first row, or one behind the cache where it has no keys
        const int pos = WIN ? g.span.block(i0 + lane / per) * kStage + lane % per * box : i0 * kStage + lane * box;
        int row = none;
        // (pages that no row's window reaches may be gone: they are not looked up)
        const bool reached = !WIN || paged_sees(p, g.span.low, pos) || pos + box > g.span.low;
        if (pos < g.seq.lk && reached && i0 + lane / per < g.blk1) {
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
          __syncwarp();
          expect_elected(bar, L::KB + L::VB);
          for (int s = 0; s < per; ++s) {
            const int r = __shfl_sync(0xffffffffu, row, i * per + s);
#pragma unroll
            for (int h = 0; h < (DQK * E + 127) / 128; ++h)
              load_elected(tile + h * kStage * 128 + s * box * (DQK * E < 128 ? DQK * E : 128), &tm_k, h * (128 / E), r,
                           bar);
#pragma unroll
            for (int h = 0; h < (DV * E + 127) / 128; ++h)
              load_elected(tile + L::KB + h * kStage * 128 + s * box * (DV * E < 128 ? DV * E : 128), &tm_v,
                           h * (128 / E), r, bar);
          }
          if constexpr (MX) {
            // the scales, 16 bytes a lane: first the keys', then the values'; zeros for keys that
            // are not there
            constexpr int CK = kStage * (DQK / 32) / 16, CV = kStage * (DV / 32) / 16;
            static_assert(CK + CV <= 32, "a piece a lane");
            const bool val = lane >= CK;
            const int c = val ? lane - CK : lane, nb = val ? DV / 32 : DQK / 32, key = c * 16 / nb;
            const int r = __shfl_sync(0xffffffffu, row, i * per + min(key / box, per - 1));
            const uint32_t sc = sb + L::SCALE0 + st * L::SCALES;
            if (lane < CK + CV)
              copy16(sc + (val ? 256 : 0) + c * 16,
                     (val ? p.vs : p.ks) + (r == none ? 0 : ((int64_t)r + key % box) * nb), r != none);
            copies_arrive(bar);
          }
        }
      }
    }
    if (lane == 0) drain_ring(full, NS, cnt, status);  // every load has landed before the CTA leaves
    __syncwarp();
    return;
  }

  // -------------------------------------------------------------------- consumers
  // Fragments: a lane's keys (or value columns) are kq and kq + 8 of 16, its rows 2 q and 2 q + 1
  // of 8; as an operand's holder of Q and P it has row kq.
  const int kq = lane >> 2, q = lane & 3;
  constexpr int G16 = kKeys / 16;  // groups of 16 keys
  constexpr int MT = DV / 16;      // output tiles
  constexpr int NBK = DQK / 32, NBV = DV / 32;
  // a consumer that gave up in a wait walks on without computing, so that its barriers still match
  bool dead = w.hold && blockIdx.x == 0 && warp == 0 && !mbar_wait(hold, 0, abort, status);
  while (walk.next<MODE>(p, t, g)) {
    const int head_k = g.unit / t.nsub, gs0 = (g.unit % t.nsub) * t.gsub;
    uint32_t qb[NT][DQK / 16][2];
    int limit[NT][2];  // keys that rows 2 q, 2 q + 1 see
    float cs[NT][2];   // their score units to log2 units
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = 8 * nt + kq, tok = g.tile * t.tokens + r / t.gsub, gh = gs0 + r % t.gsub;
      const bool row_ok = r < t.rows && tok < g.seq.lq && gh < p.group;
      const __nv_bfloat16* src = (const __nv_bfloat16*)p.q + (int64_t)(g.seq.q0 + tok) * p.sq +
                                 (int64_t)(head_k * p.group + gh) * DQK;
      const int64_t lim = g.seq.off + tok + 1;
      const int mine = !row_ok ? 0 : p.causal ? (int)max((int64_t)0, lim) : g.seq.lk;
      float c = p.scale * kLog2e;
      if constexpr (!MX) {
#pragma unroll
        for (int k = 0; k < DQK / 16; ++k) {
          qb[nt][k][0] = row_ok ? __ldg(reinterpret_cast<const uint32_t*>(src + 16 * k + 2 * q)) : 0u;
          qb[nt][k][1] = row_ok ? __ldg(reinterpret_cast<const uint32_t*>(src + 16 * k + 2 * q + 8)) : 0u;
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
        c *= exp2i(e - 14);
#pragma unroll
        for (int k = 0; k < DQK / 16; ++k) {
          qb[nt][k][0] = half2_of(__uint_as_float(v[k].x << 16) * f, __uint_as_float(v[k].x & 0xffff0000u) * f);
          qb[nt][k][1] = half2_of(__uint_as_float(v[k].y << 16) * f, __uint_as_float(v[k].y & 0xffff0000u) * f);
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        limit[nt][e] = __shfl_sync(0xffffffffu, mine, (2 * q + e) * 4);
        cs[nt][e] = __shfl_sync(0xffffffffu, c, (2 * q + e) * 4);
      }
    }
    float o[NT][MT][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < MT; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
    }
    // MXFP8: the blocks' reference scales (biased, at most 254; O of block b is in units of
    // 2^(ref - 127))
    int ref_scale[NBV];
#pragma unroll
    for (int i = 0; i < NBV; ++i) ref_scale[i] = 0;

    for (int blk = g.blk0; blk < g.blk1; ++blk, ++cnt) {
      if ((int)(cnt & 1) != warp >> 1) continue;
      const uint32_t st = cnt % NS;
      if (dead || !mbar_wait(full + 8 * st, (cnt / NS) & 1, abort, status)) {
        dead = true;
        continue;
      }
      const uint32_t kt = sb + L::TILES + st * L::STAGE, vt = kt + L::KB;
      const int rb = (warp & 1) * kKeys;  // this warp's rows of the stage
      const uint32_t sck = sb + L::SCALE0 + st * L::SCALES + rb * NBK, scv = sb + L::SCALE0 + st * L::SCALES + 256 + rb * NBV;
      const int k0 = (WIN ? g.span.block(blk) : blk) * kStage + rb, nk = g.seq.lk - k0;
      // keys [front, back) of this half are in front of every row's window and none of the sinks
      const int front = WIN ? max(p.sinks - k0, 0) : 0, back = WIN ? min(g.span.low - k0, kKeys) : 0;
      if (nk <= 0) {  // the sequence ends in the other half
        if (lane == 0) mbar_arrive(empty + 8 * st);
        continue;
      }
      if (nk < kKeys || (WIN && front < back)) {
        // values behind the sequence's end may be anything: as zeros they meet zero weights
        for (int i = lane; i < kKeys * DV * E / 16; i += 32) {
          constexpr int per = DV * E >= 128 ? 8 : 4;  // pieces of 16 bytes in a row of a box
          const int row = i / per % kKeys, half = i / (per * kKeys);
          if (row >= nk || (WIN && row >= front && row < back)) st_shared_v4(vt + half * kStage * 128 + (rb + row) * per * 16 + i % per * 16, 0u, 0u, 0u, 0u);
        }
        if constexpr (MX) {  // and their scales, which have to be numbers: the first key's
          uint32_t first = NBV == 4 ? ld_shared_u32(scv) : ld_shared_u32(scv) & 0xffffu;
          if (WIN && front == 0 && back > 0) first = 0u;  // (which is hidden too: none)
          if constexpr (WIN) __syncwarp();  // all have read it
          if (lane >= nk || (WIN && lane >= front && lane < back)) {
            if constexpr (NBV == 4) asm volatile("st.shared.u32 [%0], %1;" ::"r"(scv + lane * 4), "r"(first) : "memory");
            else asm volatile("st.shared.u16 [%0], %1;" ::"r"(scv + lane * 2), "h"((uint16_t)first) : "memory");
          }
        }
        fence_proxy_async_smem();  // the stage's next loads come through the async proxy
        __syncwarp();
      }
      // the four 8 x 8 matrices that a lane's address names: halves of 16 keys, chunks
      const int mi = lane >> 3, mr = lane & 7;
      // ---- scores
      float s[G16][NT][4];
#pragma unroll
      for (int ks = 0; ks < G16; ++ks) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[ks][nt][0] = s[ks][nt][1] = s[ks][nt][2] = s[ks][nt][3] = 0.f;
        if constexpr (!MX) {
#pragma unroll
          for (int k4 = 0; k4 < DQK / 16; k4 += 4) {  // four loads on their way
            uint32_t a[4][4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              ldsm4(a[k], kt + chunk_at<DQK, E, kStage>(rb + ks * 16 + (mi & 1) * 8 + mr, 2 * (k4 + k) + (mi >> 1)));
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_16816_bf16(s[ks][nt], a[k], qb[nt][k4 + k][0], qb[nt][k4 + k][1]);
          }
        } else {
          uint32_t sk[2];  // scales of keys kq, kq + 8
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int key = ks * 16 + kq + 8 * i;
            if constexpr (NBK == 4) sk[i] = ld_shared_u32(sck + key * 4);
            else sk[i] = ld_shared_u32(sck + (key & ~1) * 2) >> (16 * (key & 1));
          }
          uint32_t kb[NBK][4];  // the group's codes, all on their way before the first is needed
#pragma unroll
          for (int c2 = 0; c2 < NBK; ++c2)
            ldsm4(kb[c2], kt + chunk_at<DQK, E, kStage>(rb + ks * 16 + (mi & 1) * 8 + mr, 2 * c2 + (mi >> 1)));
          auto block = [&](int c2, float f0, float f1) {  // a block: two chunks of 16 columns
            const uint32_t (&b)[4] = kb[c2];
            uint32_t a[2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              a[j][0] = e4m3_half2(b[2 * j] & 0xffffu);
              a[j][1] = e4m3_half2(b[2 * j + 1] & 0xffffu);
              a[j][2] = e4m3_half2(b[2 * j] >> 16);
              a[j][3] = e4m3_half2(b[2 * j + 1] >> 16);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float x[4];
              mma_16816_f16_zero(x, a[0], qb[nt][2 * c2][0], qb[nt][2 * c2][1]);
              mma_16816_f16(x, a[1], qb[nt][2 * c2 + 1][0], qb[nt][2 * c2 + 1][1]);
              // the key's scale and the row's units in one factor: neither product alone leaves fp32
              // where the score does not
              const float2 c = make_float2(cs[nt][0], cs[nt][1]);
              const float2 y0 = ffma2(make_float2(x[0], x[1]), fmul2(make_float2(f0, f0), c),
                                      make_float2(s[ks][nt][0], s[ks][nt][1]));
              const float2 y1 = ffma2(make_float2(x[2], x[3]), fmul2(make_float2(f1, f1), c),
                                      make_float2(s[ks][nt][2], s[ks][nt][3]));
              s[ks][nt][0] = y0.x;
              s[ks][nt][1] = y0.y;
              s[ks][nt][2] = y1.x;
              s[ks][nt][3] = y1.y;
            }
          };
          block(0, scale_byte<0>(sk[0]), scale_byte<0>(sk[1]));
          block(1, scale_byte<1>(sk[0]), scale_byte<1>(sk[1]));
          if constexpr (NBK == 4) {
            block(2, scale_byte<2>(sk[0]), scale_byte<2>(sk[1]));
            block(3, scale_byte<3>(sk[0]), scale_byte<3>(sk[1]));
          }
        }
      }
      // ---- weights
      // A row's reference moves, with its sum and output, only when a score passes it far enough:
      // then alone the lanes exchange their maxima.
      constexpr float kMost = kUp<KIND> + kRescale<KIND>;
      bool need = false;
      float top[NT][2], low[NT][2];  // low: MXFP8, of the keys the row sees
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int seen = min(limit[nt][e], g.seq.lk) - k0;  // keys of this stage the row sees
          const int from = WIN ? max(limit[nt][e] - p.window, 0) - k0 : 0;
          top[nt][e] = -INFINITY;
          low[nt][e] = INFINITY;
#pragma unroll
          for (int ks = 0; ks < G16; ++ks)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float& v = s[ks][nt][2 * h + e];
              const int key = ks * 16 + 8 * h + kq;
              const bool sees = key < seen && (!WIN || key >= from || key < front);
              if constexpr (!MX) v *= cs[nt][e];
              if constexpr (MX) low[nt][e] = fminf(low[nt][e], sees ? v : INFINITY);
              v = sees ? v : -INFINITY;
              top[nt][e] = fmaxf(top[nt][e], v);
            }
          need |= top[nt][e] > m[nt][e] + kMost;  // m = -inf: any key
        }
      if (__any_sync(0xffffffffu, need)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = top[nt][e];
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            if (x > m[nt][e] + kMost) {
              x -= kUp<KIND>;
              const float a = ex2(m[nt][e] - x);  // m = -inf: 0
              l[nt][e] *= a;
#pragma unroll
              for (int i = 0; i < MT; ++i) {
                o[nt][i][e] *= a;
                o[nt][i][2 + e] *= a;
              }
              m[nt][e] = x;
            }
          }
      }
      float ref[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) ref[nt][e] = m[nt][e] == -INFINITY ? 0.f : m[nt][e];
#pragma unroll
      for (int ks = 0; ks < G16; ++ks)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s[ks][nt][i] = ex2(s[ks][nt][i] - ref[nt][i & 1]);
            l[nt][i & 1] += s[ks][nt][i];
          }
      // The weights as the products' operand: rounded to bf16 (2^-9 of a weight on average, signs
      // mixed) or, against fp16 codes, to fp16.
      bool wide = false;  // MXFP8: a product of weight and scale may be too small for fp16
      if constexpr (MX) {
        const uint32_t mine = NBV == 4 ? ld_shared_u32(scv + lane * 4)
                                       : (ld_shared_u32(scv + (lane & ~1) * 2) >> (16 * (lane & 1))) & 0xffffu;
        const uint32_t fac = sb + L::FAC + warp * NBV * 64;
        float deep = -INFINITY;  // how far (log2) a weight lies under 1
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) deep = fmaxf(deep, m[nt][e] - low[nt][e]);
        // a scale above its reference, or one or a weight so small that their product may be
        bool out = deep > 11.f;
#pragma unroll
        for (int i = 0; i < NBV; ++i) out |= (uint32_t)(ref_scale[i] - (int)((mine >> (8 * i)) & 255)) > 4u;
        if (__any_sync(0xffffffffu, out)) {
          bool above = false;
#pragma unroll
          for (int i = 0; i < NBV; ++i) above |= (int)((mine >> (8 * i)) & 255) > ref_scale[i];
          if (__any_sync(0xffffffffu, above)) {
#pragma unroll
            for (int i = 0; i < NBV; ++i) {
              const int most = __reduce_max_sync(0xffffffffu, min((mine >> (8 * i)) & 255, 254u));
              if (most > ref_scale[i]) {  // O of the block goes to the new units, with a step to spare
                const int to = min(most + 1, 254);
                const float f = ref_scale[i] == 0 ? 1.f : exp2i(max(ref_scale[i] - to, -126));
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int k = 0; k < 4; ++k) {
                    o[nt][2 * i][k] *= f;
                    o[nt][2 * i + 1][k] *= f;
                  }
                ref_scale[i] = to;
              }
            }
          }
          int gap = 0;  // steps (log2) of this key's scales under their references
#pragma unroll
          for (int i = 0; i < NBV; ++i) {
            const int e = (mine >> (8 * i)) & 255;
            if (e != 0) gap = max(gap, ref_scale[i] - e);
          }
          gap = __reduce_max_sync(0xffffffffu, gap);
          wide = gap > 14 || __any_sync(0xffffffffu, deep + (float)gap > 15.f);
        }
#pragma unroll
        for (int i = 0; i < NBV; ++i) {
          // the key's scale over the reference, 2^-14 to 1 as a half; a scale of 0 makes zeros, so that O
          // is zero until a block has a reference
          const int e = (mine >> (8 * i)) & 255;
          const uint16_t h = e == 0 ? 0 : (uint16_t)((e - ref_scale[i] + 15) << 10);
          asm volatile("st.shared.u16 [%0], %1;" ::"r"(fac + (i * 32 + lane) * 2), "h"(h) : "memory");
        }
        __syncwarp();
      }
      uint32_t pb[G16][NT][2];
#pragma unroll
      for (int ks = 0; ks < G16; ++ks)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float a = s[ks][nt][2 * h], b = s[ks][nt][2 * h + 1];
            pb[ks][nt][h] = movmatrix(MX && !wide ? half2_of(a, b) : pack_bf16(a, b));
          }
      // ---- output
#pragma unroll
      for (int ks = 0; ks < G16; ++ks) {
        if constexpr (!MX) {
#pragma unroll
          for (int m4 = 0; m4 < MT; m4 += 4) {
            uint32_t a[4][4];
#pragma unroll
            for (int mt = 0; mt < 4; ++mt)
              ldsm4t(a[mt], vt + chunk_at<DV, E, kStage>(rb + ks * 16 + (mi >> 1) * 8 + mr, 2 * (m4 + mt) + (mi & 1)));
#pragma unroll
            for (int mt = 0; mt < 4; ++mt)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_16816_bf16(o[nt][m4 + mt], a[mt], pb[ks][nt][0], pb[ks][nt][1]);
          }
        } else if (!wide) {
          const uint32_t fac = sb + L::FAC + warp * NBV * 64 + (ks * 16 + 2 * q) * 2;
          uint32_t vb[NBV][4], fv[NBV][2];
#pragma unroll
          for (int cp = 0; cp < NBV; ++cp) {
            ldsm4t(vb[cp], vt + chunk_at<DV, E, kStage>(rb + ks * 16 + (mi & 1) * 8 + mr, 2 * cp + (mi >> 1)));
            fv[cp][0] = ld_shared_u32(fac + cp * 64);
            fv[cp][1] = ld_shared_u32(fac + cp * 64 + 16);
          }
#pragma unroll
          for (int cp = 0; cp < NBV; ++cp) {  // two chunks of 16 columns: one block
            const uint32_t (&b)[4] = vb[cp];
            const uint32_t f0 = fv[cp][0], f1 = fv[cp][1];
            uint32_t pw[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              pw[nt][0] = hmul2(pb[ks][nt][0], f0);
              pw[nt][1] = hmul2(pb[ks][nt][1], f1);
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              // codes of keys 2 q, 2 q + 1: even columns to the low half, odd ones to the high, as
              // rows kq and kq + 8 of the tile
              const uint32_t r0 = __byte_perm(b[2 * c], 0, 0x3120), r1 = __byte_perm(b[2 * c + 1], 0, 0x3120);
              const uint32_t a[4] = {e4m3_half2(r0 & 0xffffu), e4m3_half2(r0 >> 16), e4m3_half2(r1 & 0xffffu),
                                     e4m3_half2(r1 >> 16)};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_16816_f16(o[nt][2 * cp + c], a, pw[nt][0], pw[nt][1]);
            }
          }
        } else {
#pragma unroll
          for (int cp = 0; cp < NBV; ++cp) {
            uint32_t b[4];
            ldsm4t(b, vt + chunk_at<DV, E, kStage>(rb + ks * 16 + (mi & 1) * 8 + mr, 2 * cp + (mi >> 1)));
            // 2^(127 - reference), of which 2^-127 is no normal number, and its product with the
            // scale 2^127 is exact all the same
            const float unit = ref_scale[cp] == 254 ? __uint_as_float(0x00400000u) : exp2i(127 - ref_scale[cp]);
            float f[4];  // of keys 2 q, 2 q + 1, 2 q + 8, 2 q + 9
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int key = ks * 16 + 2 * q + (i & 1) + 8 * (i >> 1);
              const uint32_t x = NBV == 4 ? ld_shared_u32(scv + key * 4)
                                          : ld_shared_u32(scv + (key & ~1) * 2) >> (16 * (key & 1));
              f[i] = unit * __uint_as_float(((x >> (8 * cp)) & 255u) << 23);
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t a[4];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const uint32_t r = b[2 * c + i];
                const float2 x = fmul2(e4m3_values(r & 0xffffu), make_float2(f[2 * i], f[2 * i]));
                const float2 y = fmul2(e4m3_values(r >> 16), make_float2(f[2 * i + 1], f[2 * i + 1]));
                a[2 * i] = pack_bf16(x.x, y.x);
                a[2 * i + 1] = pack_bf16(x.y, y.y);
              }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_16816_bf16(o[nt][2 * cp + c], a, pb[ks][nt][0], pb[ks][nt][1]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + 8 * st);
    }

    // the rows that this thread adds up at the end
    constexpr int CW = L::R / 4, PER = 32 / CW;  // columns a thread adds up in a round, threads of a row
    const int tid = threadIdx.x, jr = tid / PER, jc = tid % PER * CW;
    const int tok = g.tile * t.tokens + jr / t.gsub, gh = gs0 + jr % t.gsub;
    const bool jrow_ok = jr < t.rows && tok < g.seq.lq && gh < p.group;
    const int64_t out_row = (int64_t)(g.seq.q0 + tok) * p.heads_q + head_k * p.group + gh;
    // a shared prefix: what phase 1 left of them is on its way through the rounds below
    const bool joins = MODE == kShared && p.phase == 2 && g.slot < 0 && jrow_ok;
    float2 prior[MODE == kShared ? DV / 32 : 1][CW / 2];
    float prior_lse = 0.f;
    if constexpr (MODE == kShared) {
      if (joins) prior_lse = p.prior_lse[out_row];
#pragma unroll
      for (int rd = 0; rd < DV / 32; ++rd)
#pragma unroll
        for (int c = 0; c < CW / 2; ++c)
          if (joins) prior[rd][c] = *reinterpret_cast<const float2*>(p.prior_o + out_row * DV + 32 * rd + jc + 2 * c);
    }
    // ---- the warps' parts of the tile become one
    const uint32_t ml = sb + L::ML;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 4);
        l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 8);
        l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 16);
        l[nt][e] *= exp2i(-(int)kUp<KIND>);  // back to weights of at most about 1
        m[nt][e] += kUp<KIND>;
        if (kq == 0) {
          const uint32_t at = ml + ((warp * L::R + 8 * nt + 2 * q + e) * 2) * 4;
          st_shared_f32(at, m[nt][e]);
          st_shared_f32(at + 4, l[nt][e]);
        }
      }
    consumers_sync<32 * kConsumers>();
    const float* mls = (const float*)(smem_raw + (ml - smem_u32(smem_raw)));
    auto joined = [&](int r, float& M, float& Ls) {
      M = -INFINITY;
#pragma unroll
      for (int i = 0; i < kConsumers; ++i) M = fmaxf(M, mls[(i * L::R + r) * 2]);
      const float ref = M == -INFINITY ? 0.f : M;
      Ls = 0.f;
#pragma unroll
      for (int i = 0; i < kConsumers; ++i) Ls = fmaf(mls[(i * L::R + r) * 2 + 1], ex2(mls[(i * L::R + r) * 2] - ref), Ls);
    };
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float M, Ls;
        joined(8 * nt + 2 * q + e, M, Ls);
        const float a = ex2(m[nt][e] - (M == -INFINITY ? 0.f : M)) * exp2i(-(int)kUp<KIND>);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const float f = MX && ref_scale[i / 2] > 0 ? exp2i(ref_scale[i / 2] - 127) : 1.f;
          o[nt][i][e] = o[nt][i][e] * a * f;
          o[nt][i][2 + e] = o[nt][i][2 + e] * a * f;
        }
      }
    float M, Ls;
    joined(jr, M, Ls);
    const int64_t part_row = ((int64_t)blockIdx.x * 2 + g.slot) * t.rows + jr;
    float inv = Ls > 0.f ? 1.f / Ls : (Ls == 0.f ? 0.f : Ls);
    PagedJoin join{};
    if (joins) {
      join = paged_join_prior(M, Ls, prior_lse);
      inv = join.own;
    }
    const float* jb = (const float*)(smem_raw + (sb + L::JOIN - smem_u32(smem_raw)));
#pragma unroll
    for (int rd = 0; rd < DV / 32; ++rd) {
      const uint32_t mine = sb + L::JOIN + warp * L::R * L::JOIN_LD * 4;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = 8 * nt + 2 * q + (e & 1);
            // a tile's rows are columns in order; with MXFP8 rows kq, kq + 8 are columns 2 kq, 2 kq + 1
            const int c = 16 * i + (MX ? 2 * kq + (e >> 1) : kq + 8 * (e >> 1));
            st_shared_f32(mine + (r * L::JOIN_LD + c) * 4, o[nt][2 * rd + i][e]);
          }
      consumers_sync<32 * kConsumers>();
      float x[CW];
#pragma unroll
      for (int c = 0; c < CW; ++c) x[c] = 0.f;
#pragma unroll
      for (int v = 0; v < kConsumers; ++v)
#pragma unroll
        for (int c = 0; c < CW; c += 2) {
          const float2 y = *reinterpret_cast<const float2*>(jb + (v * L::R + jr) * L::JOIN_LD + jc + c);
          x[c] += y.x;
          x[c + 1] += y.y;
        }
#pragma unroll
      for (int c = 0; c < CW; c += 2) {
        if (g.slot >= 0) {
          if (jr < t.rows)
            *reinterpret_cast<float2*>(w.part_o + part_row * DV + 32 * rd + jc + c) = make_float2(x[c], x[c + 1]);
        } else if (MODE == kShared && jrow_ok) {
          const int64_t at = out_row * DV + 32 * rd + jc + c;
          if (p.phase == 1) {
            *reinterpret_cast<float2*>(p.prior_o + at) = make_float2(x[c] * inv, x[c + 1] * inv);
          } else {
            const float2 y = prior[rd][c / 2];
            *reinterpret_cast<uint32_t*>((__nv_bfloat16*)p.o + at) =
                pack_bf16(fmaf(y.x, join.prior, x[c] * inv), fmaf(y.y, join.prior, x[c + 1] * inv));
          }
        } else if (jrow_ok) {
          *reinterpret_cast<uint32_t*>((__nv_bfloat16*)p.o + out_row * DV + 32 * rd + jc + c) =
              pack_bf16(x[c] * inv, x[c + 1] * inv);
        }
      }
      consumers_sync<32 * kConsumers>();
    }
    if (tid % PER == 0) {
      if (g.slot >= 0) {
        if (jr < t.rows) {
          w.part_ml[2 * part_row] = M;
          w.part_ml[2 * part_row + 1] = Ls;
        }
      } else if (MODE == kShared && jrow_ok) {
        if (p.phase == 1) p.prior_lse[out_row] = Ls == 0.f ? -INFINITY : M + log2f(Ls);
        else p.lse[out_row] = join.lse;
      } else if (jrow_ok) {
        p.lse[out_row] = Ls == 0.f ? -INFINITY : (M + log2f(Ls)) * kLn2;
      }
    }
  }
}

template <int DQK, int DV, int KIND, int NT, int MODE>
cudaError_t launch_t(const Paged& p, const TileShape& t, int ctas, const PagedWs& w, cudaStream_t s) {
  using L = Layout<DQK, DV, KIND, NT>;
  auto kern = paged_rows16_kernel<DQK, DV, KIND, NT, MODE>;
  cudaError_t e = kernel_setup((const void*)kern, L::kThreads, L::SMEM);
  if (e != cudaSuccess) return e;
  const int64_t rows = (p.pages * p.heads_k) << p.page_shift;
  const int box = (1 << p.page_shift) < L::kStage ? (1 << p.page_shift) : L::kStage;
  CUtensorMap mk, mv;
  if (!make_rows_map(&mk, p.kc, L::E, rows, DQK, DQK * L::E < 128 ? DQK : 128 / L::E, box) ||
      !make_rows_map(&mv, p.vc, L::E, rows, DV, DV * L::E < 128 ? DV : 128 / L::E, box))
    return cudaErrorInvalidValue;
  kern<<<ctas, L::kThreads, L::SMEM, s>>>(p, t, w, mk, mv);
  return cudaGetLastError();
}
template <int DQK, int DV, int KIND, int MODE>
cudaError_t launch_rows(const Paged& p, const TileShape& t, int ctas, const PagedWs& w, cudaStream_t s) {
  return t.rows <= 8 ? launch_t<DQK, DV, KIND, 1, MODE>(p, t, ctas, w, s)
                     : launch_t<DQK, DV, KIND, 2, MODE>(p, t, ctas, w, s);
}
template <int KIND, int MODE>
cudaError_t launch_dims(const Paged& p, const TileShape& t, int ctas, const PagedWs& w, cudaStream_t s) {
  if (p.dim_qk == 128)
    return p.dim_v == 128 ? launch_rows<128, 128, KIND, MODE>(p, t, ctas, w, s)
                          : launch_rows<128, 64, KIND, MODE>(p, t, ctas, w, s);
  return p.dim_v == 128 ? launch_rows<64, 128, KIND, MODE>(p, t, ctas, w, s)
                        : launch_rows<64, 64, KIND, MODE>(p, t, ctas, w, s);
}
template <int MODE>
cudaError_t launch_rows16(const Paged& p, const TileShape& t, int ctas, const PagedWs& w, cudaStream_t s) {
  return p.kind == kCacheMx ? launch_dims<kCacheMx, MODE>(p, t, ctas, w, s)
                            : launch_dims<kCacheBf16, MODE>(p, t, ctas, w, s);
}

}  // namespace

}  // namespace jfa
