// Attention over a paged cache for many query rows: chunks of prompts and whole prompts, on
// tcgen05.
//
// Bound: the tensor cores on long chunks (4 D flops a query row and key), HBM on short ones.
// One CTA per SM walks its share of the work (paged.cuh).  A tile is two 128-row MMA tiles A
// and B of the same key head, rows = consecutive tokens by the group's heads, so a key block
// loaded once serves 256 rows.  A and B are two streams of steps, one per block of 128 keys:
//   S = Q K^T -> softmax -> P -> O += P V,
// so that the softmax of one stream runs under the products of the other.  Where B has no rows
// (a chunk of at most 128 rows, the last tile of an odd number) the streams share A's queries
// and take the key blocks in turn, and A joins both outputs: two loads and two softmaxes in
// flight instead of one.
// Warps (a softmax thread owns a row: no exchange of row statistics):
//   0-3, 4-7  softmax of A and B, and their epilogues
//   8, 10     issue the MMAs of A and of B.  An issue holds its thread for most of the MMA's own
//             time, so one issuer for both left the tensor pipe idle at every wait and commit
//             (3,990 cycles for a block of both streams, of which the MMAs take 2,048).
//   9         loads Q, K and V by TMA; looks up 32 page table entries at a time
//   11        zeroes the rows of a V tile that lie behind the sequence's end, or in front of the
//             window and behind the sinks
//   12-19     MXFP8 only: turn codes and scales into bf16 tiles (exact)
// Tiles of K and V go round one ring (K0, V0, K1, ...).  Both issuers pass every stage in order
// and free it once, whether they use it or not: an mbarrier's phase is known by its parity
// alone, so a role that left phases out could take an older one for its own.
// TMEM: S_A, S_B at columns 0, 128; O_A, O_B at 256, 384.  P (bf16) replaces the first half of
// its S.  S of a stream's next step is issued behind PV of this one by the same thread, so by
// its commit PV has completed: O may then be rescaled without a further wait.
// The row maximum is kept lazily: O and the sum are rescaled only when it grows by more
// than 2^8.
// Measured: 8 prompts of 1024 to 4096 tokens, 32 heads on 8 of 128, causal, bf16: 412 us, 1110
// TFLOP/s; 13 chunks of up to 512 tokens over caches of up to 16384, 32 heads on 4, MXFP8: 451 us,
// 995 TFLOP/s.  The prompts without any softmax take 335 us, with its TMEM loads and stores 343:
// a stream's softmax and its products follow one another, since its S and P share their columns
// of TMEM, and both streams' tiles fill the 512.  Not faster: the weights handed over in halves
// (433 us), two threads a row (495; they share a scheduler), the exponentials begun against an
// older maximum (496), a rolled softmax that reads TMEM twice (445).
// Windows and shared prefixes are instances of their own (MODE): 13 chunks of up to 1,024 tokens over
// MXFP8 caches of up to 16,384, window 2,048, 16 sinks: 326 us (and 20 for the join), 37% of the MMAs' rate in visible
// pairs (no window, 451 us above: 52%); a window's masks and a third more exponentials than visible pairs
// are the rest.  64 candidates of 1 to 4 tokens behind each of 16 histories of 512 to 8,192 keys: phase 1
// 197 us, 42%; 128 single tokens behind one prefix of 6,011 MXFP8 keys: 39 us.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "paged.cuh"
#include "paged_join.cuh"
#include "serve_maps.h"
#include "tc_ptx.cuh"

namespace jfa {
namespace {
using namespace tc;

constexpr int kKeys = 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleLog2 = 8.0f;
constexpr int kIssuerA = 8, kLoader = 9, kIssuerB = 10, kCleaner = 11;

template <int DQK, int DV, int KIND>
struct Layout {
  static constexpr bool MX = KIND == kCacheMx;
  static constexpr int kThreads = MX ? 640 : 384;
  static constexpr int kConverters = 8;  // warps (MXFP8)
  static constexpr uint32_t Q_BYTES = DQK / 64 * 16384, K_BYTES = DQK / 64 * 16384, V_BYTES = DV / 64 * 16384;
  static constexpr uint32_t STAGE = K_BYTES > V_BYTES ? K_BYTES : V_BYTES;  // bf16 tile, K or V
  // MXFP8: tiles of codes and their scales as loaded
  static constexpr uint32_t RAW = MX ? kKeys * (DQK > DV ? DQK : DV) : 0, RAW_SC = MX ? 512 : 0;
  static constexpr int NR = MX ? 3 : 0;
  static constexpr uint32_t kMaxSmem = 232448;
  // in front: barriers, TMEM address, abort flag (1 KB); the statistics that B hands to A
  static constexpr uint32_t XCH = 1024, FRONT = XCH + 128 * 2 * 4;
  static constexpr uint32_t SC0 = FRONT, TILE0 = (SC0 + NR * RAW_SC + 1023) / 1024 * 1024;
  static constexpr uint32_t RAW0 = TILE0 + 2 * Q_BYTES, ST0 = RAW0 + NR * RAW;
  static constexpr int NS_ = (kMaxSmem - 1024 - ST0) / STAGE;
  static constexpr int NS = NS_ > 8 ? 8 : NS_;
  static constexpr uint32_t SMEM = ST0 + NS * STAGE + 1024;
  static_assert(NS >= 3 && SMEM <= kMaxSmem && SMEM >= 122880, "stages; one CTA owns the SM's TMEM");
};
enum : uint32_t {
  B_QFULL = 0, B_QEMPTY = 2, B_SFULL = 4, B_PFULL = 6, B_OFULL = 8, B_OEMPTY = 10, B_XCH = 12, B_DRAIN = 13,
  B_FULL = 15, B_EMPTY = 23, B_RFULL = 31, B_REMPTY = 35, B_VTAIL = 39, B_TURN = 47, B_HOLD = 49, B_COUNT = 50
};
static_assert(8 * B_COUNT + 8 <= 1024 - 32, "front: barriers, then the share");
constexpr uint32_t T_S = 0, T_O = 256;

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"((uint64_t)map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ uint32_t ld_shared_u8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void few_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// The steps of a segment of `blocks` key blocks: stream x takes n(x) of them.
struct Streams {
  int blocks, n0, n1;
  bool split;  // B works on A's rows, the streams take the blocks in turn
  __device__ __forceinline__ int n(int x) const { return x ? n1 : n0; }
  // block of stream x's step i
  __device__ __forceinline__ int block(int x, int i) const { return split ? 2 * i + x : i; }
};
template <bool WIN>
__device__ __forceinline__ Streams streams_of(const Paged& p, const TileShape& t, const PagedSegment& g) {
  Streams s;
  const int half = t.tokens / 2, tok0 = g.tile * t.tokens;
  s.blocks = g.blk1 - g.blk0;
  s.split = tok0 + half >= g.seq.lq;
  if (s.split) {
    s.n0 = (s.blocks + 1) / 2;
    s.n1 = s.blocks / 2;
  } else {
    // blocks that A's last row sees (all of A's tokens exist); B's last row is the tile's
    const int64_t last = p.causal ? g.seq.off + tok0 + half : (int64_t)g.seq.lk;
    int nb = last < 0 ? 0 : (int)((last + kKeys - 1) / kKeys);
    if (WIN && p.window > 0) nb = nb > g.span.first ? nb - g.span.first + g.span.ns : min(nb, g.span.ns);
    s.n0 = max(0, min(g.blk1, nb) - g.blk0);
    s.n1 = s.blocks;
  }
  return s;
}

// Whether some keys of the block from `k0` on are hidden from every row of the tile: behind the
// sequence's end, or in front of the window and behind the sinks.
template <bool WIN>
__device__ __forceinline__ bool has_hidden(const Paged& p, const PagedSegment& g, int k0) {
  return g.seq.lk < k0 + kKeys || (WIN && k0 < g.span.low && p.sinks < min(k0 + kKeys, g.span.low));
}

template <int DQK, int DV, int KIND, int MODE>
__global__ void __launch_bounds__(Layout<DQK, DV, KIND>::kThreads, 1)
paged_tc_kernel(const __grid_constant__ Paged p, const TileShape t, const PagedWs w,
                const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v) {
  using L = Layout<DQK, DV, KIND>;
  constexpr bool MX = L::MX, WIN = MODE == kWindow;
  constexpr int NS = L::NS, NR = MX ? L::NR : 1;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sb = (raw + 1023u) & ~1023u;
  uint8_t* const sp = smem_raw + (sb - raw);
  PagedPos* share = reinterpret_cast<PagedPos*>(sp + L::XCH - 32);
  int* status = paged_share<MODE>(p, t, w, share, sp + L::TILE0);  // in the queries' place, before any load
  auto bar = [&](uint32_t i) { return sb + 8u * i; };
  uint32_t* tmem_slot = (uint32_t*)(sp + 8 * B_COUNT);
  volatile int* abort = (volatile int*)(sp + 8 * B_COUNT + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(bar(B_QFULL + x), 1);
      mbar_init(bar(B_QEMPTY + x), x ? 1 : 2);  // A's queries: both issuers, B's: B's
      mbar_init(bar(B_SFULL + x), 1);
      mbar_init(bar(B_PFULL + x), 4);  // a warp arrives once
      mbar_init(bar(B_OFULL + x), 1);
      mbar_init(bar(B_OEMPTY + x), 4);
      mbar_init(bar(B_DRAIN + x), 1);
      mbar_init(bar(B_TURN + x), 1);
    }
    mbar_init(bar(B_XCH), 4);
    mbar_init(bar(B_HOLD), 1);  // test hook: nothing arrives on it
    for (int s = 0; s < NS; ++s) {
      mbar_init(bar(B_FULL + s), MX ? L::kConverters : 1);
      mbar_init(bar(B_EMPTY + s), 2);  // both issuers
      mbar_init(bar(B_VTAIL + s), 1);
    }
    for (int s = 0; s < NR; ++s) {
      mbar_init(bar(B_RFULL + s), 1);
      mbar_init(bar(B_REMPTY + s), L::kConverters);
    }
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == kIssuerA) tmem_alloc(smem_u32(tmem_slot), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int rows1 = t.rows / 2;  // rows of an MMA tile

  // The softmax warpgroups take registers that the others do not need: (2 x 208 + 88) x 128 of
  // the launch's 384 x 168, with MXFP8 (2 x 168 + 64 + 2 x 40) x 128 of its 640 x 96.
  if (warp >= 8 && warp < 12) few_registers<MX ? 64 : 88>();
  if (warp == kLoader) {
    // ---------------------------------------------------------------- loads
    PagedWalk walk;
    walk.init(share);
    PagedSegment g;
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    const int box = min(1 << p.page_shift, kKeys), per = kKeys / box;
    const int none = (int)((p.pages * p.heads_k) << p.page_shift);
    const uint32_t qbytes = DQK * 2 * (uint32_t)rows1;
    uint32_t it = 0, q_it[2] = {0, 0};
    bool ok = true;
    while (ok && walk.next<MODE>(p, t, g)) {
      const Streams s = streams_of<WIN>(p, t, g);
      if (s.blocks == 0) continue;
      const int head = g.unit;
      // In bf16 the queries go behind the first keys: their place is free only when the last tile's last
      // products are done, and the keys need not wait for that (prompts 420 us, 434 with the queries
      // first).  MXFP8's keys are still to be converted, from stages that run full ahead of the tile's end
      // anyway: there the queries go first (chunks 457 us, 479 with the keys first).
      auto queries = [&]() {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (s.n(x) == 0 || (s.split && x == 1)) continue;
          if (!mbar_wait(bar(B_QEMPTY + x), (q_it[x] & 1) ^ 1, abort, status)) return false;
          if (lane == 0) {
            mbar_expect_tx(bar(B_QFULL + x), qbytes);
#pragma unroll
            for (int a = 0; a < DQK / 64; ++a)
              tma_load_3d(sb + L::TILE0 + x * L::Q_BYTES + a * 16384, &tm_q, a * 64, head * p.group,
                          g.seq.q0 + g.tile * t.tokens + x * (t.tokens / 2), bar(B_QFULL + x));
          }
          ++q_it[x];
        }
        return true;
      };
      if (MX) ok = queries();
      for (int i0 = g.blk0; ok && i0 < g.blk1; i0 += 32 / per) {
        const int pos = WIN ? g.span.block(i0 + lane / per) * kKeys + lane % per * box : i0 * kKeys + lane * box;
        int row = none;
        // (pages that no row's window reaches may be gone: they are not looked up)
        const bool reached = !WIN || paged_sees(p, g.span.low, pos) || pos + box > g.span.low;
        if (pos < g.seq.lk && reached && i0 + lane / per < g.blk1) {
          const int page = paged_page(p, g.b, pos, status);
          if (page >= 0) row = (int)paged_row(p, page, head, pos);
        }
        const int n = min(32 / per, g.blk1 - i0);
        for (int i = 0; ok && i < n; ++i)
#pragma unroll
          for (int kv = 0; kv < 2; ++kv, ++it) {
            constexpr int ring = MX ? NR : NS;
            const uint32_t st = it % ring;
            const uint32_t full = bar((MX ? B_RFULL : B_FULL) + st), empty = bar((MX ? B_REMPTY : B_EMPTY) + st);
            if ((!MX && kv == 1 && i0 + i == g.blk0 && !queries()) || !mbar_wait(empty, ((it / ring) & 1) ^ 1, abort, status)) {
              ok = false;
              break;
            }
            const int D = kv ? DV : DQK;
            const CUtensorMap* tm = kv ? &tm_v : &tm_k;
            const uint32_t dst = MX ? sb + L::RAW0 + st * L::RAW : sb + L::ST0 + st * L::STAGE;
            // values of which some are to be cleaned land on a barrier of their own and become full then
            const int k0 = (WIN ? g.span.block(i0 + i) : i0 + i) * kKeys;
            const uint32_t lands = !MX && kv == 1 && has_hidden<WIN>(p, g, k0) ? bar(B_VTAIL + st) : full;
            if (lane == 0) mbar_expect_tx(lands, MX ? kKeys * D + kKeys * D / 32 : kKeys * D * 2);
            for (int s2 = 0; s2 < per; ++s2) {
              const int r = __shfl_sync(0xffffffffu, row, i * per + s2);
              if (lane == 0) {
                if constexpr (MX) {
                  tma_load_2d(dst + s2 * box * D, tm, 0, r, full);
                  const int64_t rs = r == none ? 0 : r;  // no row: any scales do, its codes are zeros
                  bulk_load(sb + L::SC0 + st * L::RAW_SC + s2 * box * (D / 32), (kv ? p.vs : p.ks) + rs * (D / 32),
                            box * (D / 32), full);
                } else {
                  for (int a = 0; a < D / 64; ++a)
                    tma_load_2d(dst + a * 16384 + s2 * box * 128, tm, a * 64, r, lands);
                }
              }
            }
          }
      }
    }
    if (lane == 0) {  // every load has landed before the CTA leaves
      if (MX) drain_ring(bar(B_RFULL), NR, it, status);
      else drain_ring(bar(B_FULL), NS, it, status);
      drain_ring(bar(B_QFULL), 1, q_it[0], status);
      drain_ring(bar(B_QFULL + 1), 1, q_it[1], status);
    }
    __syncwarp();
  } else if (warp == kIssuerA || warp == kIssuerB) {
    // ---------------------------------------------------------------- products of one stream
    PagedWalk walk;
    walk.init(share);
    PagedSegment g;
    constexpr uint32_t idesc_s = idesc_bf16(128, kKeys, 0, 0), idesc_o = idesc_bf16(128, DV, 0, 1);
    const int x = warp == kIssuerB;
    const uint32_t t_s = tmem + T_S + x * 128, t_o = tmem + T_O + x * 128;
    uint32_t it = 0, qa_it = 0, qb_it = 0, p_it = 0, o_it = 0, turn = 0;
    bool ok = !(w.hold && blockIdx.x == 0 && x == 0) || mbar_wait(bar(B_HOLD), 0, abort, status);
    while (ok && walk.next<MODE>(p, t, g)) {
      const Streams s = streams_of<WIN>(p, t, g);
      if (s.blocks == 0) continue;
      const int n = s.n(x);
      // B may work on A's queries: it passes every phase of both tiles, and frees A's at once where
      // it does not use them
      if (s.n0 > 0) {
        if (!(ok = mbar_wait(bar(B_QFULL), qa_it++ & 1, abort, status))) break;
        if (x == 1 && (!s.split || n == 0) && lane == 0) mbar_arrive(bar(B_QEMPTY));
      }
      if (x == 1 && !s.split && !(ok = mbar_wait(bar(B_QFULL + 1), qb_it++ & 1, abort, status))) break;
      const uint32_t qx = s.split ? 0 : x, q_tile = sb + L::TILE0 + qx * L::Q_BYTES;
      int i = 0;  // steps of the stream
      for (int d = 0; ok && d < s.blocks; ++d) {
        const bool mine = s.split ? (d & 1) == x : d < n;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv, ++it) {
          const uint32_t st = it % NS, tile = sb + L::ST0 + st * L::STAGE;
          // The streams take turns, block by block: a turn is P V of a block and S of the next.
          // Their MMAs then run one behind the other and each softmax under the other's products;
          // left alone, streams that start together stay in step, and both pipes wait by turns.
          if (kv == 1 && !mbar_wait(bar(B_TURN + x), (turn++ & 1) ^ (x == 0), abort, status)) {
            ok = false;
            break;
          }
          if (mine && kv == 1 &&
              (!mbar_wait(bar(B_PFULL + x), p_it & 1, abort, status) ||
               (i == 0 && !mbar_wait(bar(B_OEMPTY + x), (o_it & 1) ^ 1, abort, status)))) {
            ok = false;
            break;
          }
          if (!mbar_wait(bar(B_FULL + st), (it / NS) & 1, abort, status)) {
            ok = false;
            break;
          }
          __syncwarp();  // converged for elect.sync
          const bool passes = kv == 0 ? d > 0 : d == s.blocks - 1;  // the turn ends here
          if (!mine) {
            if (lane == 0) {
              mbar_arrive(bar(B_EMPTY + st));
              if (passes) mbar_arrive(bar(B_TURN + (x ^ 1)));
            }
            continue;
          }
          tc_fence_after();
          if (kv == 0) {
#pragma unroll
            for (int kk = 0; kk < DQK / 16; ++kk) {
              const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
              mma_bf16(t_s, sw128_desc(q_tile + off, 16, 1024), sw128_desc(tile + off, 16, 1024), idesc_s,
                       kk > 0 ? 1u : 0u);
            }
            if (passes && lane == 0) mbar_arrive(bar(B_TURN + (x ^ 1)));
            __syncwarp();
            mma_commit(bar(B_SFULL + x));
            mma_commit(bar(B_EMPTY + st));
            if (i == n - 1) mma_commit(bar(B_QEMPTY + qx));  // the queries' last use here
          } else {
#pragma unroll
            for (int kk = 0; kk < kKeys / 16; ++kk)
              mma_bf16_tmem_a(t_o, t_s + kk * 8, sw128_desc(tile + kk * 2048, 16384, 1024), idesc_o,
                              (i > 0 || kk > 0) ? 1u : 0u);
            if (passes && lane == 0) mbar_arrive(bar(B_TURN + (x ^ 1)));
            __syncwarp();
            if (i == n - 1) {
              mma_commit(bar(B_OFULL + x));
              ++o_it;
            }
            mma_commit(bar(B_EMPTY + st));
            ++p_it;
            ++i;
          }
        }
      }
    }
    __syncwarp();
    mma_drain(bar(B_DRAIN + x), status);  // every MMA issued has completed
    __syncwarp();
  } else if (warp == kCleaner) {
    // ---------------------------------------------------------------- ends of sequences
    if constexpr (!MX) {
      PagedWalk walk;
      walk.init(share);
      PagedSegment g;
      uint32_t it = 0, phase = 0;  // phase: a bit a stage
      bool ok = true;
      while (ok && walk.next<MODE>(p, t, g)) {
        // without a window, the segment's last block alone may have hidden keys
        for (int blk = WIN ? g.blk0 : max(g.blk0, g.blk1 - 1); ok && blk < g.blk1; ++blk) {
          const int k0 = (WIN ? g.span.block(blk) : blk) * kKeys;
          if (!has_hidden<WIN>(p, g, k0)) continue;
          // values of hidden keys may be anything: as zeros they meet zero weights
          const uint32_t st = (it + 2 * (blk - g.blk0) + 1) % NS, tile = sb + L::ST0 + st * L::STAGE;
          ok = mbar_wait(bar(B_VTAIL + st), (phase >> st) & 1, abort, status);
          if (!ok) break;
          phase ^= 1u << st;
          auto clean = [&](int r0, int r1) {
            for (int c = r0 * (DV / 8) + lane; c < r1 * (DV / 8); c += 32) {
              const int row = c / (DV / 8), ch = c % (DV / 8);
              st_shared_v4(tile + (ch >> 3) * 16384 + row * 128 + (ch & 7) * 16, 0u, 0u, 0u, 0u);
            }
          };
          if constexpr (WIN) clean(max(p.sinks - k0, 0), min(g.span.low - k0, kKeys));
          clean(max(g.seq.lk - k0, 0), kKeys);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B_FULL + st));
        }
        it += 2 * (g.blk1 - g.blk0);
      }
    }
  } else if (warp < 8) {
    // ---------------------------------------------------------------- softmax and epilogue
    more_registers<MX ? 168 : 208>();
    PagedWalk walk;
    walk.init(share);
    PagedSegment g;
    const int x = warp >> 2;
    const int r = 32 * (warp & 3) + lane;  // TMEM lane: row of the MMA tile
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t t_s = tmem + lane_base + T_S + x * 128, t_o = tmem + lane_base + T_O;
    const float c_score = p.scale * kLog2e;
    float2* xch = reinterpret_cast<float2*>(sp + L::XCH);
    const int half = t.tokens / 2;
    const int rt = r / t.gsub, rg = r - rt * t.gsub;
    uint32_t s_it = 0, o_it = 0, x_it = 0;
    bool ok = true;
    while (ok && walk.next<MODE>(p, t, g)) {
      const Streams s = streams_of<WIN>(p, t, g);
      const int n = s.n(x);
      const int tok = g.tile * t.tokens + (s.split ? 0 : x * half) + rt;
      const bool row_ok = r < rows1 && tok < g.seq.lq;
      const int64_t lim = !row_ok ? 0 : p.causal ? g.seq.off + tok + 1 : (int64_t)g.seq.lk;
      const int limit = lim < 0 ? 0 : (int)min(lim, (int64_t)g.seq.lk);  // keys the row sees
      float m = -INFINITY, l = 0.f;
      for (int i = 0; i < n; ++i, ++s_it) {
        if (!mbar_wait(bar(B_SFULL + x), s_it & 1, abort, status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        float sv[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(t_s + 32 * c, sv + 32 * c);
        tmem_wait_ld();
        const int blk = g.blk0 + s.block(x, i), k0 = (WIN ? g.span.block(blk) : blk) * kKeys;
        const int seen = limit - k0;
        if constexpr (WIN) {
          // of the block's keys: the row's window, and the sinks
          const int from = max(limit - p.window, 0) - k0, front = p.sinks - k0;
          if (seen < kKeys || (from > 0 && front < kKeys)) {
#pragma unroll
            for (int c = 0; c < kKeys; c += 32) {
              const uint32_t bits = window_bits(c, from, front, seen);
#pragma unroll
              for (int k = 0; k < 32; ++k) sv[c + k] = (bits >> k) & 1 ? sv[c + k] : -INFINITY;
            }
          }
        } else if (seen < kKeys) {
#pragma unroll
          for (int k = 0; k < kKeys; ++k) sv[k] = k < seen ? sv[k] : -INFINITY;
        }
        float mx[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) mx[k] = fmaxf(sv[2 * k], sv[2 * k + 1]);
#pragma unroll
        for (int k = 16; k < kKeys; k += 16)
#pragma unroll
          for (int c = 0; c < 8; ++c) mx[c] = fmax3(mx[c], sv[k + 2 * c], sv[k + 2 * c + 1]);
        const float mt = fmax3(fmax3(mx[0], mx[1], mx[2]), fmax3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7])) * c_score;
        const bool need = mt > m + kRescaleLog2;  // m = -inf: any key
        if (__any_sync(0xffffffffu, need)) {
          float alpha = 1.f;
          if (need) {
            alpha = ex2(m - mt);
            m = mt;
            l *= alpha;
          }
          if (i > 0) {  // S(i) committed behind PV(i - 1): O is at rest
            float ov[16];  // few at a time: the scores stay in registers
#pragma unroll 1
            for (int c = 0; c < DV / 16; ++c) {
              tmem_ld16(t_o + x * 128 + 16 * c, ov);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) ov[k] *= alpha;
              tmem_st16(t_o + x * 128 + 16 * c, reinterpret_cast<const uint32_t*>(ov));
            }
          }
        }
        const float ref = m == -INFINITY ? 0.f : m;
        const float2 cc = make_float2(c_score, c_score), nm = make_float2(-ref, -ref);
        float2 rs0 = make_float2(0.f, 0.f), rs1 = make_float2(0.f, 0.f);
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          uint32_t pk[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float2 e = ffma2(make_float2(sv[32 * h + 2 * k], sv[32 * h + 2 * k + 1]), cc, nm);
            const float2 pv = make_float2(ex2(e.x), ex2(e.y));
            if (k & 1) rs1 = fadd2(rs1, pv);
            else rs0 = fadd2(rs0, pv);
            pk[k] = pack_bf16(pv.x, pv.y);  // the operand's type: 2^-9 of a weight on average
          }
          tmem_st16(t_s + 16 * h, pk);
        }
        const float2 rr = fadd2(rs0, rs1);
        l += rr.x + rr.y;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_PFULL + x));
      }
      if (!ok) break;
      // ------------------------------------------------------------ the tile's end
      const bool joins = s.split && s.n1 > 0;  // A adds B's part
      if (s.split && x == 1) {
        if (n > 0) {
          if (!mbar_wait(bar(B_OFULL + 1), o_it & 1, abort, status)) break;
          ++o_it;
          // only now: B's first product has waited for A to have read the last tile's
          xch[r] = make_float2(m, l);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B_XCH));
        }
        continue;
      }
      float m2 = -INFINITY, l2 = 0.f;
      if (n > 0) {
        if (!mbar_wait(bar(B_OFULL + x), o_it & 1, abort, status)) break;
        ++o_it;
      }
      if (joins) {
        if (!mbar_wait(bar(B_XCH), x_it & 1, abort, status)) break;
        ++x_it;
        m2 = xch[r].x;
        l2 = xch[r].y;
      }
      tc_fence_after();
      const float M = fmaxf(m, m2), ref = M == -INFINITY ? 0.f : M;
      const float f1 = ex2(m - ref), f2 = ex2(m2 - ref);
      const float lt = l * f1 + l2 * f2;
      const int64_t orow = (int64_t)(g.seq.q0 + tok) * p.heads_q + g.unit * p.group + rg;
      const int64_t prow = ((int64_t)blockIdx.x * 2 + g.slot) * t.rows + x * rows1 + r;
      const bool whole = g.slot < 0;
      float inv = !whole ? 1.f : lt > 0.f ? 1.f / lt : (lt == 0.f ? 0.f : lt);
      // a shared prefix: phase 1 leaves fp32, phase 2 adds that to its own
      const bool prior = MODE == kShared && whole && p.phase == 2;
      PagedJoin join{};
      if (prior && row_ok) {
        join = paged_join_prior(M, lt, p.prior_lse[orow]);
        inv = join.own;
      }
      if (n > 0) {
#pragma unroll 1
        for (int c = 0; c < DV / 32; ++c) {
          float ov[32];
          tmem_ld32(t_o + x * 128 + 32 * c, ov);
          if (joins) {
            float o2[32];
            tmem_ld32(t_o + 128 + 32 * c, o2);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) ov[k] = ov[k] * f1 + o2[k] * f2;
          } else {
            tmem_wait_ld();
          }
          if (MODE == kShared && whole) {
            if (row_ok) {
              float4* at = reinterpret_cast<float4*>(p.prior_o + orow * DV + 32 * c);
#pragma unroll
              for (int k = 0; k < 32; ++k) ov[k] *= inv;
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                if (!prior) {
                  at[k] = make_float4(ov[4 * k], ov[4 * k + 1], ov[4 * k + 2], ov[4 * k + 3]);
                } else {
                  const float4 y = at[k];
                  ov[4 * k] = fmaf(y.x, join.prior, ov[4 * k]);
                  ov[4 * k + 1] = fmaf(y.y, join.prior, ov[4 * k + 1]);
                  ov[4 * k + 2] = fmaf(y.z, join.prior, ov[4 * k + 2]);
                  ov[4 * k + 3] = fmaf(y.w, join.prior, ov[4 * k + 3]);
                }
              }
              if (prior) store32_bf16((__nv_bfloat16*)p.o + orow * DV + 32 * c, ov, 1.f);
            }
          } else if (whole) {
            if (row_ok) store32_bf16((__nv_bfloat16*)p.o + orow * DV + 32 * c, ov, inv);
          } else if (r < rows1) {
            float4* dst = reinterpret_cast<float4*>(w.part_o + prow * DV + 32 * c);
#pragma unroll
            for (int k = 0; k < 8; ++k) dst[k] = make_float4(ov[4 * k], ov[4 * k + 1], ov[4 * k + 2], ov[4 * k + 3]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(B_OEMPTY + x));
          if (joins) mbar_arrive(bar(B_OEMPTY + 1));
        }
      } else if (MODE == kShared && whole && row_ok) {  // no keys: zeros, or phase 1's result alone
        for (int c = 0; c < DV / 32; ++c) {
          float4* at = reinterpret_cast<float4*>(p.prior_o + orow * DV + 32 * c);
          float z[32];
          for (int k = 0; k < 8; ++k) {
            if (!prior) at[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            const float4 y = at[k];
            z[4 * k] = y.x;
            z[4 * k + 1] = y.y;
            z[4 * k + 2] = y.z;
            z[4 * k + 3] = y.w;
          }
          if (prior) store32_bf16((__nv_bfloat16*)p.o + orow * DV + 32 * c, z, join.prior);
        }
      } else if (whole && row_ok) {
        const float z[32] = {0.f};
        for (int c = 0; c < DV / 32; ++c) store32_bf16((__nv_bfloat16*)p.o + orow * DV + 32 * c, z, 1.f);
      }
      if (MODE == kShared && whole) {
        if (row_ok && prior) p.lse[orow] = join.lse;
        if (row_ok && !prior) p.prior_lse[orow] = lt == 0.f ? -INFINITY : M + log2f(lt);
      } else if (whole) {
        if (row_ok) p.lse[orow] = lt == 0.f ? -INFINITY : (M + log2f(lt)) * kLn2;
      } else if (r < rows1) {
        // a part without keys has no output: its maximum says so
        w.part_ml[2 * prow] = joins ? M : m;
        w.part_ml[2 * prow + 1] = joins ? lt : l;
      }
    }
  } else if (MX && warp >= 12) {
    // ---------------------------------------------------------------- MXFP8 to bf16 tiles
    few_registers<40>();
    if constexpr (MX) {
      PagedWalk walk;
      walk.init(share);
      PagedSegment g;
      const int row = threadIdx.x & 127, part = (threadIdx.x - 384) >> 7;  // key of the block, half of its columns
      uint32_t it = 0;
      bool ok = true;
      while (ok && walk.next<MODE>(p, t, g)) {
        for (int blk = g.blk0; ok && blk < g.blk1; ++blk) {
          // hidden rows become zeros
          const int at = (WIN ? g.span.block(blk) : blk) * kKeys + row;
          const bool live = at < g.seq.lk && (!WIN || paged_sees(p, g.span.low, at));
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv, ++it) {
            const int D = kv ? DV : DQK;
            const uint32_t rs = it % NR, st = it % NS;
            if (!mbar_wait(bar(B_RFULL + rs), (it / NR) & 1, abort, status) ||
                !mbar_wait(bar(B_EMPTY + st), ((it / NS) & 1) ^ 1, abort, status)) {
              ok = false;
              break;
            }
            const uint32_t src = sb + L::RAW0 + rs * L::RAW, sc = sb + L::SC0 + rs * L::RAW_SC + row * (D / 32);
            const uint32_t dst = sb + L::ST0 + st * L::STAGE;
            const int c0 = part * (D / 32), c1 = c0 + D / 32;  // 16-byte chunks of codes
#pragma unroll 1  // in 40 registers: 459 us for the chunked prompts, 486 with two chunks at once, 515 with four
            for (int c = c0; c < c1; ++c) {
              const uint32_t chunk = D == 128 ? src + row * 128 + ((c ^ (row & 7)) << 4)
                                              : src + row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
              const uint4 v = ld_shared_v4(chunk);
              // scale byte of the chunk's block; 255 counts as the largest, so zeros stay zeros
              const float f = __uint_as_float(min(ld_shared_u8(sc + c / 2), 254u) << 23);
              const float2 ff = make_float2(f, f);
              const uint32_t in[4] = {v.x, v.y, v.z, v.w};
              uint32_t o[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const float2 y = fmul2(e4m3_values((in[k >> 1] >> (16 * (k & 1))) & 0xffffu), ff);
                o[k] = live ? pack_bf16(y.x, y.y) : 0u;  // exact: 3-bit mantissas
              }
              const uint32_t d0 = dst + (c >> 2) * 16384;
              st_shared_v4(d0 + sw128_offset(row, (2 * c) & 7), o[0], o[1], o[2], o[3]);
              st_shared_v4(d0 + sw128_offset(row, (2 * c + 1) & 7), o[4], o[5], o[6], o[7]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(bar(B_FULL + st));
              mbar_arrive(bar(B_REMPTY + rs));
            }
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kIssuerA) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Queries as [token][head][dim], read in boxes of `tokens` x group x 64 columns.
bool make_query_map(CUtensorMap* map, const Paged& p, int tokens) {
  void* ptr = nullptr;
  cudaDriverEntryPointQueryResult q;
  static const PFN_cuTensorMapEncodeTiled_v12000 fn =
      cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
              q == cudaDriverEntryPointSuccess
          ? (PFN_cuTensorMapEncodeTiled_v12000)ptr
          : nullptr;
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)p.dim_qk, (cuuint64_t)p.heads_q, (cuuint64_t)p.total_q};
  // one token has no stride of its own
  const int64_t st = p.total_q > 1 ? p.sq : (int64_t)p.heads_q * p.dim_qk;
  const cuuint64_t strides[2] = {(cuuint64_t)p.dim_qk * 2, (cuuint64_t)st * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)p.group, (cuuint32_t)tokens};
  const cuuint32_t elem[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p.q), dims, strides, box, elem,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DQK, int DV, int KIND, int MODE>
cudaError_t launch_t(const Paged& p, const TileShape& t, int ctas, const PagedWs& w, cudaStream_t s) {
  using L = Layout<DQK, DV, KIND>;
  auto kern = paged_tc_kernel<DQK, DV, KIND, MODE>;
  cudaError_t e = kernel_setup((const void*)kern, L::kThreads, L::SMEM);
  if (e != cudaSuccess) return e;
  const int64_t rows = (p.pages * p.heads_k) << p.page_shift;
  const int box = (1 << p.page_shift) < kKeys ? (1 << p.page_shift) : kKeys;
  constexpr int E = L::MX ? 1 : 2;
  CUtensorMap mq, mk, mv;
  if (!make_query_map(&mq, p, t.tokens / 2) ||
      !make_rows_map(&mk, p.kc, E, rows, DQK, L::MX ? DQK : 64, box) ||
      !make_rows_map(&mv, p.vc, E, rows, DV, L::MX ? DV : 64, box))
    return cudaErrorInvalidValue;
  kern<<<ctas, L::kThreads, L::SMEM, s>>>(p, t, w, mq, mk, mv);
  return cudaGetLastError();
}
template <int KIND, int MODE>
cudaError_t launch_dims(const Paged& p, const TileShape& t, int ctas, const PagedWs& w, cudaStream_t s) {
  if (p.dim_qk == 128)
    return p.dim_v == 128 ? launch_t<128, 128, KIND, MODE>(p, t, ctas, w, s)
                          : launch_t<128, 64, KIND, MODE>(p, t, ctas, w, s);
  return p.dim_v == 128 ? launch_t<64, 128, KIND, MODE>(p, t, ctas, w, s)
                        : launch_t<64, 64, KIND, MODE>(p, t, ctas, w, s);
}
template <int MODE>
cudaError_t launch_tc(const Paged& p, const TileShape& t, int ctas, const PagedWs& w, cudaStream_t s) {
  return p.kind == kCacheMx ? launch_dims<kCacheMx, MODE>(p, t, ctas, w, s)
                            : launch_dims<kCacheBf16, MODE>(p, t, ctas, w, s);
}

}  // namespace
}  // namespace jfa
