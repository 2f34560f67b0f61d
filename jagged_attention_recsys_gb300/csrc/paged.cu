// Attention of new tokens over a paged cache: the work plan, the CUDA-core kernel and the
// kernel that joins split tiles.
//
// Work.  A tile is the query rows of consecutive new tokens that share a key head (grouped
// heads read each key once); its cost is the keys its last row sees plus a fixed overhead.
// The plan lays all tiles end to end (sequence, key head, tile) and cuts their total cost into
// equal shares, one per CTA, at key-block boundaries: every CTA has the same work whatever the
// lengths, from one user with a long history to many with short ones.  A tile that a cut
// falls into is computed in parts: each CTA leaves its unnormalised output and softmax
// statistics in its slot of the workspace (a CTA has at most two such parts, its first and its
// last), and the join kernel adds a tile's parts in CTA order, so the results repeat bit for
// bit and no atomics are used.
//
// The cost of the tiles in front of tile t of a sequence is a closed form (an arithmetic
// series under the causal mask), so the plan needs one scan over the sequences and one binary
// search per CTA, and no list of tiles.  Batches of at most kPlanInCta sequences need no launch
// for it unless the caller asks for a plan: each CTA scans the lengths itself (1 us of loads and
// shuffles) and the join gathers the CTAs' statuses.  A step of four users over short caches
// takes 24 us a call instead of 33 by that and lighter argument handling.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "paged.cuh"

namespace jfa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// ------------------------------------------------------------------------------- plan
constexpr int kPlanThreads = 1024;
constexpr int kPlanSmemSeqs = 4096;  // scan kept in shared memory up to this batch

__global__ void __launch_bounds__(kPlanThreads)
paged_plan_kernel(const __grid_constant__ Paged p, const TileShape t, int ctas, const PagedWs w) {
  extern __shared__ int64_t smem_cum[];
  __shared__ int64_t warp_sum[32];
  __shared__ int64_t carry_s;
  __shared__ int bad_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t B = p.batch;
  int64_t* cum = B <= kPlanSmemSeqs ? smem_cum : w.cum;
  if (tid == 0) {
    carry_s = 0;
    bad_s = B == 0 && p.offs[0] != 0;
    cum[0] = 0;
  }
  __syncthreads();
  for (int64_t base = 0; base < B; base += kPlanThreads) {
    const int64_t b = base + tid;
    int64_t x = b < B ? checked_cost(p, t, b) : 0;
    if (x < 0) {
      bad_s = 1;
      x = 0;
    }
    for (int m = 1; m < 32; m <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, m);
      if (lane >= m) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    if (warp == 0) {
      int64_t y = warp_sum[lane];
      for (int m = 1; m < 32; m <<= 1) {
        const int64_t z = __shfl_up_sync(0xffffffffu, y, m);
        if (lane >= m) y += z;
      }
      warp_sum[lane] = y;
    }
    __syncthreads();
    const int64_t carry = carry_s;
    if (warp > 0) x += warp_sum[warp - 1];
    if (b < B) cum[b + 1] = carry + x;
    __syncthreads();
    if (tid == kPlanThreads - 1) carry_s = carry + x;
    __syncthreads();
  }
  const int64_t W = carry_s;
  const bool bad = bad_s != 0;
  if (tid == 0) w.hdr->status = bad ? JFA_ERR_BAD_OFFSETS : JFA_OK;
  for (int c = tid; c <= ctas; c += kPlanThreads) w.pos[c] = paged_cut(p, t, ctas, c, cum, W, bad);
}

// ------------------------------------------------------------------- the CUDA-core kernel
// Any types and any dims that are multiples of 8: fp32 arithmetic throughout.  A CTA holds a
// tile of up to 16 rows and blocks of 32 keys in shared memory as fp32; eight threads share a
// row.  It serves fp32 and the shapes the tensor-core kernels do not take.
constexpr int kRows = 16, kKeys = 32, kSimtThreads = 128;

template <typename T>
__device__ __forceinline__ float value(const T* x) { return (float)*x; }
template <>
__device__ __forceinline__ float value(const __nv_bfloat16* x) { return __bfloat162float(*x); }

template <typename T>
__device__ __forceinline__ T result(float x) { return (T)x; }
template <>
__device__ __forceinline__ __nv_bfloat16 result(float x) { return __float2bfloat16_rn(x); }

// Column c of a cache row
template <int KIND>
__device__ __forceinline__ float cache_value(const void* codes, const uint8_t* scales, int64_t row, int dim, int c) {
  if constexpr (KIND == kCacheF32) return ((const float*)codes)[row * dim + c];
  if constexpr (KIND == kCacheBf16) return __bfloat162float(((const __nv_bfloat16*)codes)[row * dim + c]);
  const float f = __uint_as_float((uint32_t)scales[row * (dim >> 5) + (c >> 5)] << 23);
  return e4m3_values(((const uint8_t*)codes)[row * dim + c]).x * f;
}

template <typename T, int KIND>
__global__ void __launch_bounds__(kSimtThreads)
paged_simt_kernel(const __grid_constant__ Paged p, const TileShape t, const PagedWs w) {
  extern __shared__ __align__(16) float sm[];
  const int dq = p.dim_qk, dv = p.dim_v, ldq = dq + 1, ldv = dv + 1;
  float* Q = sm;                  // [16][dq + 1]
  float* K = Q + kRows * ldq;     // [32][dq + 1]
  float* V = K + kKeys * ldq;     // [32][dv + 1]
  float* S = V + kKeys * ldv;     // [16][33]
  __shared__ int64_t row_of[kKeys];
  const int tid = threadIdx.x, r = tid >> 3, sub = tid & 7;
  __shared__ PagedPos share[2];
  int* status = paged_share(p, t, w, share, sm);
  PagedWalk walk;
  walk.init(share);
  PagedSegment g;
  while (walk.next(p, t, g)) {
    const int head_k = g.unit / t.nsub, gs0 = (g.unit % t.nsub) * t.gsub;
    // this thread's row
    const int tok = g.tile * t.tokens + r / t.gsub, gh = gs0 + r % t.gsub;
    const bool row_ok = r < t.rows && tok < g.seq.lq && gh < p.group;
    const int head = head_k * p.group + gh;
    for (int i = tid; i < t.rows * dq; i += kSimtThreads) {
      const int rr = i / dq, c = i - rr * dq;
      const int tk = g.tile * t.tokens + rr / t.gsub, hh = gs0 + rr % t.gsub;
      Q[rr * ldq + c] = tk < g.seq.lq && hh < p.group
                            ? value((const T*)p.q + (int64_t)(g.seq.q0 + tk) * p.sq + (int64_t)(head_k * p.group + hh) * dq + c)
                            : 0.f;
    }
    for (int i = tid + t.rows * ldq; i < kRows * ldq; i += kSimtThreads) Q[i] = 0.f;
    const int64_t limit = !row_ok ? 0 : p.causal ? g.seq.off + tok + 1 : g.seq.lk;  // keys the row sees
    float m = -INFINITY, l = 0.f, acc[16];
#pragma unroll
    for (int c = 0; c < 16; ++c) acc[c] = 0.f;
    for (int blk = g.blk0; blk < g.blk1; ++blk) {
      const int k0 = blk * kKeys, nk = min(kKeys, g.seq.lk - k0);
      __syncthreads();
      if (tid < kKeys) {
        int64_t row = -1;
        if (tid < nk) {
          const int page = paged_page(p, g.b, k0 + tid, status);
          if (page >= 0) row = paged_row(p, page, head_k, k0 + tid);
        }
        row_of[tid] = row;
      }
      __syncthreads();
      // slots behind the sequence's end are never read
      for (int i = tid; i < kKeys * dq; i += kSimtThreads) {
        const int j = i / dq, c = i - j * dq;
        K[j * ldq + c] = row_of[j] >= 0 ? cache_value<KIND>(p.kc, p.ks, row_of[j], dq, c) : 0.f;
      }
      for (int i = tid; i < kKeys * dv; i += kSimtThreads) {
        const int j = i / dv, c = i - j * dv;
        V[j * ldv + c] = row_of[j] >= 0 ? cache_value<KIND>(p.vc, p.vs, row_of[j], dv, c) : 0.f;
      }
      __syncthreads();
      float s[kKeys / 8], mt = -INFINITY;
#pragma unroll
      for (int i = 0; i < kKeys / 8; ++i) {
        const int j = sub + 8 * i;
        float x = 0.f;
        for (int c = 0; c < dq; ++c) x = fmaf(Q[r * ldq + c], K[j * ldq + c], x);
        s[i] = k0 + j < limit && j < nk ? x * p.scale * kLog2e : -INFINITY;
        mt = fmaxf(mt, s[i]);
      }
      for (int o = 4; o > 0; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
      const float mn = fmaxf(m, mt), ref = mn == -INFINITY ? 0.f : mn;
      const float alpha = exp2f(m - ref);
      float ls = 0.f;
#pragma unroll
      for (int i = 0; i < kKeys / 8; ++i) {
        const float e = exp2f(s[i] - ref);
        S[r * 33 + sub + 8 * i] = e;
        ls += e;
      }
      for (int o = 4; o > 0; o >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
      l = fmaf(l, alpha, ls);
      m = mn;
      __syncwarp();
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        if (sub + 8 * c < dv) {
          float x = acc[c] * alpha;
          for (int j = 0; j < nk; ++j) {
            // a value behind the row's mask counts for nothing, whatever it is
            const float e = S[r * 33 + j];
            if (e > 0.f) x = fmaf(e, V[j * ldv + sub + 8 * c], x);
          }
          acc[c] = x;
        }
      }
    }
    __syncthreads();
    if (g.slot >= 0) {
      if (r < t.rows) {
        const int64_t pr = ((int64_t)blockIdx.x * 2 + g.slot) * t.rows + r;
        if (sub == 0) {
          w.part_ml[2 * pr] = m;
          w.part_ml[2 * pr + 1] = l;
        }
#pragma unroll
        for (int c = 0; c < 16; ++c)
          if (sub + 8 * c < dv) w.part_o[pr * dv + sub + 8 * c] = acc[c];
      }
    } else if (row_ok) {
      const int64_t orow = (int64_t)(g.seq.q0 + tok) * p.heads_q + head;
      const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // no key: 0; NaN stays NaN
#pragma unroll
      for (int c = 0; c < 16; ++c)
        if (sub + 8 * c < dv) ((T*)p.o)[orow * dv + sub + 8 * c] = result<T>(acc[c] * inv);
      if (sub == 0) p.lse[orow] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    }
  }
}

// --------------------------------------------------------------------------- the join
// A warp a row: the parts of a split tile, rescaled to their common maximum and added in CTA
// order.  CTA x of the grid serves the tile whose parts begin with CTA x's last one.
constexpr int kJoinWarps = 4;

template <typename T>
__global__ void __launch_bounds__(kJoinWarps * 32)
paged_join_kernel(const __grid_constant__ Paged p, const TileShape t, int ctas, const PagedWs w) {
  const int c = blockIdx.x, lane = threadIdx.x & 31;
  if (w.ctas > 0 && c == 0 && blockIdx.y == 0 && threadIdx.x < 32) {
    // the call's error: a timeout of any CTA, else an invalid batch, else a bad page
    static_assert(JFA_OK < 1 && 1 < JFA_ERR_BAD_OFFSETS && JFA_ERR_BAD_OFFSETS < JFA_ERR_TIMEOUT, "ranks");
    int st = 0;
    for (int i = lane; i < w.ctas; i += 32) st = max(st, w.cta_status[i] == JFA_ERR_BAD_PAGES ? 1 : w.cta_status[i]);
    st = __reduce_max_sync(0xffffffffu, st);
    if (lane == 0) w.hdr->status = st == 1 ? (int)JFA_ERR_BAD_PAGES : st;
  }
  // the CTAs that hold the tile's parts: c (slot 1), then c + 1 .. last (slot 0)
  PagedCutTile cut;
  if (!cut.find(p, t, w, ctas, c)) return;
  const PagedSeq& seq = cut.seq;
  const int last = cut.last;
  for (int r = blockIdx.y * kJoinWarps + (threadIdx.x >> 5); r < t.rows; r += gridDim.y * kJoinWarps) {
    int tok, head;
    if (!cut.row(p, t, r, tok, head)) continue;
    auto slot_row = [&](int i) { return ((int64_t)i * 2 + (i == c ? 1 : 0)) * t.rows + r; };
    auto empty = [&](int i) {  // a CTA without work inside the tile
      const PagedPos a = paged_pos(p, t, w, i), e = paged_pos(p, t, w, i + 1);
      return i != c && cut.same(e) && a.blk >= e.blk;
    };
    float m = -INFINITY;
    for (int i = c + lane; i <= last; i += 32)
      if (!empty(i)) m = fmaxf(m, w.part_ml[2 * slot_row(i)]);
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float ref = m == -INFINITY ? 0.f : m;
    float l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};  // columns lane + 32 i
    for (int i = c; i <= last; ++i) {
      if (empty(i)) continue;
      const int64_t pr = slot_row(i);
      const float f = exp2f(w.part_ml[2 * pr] - ref);
      l = fmaf(w.part_ml[2 * pr + 1], f, l);
      if (w.part_ml[2 * pr] == -INFINITY) continue;  // no keys: the part has no output
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (lane + 32 * k < p.dim_v) acc[k] = fmaf(w.part_o[pr * p.dim_v + lane + 32 * k], f, acc[k]);
    }
    const int64_t orow = (int64_t)(seq.q0 + tok) * p.heads_q + head;
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (lane + 32 * k < p.dim_v) ((T*)p.o)[orow * p.dim_v + lane + 32 * k] = result<T>(acc[k] * inv);
    if (lane == 0) p.lse[orow] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
  }
}

template <typename T, int KIND>
cudaError_t simt_t(const Paged& p, const TileShape& t, int ctas, const PagedWs& w, cudaStream_t s) {
  auto kern = paged_simt_kernel<T, KIND>;
  size_t smem = sizeof(float) * ((kRows + kKeys) * (p.dim_qk + 1) + kKeys * (p.dim_v + 1) + kRows * 33);
  if (smem < kPlanScratch) smem = kPlanScratch;
  constexpr size_t most = sizeof(float) * ((kRows + kKeys) * 129 + kKeys * 129 + kRows * 33);
  cudaError_t e = kernel_setup((const void*)kern, kSimtThreads, most);
  if (e != cudaSuccess) return e;
  kern<<<ctas, kSimtThreads, smem, s>>>(p, t, w);
  return cudaGetLastError();
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

// The tensor-core kernels take bf16 queries at dims 64 and 128 whose cache rows a 32-bit index
// reaches (TMA coordinates); everything else runs on CUDA cores.
int paged_kernel(const Paged& p, int dtype) {
  const bool dims = (p.dim_qk == 64 || p.dim_qk == 128) && (p.dim_v == 64 || p.dim_v == 128);
  const int64_t rows = (p.pages * p.heads_k) << p.page_shift;
  if (dtype != JFA_BF16 || !dims || p.pages == 0 || p.total_q == 0 || rows >= INT32_MAX) return kPagedSimt;
  // Rows that share a key head, a sequence on average: few go to mma.sync tiles of at most 16, more
  // to tcgen05's 128-row tiles (groups larger than one would split them).  Measured, 64 users of
  // 2048 keys, 8 key heads of 128, us, few-row kernel against tcgen05: bf16 pages 16 rows 115 to
  // 121, 24 rows 195 to 121; MXFP8, where tcgen05 waits for the tiles in bf16, 16 rows 84 to 156,
  // 32 rows 141 to 162, 48 rows 191 to 164.
  const int64_t rows_per_seq = p.total_q * p.group / p.batch;
  return rows_per_seq <= (p.kind == kCacheMx ? 32 : 16) || p.group > 128 ? kPagedRows16 : kPagedTc;
}

TileShape paged_shape(const Paged& p, int kernel) {
  TileShape t;
  if (kernel == kPagedTc) {
    t.gsub = p.group;
    t.nsub = 1;
    t.tokens = 2 * (128 / p.group);  // two MMA tiles
    t.rows = t.tokens * t.gsub;
    t.keys = 128;
    t.overhead = 192;
    t.share = 512;
    return t;
  }
  // the few-row kernel's tiles of 8 rows where a sequence's rows of a key head fit them (the users
  // above, 8 rows: bf16 109 us to 115 in tiles of 16, MXFP8 72 to 82)
  const int most = kernel == kPagedRows16 && p.group <= 8 && p.total_q * p.group <= 8 * p.batch ? 8 : kRows;
  t.gsub = p.group < most ? p.group : most;
  t.nsub = (p.group + t.gsub - 1) / t.gsub;
  t.tokens = most / t.gsub;
  t.rows = t.tokens * t.gsub;
  t.keys = kernel == kPagedRows16 ? paged_rows16_keys(p.dim_qk, p.dim_v, p.kind) : kKeys;
  t.overhead = kernel == kPagedRows16 ? 64 : kKeys;
  t.share = kernel == kPagedRows16 ? 192 : kKeys;
  return t;
}

int paged_ctas(const Paged& p, int kernel) {
  if (kernel == kPagedTc) return num_sms() < kMaxTcCtas ? num_sms() : kMaxTcCtas;
  const int n = num_sms() * (kernel == kPagedRows16 && paged_shape(p, kernel).rows > 8 ? 2 : 3);
  return n < kMaxPagedCtas ? n : kMaxPagedCtas;
}

// Large enough for every kernel that may serve the request.
size_t paged_layout(const Paged& p, void* base, PagedWs* out) {
  char* b = (char*)base;
  size_t off = 0;
  PagedWs w{};
  w.hdr = (PagedHeader*)b;
  off = 256;
  w.pos = (PagedPos*)(b + off);
  off = up256(off + sizeof(PagedPos) * (kMaxPagedCtas + 2));
  w.cum = (int64_t*)(b + off);
  off = up256(off + sizeof(int64_t) * (size_t)(p.batch + 1));
  w.cta_status = (int*)(b + off);
  off = up256(off + sizeof(int) * kMaxPagedCtas);
  constexpr size_t rows = 2 * (kMaxPagedCtas * 16 > kMaxTcCtas * 256 ? kMaxPagedCtas * 16 : kMaxTcCtas * 256);
  w.part_ml = (float*)(b + off);
  off = up256(off + sizeof(float) * 2 * rows);
  w.part_o = (float*)(b + off);
  off = up256(off + sizeof(float) * rows * (size_t)p.dim_v);
  if (out) *out = w;
  return off;
}

cudaError_t launch_paged_plan(const Paged& p, const TileShape& t, int ctas, const PagedWs& w, cudaStream_t s) {
  const size_t smem = p.batch <= kPlanSmemSeqs ? sizeof(int64_t) * (size_t)(p.batch + 1) : 0;
  paged_plan_kernel<<<1, kPlanThreads, smem, s>>>(p, t, ctas, w);
  return cudaGetLastError();
}

cudaError_t launch_paged_simt(const Paged& p, const TileShape& t, int ctas, int dtype, const PagedWs& w,
                              cudaStream_t s) {
  if (dtype == JFA_BF16)
    return p.kind == kCacheMx ? simt_t<__nv_bfloat16, kCacheMx>(p, t, ctas, w, s)
                              : simt_t<__nv_bfloat16, kCacheBf16>(p, t, ctas, w, s);
  return p.kind == kCacheMx ? simt_t<float, kCacheMx>(p, t, ctas, w, s) : simt_t<float, kCacheF32>(p, t, ctas, w, s);
}

cudaError_t launch_paged_combine(const Paged& p, const TileShape& t, int ctas, int dtype, const PagedWs& w,
                                 cudaStream_t s) {
  int gy = (t.rows + kJoinWarps - 1) / kJoinWarps;
  if (gy > 8) gy = 8;
  if (dtype == JFA_BF16)
    paged_join_kernel<__nv_bfloat16><<<dim3(ctas, gy), kJoinWarps * 32, 0, s>>>(p, t, ctas, w);
  else
    paged_join_kernel<float><<<dim3(ctas, gy), kJoinWarps * 32, 0, s>>>(p, t, ctas, w);
  return cudaGetLastError();
}

}  // namespace jfa
