/*
 * jfa.h -- C ABI of libjfa, Jagged Flash Attention for one NVIDIA GB300 (sm_103a).
 *
 * Source of the method.  Meta GEM MFU co-design write-up
 * (piletech.kr/articles/112134), "상세 정리" (details) section:
 *   - jagged-input bullet: per-request sequences have different lengths, and
 *     padding them wastes up to half of the attention compute; the attention
 *     patterns are self, cross, pooled multi-head and asymmetric QKV;
 *   - Jagged Flash Attention bullet: attention that works directly on the
 *     variable-length tensors, masks by subtraction instead of -inf fill, and
 *     parallelises the backward pass without atomic operations;
 *   - Generalized Dot-Product Attention bullet: the same pipeline for
 *     non-softmax activations, with software tile scheduling over jagged
 *     tensors.
 * The pages give no formulas; the ones below are the plain definitions.
 *
 * Jagged tensors.  B sequences are concatenated without padding.  Sequence b
 * owns query rows offs_q[b] .. offs_q[b+1]-1 and key/value rows
 * offs_k[b] .. offs_k[b+1]-1.  Offsets are int64 [B+1] in DEVICE memory,
 * offs[0] == 0, non-decreasing, offs[B] == total rows.
 *
 * Layouts (row-major, contiguous, every pointer 16-byte aligned):
 *   Q  [T_q, H, Dqk]   K [T_k, H, Dqk]   V [T_k, H, Dv]
 *   O  [T_q, H, Dv]    dO [T_q, H, Dv]   lse [T_q, H] fp32 (natural log)
 *   dQ/dK/dV have the shapes of Q/K/V.  Values are fp32 or bf16 (params.dtype),
 *   lse is always fp32.
 *
 * Math, per sequence b and head h (i < Lq_b query rows, j < Lk_b key rows):
 *   s_ij = scale * <q_i, k_j>; valid pairs: j < Lk_b, and j <= i when causal.
 *   softmax:  P_ij = exp(s_ij - lse_i) over the valid j, o_i = sum_j P_ij v_j,
 *             lse_i = log sum_{valid j} exp(s_ij).  A row with no valid key
 *             (cross-attention with Lk_b == 0) gets o_i = 0, lse_i = -inf.
 *   SiLU/L:   P_ij = SiLU(s_ij) / Lq_b over the valid j, o_i = sum_j P_ij v_j.
 *   Backward: the analytic gradients of a loss whose gradient w.r.t. O is dO.
 *
 * Ownership and threading.  The caller owns every buffer.  The library never
 * allocates device memory on these paths and keeps no per-call state; its
 * only scratch is the caller's workspace (size from jfa_workspace_size).
 * One workspace must not be used by two calls that may run concurrently.
 * The one exception is jfa_fwd_noalloc below, whose scratch is a fixed array
 * inside the library shared by all of its calls.
 *
 * Asynchrony and errors.  Every compute call only enqueues work on `stream`
 * (NULL = the legacy default stream) and returns.  Argument errors are
 * detected on the host before anything is launched, and returned.  Errors
 * found on the device are written to a status word inside the workspace:
 * offsets that are not a valid jagged layout (the call then computes nothing
 * and leaves its outputs untouched), or a bounded wait inside a kernel that
 * gave up (the outputs are then incomplete).  jfa_status_check()
 * synchronises the stream and returns that word.  The library never aborts,
 * traps or prints.
 */
#ifndef JFA_H_
#define JFA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same object as cudaStream_t; declared here so this header needs no CUDA headers. */
typedef struct CUstream_st* jfa_stream_t;

typedef enum {
  JFA_OK = 0,
  JFA_ERR_INVALID_ARG = 1, /* null pointer, bad size, misaligned pointer */
  JFA_ERR_UNSUPPORTED = 2, /* valid request the library does not implement */
  JFA_ERR_WORKSPACE = 3,   /* workspace missing, misaligned or too small */
  JFA_ERR_BAD_OFFSETS = 4, /* (device) offsets are not a jagged layout of the given totals */
  JFA_ERR_TIMEOUT = 5,     /* (device) a bounded wait inside a kernel gave up */
  JFA_ERR_CUDA = 6,        /* a CUDA runtime or driver call failed */
  JFA_ERR_BAD_PAGES = 7    /* (device) a page table names a page outside the cache */
} jfa_status;

typedef enum {
  JFA_F32 = 0,
  JFA_BF16 = 1,
  JFA_MXFP8 = 2 /* caches only: e4m3 codes, one power-of-two scale per 32 columns */
} jfa_dtype;

typedef struct {
  int64_t batch;   /* B >= 0 */
  int64_t total_q; /* T_q = offs_q[B] <= 2^31 - 1 */
  int64_t total_k; /* T_k = offs_k[B] <= 2^31 - 1; equal to total_q for self-attention */
  int32_t heads;   /* H >= 1; H * (max(T_q, T_k) / 32 + B + 1) <= 2^31 - 1 (work-list
                      items), else JFA_ERR_UNSUPPORTED */
  int32_t dim_qk;  /* Dqk: bf16 supports 64 and 128; fp32 supports 1..128 */
  int32_t dim_v;   /* Dv:  bf16 supports 64 and 128; fp32 supports 1..128 */
  float scale;     /* score scale > 0, normally 1/sqrt(Dqk) */
  int32_t causal;  /* 1: key j visible to query i only if j <= i (self-attention only) */
  int32_t dtype;   /* jfa_dtype of Q, K, V, O, dO, dQ, dK, dV */
  int32_t flags;   /* 0, or JFA_PLANNED (see jfa_plan); other bits: JFA_ERR_INVALID_ARG */
} jfa_params;

#define JFA_PLANNED 1

/*
 * Bytes of device workspace the calls below need for these params (work lists
 * of the jagged tile scheduler, the backward row term D, the status word).
 * Any call may be given a larger workspace.  Depends on batch, total_q,
 * total_k and heads only.  Returns 0 for a null pointer.
 */
size_t jfa_workspace_size(const jfa_params* p);

/*
 * Work lists built once for several calls (the jagged tile scheduler of the
 * Generalized Dot-Product Attention bullet, run once per batch instead of once
 * per call).  Every compute call starts by validating its offsets and building
 * its heavy-first work lists in the workspace.  jfa_plan does that once, for
 * the forward and the backward calls of these params: the same offsets serve
 * every call of a training step, and the plan serves every layer whose params
 * differ from the plan's only in scale, dim_qk, dim_v or dtype, as long as
 * jfa_path_for gives the same kernel family (and, for jfa_block_rope_*, dim_qk
 * is the plan's: the rotary table depends on it).
 *
 * A later call then passes params with flags = JFA_PLANNED, the same offsets
 * (the same pointers, their contents unchanged) and the same workspace; it
 * launches no scheduler and reads the planned lists.  Calls ordered after the
 * plan on the GPU (the same stream, or an event) may use it any number of
 * times, one at a time; it stays valid until the workspace is used by a call
 * without JFA_PLANNED or by another plan.  A planned call does not reset the
 * status word: it keeps the plan's status (JFA_ERR_BAD_OFFSETS makes every
 * planned call compute nothing), and after JFA_ERR_TIMEOUT the lists must be
 * planned again.  Nothing checks that a planned call's offsets are the plan's:
 * other offsets with the same totals produce wrong results, within the
 * buffers' bounds.
 *
 * jfa_plan serves jfa_fwd, jfa_bwd, jfa_cross_fwd, jfa_cross_bwd, jfa_gdpa_fwd
 * and jfa_gdpa_bwd (pass offs_q == offs_k for self-attention; causal needs
 * Lq_b == Lk_b, checked on the device); jfa_block_plan serves the four
 * BlockAttention calls (it also writes their block offsets and, where
 * jfa_block_rope_* is supported, the rotary table).  The pooled calls and
 * jfa_fwd_noalloc return JFA_ERR_UNSUPPORTED for JFA_PLANNED.  Argument errors
 * are those of the calls served; p->flags may be 0 or JFA_PLANNED and does not
 * change what is built.
 */
jfa_status jfa_plan(const jfa_params* p, const int64_t* offs_q, const int64_t* offs_k, void* ws,
                    size_t ws_bytes, jfa_stream_t stream);
jfa_status jfa_block_plan(const jfa_params* p, const int64_t* offs, void* ws, size_t ws_bytes,
                          jfa_stream_t stream);

/*
 * Softmax self-attention forward (Jagged Flash Attention bullet).  One offsets
 * array serves queries and keys (total_k must equal total_q).  Writes O and lse.
 * Causal masking is allowed.
 */
jfa_status jfa_fwd(const jfa_params* p, const void* q, const void* k, const void* v,
                   const int64_t* offs, void* o, float* lse, void* ws, size_t ws_bytes,
                   jfa_stream_t stream);

/*
 * Softmax self-attention backward, without atomics (Jagged Flash Attention
 * bullet): a key-tile-major pass writes dK and dV, a query-tile-major pass
 * writes dQ, each output element is written exactly once.  o and lse are the
 * outputs of jfa_fwd on the same inputs; dout is dL/dO.
 */
jfa_status jfa_bwd(const jfa_params* p, const void* q, const void* k, const void* v,
                   const void* o, const float* lse, const void* dout, const int64_t* offs,
                   void* dq, void* dk, void* dv, void* ws, size_t ws_bytes,
                   jfa_stream_t stream);

/*
 * Softmax cross-attention forward with independent query and key offsets and
 * possibly Dv != Dqk (jagged-input bullet: cross and asymmetric-QKV patterns).
 * Causal must be 0.  A sequence with Lk_b == 0 yields o = 0 and lse = -inf.
 */
jfa_status jfa_cross_fwd(const jfa_params* p, const void* q, const void* k, const void* v,
                         const int64_t* offs_q, const int64_t* offs_k, void* o, float* lse,
                         void* ws, size_t ws_bytes, jfa_stream_t stream);

/* Backward of jfa_cross_fwd; same passes as jfa_bwd. */
jfa_status jfa_cross_bwd(const jfa_params* p, const void* q, const void* k, const void* v,
                         const void* o, const float* lse, const void* dout,
                         const int64_t* offs_q, const int64_t* offs_k, void* dq, void* dk,
                         void* dv, void* ws, size_t ws_bytes, jfa_stream_t stream);

/*
 * Non-softmax (Generalized Dot-Product Attention bullet) forward:
 * P_ij = SiLU(s_ij) / Lq_b on the valid pairs, O = P V.  No lse is produced.
 * Pass the same pointer as offs_q and offs_k for self-attention; causal is
 * allowed only then (Lq_b == Lk_b is checked on the device).
 */
jfa_status jfa_gdpa_fwd(const jfa_params* p, const void* q, const void* k, const void* v,
                        const int64_t* offs_q, const int64_t* offs_k, void* o, void* ws,
                        size_t ws_bytes, jfa_stream_t stream);

/* Backward of jfa_gdpa_fwd (no D term, no lse); same two atomic-free passes. */
jfa_status jfa_gdpa_bwd(const jfa_params* p, const void* q, const void* k, const void* v,
                        const void* dout, const int64_t* offs_q, const int64_t* offs_k,
                        void* dq, void* dk, void* dv, void* ws, size_t ws_bytes,
                        jfa_stream_t stream);

/*
 * Allocation-free variant of jfa_fwd.  The pages describe no such call; it
 * exists for callers that cannot allocate device memory at all -- for example
 * a plugin running inside a host application that owns the device allocator
 * and forbids other allocations, or a serving process that must not allocate
 * once it has started -- and so cannot provide the workspace jfa_fwd needs.
 *
 * Same arguments, layouts and results as jfa_fwd, minus the workspace: the
 * scratch (work lists and status word) lives in one 64 MiB array compiled
 * into the library, which every GPU that loads the library holds until the
 * process exits.  Requests whose workspace (jfa_workspace_size) would exceed
 * 64 MiB are rejected with JFA_ERR_WORKSPACE before anything is launched.
 * The call itself never allocates: no cudaMalloc, no cudaFree, no allocating
 * library routine.  The first call on a device looks up the array's device
 * address (cudaGetSymbolAddress, with that device current) and caches it;
 * make that first call before any stream capture.  The cache is keyed on the
 * CUDA context, not the device number: after cudaDeviceReset, or under another
 * context on the same device, the first call looks the address up again (and
 * that call, too, should come before any capture).  All calls share the one
 * array, which keeps the last call's contents, so calls that may overlap on
 * the GPU (different streams, or different host threads) race and must be
 * serialised by the caller.  Errors found on the device are silent here:
 * offsets that are not a valid jagged layout make the call compute nothing,
 * as in jfa_fwd, and a bounded wait inside a kernel that gives up leaves the
 * outputs incomplete; the status word that jfa_fwd's caller reads with
 * jfa_status_check lives in the shared array, which this variant's caller
 * cannot name.
 */
jfa_status jfa_fwd_noalloc(const jfa_params* p, const void* q, const void* k, const void* v,
                           const int64_t* offs, void* o, float* lse, jfa_stream_t stream);

/*
 * Pooled multi-head attention (Meta GEM MFU write-up,
 * piletech.kr/articles/112134, details section, jagged-input bullet: pooled
 * multi-head attention is one of the attention patterns over jagged
 * sequences).  m learned query rows per head, q [m, H, Dqk], are shared by
 * every sequence: sequence b's m outputs are the softmax attention of those
 * rows over its own keys and values, k/v rows offs_k[b] .. offs_k[b+1]-1
 * (non-causal, scale = p->scale).
 *   o   [B*m, H, Dv], lse [B*m, H]: sequence b's rows are b*m .. b*m+m-1;
 *       a sequence without keys gets o = 0, lse = -inf.
 *   dq  [m, H, Dqk]: the sum over sequences of each sequence's gradient of the
 *       shared rows (fixed order, bitwise reproducible); dk, dv as in
 *       jfa_cross_bwd.
 * p->batch = B, p->total_q = B*m (the rows of o), p->total_k = offs_k[B],
 * p->causal = 0.  The workspace (size from jfa_pooled_workspace_size, 256-byte
 * aligned) also holds the query rows broadcast to every sequence and their
 * per-sequence gradients, kept in fp32 until they are summed; it is used as by
 * jfa_cross_fwd / jfa_cross_bwd otherwise, and errors are reported the same
 * way.  Runs on the cross-attention kernels.
 */
size_t jfa_pooled_workspace_size(const jfa_params* p, int32_t m);
jfa_status jfa_pooled_fwd(const jfa_params* p, int32_t m, const void* q, const void* k,
                          const void* v, const int64_t* offs_k, void* o, float* lse, void* ws,
                          size_t ws_bytes, jfa_stream_t stream);
jfa_status jfa_pooled_bwd(const jfa_params* p, int32_t m, const void* q, const void* k,
                          const void* v, const void* o, const float* lse, const void* dout,
                          const int64_t* offs_k, void* dq, void* dk, void* dv, void* ws,
                          size_t ws_bytes, jfa_stream_t stream);

/*
 * BlockAttention (Meta GEM MFU write-up, piletech.kr/articles/112134, details
 * section, BlockAttention bullet: fixed 64-token blocks make attention linear
 * in the sequence length).  Softmax self-attention in which row i of a
 * sequence sees only the keys of its own block, rows 64*floor(i/64) ..
 * 64*floor(i/64)+63 of the same sequence (the last block may be shorter), and
 * with p->causal = 1 only those not after it.  Arguments and outputs as for
 * jfa_fwd / jfa_bwd.  The offsets are cut into blocks on the device and the
 * self-attention kernels run on the blocks as sequences of their own; the
 * workspace (jfa_block_workspace_size) holds the block offsets and room for up
 * to B + ceil(T/64) block sequences.  The pages combine the blocks with a fused
 * rotary position embedding: see jfa_block_rope_fwd / jfa_block_rope_bwd below.
 */
size_t jfa_block_workspace_size(const jfa_params* p);
jfa_status jfa_block_fwd(const jfa_params* p, const void* q, const void* k, const void* v,
                         const int64_t* offs, void* o, float* lse, void* ws, size_t ws_bytes,
                         jfa_stream_t stream);
jfa_status jfa_block_bwd(const jfa_params* p, const void* q, const void* k, const void* v,
                         const void* o, const float* lse, const void* dout, const int64_t* offs,
                         void* dq, void* dk, void* dv, void* ws, size_t ws_bytes,
                         jfa_stream_t stream);

/*
 * BlockAttention with the fused rotary position embedding (same bullet: the 64-token
 * blocks are combined with a fused rotary position embedding).  The page gives none of
 * the embedding's parameters; this library follows RoFormer's definition: columns
 * (2i, 2i+1) of every q and k row, at position p, turn by the angle p * 10000^(-2i/D)
 * (D = dim_qk), with p the row's index inside its sequence.  Inside one block the scores
 * depend only on the difference of positions, so this equals counting positions from
 * each block's first row, which is how the kernels do it.  q and k are the unrotated
 * inputs; dq and dk are the gradients with respect to them.  The rotation is applied to
 * the Q and K tiles in shared memory between their load and the MMAs (no extra pass over
 * HBM), and its transpose to dQ and dK before they are stored.  Arguments, outputs,
 * workspace (jfa_block_workspace_size) and errors as for jfa_block_fwd / jfa_block_bwd;
 * bf16 with dim_qk == dim_v (64 or 128) only, else JFA_ERR_UNSUPPORTED.
 */
jfa_status jfa_block_rope_fwd(const jfa_params* p, const void* q, const void* k, const void* v,
                              const int64_t* offs, void* o, float* lse, void* ws, size_t ws_bytes,
                              jfa_stream_t stream);
jfa_status jfa_block_rope_bwd(const jfa_params* p, const void* q, const void* k, const void* v,
                              const void* o, const float* lse, const void* dout, const int64_t* offs,
                              void* dq, void* dk, void* dv, void* ws, size_t ws_bytes,
                              jfa_stream_t stream);

/*
 * RMS norm of every query and key head with the rotary position embedding, in one
 * pass over the values (training and serving; q and k may be slices of one
 * projection's output).  Per row x of D = dim values (one token, one head), with
 * r = 1 / sqrt(mean(x^2) + eps) and weight w (wq or wk, fp32 [D]; NULL: ones):
 *   n = x r w (norm = 1) or n = x (norm = 0; the weights and their gradients are
 *   then NULL);
 *   pair i < rope.dim / 2 of columns (a, b) = (i, i + rope.dim/2) (JFA_ROPE_HALVES) or
 *   (2i, 2i + 1) (JFA_ROPE_PAIRS) turns by the angle pos[t] theta_i:
 *     y_a = amp (n_a cos - n_b sin), y_b = amp (n_a sin + n_b cos);
 *   the columns from rope.dim on are y = n.  rope.dim = 0: no rotation, pos may be NULL.
 * Frequencies: theta_i = base^(-2i / rope.dim), for contexts `factor` times longer than
 * the model was trained on changed by `scaling`:
 *   JFA_ROPE_LINEAR  theta_i / factor (positions squeezed);
 *   JFA_ROPE_NTK     base * factor^(rope.dim / (rope.dim - 2)) in place of base;
 *   JFA_ROPE_YARN    theta_i (g + (1 - g) / factor), g = clamp((n_i - turns_slow) /
 *                    (turns_fast - turns_slow), 0, 1), n_i = orig_len theta_i / 2 pi the
 *                    turns pair i makes over the trained context; the method's
 *                    temperature is the caller's choice of amp.  (The ramp is over turns;
 *                    a ramp over the pair's index between rounded bounds, which some models
 *                    were trained with, cannot be expressed, nor a table of frequencies.)
 * pos is int64 [T] on the device, any values (negative too).  Frequencies are worked out in
 * 64-bit floating point, so an angle is within |pos| 2^-53 turns (7e-10 rad at position 10^6,
 * 7e-7 at 10^9) besides fp32 rounding.
 *
 * Strides are in elements between tokens; a token's heads are contiguous, [heads, dim].
 * heads_q or heads_k may be 0 (that tensor is then absent).  yq may be q (and yk be k)
 * with the same stride; outputs overlap inputs in no other way.
 *
 * Backward: dyq, dyk are the gradients of yq, yk (strides stride_yq, stride_yk); dq, dk
 * (strides stride_dq, stride_dk) those of q, k; dwq, dwk (fp32 [D], or NULL: not wanted)
 * the weights', summed over tokens and heads in a fixed order without atomics (bitwise
 * reproducible on one GPU).  The row's r is recomputed from q, k.  dq may be dyq or q
 * with the same stride.  q, k may be NULL when norm = 0.  Without tokens, or heads of its
 * tensor, dwq or dwk is zeroed.
 *
 * Values are fp32 or bf16 (dtype), pointers aligned to a value; pointers and strides of
 * whole 16 bytes (fp32: 32) with dim and rope.dim multiples of 16 take the fast kernels.
 * Sums are fp32: a row's sum of squares has to stay in its range (with larger values y is 0,
 * and with eps = 0 rows of values under 2^-63 lose precision).
 * dim <= 256 and tokens <= 2^31 - 1, else JFA_ERR_UNSUPPORTED.  The forward needs no
 * workspace; the backward's (256-byte aligned, jfa_norm_rope_workspace_size; 0 for bad params) is scratch
 * without a status word.  The library finds no errors on the device here.
 */
enum { JFA_ROPE_HALVES = 0, JFA_ROPE_PAIRS = 1 };
enum { JFA_ROPE_PLAIN = 0, JFA_ROPE_LINEAR = 1, JFA_ROPE_NTK = 2, JFA_ROPE_YARN = 3 };
typedef struct {
  int32_t dim;     /* rotated columns of a head: even, 0 .. head dim */
  int32_t layout;  /* JFA_ROPE_HALVES or JFA_ROPE_PAIRS */
  int32_t scaling; /* JFA_ROPE_PLAIN, _LINEAR, _NTK (dim >= 4) or _YARN */
  float amp;       /* factor of the rotated columns, normally 1 */
  double base;     /* >= 1, normally 10000 */
  double factor;   /* >= 1 (LINEAR, NTK, YARN) */
  double orig_len, turns_fast, turns_slow; /* YARN: > 0, > turns_slow, >= 0 */
} jfa_rope;
typedef struct {
  int64_t tokens;
  int64_t stride_q, stride_k;   /* q, k */
  int64_t stride_yq, stride_yk; /* yq, yk; backward: dyq, dyk */
  int64_t stride_dq, stride_dk; /* backward: dq, dk */
  int32_t heads_q, heads_k, dim;
  int32_t dtype; /* JFA_F32 or JFA_BF16 */
  int32_t norm;  /* 1: RMS norm, 0: rotation only */
  float eps;     /* >= 0 */
  jfa_rope rope;
} jfa_norm_rope_params;

size_t jfa_norm_rope_workspace_size(const jfa_norm_rope_params* p);
jfa_status jfa_norm_rope_fwd(const jfa_norm_rope_params* p, const void* q, const void* k,
                             const int64_t* pos, const float* wq, const float* wk, void* yq,
                             void* yk, jfa_stream_t stream);
jfa_status jfa_norm_rope_bwd(const jfa_norm_rope_params* p, const void* q, const void* k,
                             const int64_t* pos, const float* wq, const float* wk,
                             const void* dyq, const void* dyk, void* dq, void* dk, float* dwq,
                             float* dwk, void* ws, size_t ws_bytes, jfa_stream_t stream);

/*
 * Paged cache.  Keys and values of sequences that grow are kept in pages of page_size
 * positions (16, 32, 64, 128 or 256):
 *   k_cache [pages, Hk, page_size, Dqk], v_cache [pages, Hk, page_size, Dv], contiguous.
 * Position x of sequence b is row x % page_size of page table[b, x / page_size] (int32
 * [B, max_pages]; sequences may share pages).  lens [B] (int64) holds the sequences'
 * cached lengths, the new tokens of the call among them: a call's T = offs[B] new tokens
 * (offs int64 [B+1], a jagged layout as elsewhere) are the last ones of their sequences,
 * token i of sequence b at position lens[b] - L_b + i, L_b = offs[b+1] - offs[b].
 * Where L_b > lens[b] the first tokens come before the cache's start: they are not
 * written, read back as zeros, and see no keys under the causal mask.
 *
 * The cache holds the values' own type, or MXFP8 (cache_dtype JFA_MXFP8): e4m3 codes,
 * one byte a value, with k_scale [pages, Hk, page_size, Dqk / 32] and v_scale likewise,
 * biased E8M0 exponents (2^(s - 127)) per 32 columns.  Writing takes the smallest power
 * of two with max|x| <= 448 * scale, exponent kept in [-100, 119], and rounds x / scale
 * to the nearest code, ties to even, saturating (NaN stays NaN).  Scales read may be any
 * in [1, 254]; 0 reads as zeros.
 *
 * Index arrays live on the device.  jfa_paged_plan and every call without JFA_PLANNED
 * reset the workspace's status word; invalid offs or lens outside [0, max_pages *
 * page_size] give JFA_ERR_BAD_OFFSETS, and a page index outside [0, pages) that a call
 * meets JFA_ERR_BAD_PAGES, unless it has the former or JFA_ERR_TIMEOUT to report.  jfa_paged_fwd
 * computes nothing on the former.  Rows behind a
 * bad page are not written, are read as zeros, and count as zero keys and values.  Nothing
 * outside the buffers is touched.  Pages' rows behind a sequence's length are never
 * read as values (they may hold anything).
 *
 * jfa_cache_write puts the new keys and values k [T, Hk, Dqk], v [T, Hk, Dv] (token
 * strides stride_k, stride_v; any slice of a projection's output) into their pages.  Two
 * tokens of a call that share a slot leave either's row, in parts.  jfa_cache_read
 * gathers the same tokens' rows back into contiguous k [T, Hk, Dqk], v [T, Hk, Dv]
 * (L_b = lens[b] reads whole sequences); MXFP8 values are exact in fp32, and
 * in bf16 with scales of at least 3; values past fp32 (scales above 246) become infinite.
 *
 * jfa_paged_fwd: softmax attention of the new tokens' queries q [T, Hq, Dqk] (token
 * stride stride_q) over their sequences' cached keys, from one token a sequence to whole
 * prompts.  Query head h reads key head h / (Hq / Hk).  With causal = 1 token i of
 * sequence b sees positions <= lens[b] - L_b + i, else all lens[b].  o [T, Hq, Dv] and
 * lse [T, Hq] as in jfa_fwd; a row that sees no key gets o = 0, lse = -inf.  Scores,
 * statistics and sums are fp32; on the tensor-core kernels (bf16, dims 64 and 128) the
 * weights are rounded to bf16 (over MXFP8 also fp16, where that is as close) for the product
 * with the values, and over MXFP8 values of a query row under 2^-31 of its largest may be off by
 * 2^-39 of that.  A score has to stay in fp32's range before and after its scale.  The
 * sums run before they are divided by the weights' sum: a row's keys times its largest |v|
 * has to stay below 2^128.  Keys and values of positions that a sequence's other queries
 * see must be finite where a row's own mask hides them.  Results repeat bit for bit on one
 * GPU.
 *
 * Every call cuts its work into equal shares on the device (jfa_paged_plan does it once for
 * several calls, which then pass flags = JFA_PLANNED, the same params but for scale and
 * strides, the same offs and lens, unchanged, and the same workspace; on another request's plan
 * a call's outputs are undefined, and nothing outside them is touched).  The plan serves
 * jfa_cache_write, jfa_cache_read and jfa_paged_fwd.  One workspace must not be used by
 * calls that may run concurrently.
 *
 * Limits (JFA_ERR_UNSUPPORTED): dims multiples of 8 (MXFP8: 32), at most 256, in
 * jfa_paged_fwd 128; cache_dtype the values' type or JFA_MXFP8; max_pages * page_size and
 * total_q at most 2^31 - 256, batch and pages 2^31 - 1.  k, v, q, o, lse and the caches are 16-byte
 * aligned, with strides of whole 16 bytes.  The tensor-core kernels serve bf16 at dims of 64 and
 * 128; fp32 and other dims take a CUDA-core kernel, some 40 times slower for single tokens and
 * 200 to 360 times for prompts.  The workspace is
 * about 22 MB for values of 64 columns and 43 MB for 128, whatever the batch.
 */
typedef struct {
  int64_t batch;   /* B >= 0 */
  int64_t total_q; /* T = offs[B] */
  int64_t pages;   /* pages of the cache */
  int64_t stride_q, stride_k, stride_v; /* elements between tokens (>= heads * dim) */
  int32_t heads_q; /* Hq, a multiple of Hk (attention) */
  int32_t heads_k; /* Hk */
  int32_t dim_qk, dim_v;
  int32_t page_size, max_pages;
  float scale;         /* score scale > 0 (attention) */
  int32_t causal;      /* 0 or 1 (attention) */
  int32_t dtype;       /* of q, k, v, o: JFA_F32 or JFA_BF16 */
  int32_t cache_dtype; /* dtype or JFA_MXFP8 */
  int32_t flags;       /* 0 or JFA_PLANNED */
} jfa_paged_params;

/* Bytes of workspace (256-byte aligned) of all four calls; 0 for bad params. */
size_t jfa_paged_workspace_size(const jfa_paged_params* p);
jfa_status jfa_cache_write(const jfa_paged_params* p, const void* k, const void* v,
                           const int64_t* offs, const int64_t* lens, const int32_t* table,
                           void* k_cache, void* v_cache, uint8_t* k_scale, uint8_t* v_scale,
                           void* ws, size_t ws_bytes, jfa_stream_t stream);
jfa_status jfa_cache_read(const jfa_paged_params* p, const void* k_cache, const void* v_cache,
                          const uint8_t* k_scale, const uint8_t* v_scale, const int64_t* offs,
                          const int64_t* lens, const int32_t* table, void* k, void* v, void* ws,
                          size_t ws_bytes, jfa_stream_t stream);
jfa_status jfa_paged_plan(const jfa_paged_params* p, const int64_t* offs, const int64_t* lens,
                          void* ws, size_t ws_bytes, jfa_stream_t stream);
jfa_status jfa_paged_fwd(const jfa_paged_params* p, const void* q, const void* k_cache,
                         const void* v_cache, const uint8_t* k_scale, const uint8_t* v_scale,
                         const int64_t* offs, const int64_t* lens, const int32_t* table, void* o,
                         float* lse, void* ws, size_t ws_bytes, jfa_stream_t stream);

/*
 * Synchronises `stream`, then returns the device status word of the last
 * call that used `ws` (JFA_OK, JFA_ERR_BAD_OFFSETS, JFA_ERR_BAD_PAGES or
 * JFA_ERR_TIMEOUT), or JFA_ERR_CUDA if the synchronisation itself failed.
 */
jfa_status jfa_status_check(const void* ws, jfa_stream_t stream);

/* Static, human-readable name of a status code. */
const char* jfa_status_string(jfa_status s);

/*
 * Kernel timing, for benchmarks.  While enabled, every kernel the library
 * launches is bracketed by CUDA events recorded on its launch stream.
 * jfa_profile_read synchronises those events and returns, for kernel kind
 * `kind` (a JFA_KERNEL_* value), the number of launches and their summed
 * device time in milliseconds since the last reset.  Not thread-safe.
 */
enum {
  JFA_KERNEL_SCHEDULE = 0, /* jagged tile scheduler: offsets -> heavy-first work lists */
  JFA_KERNEL_FWD = 1,      /* forward tile loop */
  JFA_KERNEL_BWD_D = 2,    /* backward row term D = rowsum(dO * O) */
  JFA_KERNEL_BWD_DKDV = 3, /* key-tile-major dK/dV pass */
  JFA_KERNEL_BWD_DQ = 4,   /* query-tile-major dQ pass */
  JFA_KERNEL_AUX = 5,      /* pooled query broadcast and gradient sum; block offsets */
  JFA_KERNEL_NORM_ROPE = 6, /* norms with rotary positions (backward: with its weight sums) */
  JFA_KERNEL_CACHE = 7,     /* paged cache written or read */
  JFA_KERNEL_PAGED = 8,     /* attention over a paged cache, with the join of split tiles */
  JFA_KERNEL_KINDS = 9
};
jfa_status jfa_profile_enable(int on);
jfa_status jfa_profile_reset(void);
jfa_status jfa_profile_read(int kind, int64_t* launches, double* total_ms);

/*
 * Test hook for the bounded waits inside the tensor-core kernels.  Every wait on
 * an mbarrier in those kernels gives up after about two seconds, records
 * JFA_ERR_TIMEOUT in the workspace's status word, lets the CTA's other roles
 * leave, waits for the CTA's own copies and MMAs in flight and frees its
 * tensor memory, so the context stays usable.  While `on` is nonzero, every
 * bf16 forward launch in the calling thread's current context (jfa_fwd,
 * jfa_cross_fwd, jfa_gdpa_fwd and the calls built on them) starts with its MMA
 * issuer waiting on a barrier that nothing arrives on, before any MMA is
 * issued; in the tensor-core kernels of jfa_paged_fwd one role of the first CTA
 * waits in the same way (a consumer warp of the few-row kernel, an MMA issuer of
 * the other) while its copies are in flight, in launches of the whole process.
 * The call then reports JFA_ERR_TIMEOUT through jfa_status_check and leaves its
 * outputs incomplete.  Off by default; turn it off again before
 * normal use.  Synchronises the device.
 */
jfa_status jfa_test_hold(int on);

/*
 * Which kernel family serves a request with these params: 1 = tcgen05/TMA
 * tensor-core kernels (bf16), 0 = CUDA-core fp32 kernels, -1 = unsupported.
 */
int jfa_path_for(const jfa_params* p);

/*
 * Base Batch Shuffling: a plan that spreads a global batch over `ranks`
 * data-parallel ranks with balanced attention work and no data exchanged
 * between ranks (Meta GEM MFU write-up, piletech.kr/articles/112134, details
 * section, Base Batch Shuffling bullet: sub-batches of 128 samples sorted by
 * sequence length, the heaviest merged with the lightest in turn).  Host
 * function; touches no GPU.  Every rank calls it with the same per-sample
 * costs and gets the same plan, then loads only the sub-batches assigned to
 * it.
 *
 * Plan (readings where the pages are silent):
 *   - sub-batch s holds samples s*sub .. min((s+1)*sub, n_samples)-1, and costs
 *     the sum of their `cost` (the caller's measure, e.g. useful attention
 *     FLOPs: Lq*Lk, or L(L+1)/2 when causal);
 *   - sub-batches are sorted by cost, heaviest first, ties by index;
 *   - pair i merges the i-th heaviest with the i-th lightest (the middle one of
 *     an odd count stays single);
 *   - pairs go to ranks in serpentine order 0, 1, .., R-1, R-1, .., 0, 0, ..,
 *     so ranks receive equally many pairs, within one.
 *
 * cost       host int64 [n_samples], every value >= 0
 * sub        samples per sub-batch (the pages use 128), >= 1
 * ranks      number of ranks, >= 1
 * sub_rank   host int32 [ceil(n_samples/sub)], out: rank of each sub-batch
 * sub_slot   host int32 [ceil(n_samples/sub)], out: its position in that
 *            rank's list (heavy member of a pair first)
 * rank_cost  host int64 [ranks] or NULL, out: each rank's total cost
 * Returns JFA_ERR_INVALID_ARG (and writes nothing) for n_samples < 0, sub < 1,
 * ranks < 1, a negative cost, or a NULL array with n_samples > 0.
 */
jfa_status jfa_bbs_plan(const int64_t* cost, int64_t n_samples, int32_t sub, int32_t ranks,
                        int32_t* sub_rank, int32_t* sub_slot, int64_t* rank_cost);

#ifdef __cplusplus
}
#endif

#endif /* JFA_H_ */
