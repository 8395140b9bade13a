/*
 * nvfp4moe — NVFP4 block-scaled Mixture-of-Experts layer for AMD MI355X (gfx950).
 *
 * Plain C ABI.  Every pointer argument is a DEVICE pointer unless stated
 * otherwise; sizes are host integers.  Every compute call enqueues its kernels
 * on `stream` (a hipStream_t passed as void*, NULL = the null stream), returns
 * without synchronising the host, and allocates nothing: the caller owns every
 * buffer, including workspaces.  The library keeps no pointer past the work it
 * enqueued and holds no global state, so calls on different streams may run
 * concurrently (calls that share a workspace or an output must not overlap).
 *
 * Number format (the block-scaled MMA described in "From Empirical Limits to
 * Research-Driven Optimization: The SM120 FP4 Kernel Research Campaign",
 * section "Section 1: CUTLASS Kernels - The Foundation": E2M1 operands, one
 * unsigned E4M3 block scale per 16 elements along K, FP32 accumulation), plus a
 * float32 per-tensor scale:
 *   codes   uint8 [rows, cols/2]   two E2M1 codes per byte, element 2i in the
 *                                  low nibble of byte i, row-major, blocks run
 *                                  along the last (reduction) axis
 *   scales  uint8 [rows, cols/16]  one E4M3 code per 16-element block
 *   g       float32 (device)       per-tensor scale; value = E2M1*E4M3*g
 *
 * Quantiser (a reading of the pages, which print none):
 *   g = amax/2688, block scale = E4M3_satfinite((absmax_b/6)/g) (nearest even),
 *   code = E2M1(x / (scale*g)) (nearest even, saturating at 6, sign copied from
 *   x, a zero block scale gives code 0).  All decisions in float32 with correctly
 *   rounded division, so codes are reproducible bit for bit.
 *
 * Errors: every call validates its arguments on the host BEFORE enqueuing
 * anything.  A non-OK status means nothing was enqueued, except
 * NVFP4MOE_ERR_HIP, which reports a failed kernel launch (earlier kernels of
 * the same call may have been enqueued).  nvfp4moe_last_error_detail() gives a
 * thread-local explanation of the last failure on the calling thread.  The
 * *_workspace_size() and *_packed_size() queries return 0 for arguments the
 * matching call rejects.
 */
#ifndef NVFP4MOE_H
#define NVFP4MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum nvfp4moe_status {
  NVFP4MOE_OK = 0,
  NVFP4MOE_ERR_INVALID = 1,      /* null pointer, negative/zero size, k > E, K % 32 != 0, misaligned pointer */
  NVFP4MOE_ERR_UNSUPPORTED = 2,  /* valid request outside what the compiled kernels cover (size limits) */
  NVFP4MOE_ERR_WORKSPACE = 3,    /* workspace missing or smaller than the *_workspace_size() query */
  NVFP4MOE_ERR_HIP = 4           /* the HIP runtime rejected a kernel launch */
} nvfp4moe_status;

/* Index arrays that live on the device (expert offsets, gathered rows,
 * combine rows) are not read by the host: the kernels clamp entries that
 * break the documented ranges, which then gives wrong rows but never an
 * access outside a buffer.  With the environment variable NVFP4MOE_DEBUG set
 * (to anything but "" or "0"; read at every call) the grouped GEMMs,
 * moe_expert_ffn and moe_unpermute_combine first copy those arrays to the
 * host and check them (offsets non-decreasing from 0 to at most m_total,
 * gathered rows in [0, a_rows_total), combine rows in [0, T * k) or
 * [0, out_rows)), returning NVFP4MOE_ERR_INVALID with the first bad entry in
 * nvfp4moe_last_error_detail() before any launch.  The copies synchronise
 * the stream: a debugging aid, not for use under graph capture. */

typedef enum nvfp4moe_dtype {
  NVFP4MOE_F32 = 0,
  NVFP4MOE_BF16 = 1,
  NVFP4MOE_F16 = 2               /* the 16-bit expert FFN, the router with scores and INT4 only */
} nvfp4moe_dtype;

/* activation of the gated feed-forward block */
typedef enum nvfp4moe_activation {
  NVFP4MOE_ACT_SILU = 0,         /* g / (1 + exp(-g)) */
  NVFP4MOE_ACT_GELU = 1          /* g/2 (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))) */
} nvfp4moe_activation;

/* scores of moe_route_scored */
typedef enum nvfp4moe_score {
  NVFP4MOE_SCORE_SOFTMAX = 0,    /* softmax over the token's logits (-inf and NaN left out) */
  NVFP4MOE_SCORE_SIGMOID = 1     /* 1 / (1 + exp(-l)) */
} nvfp4moe_score;

typedef enum nvfp4moe_epilogue {
  /* y[p, n] = acc * (g_a * g_b[e]) written as float32 to out[p*N + n], p < m_total */
  NVFP4MOE_EPI_F32 = 0,
  /* same, rounded to bfloat16 (nearest even) */
  NVFP4MOE_EPI_BF16 = 1,
  /* SwiGLU + NVFP4 re-quantisation of the gate_up output (N = 2I):
   * h[p, i] = silu(y[p, i]) * y[p, I + i]  (rows [0,I) of each expert's B are the
   * gate, rows [I,2I) the up projection), quantised with the caller's per-tensor
   * scale *out_g into out_codes [m_total, I/2] and out_scales [m_total, I/16].
   * Requires I % 16 == 0. */
  NVFP4MOE_EPI_SWIGLU_NVFP4 = 2,
  /* weighted scatter-add (the combine fused into the down GEMM):
   * out[row_token[p]*N + n] += row_weight[p] * y[p, n]   (float32 atomics;
   * out is float32 [out_rows, N] and must be zeroed by the caller; the order of
   * the additions is not fixed, so results may differ in the last bits between
   * runs). */
  NVFP4MOE_EPI_COMBINE_F32 = 3,
  /* int8_grouped_gemm only: SwiGLU of the gate_up output (N = 2I, halves as
   * above), h = silu(y[:, :I]) * y[:, I:] rounded to bfloat16 into out
   * [m_total, I] (nearest even). */
  NVFP4MOE_EPI_SWIGLU_BF16 = 4
} nvfp4moe_epilogue;

/* Arguments of nvfp4_grouped_gemm (a struct keeps the ABI stable). */
typedef struct nvfp4moe_gemm_args {
  /* A operand: NVFP4 rows (activations). */
  const uint8_t* a_codes;     /* [a_rows_total, K/2], 16-byte aligned */
  const uint8_t* a_scales;    /* [a_rows_total, K/16] */
  const float* a_g;           /* device, 1 float */
  const int32_t* a_rows;      /* device [m_total]: A row read by GEMM row p, or NULL for row p.
                                 Every entry must lie in [0, a_rows_total). */
  int64_t a_rows_total;
  /* B operand: per-expert NVFP4 weights, row n of expert e is output column n. */
  const uint8_t* b_codes;     /* [E, N, K/2], 16-byte aligned */
  const uint8_t* b_scales;    /* [E, N, K/16] */
  const float* b_g;           /* device [E]: one per-tensor scale per expert */
  /* grouping: rows [offsets[e], offsets[e+1]) of the GEMM belong to expert e. */
  const int32_t* offsets;     /* device [E+1], non-decreasing, offsets[0] = 0, offsets[E] <= m_total */
  int32_t E;
  int32_t N;                  /* multiple of 16 */
  int32_t K;                  /* multiple of 32 */
  int64_t m_total;            /* host-side bound on offsets[E] (rows of out) */
  int32_t epilogue;           /* nvfp4moe_epilogue */
  void* out;                  /* EPI_F32: float [m_total, N]; EPI_BF16: bf16 [m_total, N]
                                 (16-byte aligned: rows leave as 16-byte stores);
                                 EPI_COMBINE_F32: float [out_rows, N]; unused for SWIGLU */
  int64_t out_rows;           /* EPI_COMBINE_F32: rows of the accumulator (tokens) */
  uint8_t* out_codes;         /* EPI_SWIGLU_NVFP4 */
  uint8_t* out_scales;        /* EPI_SWIGLU_NVFP4 */
  const float* out_g;         /* EPI_SWIGLU_NVFP4: device, 1 float, > 0 */
  const int32_t* row_token;   /* EPI_COMBINE_F32: device [m_total], values in [0, out_rows) */
  const float* row_weight;    /* EPI_COMBINE_F32: device [m_total] */
  int32_t max_rows_per_expert_hint;  /* rows per expert the caller expects (the pages' tune_max_num_tokens);
                                        0: m_total / E.  Picks the tile shape (>= 128: the large-M tile)
                                        and the weight-load cache policy (>= 64: cached, else
                                        non-temporal); never changes the result. */
  /* Optional: B in the packed tile layout written by nvfp4_weight_repack (16-byte
     aligned).  When set, b_codes / b_scales are not read (and may be NULL). */
  const uint8_t* b_packed;
} nvfp4moe_gemm_args;

/* ---------------------------------------------------------------- route + permute
 * Top-k routing and the expert-first permutation ("Discovering SM120-Specific
 * CUTLASS MoE Kernels", section "Input Knowledge Required": a router picks
 * experts per token; "From Empirical Limits ...", section "Sections 5-6:
 * Algorithmic Techniques": expert-first layout, token reordering).
 *   logits             float32 [T, E]
 *   topk_ids   (out)   int32 [T, k]   k largest logits by descending value, ties to the lower id
 *   topk_w     (out)   float32 [T, k] exp(l_j - l_max) / sum over the k chosen (softmax over E,
 *                                     renormalised over the k), computed in float64
 *   counts     (out)   int32 [E]      assignments per expert
 *   offsets    (out)   int32 [E+1]    exclusive prefix sum of counts
 *   perm_src_token     (out) int32 [T*k]  token of permuted row p
 *   perm_of_assignment (out) int32 [T*k]  permuted row of assignment t*k+j
 *   perm_weight        (out, nullable) float32 [T*k]  topk_w of permuted row p
 * Rows of one expert keep ascending t*k+j (stable): every output is
 * deterministic and bit-exact.  Limits: 1 <= k <= min(E, 32), E <= 4096,
 * T*k < 2^30.  Logits must be finite. */
size_t moe_route_permute_workspace_size(int32_t T, int32_t E, int32_t k);
int moe_route_permute(const float* logits, int32_t T, int32_t E, int32_t k,
                      int32_t* topk_ids, float* topk_w, int32_t* counts, int32_t* offsets,
                      int32_t* perm_src_token, int32_t* perm_of_assignment, float* perm_weight,
                      void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------- router with scores
 * moe_route_permute with the choices of a trained router (the router of
 * "Discovering SM120-Specific CUTLASS MoE Kernels", section "Input Knowledge
 * Required", whose form the pages leave open):
 *   scores   s [T, E] of the logits l (float32, bf16 or f16), by `score`, whatever
 *            the bias; 0 where the logit is -inf or NaN
 *   keys     s + bias[e] (the balance bias enters the choice, not the weights)
 *   groups   the E experts are n_group groups of neighbours; a group's value is the
 *            sum of its group_top (1 or 2) largest keys; the topk_group best stay
 *            (ties: the lower group)
 *   choice   the k largest keys of the groups that stay, descending, ties to the
 *            lower id; without a bias by the logits themselves (the scores' order
 *            without their saturation)
 *   weights  the chosen scores u_j, as they are or (renormalize) u_j / sum(u), also
 *            where the scores underflow together, times `scale`, rounded to float32 once
 * Scores, keys and weights are float64 up to there, so near-equal keys are ordered
 * as defined (values that differ by float64's own rounding, as sums of a group's keys
 * can, may come in either order).  An expert is closed to the choice if its logit is
 * -inf or NaN, or its key -inf or NaN.  Closed experts count nothing in their group (a
 * group without an open expert comes last), and are chosen, by ascending id and with
 * weight 0, only where the groups that stay have fewer than k open ones; a row without
 * any open expert has weights 0.  A bias of -inf or NaN closes an expert to the choice
 * alone: its score and its share of a softmax's sum remain, and its logit's gradient.
 * +inf counts as the largest float32.
 * Outputs, permutation and workspace as for moe_route_permute, none of them over the
 * logits or the bias; `scores` (nullable) receives s as float32.  Limits as there, and
 * n_group divides E, n_group <= 64, k <= topk_group * E / n_group,
 * group_top <= E / n_group. */
typedef struct nvfp4moe_route_args {
  const void* logits;         /* [T, E] */
  int32_t dtype;              /* nvfp4moe_dtype of the logits */
  int32_t T, E, k;
  int32_t score;              /* nvfp4moe_score */
  int32_t renormalize;        /* 0 or 1 */
  float scale;
  const float* bias;          /* [E] or NULL */
  int32_t n_group;            /* 1: no groups (then topk_group and group_top are 1) */
  int32_t topk_group;
  int32_t group_top;
  int32_t* topk_ids;          /* out [T, k] */
  float* topk_w;              /* out [T, k] */
  int32_t* counts;            /* out [E] */
  int32_t* offsets;           /* out [E+1] */
  int32_t* perm_src_token;    /* out [T*k] */
  int32_t* perm_of_assignment;/* out [T*k] */
  float* perm_weight;         /* out [T*k] or NULL */
  float* scores;              /* out [T, E] or NULL */
} nvfp4moe_route_args;
int moe_route_scored(const nvfp4moe_route_args* args, void* workspace, size_t workspace_bytes, void* stream);

/* Gradient of the logits from d_topk_w [T, k], that of the weights, and (nullable)
 * d_scores, that of the scores (a balance loss): [T, E] with d_scores_ld = E, or one
 * row for all tokens with d_scores_ld = 0.  logits, topk_ids and the options are
 * those of the forward call (bias: only its -inf and NaN matter).  The choice and
 * the bias have no gradient; logits of -inf or NaN get 0.  Ids outside [0, E) are left out;
 * an id that stands twice in a row counts twice.  dlogits has the logits' type;
 * float32 arithmetic, rounded once. */
typedef struct nvfp4moe_route_grad_args {
  const void* logits;
  int32_t dtype;
  int32_t T, E, k;
  int32_t score;
  int32_t renormalize;
  float scale;
  const float* bias;
  const int32_t* topk_ids;
  const float* d_topk_w;
  const float* d_scores;      /* or NULL */
  int64_t d_scores_ld;        /* E or 0 */
  void* dlogits;              /* out [T, E] */
} nvfp4moe_route_grad_args;
int moe_route_scored_backward(const nvfp4moe_route_grad_args* args, void* stream);

/* ---------------------------------------------------------------- quantise
 * The NVFP4 encoding of an operand (e2m1 values with one ue4m3 scale per 16
 * along the reduction axis: "From Empirical Limits ...", section "Section 1:
 * CUTLASS Kernels - The Foundation"; the quantiser rule is the reading given
 * at the top of this file).
 * x [rows, cols] (bf16 or float32, finite) -> NVFP4 codes/scales as described
 * above.  g_in (device, nullable): a caller-supplied per-tensor scale; NULL
 * computes g = amax/2688 (1 if the tensor is zero) on the device.  g_out
 * (device, nullable) receives the scale used.  cols % 32 == 0, x 16-byte
 * aligned. */
size_t nvfp4_quantize_workspace_size(void);
int nvfp4_quantize(const void* x, int32_t x_dtype, int64_t rows, int64_t cols,
                   const float* g_in, float* g_out, uint8_t* codes, uint8_t* scales,
                   void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------- route + quantise
 * moe_route_permute and nvfp4_quantize of the layer's activations in one
 * call, with the same arguments and the same, bit-identical outputs (x has
 * T rows).  The two steps read different inputs; their kernels share launches,
 * so their short launches overlap instead of running one after another.
 * workspace: moe_route_quantize_workspace_size(T, E, k) bytes, 16-byte
 * aligned, caller-owned (the routing scratch followed by the quantiser's amax
 * partials).  Errors as for the two calls. */
size_t moe_route_quantize_workspace_size(int32_t T, int32_t E, int32_t k);
int moe_route_quantize(const float* logits, int32_t T, int32_t E, int32_t k,
                       int32_t* topk_ids, float* topk_w, int32_t* counts, int32_t* offsets,
                       int32_t* perm_src_token, int32_t* perm_of_assignment, float* perm_weight,
                       const void* x, int32_t x_dtype, int64_t cols, const float* g_in, float* g_out,
                       uint8_t* codes, uint8_t* scales,
                       void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------- route + quantise, no allocation
 * For callers that cannot allocate device memory or pass a workspace: code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc.  Same arguments, kernels and bit-identical outputs as
 * moe_route_quantize, minus the workspace: the scratch comes from one fixed
 * block of device memory that the library holds on each GPU it runs on until
 * the process ends (moe_route_quantize_noalloc_max_workspace() bytes, 4 MiB).
 * A call whose moe_route_quantize_workspace_size(T, E, k) exceeds that block
 * returns NVFP4MOE_ERR_UNSUPPORTED (about T*k <= 900k at E = 256).  Nothing is
 * allocated: the device address of the block is looked up once per device, on
 * the first call with that device current.  Every call on one GPU shares the
 * block, so calls that overlap on one GPU (concurrent streams, or threads)
 * race and must be serialised by the caller.  Other errors as for
 * moe_route_quantize. */
size_t moe_route_quantize_noalloc_max_workspace(void);
int moe_route_quantize_noalloc(const float* logits, int32_t T, int32_t E, int32_t k,
                               int32_t* topk_ids, float* topk_w, int32_t* counts, int32_t* offsets,
                               int32_t* perm_src_token, int32_t* perm_of_assignment, float* perm_weight,
                               const void* x, int32_t x_dtype, int64_t cols, const float* g_in, float* g_out,
                               uint8_t* codes, uint8_t* scales, void* stream);

/* ---------------------------------------------------------------- grouped GEMM
 * For expert e and GEMM row p in [offsets[e], offsets[e+1]) with A row
 * r = a_rows ? a_rows[p] : p:
 *   y[p, n] = (g_a * g_b[e]) * sum_kb s_a[r,kb] s_b[e,n,kb] sum_{i<16} q_a[r,16kb+i] q_b[e,n,16kb+i]
 * FP32 accumulation; the block products are formed exactly (E2M1*E4M3 values
 * are exact in FP16 and their products exact in FP32).  The MoE grouped GEMM of
 * "From Empirical Limits ...", section "Sections 2-4: Framework and Community
 * Landscape", with the epilogues listed in nvfp4moe_epilogue (the "finalize"
 * epilogue of "The Critical Search: Uncovering SM120 CUTLASS Collective
 * Implementations", section "Context: The Optimization Journey", is
 * NVFP4MOE_EPI_COMBINE_F32).  Rows p >= offsets[E] are not written.  Experts
 * with no rows read no weight bytes.  Size limits (NVFP4MOE_ERR_UNSUPPORTED
 * beyond them): A codes (a_rows_total * K / 2 bytes) below 2 GiB; fewer than
 * 2^31 rows. */
int nvfp4_grouped_gemm(const nvfp4moe_gemm_args* args, void* stream);

/* ---------------------------------------------------------------- expert FFN in one call
 * gate_up grouped GEMM + SwiGLU + NVFP4 requantisation of h, then the down
 * grouped GEMM, for all experts: the two nvfp4_grouped_gemm calls of the
 * layer (EPI_SWIGLU_NVFP4 on gathered x rows, then EPI_BF16 on h), with the
 * same results bit for bit.  From 48 rows per expert (the hint, else
 * m_total / E) both run in ONE persistent launch whose down tasks start as soon
 * as the gate_up tasks of their row chunk are done, filling the slots the light
 * chunks leave free ("From Empirical Limits ...", section "Sections 5-6:
 * Algorithmic Techniques": adaptive grid sizing; section "Key Findings and
 * Their Impact": fusion; "Discovering SM120-Specific CUTLASS MoE Kernels",
 * section "The Discovery": a min-latency kernel for small batches, tuned to the
 * expected tokens).  The tile table, by rows per expert (measured):
 *   < 48       two launches, decode tile, non-temporal weight loads (while
 *              every expert fits one 64-row chunk gate_up fills every slot in
 *              one round: no tail to fill)
 *   48 .. 63   one launch, decode tile, non-temporal weight loads
 *   >= 64      one launch, decode tile, cached weight loads (from 128 rows
 *              the MFMA-bound regime, where it still beats two launches of
 *              the large-M tile: down overlaps gate_up's tail)
 * Arguments (device pointers):
 *   x_codes/x_scales/x_g   NVFP4 activations [x_rows, H/2], [x_rows, H/16], g
 *   perm_src_token         [m_total]: x row of GEMM row p (moe_route_permute)
 *   offsets                [E+1] expert offsets (moe_route_permute)
 *   w_gu_packed, g_gu      gate_up weights [E, 2I, H] repacked by
 *                          nvfp4_weight_repack, per-expert scales [E]
 *   w_dn_packed, g_dn      down weights [E, H, I] repacked, scales [E]
 *   g_h                    per-tensor scale of h (1 float)
 *   h_codes, h_scales      (out) h [m_total, I/2], [m_total, I/16]
 *   y                      (out) bf16 [m_total, H], the down rows (then
 *                          moe_unpermute_combine, or the fused combine below)
 *   out, perm_of_assignment, topk_w, T, k   optional weighted top-k combine
 *                          of the down rows, with moe_unpermute_combine's
 *                          arithmetic and result bit for bit (bf16 in, bf16
 *                          out): out [T, H] bf16, perm_of_assignment and topk_w
 *                          [T, k] from moe_route_permute, T * k == m_total,
 *                          m_total * H * 2 < 2^31.  out == NULL: no combine
 *                          (y holds the result).  In the one-launch regime the
 *                          combine runs inside the launch - the down task that
 *                          writes the last of a token's k rows of a column
 *                          group combines that group (the pages' finalize:
 *                          "The Critical Search ...", section "Context: The
 *                          Optimization Journey") - otherwise as one more
 *                          kernel on the stream after the down GEMM.
 * I % 32 == 0, I <= 256 (one K step of the down GEMM), H % 32 == 0, E <= 4096.
 * workspace: moe_expert_ffn_workspace_size(E, m_total, H, I) bytes, 256-byte
 * aligned, caller-owned; it holds the task lists and chunk counters, which the
 * call rewrites (a planning kernel, no memset).  Its first 64 int32 words are a
 * header; word 8 is nonzero after a launch in which a down task stopped waiting
 * for its h rows past a bounded spin (a fault of the scheduling, never expected:
 * the results of that launch are then invalid).  Calls sharing a workspace must
 * not overlap. */
typedef struct nvfp4moe_ffn_args {
  const uint8_t* x_codes;
  const uint8_t* x_scales;
  const float* x_g;
  int64_t x_rows;
  const int32_t* perm_src_token;
  const int32_t* offsets;
  int32_t E;
  int32_t H;
  int32_t I;
  int64_t m_total;
  const uint8_t* w_gu_packed;
  const float* g_gu;
  const uint8_t* w_dn_packed;
  const float* g_dn;
  const float* g_h;
  uint8_t* h_codes;
  uint8_t* h_scales;
  void* y;
  int32_t max_rows_per_expert_hint;
  void* out;
  const int32_t* perm_of_assignment;
  const float* topk_w;
  int32_t T;
  int32_t k;
} nvfp4moe_ffn_args;
size_t moe_expert_ffn_workspace_size(int32_t E, int64_t m_total, int32_t H, int32_t I);
int moe_expert_ffn(const nvfp4moe_ffn_args* args, void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------- MXFP4 variant
 * The MXFP4 format: E2M1 values with one E8M0 scale (a power of two, code c =
 * 2^(c-127)) per 32 consecutive values along the reduction axis and no
 * per-tensor scale (the OCP MX format; the pages list an MXFP4 grouped GEMM
 * with 128x128x128 tiles among the kernels they survey: "From Empirical Limits
 * ...", section "Sections 2-4: Framework and Community Landscape").  It maps
 * onto gfx950's block-scaled MFMA with no decode in registers.
 *   codes  uint8 [rows, cols/2]   as NVFP4 (element 2i in the low nibble of byte i)
 *   scales uint8 [rows, cols/32]  E8M0 codes
 * Quantiser: X = floor(log2(absmax_block)) - 2 clamped to [-127, 127], scale
 * code X + 127, code = E2M1 nearest-even of x / 2^X (exact), saturating at 6,
 * sign copied from x; an all-zero block gets scale code 0 and codes 0.
 * x: bf16 or float32 [rows, cols], finite, 16-byte aligned, cols % 32 == 0. */
int mxfp4_quantize(const void* x, int32_t x_dtype, int64_t rows, int64_t cols, uint8_t* codes, uint8_t* scales,
                   void* stream);
/* Grouped MXFP4 GEMM with the nvfp4_grouped_gemm argument struct, read as:
 *   y[p, n] = a_g * b_g[e] * sum_k A^[r, k] B^[e, n, k]   (A^, B^ dequantised MX values)
 * a_scales [a_rows_total, K/32], b_scales [E, N, K/32] (E8M0); a_g, b_g are
 * float32 multipliers (pass 1.0 for plain MX tensors); b_packed: optional B in
 * the layout written by mxfp4_weight_repack (then b_codes/b_scales are not read).  Epilogues: EPI_F32, EPI_BF16, and EPI_SWIGLU_NVFP4
 * read as SwiGLU + MXFP4 requantisation of h: out_codes [m_total, I/2],
 * out_scales [m_total, I/32] (out_g unused; I % 32 == 0).  EPI_COMBINE_F32 is
 * NVFP4MOE_ERR_UNSUPPORTED.  K % 32 == 0.  FP32 accumulation of exact
 * E2M1 x E2M1 x 2^k products; other limits as for nvfp4_grouped_gemm. */
int mxfp4_grouped_gemm(const nvfp4moe_gemm_args* args, void* stream);
/* MXFP4 weights [E, N, K] repacked once into streaming tiles of 16 rows x 256
 * K (2176 bytes: each lane's 32 code bytes and 2 scale bytes, in the order the
 * kernel's lanes read them; zero codes past N and K).  Private layout, pure
 * data movement.  K % 32 == 0; 16-byte aligned codes and packed. */
size_t mxfp4_weight_packed_size(int32_t E, int32_t N, int32_t K);
int mxfp4_weight_repack(const uint8_t* codes, const uint8_t* scales, int32_t E, int32_t N, int32_t K,
                        uint8_t* packed, size_t packed_bytes, void* stream);

/* ---------------------------------------------------------------- FP8 block-scaled variant
 * FP8 E4M3 operands with float32 block scales along K (the FP8 grouped GEMM
 * the pages list beside the FP4 ones: "From Empirical Limits ...", section
 * "Sections 2-4: Framework and Community Landscape"; the blockwise-scaled
 * FP8 collective: "The Critical Search: Uncovering SM120 CUTLASS Collective
 * Implementations", section "Output Knowledge Created").  Blocks of 128
 * values along K: one scale per row and block for activations (1 x 128), one
 * per 128 x 128 tile for weights.
 *   codes  uint8 [rows, cols]   E4M3 (OCP E4M3FN) bytes, sign in bit 7
 *   scales float [ceil(rows/block_rows), cols/128]
 * Quantiser: s = absmax_block / 448 (float32 division; 1 for an all-zero
 * block), code = E4M3 nearest-even of |x| / s (correctly rounded float32
 * quotient), saturating at 448, sign copied from x.
 * fp8_quantize: x bf16 or float32 [batch, rows, cols] (finite, 16-byte aligned,
 * cols % 128 == 0); block_rows 1 (activations: batch is folded into rows) or
 * 128 (weights: each of the batch matrices has its own row blocks, scales
 * [batch, ceil(rows/128), cols/128]; rows <= 8388480, batch <= 65535,
 * cols < 2^31).  Block rows 1: fewer than 2^26 blocks in all.  codes 16-byte,
 * scales 4-byte aligned. */
int fp8_quantize(const void* x, int32_t x_dtype, int64_t batch, int64_t rows, int64_t cols, int32_t block_rows,
                 uint8_t* codes, float* scales, void* stream);
/* SwiGLU between the FP8 grouped GEMMs: h = silu(gate) * up of gate_up [M, 2I]
 * (float32 or bf16; gate = columns [0, I), up = [I, 2I), as moe_swiglu), in
 * float32, quantised as fp8_quantize with 1 x 128 blocks: codes [M, I], scales
 * [M, I/128].  I % 128 == 0; gate_up 8-byte, codes 2-byte, scales 4-byte
 * aligned. */
int fp8_swiglu_quantize(const void* gate_up, int32_t dtype, int64_t M, int32_t I, uint8_t* codes, float* scales,
                        void* stream);
/* FP8 weights [E, N, K] repacked once into tiles of 16 rows x 128 K (2048
 * bytes, each lane's 32 bytes in the order the kernel's lanes read them; zero
 * codes past N).  Private layout, pure data movement.  K % 128 == 0, N % 16 ==
 * 0, 16-byte aligned codes and packed. */
size_t fp8_weight_packed_size(int32_t E, int32_t N, int32_t K);
int fp8_weight_repack(const uint8_t* codes, int32_t E, int32_t N, int32_t K, uint8_t* packed, size_t packed_bytes,
                      void* stream);
/* Grouped FP8 GEMM, per expert e and GEMM row p in [offsets[e], offsets[e+1])
 * with A row r = a_rows[p] (or p):
 *   y[p, n] = sum_kb sa[r, kb] * sb[e, n / 128, kb] * sum_{k in block kb} A[r, k] B[e, n, k]
 * Each block's partial sum comes from the FP8 matrix instruction in float32
 * and enters the float32 accumulator scaled by sa * sb.  Same grouping and
 * bounds rules as nvfp4_grouped_gemm; epilogues EPI_F32, EPI_BF16, and
 * EPI_SWIGLU_NVFP4 read as SwiGLU + FP8 requantisation of h (the gate_up GEMM
 * with fp8_swiglu_quantize fused into it, the same bits): N = 2I with
 * I % 128 == 0, h = silu(y[:, :I]) * y[:, I:], out_codes [m_total, I] E4M3 and
 * out_scales float32 [m_total, I/128] as fp8_swiglu_quantize writes them.
 * This epilogue runs the decode tile at every size (the large tile has no
 * SwiGLU epilogue). */
typedef struct nvfp4moe_fp8_gemm_args {
  const uint8_t* a_codes;     /* [a_rows_total, K] E4M3, 16-byte aligned */
  const float* a_scales;      /* [a_rows_total, K/128] */
  const int32_t* a_rows;      /* device [m_total] or NULL; entries in [0, a_rows_total) */
  int64_t a_rows_total;
  const uint8_t* b_packed;    /* fp8_weight_repack layout of [E, N, K], 16-byte aligned */
  const float* b_scales;      /* [E, ceil(N/128), K/128] */
  const int32_t* offsets;     /* device [E+1], as for nvfp4_grouped_gemm */
  int32_t E;
  int32_t N;                  /* multiple of 16 */
  int32_t K;                  /* multiple of 128 */
  int64_t m_total;
  int32_t epilogue;           /* NVFP4MOE_EPI_F32, NVFP4MOE_EPI_BF16 or NVFP4MOE_EPI_SWIGLU_NVFP4 (see above) */
  void* out;                  /* float or bf16 [m_total, N], 16-byte aligned; unused for SwiGLU */
  int32_t max_rows_per_expert_hint;  /* as for nvfp4_grouped_gemm: < 64 streams weights non-temporally */
  uint8_t* out_codes;         /* SwiGLU: h codes [m_total, N/2] */
  float* out_scales;          /* SwiGLU: h block scales [m_total, N/256], 4-byte aligned */
} nvfp4moe_fp8_gemm_args;
int fp8_grouped_gemm(const nvfp4moe_fp8_gemm_args* args, void* stream);

/* ---------------------------------------------------------------- 16-bit expert FFN
 * The experts' feed-forward block on bfloat16 or float16 operands, with its
 * gradients: the form the experts are trained in before they are quantised
 * for the calls above (same grouping, gate_up row order and layer shape: "From
 * Empirical Limits ...", section "Sections 5-6: Algorithmic Techniques").  All
 * operands row-major; `dtype` (NVFP4MOE_BF16 or NVFP4MOE_F16) is the type of
 * every 16-bit operand and result of a call.  Sums run in float32 in a fixed
 * order (no atomics: results are the same from run to run) and are rounded
 * once, nearest even.  The grouping rules of nvfp4_grouped_gemm hold: rows
 * [offsets[e], offsets[e+1]) belong to expert e, rows p >= offsets[E] of a
 * result are not written, E = 1 is a dense product.  m_total may be 0 (then
 * the row operands may be NULL; a weight gradient is still written, as zeros).
 * Pointers 16-byte aligned; H, I, N and K multiples of 8 up to 2^26; E <= 4096;
 * m_total < 2^30; an operand or result may exceed 4 GiB.  A hint is the rows
 * per expert the caller expects (0: m_total over the experts that can have
 * rows): it picks the kernel, never the result's definition.  Results must not
 * overlap operands.  Index arrays: see NVFP4MOE_DEBUG above (bad a_rows entries
 * read row 0). */

/* h[p, i] = act(g[p, i]) * u[p, i] with g = x[r] w[e, :I]^T, u = x[r] w[e, I:]^T
 * and r = a_rows ? a_rows[p] : p; gate and up projection, activation and
 * product in one kernel.  gu (nullable) receives g and u in float32
 * [m_total, 2I] for moe_gated_ffn_backward. */
typedef struct nvfp4moe_gated_args {
  const void* x;              /* [x_rows, H] */
  int32_t dtype;
  const int32_t* a_rows;      /* device [m_total] or NULL; entries in [0, x_rows) */
  int64_t x_rows;             /* without a_rows: at least m_total */
  const void* w;              /* [E, 2I, H]: rows [0, I) gate, [I, 2I) up */
  const int32_t* offsets;     /* device [E+1] */
  int32_t E, H, I;
  int64_t m_total;
  int32_t activation;         /* nvfp4moe_activation */
  int32_t max_rows_per_expert_hint;
  void* h;                    /* out [m_total, I] */
  float* gu;                  /* out [m_total, 2I] or NULL */
} nvfp4moe_gated_args;
int moe_gated_ffn(const nvfp4moe_gated_args* args, void* stream);

/* Gradients of moe_gated_ffn from dh, the gradient of h, and the gu it saved:
 *   dg = dh * u * act'(g), du = dh * act(g)   (float32, rounded to dtype: the
 *                                              operand of both products; in
 *                                              float16 above 65504 infinite)
 *   dx[p, :] = dg[p] w[e, :I] + du[p] w[e, I:]         one row per row p
 *   dw[e, :I] = sum_p dg[p]^T x[r_p], dw[e, I:] = sum_p du[p]^T x[r_p]
 * dx rows are per GEMM row: for gathered x, the gradient of a token is the sum
 * of its rows, moe_unpermute_combine(dx, perm_of_assignment, NULL, ...).
 * Either of dx and dw may be NULL (not wanted).  dw of an expert without rows
 * is zero.  (m_total / 64 + min(E, m_total)) * ceil(I / 64) <= 2^24 - 8: for
 * I <= 64 about 2^30 - 64 E rows.  workspace:
 * moe_gated_ffn_backward_workspace_size bytes, 256-byte aligned, caller-owned;
 * calls sharing one must not overlap. */
typedef struct nvfp4moe_gated_grad_args {
  const void* x;              /* as in the forward call (not read when dw is NULL) */
  int32_t dtype;
  const int32_t* a_rows;
  int64_t x_rows;
  const void* w;              /* not read when dx is NULL */
  const int32_t* offsets;
  int32_t E, H, I;
  int64_t m_total;
  int32_t activation;
  int32_t max_rows_per_expert_hint;
  const float* gu;            /* [m_total, 2I] */
  const void* dh;             /* [m_total, I] */
  void* dx;                   /* out [m_total, H] or NULL */
  void* dw;                   /* out [E, 2I, H] or NULL */
} nvfp4moe_gated_grad_args;
size_t moe_gated_ffn_backward_workspace_size(int32_t E, int32_t H, int32_t I, int64_t m_total);
int moe_gated_ffn_backward(const nvfp4moe_gated_grad_args* args, void* workspace, size_t workspace_bytes,
                           void* stream);

/* y[p, n] = sum_k a[r, k] b[e, n, k], the down projection (r = a_rows ? a_rows[p]
 * : p); out in dtype, or float32. */
typedef struct nvfp4moe_product_args {
  const void* a;              /* [a_rows_total, K] */
  int32_t dtype;
  const int32_t* a_rows;      /* device [m_total] or NULL; entries in [0, a_rows_total) */
  int64_t a_rows_total;       /* without a_rows: at least m_total */
  const void* b;              /* [E, N, K] */
  const int32_t* offsets;     /* device [E+1] */
  int32_t E, N, K;
  int64_t m_total;
  int32_t out_dtype;          /* dtype or NVFP4MOE_F32 */
  int32_t max_rows_per_expert_hint;
  void* out;                  /* [m_total, N] */
} nvfp4moe_product_args;
int moe_grouped_gemm(const nvfp4moe_product_args* args, void* stream);

/* Gradients of moe_grouped_gemm from dy [m_total, N]:
 *   da[p, :] = dy[p] b[e]  (one row per row p, as dx above),  db[e] = sum_p dy[p]^T a[r_p]
 * in dtype.  Either may be NULL; db of an expert without rows is zero.
 * workspace as above (moe_grouped_gemm_backward_workspace_size; may be NULL
 * where that is 0: it holds the parts of da or db where its tiles are few). */
typedef struct nvfp4moe_product_grad_args {
  const void* a;              /* as in the forward call (not read when db is NULL) */
  int32_t dtype;
  const int32_t* a_rows;
  int64_t a_rows_total;
  const void* b;              /* not read when da is NULL */
  const int32_t* offsets;
  int32_t E, N, K;
  int64_t m_total;
  int32_t max_rows_per_expert_hint;
  const void* dy;             /* [m_total, N] */
  void* da;                   /* out [m_total, K] or NULL */
  void* db;                   /* out [E, N, K] or NULL */
} nvfp4moe_product_grad_args;
size_t moe_grouped_gemm_backward_workspace_size(int32_t E, int32_t N, int32_t K, int64_t m_total);
int moe_grouped_gemm_backward(const nvfp4moe_product_grad_args* args, void* workspace, size_t workspace_bytes,
                              void* stream);

/* ---------------------------------------------------------------- INT8 variant
 * Symmetric 8-bit integers with one float32 scale per row: per token for
 * activations, per output channel for weights (value = code * scale).
 * int8_quantize: x [rows, cols] (bf16 or float32) -> codes int8 in [-127, 127]
 * and scales [rows]: s = absmax * (1/127) (float32 product with the float32
 * nearest 1/127; 1 where that is zero), code = nearest-even integer of the
 * correctly rounded float32 quotient x / s.  A row that holds a NaN or an
 * infinity gets scale NaN and codes 0, so that products of it are NaN.
 * Reproducible bit for bit.  cols % 8 == 0; x 16-byte, codes
 * 8-byte, scales 4-byte aligned; rows < 2^31. */
int int8_quantize(const void* x, int32_t x_dtype, int64_t rows, int64_t cols, int8_t* codes, float* scales,
                  void* stream);
/* Grouped INT8 GEMM, rows and experts as in nvfp4_grouped_gemm:
 *   y[p, n] = (a_scales[r] * b_scales[e, n]) * sum_k a[r, k] b[e, n, k]
 * with an exact 32-bit integer sum, scaled in float32.  Epilogues EPI_F32,
 * EPI_BF16 and EPI_SWIGLU_BF16 (N = 2I, I % 8 == 0).  Weights row-major, as
 * int8_quantize writes them.  K % 16 == 0, K <= 131056 (the sum's range),
 * N % 8 == 0, E <= 4096. */
typedef struct nvfp4moe_int8_gemm_args {
  const int8_t* a_codes;      /* [a_rows_total, K], 16-byte aligned */
  const float* a_scales;      /* [a_rows_total] */
  const int32_t* a_rows;      /* device [m_total] or NULL; entries in [0, a_rows_total) */
  int64_t a_rows_total;       /* without a_rows: at least m_total */
  const int8_t* b_codes;      /* [E, N, K], 16-byte aligned */
  const float* b_scales;      /* [E, N], 16-byte aligned */
  const int32_t* offsets;     /* device [E+1] */
  int32_t E, N, K;
  int64_t m_total;
  int32_t epilogue;
  int32_t max_rows_per_expert_hint;
  void* out;                  /* float or bf16 [m_total, N], or bf16 [m_total, N/2]; 16-byte aligned */
} nvfp4moe_int8_gemm_args;
int int8_grouped_gemm(const nvfp4moe_int8_gemm_args* args, void* stream);

/* ---------------------------------------------------------------- INT4 variant
 * Weights in 4 bits on 16-bit activations, for few rows an expert (decode), where
 * the weights' stream is the cost.  Groups of 32, 64 or 128 values along the
 * reduction share a scale and, optionally, a zero point:
 *   codes   uint8 [rows, cols/2]      element 2i in the low nibble of byte i
 *   scales  bf16 or f16 [rows, cols/group]
 *   zeros   uint8 [rows, cols/group], 0 .. 15, or NULL (8 everywhere)
 *   value = (code - zero) * scale
 * int4_quantize: x [rows, cols] (float32, bf16 or f16).  Without zeros: scale =
 * absmax * (1/7), code = clamp(rint(x / scale), -8, 7) + 8; with: lo = min(x, 0), hi
 * = max(x, 0), scale = (hi - lo) * (1/15), zero = clamp(rint(-lo / scale), 0, 15),
 * code = clamp(rint(x / scale) + zero, 0, 15).  The scale is a float32 product (with
 * the float32 nearest 1/7 or 1/15) rounded to its type (1 where that is zero),
 * quotients are correctly rounded float32 ones, rint goes to the nearest even:
 * reproducible bit for bit.  A group that holds a NaN or an
 * infinity, or whose scale overflows its type, gets scale NaN and codes 8 (with
 * zeros: codes and zero 0).  cols % group == 0; x and codes 16-byte aligned;
 * rows * cols < 2^40. */
int int4_quantize(const void* x, int32_t x_dtype, int64_t rows, int64_t cols, int32_t group, int32_t scale_dtype,
                  uint8_t* codes, void* scales, uint8_t* zeros, void* stream);
/* The values: out [rows, cols] in scale_dtype (rounded once) or float32 (exact).
 * 16-byte aligned codes and out. */
int int4_dequantize(const uint8_t* codes, const void* scales, const uint8_t* zeros, int64_t rows, int64_t cols,
                    int32_t group, int32_t scale_dtype, int32_t out_dtype, void* out, void* stream);
/* Grouped product, rows and experts as in the 16-bit expert FFN:
 *   y[p, n] = sum_k a[r, k] value(b)[e, n, k]       (r = a_rows ? a_rows[p] : p)
 * in dtype or float32; gated (N = 2I, rows [0, I) gate): h[p, i] = act(y[p, i]) *
 * y[p, I + i] [m_total, I] in dtype.  Exact products, float32 sums in a fixed
 * order.  Any N (gated: even); K % group == 0; E <= 4096; zeros entries above 15
 * count as they are.  Activations finite, and small enough that 31 sum(|a|) over a
 * group stays in float32's range (a row with an infinity or a NaN gives NaNs in its
 * own results only).  Any number of rows gives the product; from some
 * 160 rows an expert int4_dequantize and the 16-bit products are faster.  Size limits
 * (NVFP4MOE_ERR_UNSUPPORTED beyond them) as there, fewer than 2^32 threads in all,
 * and gated (N/2 + 64) * (K/2) < 2^32 - 64. */
typedef struct nvfp4moe_int4_gemv_args {
  const void* a;              /* [a_rows_total, K], 16-byte aligned */
  int32_t dtype;              /* NVFP4MOE_BF16 or NVFP4MOE_F16: of a, b_scales and 16-bit results */
  const int32_t* a_rows;      /* device [m_total] or NULL; entries in [0, a_rows_total) */
  int64_t a_rows_total;       /* without a_rows: at least m_total */
  const uint8_t* b_codes;     /* [E, N, K/2], 16-byte aligned */
  const void* b_scales;       /* [E, N, K/group] */
  const uint8_t* b_zeros;     /* [E, N, K/group] or NULL */
  int32_t group;              /* 32, 64 or 128 */
  const int32_t* offsets;     /* device [E+1] */
  int32_t E, N, K;
  int64_t m_total;
  int32_t gated;              /* 0 or 1 */
  int32_t activation;         /* nvfp4moe_activation, gated only */
  int32_t out_dtype;          /* dtype, or NVFP4MOE_F32 (not gated) */
  int32_t max_rows_per_expert_hint;
  void* out;                  /* 16-byte aligned */
} nvfp4moe_int4_gemv_args;
int int4_grouped_gemv(const nvfp4moe_int4_gemv_args* args, void* stream);

/* ---------------------------------------------------------------- packed weights
 * Weights are static, so they can be repacked once into a tile layout that the
 * grouped GEMM streams with fully contiguous, non-temporal loads: tile
 * (e, 16-row tile rt, 256-K step st) is 2304 bytes (the 16 rows' 128 code bytes
 * and 16 scale bytes of the step, ordered by the lane that consumes them),
 * tiles ordered by (e, rt, st), zero padded past N and K.  The layout is private
 * to this library (it may change between versions; nvfp4moe_version() tells
 * them apart); the row-major NVFP4 tensors stay the reference format.
 *   codes   [E, N, K/2]  row-major NVFP4 codes (16-byte aligned)
 *   scales  [E, N, K/16] E4M3 block scales
 *   packed  (out) nvfp4_weight_packed_size(E, N, K) bytes, 16-byte aligned
 * K % 32 == 0.  Pure data movement: no rounding, bit-exact. */
size_t nvfp4_weight_packed_size(int32_t E, int32_t N, int32_t K);
int nvfp4_weight_repack(const uint8_t* codes, const uint8_t* scales, int32_t E, int32_t N, int32_t K,
                        uint8_t* packed, size_t packed_bytes, void* stream);

/* ---------------------------------------------------------------- SwiGLU (unfused)
 * The activation between the two expert GEMMs, re-quantised to NVFP4 so that
 * the down GEMM runs on e2m1 operands too (the e2m1 x e2m1 block-scaled MMA of
 * "From Empirical Limits ...", section "Section 1: CUTLASS Kernels - The
 * Foundation"; the same step fused into the gate_up epilogue is
 * NVFP4MOE_EPI_SWIGLU_NVFP4, the kind of epilogue fusion that section "Key
 * Findings and Their Impact" of that page weighs more when bandwidth is tight).
 * gate_up [M, 2I] (float32 or bf16) -> h = silu(gate) * up, gate = columns
 * [0, I), up = [I, 2I), quantised to NVFP4 codes [M, I/2], scales [M, I/16].
 * g_in (nullable): per-tensor scale of h; NULL computes amax(h)/2688 on the
 * device (two passes).  g_out (nullable) receives the scale used.  I % 16 == 0. */
size_t moe_swiglu_workspace_size(void);
int moe_swiglu(const void* gate_up, int32_t dtype, int64_t M, int32_t I,
               const float* g_in, float* g_out, uint8_t* codes, uint8_t* scales,
               void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------- combine (unfused)
 * out[t, :] = sum_{j<k} topk_w[t, j] * y[perm_of_assignment[t*k + j], :]
 * ("token reordering with fused reduction", "From Empirical Limits ...", section
 * "Sections 5-6: Algorithmic Techniques").  y [rows, H] float32 or bf16; out
 * [T, H] float32 or bf16 (nearest even); float32 accumulation in j order.
 * perm_of_assignment NULL means row t*k + j; topk_w NULL means weight 1, so
 * (perm NULL, w NULL, k = 1) converts a float32 accumulator to bf16.
 * Every perm_of_assignment entry must lie in [0, rows of y): the kernel reads
 * the rows it names without a bounds check (the routing calls produce such
 * entries).  Without perm_of_assignment, y needs at least T*k rows.
 * H % 8 == 0. */
int moe_unpermute_combine(const void* y, int32_t y_dtype, const int32_t* perm_of_assignment,
                          const float* topk_w, int32_t T, int32_t k, int32_t H,
                          void* out, int32_t out_dtype, void* stream);

/* Gradients of moe_unpermute_combine from dout [T, H]: dy[row(t, j), :] = topk_w[t, j]
 * * dout[t, :] in y's type, and d_topk_w[t, j] = <dout[t], y[row(t, j)]> in float32
 * (fixed order).  y [y_rows, H]; perm_of_assignment and topk_w as in the forward
 * call (either NULL), entries of perm_of_assignment all different: rows of dy that
 * none names are left as they are, and an entry outside [0, y_rows) is left out
 * (d_topk_w 0).  Either of dy and d_topk_w may be NULL; y is not read without
 * d_topk_w.  float32 and bf16, each of dout and y.  H % 8 == 0; T >= 1; k <= 1024;
 * T * ceil(k / 4) < 2^24. */
int moe_unpermute_combine_backward(const void* dout, int32_t dout_dtype, const void* y, int32_t y_dtype, int64_t y_rows,
                                   const int32_t* perm_of_assignment, const float* topk_w, int32_t T, int32_t k,
                                   int32_t H, void* dy, float* d_topk_w, void* stream);

/* ---------------------------------------------------------------- status */
const char* nvfp4moe_status_string(int status);
const char* nvfp4moe_last_error_detail(void);
/* library version: major*10000 + minor*100 + patch */
int nvfp4moe_version(void);   /* 101: packed weight tiles of 16 rows x 256 K */

#ifdef __cplusplus
}
#endif

#endif /* NVFP4MOE_H */
