// Internal declarations shared by the HIP sources of libnvfp4moe.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lds_budget.h"
#include "nvfp4_device.h"

namespace nvfp4 {

enum : int { EPI_F32 = 0, EPI_BF16 = 1, EPI_SWIGLU = 2, EPI_COMBINE = 3 };

// Kernel-side arguments of the grouped GEMM (validated on the host first).
struct GemmParams {
  const uint8_t* a_codes;
  const uint8_t* a_scales;
  const float* a_g;
  const int32_t* a_rows;
  const uint8_t* b_codes;
  const uint8_t* b_scales;
  const uint8_t* b_packed;   // packed weight tiles (nvfp4_weight_repack) or nullptr
  const float* b_g;
  const int32_t* offsets;
  int E, N, K;
  int n_tiles;            // column tiles per expert (set by the launcher)
  int slots;              // workgroups of the kernel resident at once (set by the launcher)
  int m_total;            // rows of the outputs indexed by GEMM row
  int a_rows_total;       // rows of A (bound for gathered row indices)
  int out_rows;           // rows of the combine accumulator
  void* out;
  uint8_t* out_codes;
  uint8_t* out_scales;
  const float* out_g;
  const int32_t* row_token;
  const float* row_weight;
};

size_t route_permute_ws_bytes(int T, int E, int k);
hipError_t launch_route_permute(const float* logits, int T, int E, int k, int* topk_ids, float* topk_w,
                                int* counts, int* offsets, int* perm_src_token, int* perm_of_assignment,
                                float* perm_weight, void* ws, hipStream_t stream);
// the permutation of given choices (the steps of launch_route_permute behind the routing itself)
hipError_t launch_permute(const int* topk_ids, const float* topk_w, int T, int E, int k, int* counts, int* offsets,
                          int* perm_src_token, int* perm_of_assignment, float* perm_weight, void* ws, hipStream_t stream);
size_t route_quantize_ws_bytes(int T, int E, int k);
hipError_t launch_route_quantize(const float* logits, int T, int E, int k, int* topk_ids, float* topk_w,
                                 int* counts, int* offsets, int* perm_src_token, int* perm_of_assignment,
                                 float* perm_weight, const void* x, int dtype, int64_t cols, const float* g_in,
                                 float* g_out, uint8_t* codes, uint8_t* scales, void* ws, hipStream_t stream);
hipError_t launch_quantize(const void* x, int dtype, int64_t rows, int64_t cols, const float* g_in, float* g_out,
                           uint8_t* codes, uint8_t* scales, void* ws, hipStream_t stream);
hipError_t launch_swiglu(const void* y, int dtype, int64_t M, int I, const float* g_in, float* g_out,
                         uint8_t* codes, uint8_t* scales, void* ws, hipStream_t stream);
hipError_t launch_combine(const void* y, int y_dtype, const int* perm, const float* w, int T, int k, int H,
                          void* out, int out_dtype, hipStream_t stream);
size_t packed_weight_bytes(int E, int N, int K);
hipError_t launch_repack(const uint8_t* codes, const uint8_t* scales, int E, int N, int K, uint8_t* packed,
                         hipStream_t stream);
hipError_t launch_grouped_gemm(const GemmParams& prm, int epilogue, int64_t m_total, int hint, hipStream_t stream);
bool gemm_large_fits(const GemmParams& prm, int64_t rows_per_expert);
hipError_t launch_gemm_large(const GemmParams& prm, int epilogue, int64_t m_total, hipStream_t stream);
hipError_t launch_mx_quantize(const void* x, int dtype, int64_t rows, int64_t cols, uint8_t* codes,
                              uint8_t* scales, hipStream_t stream);
hipError_t launch_mx_gemm(const GemmParams& prm, int epilogue, int64_t m_total, int hint, hipStream_t stream);
size_t mx_packed_weight_bytes(int E, int N, int K);

hipError_t launch_mx_repack(const uint8_t* codes, const uint8_t* scales, int E, int N, int K, uint8_t* packed,
                            hipStream_t stream);
size_t moe_ffn_ws_bytes(int E, int64_t m_total, int H, int I);
// the weighted top-k combine fused into the expert-FFN launch
struct FfnCombine {
  const int32_t* perm_of;   // [T, k] row of assignment (t, j)
  const float* topk_w;      // [T, k]
  int T, k;
  void* out;                // bf16 [T, H]
};
hipError_t launch_moe_ffn(GemmParams gu, GemmParams dn, int64_t m_total, bool cached, void* ws, int spin_limit,
                          const FfnCombine* comb, hipStream_t stream);

// Kernel-side arguments of the grouped FP8 GEMM (validated on the host first).
struct Fp8Params {
  const uint8_t* a_codes;
  const float* a_scales;       // [a_rows_total, K/128]
  const int32_t* a_rows;
  const uint8_t* b_packed;
  const float* b_scales;       // [E, ceil(N/128), K/128]
  const int32_t* offsets;
  int E, N, K, m_total, a_rows_total;
  void* out;
  uint8_t* out_codes;          // SwiGLU epilogue: h E4M3 codes [m_total, N/2]
  float* out_scales;           // SwiGLU epilogue: h block scales [m_total, N/256]
};

hipError_t launch_fp8_quantize(const void* x, int dtype, int64_t batch, int64_t rows, int64_t cols, int block_rows,
                               uint8_t* codes, float* scales, hipStream_t stream);
size_t fp8_packed_weight_bytes(int E, int N, int K);
hipError_t launch_fp8_swiglu(const void* y, int dtype, int64_t M, int I, uint8_t* codes, float* scales,
                             hipStream_t stream);
hipError_t launch_fp8_repack(const uint8_t* codes, int E, int N, int K, uint8_t* packed, hipStream_t stream);
hipError_t launch_fp8_gemm(const Fp8Params& p, int epilogue, int64_t m_total, int hint, hipStream_t stream);

// Kernel-side arguments of the products on plain operands (validated on the
// host first); what rows, columns and reduction are is said in tile_gemm.h.
enum : int { TG_ACT_SILU = 0, TG_ACT_GELU = 1 };
struct TileParams {
  const void* a;           // rows operand
  const void* b;           // columns operand
  const int32_t* a_rows;   // gathered rows (NT: of a, TN and TC: of b) or nullptr
  const float* sa;         // int8: scale per row of a
  const float* sb;         // int8: scale per expert and row of b
  const int32_t* offsets;
  int E, N, K;             // N columns of the output (gated: 2I), K values of the reduction (NT, NN) or columns of a (TC)
  int R;                   // TN, TC: rows of the output per expert
  int m_total;
  int src_rows;            // bound of the entries of a_rows
  int act;
  int rows_hint;           // expected rows per expert
  int parts, part_k;       // float32 sums by parts: parts of the reduction and (NN) their length, a multiple of 64
  int n_tiles, r_tiles;    // set by the launcher
  void* out;
  float* gu;               // gated: float32 pre-activations [m_total, N], or nullptr
};
hipError_t launch_tile_gemm_bf16(const TileParams& p, int layout, int epilogue, hipStream_t stream);
hipError_t launch_tile_gemm_f16(const TileParams& p, int layout, int epilogue, hipStream_t stream);
hipError_t launch_tile_gemm_i8(const TileParams& p, int epilogue, hipStream_t stream);
hipError_t launch_gated_grad(const float* gu, const void* dh, int dtype_f16, int I, int64_t m_total,
                             const int32_t* offsets, int E, int act, void* dgu, void* dgu_t, hipStream_t stream);
int64_t gated_grad_ld(int64_t m_total, int E);   // columns of dgu_t
int64_t gated_grad_blocks(int I, int64_t m_total, int E);   // workgroups, fewer than 2^24
// sum of `parts` float32 matrices [rows, N] in their order, rounded to 16 bits; with offsets, rows behind the last expert are left
hipError_t launch_join(const float* part, int parts, int64_t rows, int N, const int32_t* offsets, int E, int dtype_f16,
                       void* out, hipStream_t stream);
// Kernel-side arguments of the router with scores (validated on the host first).
struct ScoredParams {
  const void* logits;
  const float* bias;       // [E] or nullptr
  int T, E, k;
  int softmax, renormalize;
  int n_group, topk_group, group_top;
  float scale;
  int* topk_ids;
  float* topk_w;
  float* scores;           // [T, E] or nullptr
  // set by the launcher
  int narrow;              // 16-bit logits
  int vec, vec_bias, vec_scores;   // rows can be read or written 4 values at a time
  int lanes_per_group;     // a power of two, or 0: groups by way of LDS
  int lds_wave;            // doubles of LDS a wave
};
struct ScoredGradParams {
  const void* logits;
  const float* bias;
  int T, E, k;
  int softmax, renormalize;
  float scale;
  const int* topk_ids;
  const float* d_topk_w;
  const float* d_scores;   // or nullptr
  int64_t d_scores_ld;     // E, or 0: one row for all tokens
  void* dlogits;
  int vec, vec_d, vec_out; // set by the launcher, as above
};
hipError_t launch_route_scored(const ScoredParams& p, int dtype, int* counts, int* offsets, int* perm_src_token,
                               int* perm_of_assignment, float* perm_weight, void* ws, hipStream_t stream);
hipError_t launch_route_scored_grad(const ScoredGradParams& p, int dtype, hipStream_t stream);

// Gradients of the weighted combine.
struct CombineGradParams {
  const void* dout;        // [T, H]
  const void* y;           // [rows, H]; not read without dw
  const int* perm;         // [T * k] or nullptr
  const float* w;          // [T * k] or nullptr: 1
  int T, k, H;
  int64_t rows;
  void* dy;                // [rows, H] or nullptr
  float* dw;               // [T * k] or nullptr
};
hipError_t launch_combine_grad(const CombineGradParams& p, int dout_dtype, int y_dtype, hipStream_t stream);

// INT4 groups along the last axis.
hipError_t launch_int4_quantize(const void* x, int dtype, int64_t rows, int64_t cols, int group, int scale_f16, uint8_t* codes,
                                void* scales, uint8_t* zeros, hipStream_t stream);
hipError_t launch_int4_dequantize(const uint8_t* codes, const void* scales, const uint8_t* zeros, int64_t rows, int64_t cols,
                                  int group, int scale_f16, int out_dtype, void* out, hipStream_t stream);
struct Int4Params {
  const void* a;           // rows, 16 bit
  const int32_t* a_rows;
  const uint8_t* codes;    // [E, N, K/2]
  const void* scales;      // [E, N, K/group], 16 bit
  const uint8_t* zeros;    // [E, N, K/group] or nullptr: 8
  const int32_t* offsets;
  int E, N, K;             // N: rows of the weights (gated: 2I)
  int m_total;
  int src_rows;
  int act;
  int rows_hint;
  int n_tiles, rounds;     // set by the launcher
  void* out;
};
int64_t int4_gemv_threads(int E, int N, int K, int64_t m_total, int64_t hint, int gated);   // of the launch
hipError_t launch_int4_gemv(const Int4Params& p, int f16, int group, int gated, int out_f32, hipStream_t stream);
hipError_t launch_int8_quantize(const void* x, int dtype, int64_t rows, int64_t cols, int8_t* codes, float* scales,
                                hipStream_t stream);

}  // namespace nvfp4
