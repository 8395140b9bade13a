// Grouped matrix products on plain operands (bf16, fp16, int8) for gfx950.
//
// One tile routine serves every product of the 16-bit expert FFN, its
// gradients and the INT8 product:
//   out[r, c] = sum_k R[r, k] * C[c, k]        (r, c, k as below)
//             rows r           columns c        reduction k     R          C
//   NT  y     rows of expert   N                K               [r][k]     [c][k]   y  = a B^T
//   NN  da    rows of expert   K                N               [r][k]     [k][c]   da = dy B
//   TN  dB    N                K                rows of expert  [k][r]     [k][c]   dB = dy^T a
// An operand stored [x][k] is K-contiguous, one stored [k][x] is K-major.
//
// The matrix instruction gets C as its first operand and R as its second, so a
// lane's four results are four neighbouring columns of one output row (one
// 8- or 16-byte store).
#pragma once

#include "gemm_device.h"

namespace nvfp4 {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 half4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

enum : int { TG_BF16 = 0, TG_F16 = 1, TG_I8 = 2 };            // operand type
enum : int { TG_NT = 0, TG_NN = 1, TG_TN = 2 };               // operand layouts
enum : int { TG_OUT_16 = 0, TG_OUT_F32 = 1, TG_OUT_GATED = 2 };  // epilogue

template <int T>
struct TgType;
template <>
struct TgType<TG_BF16> {
  using acc_t = float4v;
  static constexpr int bytes = 2;
  static __device__ __forceinline__ acc_t mfma(u32x4 a, u32x4 b, acc_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint2 pack(const float4v& v) {
    const bf16x4 r = {static_cast<__bf16>(v[0]), static_cast<__bf16>(v[1]), static_cast<__bf16>(v[2]), static_cast<__bf16>(v[3])};
    return __builtin_bit_cast(uint2, r);
  }
};
template <>
struct TgType<TG_F16> {
  using acc_t = float4v;
  static constexpr int bytes = 2;
  static __device__ __forceinline__ acc_t mfma(u32x4 a, u32x4 b, acc_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, a), __builtin_bit_cast(half8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint2 pack(const float4v& v) {
    const half4 r = {static_cast<_Float16>(v[0]), static_cast<_Float16>(v[1]), static_cast<_Float16>(v[2]), static_cast<_Float16>(v[3])};
    return __builtin_bit_cast(uint2, r);
  }
};
// int8: 64 values of k per instruction, exact 32-bit sums; 16-bit results are bf16
template <>
struct TgType<TG_I8> {
  using acc_t = i32x4;
  static constexpr int bytes = 1;
  static __device__ __forceinline__ acc_t mfma(u32x4 a, u32x4 b, acc_t c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint2 pack(const float4v& v) { return TgType<TG_BF16>::pack(v); }
};

// act(g) and its derivative, float32
__device__ __forceinline__ float tg_act(float g, int act) {
  if (act == TG_ACT_SILU) return g / (1.0f + __expf(-g));
  const float z = 0.7978845608028654f * (g + 0.044715f * g * g * g);
  // 0.5 (1 + tanh z) = 1 / (1 + exp(-2 z))
  return g / (1.0f + __expf(-2.0f * z));
}
__device__ __forceinline__ float tg_act_grad(float g, int act, float& value) {
  if (act == TG_ACT_SILU) {
    const float s = 1.0f / (1.0f + __expf(-g));
    value = g * s;
    return s * (1.0f + g * (1.0f - s));
  }
  const float g2 = g * g;
  const float s = 1.0f / (1.0f + __expf(-1.5957691216057308f * (g + 0.044715f * g * g2)));
  value = g * s;
  return s + g * s * (1.0f - s) * 1.5957691216057308f * (1.0f + 0.134145f * g2);
}

constexpr int kTgBM = 128, kTgBN = 128;     // tile; a K step is 128 bytes of each K-contiguous row
constexpr int kTgStep = 128;

// 16-byte chunk `ch` of row r lies at chunk ch ^ ((r >> 1) & 7): the 16 rows
// that the lanes of one fragment read at one chunk then cover all 64 banks
__device__ __forceinline__ int tg_at(int r, int ch) { return r * kTgStep + 16 * (ch ^ ((r >> 1) & 7)); }

template <int T, int L, int EPI>
__global__ __launch_bounds__(256) void k_tile_gemm(const TileParams p) {
  using TT = TgType<T>;
  using acc_t = typename TT::acc_t;
  constexpr int EB = TT::bytes;
  constexpr int SK = kTgStep / EB;          // values of k per step
  constexpr bool RKM = L == TG_TN, CKM = L != TG_NT;
  constexpr bool GATED = EPI == TG_OUT_GATED;
  static_assert(T != TG_I8 || L == TG_NT, "int8 has the forward product only");
  __shared__ __attribute__((aligned(16))) uint8_t lds[(kTgBM + kTgBN) * kTgStep];
  uint8_t* lr_ = lds;
  uint8_t* lc_ = lds + kTgBM * kTgStep;

  int e, m0, nt;
  int row0, Me;
  if constexpr (L == TG_TN) {
    const int per = p.r_tiles * p.n_tiles;
    e = blockIdx.x / per;
    const int u = blockIdx.x - e * per;
    m0 = (u / p.n_tiles) * kTgBM;
    nt = u % p.n_tiles;
    row0 = min(max(p.offsets[e], 0), p.m_total);
    Me = max(min(max(p.offsets[e + 1], 0), p.m_total) - row0, 0);
  } else {
    bool narrow;
    GemmParams map{};
    map.offsets = p.offsets;
    map.E = p.E;
    map.m_total = p.m_total;
    map.n_tiles = p.n_tiles;
    map.slots = 1 << 30;
    if (!find_task<kTgBM / 16, false, 0>(map, e, m0, nt, narrow)) return;
    row0 = min(max(p.offsets[e], 0), p.m_total);
    Me = min(max(p.offsets[e + 1], 0), p.m_total) - row0;
  }
  const int rows = L == TG_TN ? min(kTgBM, p.R - m0) : min(kTgBM, Me - m0);
  const int kt = L == TG_TN ? Me : p.K;     // length of the reduction
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int wr = wave >> 1, wc = wave & 1, lr = lane & 15, lg = lane >> 4;
  const int c0 = nt * (GATED ? kTgBN / 2 : kTgBN);
  const int half = p.N / 2;

  const uint8_t* A = static_cast<const uint8_t*>(p.a);
  const uint8_t* B = static_cast<const uint8_t*>(p.b);
  if constexpr (L != TG_TN) B += static_cast<size_t>(e) * p.N * p.K * EB;

  auto src_row = [&](int q) {               // row q of the expert's rows in the gathered operand
    int64_t r = row0 + q;
    if (p.a_rows) {
      r = p.a_rows[r];
      r = (r >= 0 && r < p.src_rows) ? r : 0;
    }
    return r;
  };
  acc_t acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = acc_t{0, 0, 0, 0};

  for (int k0 = 0; k0 < kt; k0 += SK) {
    u32x4 ra[4], rb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int q = t + 256 * i;
      ra[i] = u32x4{0, 0, 0, 0};
      rb[i] = u32x4{0, 0, 0, 0};
      if constexpr (!RKM) {
        const int r = q >> 3, k = k0 + (q & 7) * (16 / EB);
        if (r < rows && k < kt) {
          const int64_t sr = L == TG_NT ? src_row(m0 + r) : row0 + m0 + r;
          ra[i] = *reinterpret_cast<const u32x4*>(A + (sr * p.K + k) * EB);
        }
      } else {
        const int k = k0 + (q >> 4), r = m0 + (q & 15) * 8;
        if (k < kt && r < p.R) ra[i] = *reinterpret_cast<const u32x4*>(A + (static_cast<int64_t>(row0 + k) * p.R + r) * EB);
      }
      if constexpr (!CKM) {
        const int c = q >> 3, k = k0 + (q & 7) * (16 / EB);
        int col;
        bool in;
        if constexpr (GATED) {
          in = c0 + (c & 63) < half;
          col = c0 + (c & 63) + (c >= 64 ? half : 0);
        } else {
          col = c0 + c;
          in = col < p.N;
        }
        if (in && k < kt) rb[i] = *reinterpret_cast<const u32x4*>(B + (static_cast<int64_t>(col) * p.K + k) * EB);
      } else {
        const int k = k0 + (q >> 4), c = c0 + (q & 15) * 8;
        if (k < kt && c < p.N) {
          const int64_t kr = L == TG_TN ? src_row(k) : k;
          rb[i] = *reinterpret_cast<const u32x4*>(B + (kr * p.N + c) * EB);
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int q = t + 256 * i;
      if constexpr (!RKM) {
        *reinterpret_cast<u32x4*>(lr_ + tg_at(q >> 3, q & 7)) = ra[i];
      } else {
        // transposed into the K-contiguous layout, value by value
#pragma unroll
        for (int v = 0; v < 8; ++v) {
          const int k = q >> 4, r = (q & 15) * 8 + v;
          *reinterpret_cast<uint16_t*>(lr_ + tg_at(r, k >> 3) + 2 * (k & 7)) = static_cast<uint16_t>(ra[i][v >> 1] >> (16 * (v & 1)));
        }
      }
      if constexpr (!CKM) {
        *reinterpret_cast<u32x4*>(lc_ + tg_at(q >> 3, q & 7)) = rb[i];
      } else {
#pragma unroll
        for (int v = 0; v < 8; ++v) {
          const int k = q >> 4, r = (q & 15) * 8 + v;
          *reinterpret_cast<uint16_t*>(lc_ + tg_at(r, k >> 3) + 2 * (k & 7)) = static_cast<uint16_t>(rb[i][v >> 1] >> (16 * (v & 1)));
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      u32x4 fc[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // gated: tiles 0, 1 are gate columns, 2, 3 the same columns of up
        const int ct = GATED ? (j < 2 ? 32 * wc + 16 * j : 64 + 32 * wc + 16 * (j - 2)) : 64 * wc + 16 * j;
        fc[j] = *reinterpret_cast<const u32x4*>(lc_ + tg_at(ct + lr, 4 * s + lg));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const u32x4 fr = *reinterpret_cast<const u32x4*>(lr_ + tg_at(64 * wr + 16 * i + lr, 4 * s + lg));
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = TT::mfma(fc[j], fr, acc[i][j]);
      }
    }
  }

  // lane: output row lr of a 16-row tile, columns 4 lg .. 4 lg + 3 of a 16-column tile
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 64 * wr + 16 * i + lr;
    if (r >= rows) continue;
    const int64_t orow = L == TG_TN ? static_cast<int64_t>(e) * p.R + m0 + r : static_cast<int64_t>(row0) + m0 + r;
    float sa = 1.0f;
    if constexpr (T == TG_I8) sa = p.sa[src_row(m0 + r)];
#pragma unroll
    for (int j = 0; j < (GATED ? 2 : 4); ++j) {
      const int c = c0 + (GATED ? 32 * wc : 64 * wc) + 16 * j + 4 * lg;
      if (c >= (GATED ? half : p.N)) continue;
      float4v v, w;
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = static_cast<float>(acc[i][j][q]);
      if constexpr (T == TG_I8) v = v * (*reinterpret_cast<const float4v*>(p.sb + static_cast<size_t>(e) * p.N + c) * sa);
      if constexpr (GATED) {
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] = static_cast<float>(acc[i][j + 2][q]);
        if constexpr (T == TG_I8) w = w * (*reinterpret_cast<const float4v*>(p.sb + static_cast<size_t>(e) * p.N + half + c) * sa);
        if (p.gu) {
          *reinterpret_cast<float4v*>(p.gu + orow * p.N + c) = v;
          *reinterpret_cast<float4v*>(p.gu + orow * p.N + half + c) = w;
        }
        float4v h;
#pragma unroll
        for (int q = 0; q < 4; ++q) h[q] = tg_act(v[q], p.act) * w[q];
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + orow * half + c) = TT::pack(h);
      } else if constexpr (EPI == TG_OUT_F32) {
        *reinterpret_cast<float4v*>(static_cast<float*>(p.out) + orow * p.N + c) = v;
      } else {
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + orow * p.N + c) = TT::pack(v);
      }
    }
  }
}

template <int T, int L, int EPI>
static hipError_t tg_launch(TileParams p, hipStream_t stream) {
  const int cols = EPI == TG_OUT_GATED ? p.N / 2 : p.N;
  const int bn = EPI == TG_OUT_GATED ? kTgBN / 2 : kTgBN;
  p.n_tiles = (cols + bn - 1) / bn;
  p.r_tiles = (p.R + kTgBM - 1) / kTgBM;
  int64_t blocks;
  if (L == TG_TN) {
    blocks = static_cast<int64_t>(p.E) * p.r_tiles * p.n_tiles;
  } else {
    // at most min(E, m_total) experts have rows, each with one partial chunk
    const int64_t chunks = p.m_total / kTgBM + (p.E < p.m_total ? p.E : p.m_total);
    blocks = (chunks * p.n_tiles + 7) / 8 * 8;
  }
  if (blocks >= (int64_t(1) << 31)) return hipErrorInvalidConfiguration;
  if (blocks == 0) return hipSuccess;
  hipLaunchKernelGGL((k_tile_gemm<T, L, EPI>), dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream, p);
  return hipGetLastError();
}

template <int T>
static hipError_t tg_launch16(const TileParams& p, int layout, int epilogue, hipStream_t stream) {
  if (layout == TG_NT)
    return epilogue == TG_OUT_GATED ? tg_launch<T, TG_NT, TG_OUT_GATED>(p, stream)
           : epilogue == TG_OUT_F32 ? tg_launch<T, TG_NT, TG_OUT_F32>(p, stream)
                                    : tg_launch<T, TG_NT, TG_OUT_16>(p, stream);
  if (layout == TG_NN) return tg_launch<T, TG_NN, TG_OUT_16>(p, stream);
  return tg_launch<T, TG_TN, TG_OUT_16>(p, stream);
}

}  // namespace nvfp4
