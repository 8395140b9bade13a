// The forward products (NT in tile_gemm.h) where their tiles are too few for the
// chip: single tokens, and dense products of some hundred rows.  No LDS staging:
// every lane loads its fragments straight from the row-major operands (16 bytes;
// a wave's two loads of a piece cover 128 bytes of 16 rows).
//
// A task is 16 RT rows of an expert times WC x CT column tiles of 16 weight rows
// (gated: 8 of gate and the 8 of up for the same columns, so that one token's
// experts make twice as many tasks).  WK waves share the tiles and take every
// WK-th 128-byte piece of the reduction, so that together they read contiguous
// memory and few rows still keep a chip's worth of loads in flight; their sums
// meet in LDS and are added in the order of the waves.  Bound by the weights'
// stream and, for one token, by the launch: 8 experts' 6144 -> 2 x 256 in bf16
// (50 MB) take 13.6 us a call, 3.7 TB/s.
#pragma once

#include "tile_gemm.h"

namespace nvfp4 {

constexpr int kSkPiece = 128;              // bytes of k per wave and turn: two matrix instructions a tile

template <int T, int EPI, int RT, int CT, int WK, int WC>
__global__ __launch_bounds__(64 * WK * WC) __attribute__((amdgpu_waves_per_eu(2))) void k_skinny_gemm(const TileParams p) {
  using TT = TgType<T>;
  using acc_t = typename TT::acc_t;
  constexpr int EB = TT::bytes;
  constexpr bool GATED = EPI == TG_OUT_GATED;
  constexpr int COLS = GATED ? 8 : 16;                      // output columns of a tile
  constexpr int TURNS = RT == 1 ? 6 : 3;                    // pieces loaded ahead: what the registers hold
  __shared__ acc_t red[WK][WC][RT * CT][64];
  static_assert(fits_lds(sizeof(red), 1), "partial sums exceed the LDS of a CU");
  int e, m0, nt;
  bool narrow;
  {
    GemmParams map{};
    map.offsets = p.offsets;
    map.E = p.E;
    map.m_total = p.m_total;
    map.n_tiles = p.n_tiles;
    map.slots = 1 << 30;
    if (!find_task<RT, false, 0>(map, e, m0, nt, narrow)) return;
  }
  const int row0 = min(max(p.offsets[e], 0), p.m_total);
  const int rows = min(16 * RT, min(max(p.offsets[e + 1], 0), p.m_total) - row0 - m0);
  if (rows <= 0 || m0 < 0) return;          // offsets that overlap so far that the task count does not fit
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wk = wave % WK, wc = wave / WK;
  const int width = GATED ? p.N / 2 : p.N;                  // columns of the output
  const int c0 = nt * (WC * CT * COLS);                     // of the task
  const int64_t kb = static_cast<int64_t>(p.K) * EB;        // bytes of a row
  auto src_row = [&](int r) __attribute__((always_inline)) -> int64_t {
    if (p.a_rows) {
      r = p.a_rows[r];
      r = (r >= 0 && r < p.src_rows) ? r : 0;
    }
    return r;
  };
  const uint8_t* a[RT];
  const uint8_t* b[CT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
    a[i] = static_cast<const uint8_t*>(p.a) + src_row(row0 + m0 + (16 * i + lr < rows ? 16 * i + lr : 0)) * kb + 16 * lg;
#pragma unroll
  for (int j = 0; j < CT; ++j) {
    const int wrow = min(c0 + (wc * CT + j) * COLS + (lr % COLS), width - 1) + (lr >= COLS ? width : 0);
    b[j] = static_cast<const uint8_t*>(p.b) + (static_cast<int64_t>(e) * p.N + wrow) * kb + 16 * lg;
  }
  acc_t acc[RT][CT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < CT; ++j) acc[i][j] = acc_t{0, 0, 0, 0};
  const int pieces = static_cast<int>((kb + kSkPiece - 1) / kSkPiece);
  for (int q0 = wk; q0 < pieces; q0 += WK * TURNS) {
    u32x4 fa[TURNS][2][RT], fb[TURNS][2][CT];
#pragma unroll
    for (int i = 0; i < TURNS; ++i)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int64_t o = static_cast<int64_t>(q0 + i * WK) * kSkPiece + 64 * s;
        const bool in = o + 16 * lg < kb;                   // zeros behind the end of the reduction
#pragma unroll
        for (int j = 0; j < CT; ++j) {
          fb[i][s][j] = u32x4{0, 0, 0, 0};
          // 16 rows: a weight is read once
          if (in && RT == 1) fb[i][s][j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(b[j] + o));
          if (in && RT > 1) fb[i][s][j] = *reinterpret_cast<const u32x4*>(b[j] + o);
        }
#pragma unroll
        for (int j = 0; j < RT; ++j) {
          fa[i][s][j] = u32x4{0, 0, 0, 0};
          if (in) fa[i][s][j] = *reinterpret_cast<const u32x4*>(a[j] + o);
        }
      }
#pragma unroll
    for (int i = 0; i < TURNS; ++i)
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int j = 0; j < CT; ++j) acc[r][j] = TT::mfma(fb[i][s][j], fa[i][s][r], acc[r][j]);
  }
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < CT; ++j) red[wk][wc][i * CT + j][lane] = acc[i][j];
  __syncthreads();

  // one thread per 4 neighbouring columns of a row; gated: lane groups 0, 1 hold
  // gate columns, 2, 3 the same of up
  for (int o = threadIdx.x; o < WC * RT * CT * 64; o += 64 * WK * WC) {
    const int w = o / (RT * CT * 64), ij = (o >> 6) % (RT * CT), l = o & 63;
    if (GATED && l >= 32) continue;
    const int r = 16 * (ij / CT) + (l & 15);
    const int c = c0 + (w * CT + ij % CT) * COLS + 4 * (l >> 4);
    if (r >= rows || c >= width) continue;
    acc_t sv = red[0][w][ij][l], sw = {0, 0, 0, 0};
    if constexpr (GATED) sw = red[0][w][ij][l + 32];
#pragma unroll
    for (int k = 1; k < WK; ++k) {
      sv += red[k][w][ij][l];
      if constexpr (GATED) sw += red[k][w][ij][l + 32];
    }
    float4v v, g;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[q] = static_cast<float>(sv[q]);
      g[q] = static_cast<float>(sw[q]);
    }
    const int64_t orow = static_cast<int64_t>(row0) + m0 + r;
    if constexpr (T == TG_I8) {
      const float sa = p.sa[src_row(row0 + m0 + r)];
      const float* sb = p.sb + static_cast<size_t>(e) * p.N + c;
      v = v * (*reinterpret_cast<const float4v*>(sb) * sa);
      if constexpr (GATED) g = g * (*reinterpret_cast<const float4v*>(sb + width) * sa);
    }
    if constexpr (GATED) {
      if (p.gu) {
        *reinterpret_cast<float4v*>(p.gu + orow * p.N + c) = v;
        *reinterpret_cast<float4v*>(p.gu + orow * p.N + width + c) = g;
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = tg_act(v[q], p.act) * g[q];
    }
    if constexpr (EPI == TG_OUT_F32)
      *reinterpret_cast<float4v*>(static_cast<float*>(p.out) + orow * p.N + c) = v;
    else
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + orow * width + c) = TT::pack(v);
  }
}

template <int T, int EPI, int RT, int CT, int WK, int WC>
static hipError_t sk_start(TileParams p, hipStream_t stream) {
  const int width = EPI == TG_OUT_GATED ? p.N / 2 : p.N;
  const int per = (EPI == TG_OUT_GATED ? 8 : 16) * CT * WC;
  p.n_tiles = (width + per - 1) / per;
  const int64_t chunks = p.m_total / (16 * RT) + (p.E < p.m_total ? p.E : p.m_total);
  const int64_t blocks = (chunks * p.n_tiles + 7) / 8 * 8;
  if (blocks >= (int64_t(1) << 31)) return hipErrorInvalidConfiguration;
  if (blocks == 0) return hipSuccess;
  hipLaunchKernelGGL((k_skinny_gemm<T, EPI, RT, CT, WK, WC>), dim3(static_cast<unsigned>(blocks)), dim3(64 * WK * WC), 0, stream, p);
  return hipGetLastError();
}

// `rows` of one expert.  8 waves on one set of columns; 16 rows of 1 KB and less
// (8 pieces): pairs of waves
template <int T, int EPI>
static hipError_t sk_launch(const TileParams& p, int64_t rows, hipStream_t stream) {
  const bool deep = static_cast<int64_t>(p.K) * TgType<T>::bytes > 8 * kSkPiece;
  if (rows <= 16) return deep ? sk_start<T, EPI, 1, 1, 8, 1>(p, stream) : sk_start<T, EPI, 1, 1, 2, 4>(p, stream);
  if (rows <= 32) return sk_start<T, EPI, 2, 2, 8, 1>(p, stream);
  return sk_start<T, EPI, 4, 2, 8, 1>(p, stream);
}

// ------------------------------------------------------------------ choice of the kernel
// From the sizes alone: rows of one expert (the hint, or what m_total gives each
// expert that can have any) and the tiles they make.
//   forward, up to 32 rows and fewer than 256 tiles of 128 x 128 (half the chip's
//     slots), or so few rows and columns that 64 x 32 tiles are one round of
//     workgroups: the kernel above (17 rows, 5632 -> 2048: 19 us against 48 on
//     tiles; 256 rows, 256 tasks: 35 against 48; 100 rows of 2048 -> 5632, 352
//     tasks: 29 against 20, so tiles)
//   forward, up to 32 rows and 1 KB of reduction (8 steps): 64 x 128 tiles, three
//     workgroups a CU (256 experts, 8 rows, int8 256 -> 6144: 90 us against 112 on
//     128 x 128; bf16 256 -> 6144 161 against 166; 32 rows, int8 512 -> 2048 50
//     against 58; longer ones level off, bf16 1024 -> 2048 206 against 203, and
//     64 rows lose, bf16 256 -> 6144 209 against 196)
//   192 rows of output and at least 128 tiles of 256 x 256: those, with half the
//     operand traffic a product (512 rows an expert, 512 -> 6144 row gradient:
//     995 us against 1270 on 128 x 128 tiles; 512 rows of 2048 -> 2 x 5632, 88
//     tiles: 50 us against 33, so 128 x 128)
//   else 128 x 128, two workgroups a CU
template <int T, int L, int EPI>
static hipError_t tg_launch(const TileParams& p, hipStream_t stream) {
  constexpr bool WEIGHT = L == TG_TN || L == TG_TC;
  constexpr bool GATED = EPI == TG_OUT_GATED;
  const int64_t experts = WEIGHT ? p.E : (p.E < p.m_total ? p.E : p.m_total);
  if (experts == 0) return hipSuccess;
  const int64_t share = (p.m_total + experts - 1) / experts;
  const int64_t rows = WEIGHT ? p.R : (p.rows_hint > share ? p.rows_hint : share);
  const int64_t width = GATED ? p.N / 2 : p.N;
  auto tiles = [&](int64_t bm, int64_t bn) { return experts * ((rows + bm - 1) / bm) * ((width + bn - 1) / bn); };
  if constexpr (L == TG_NT) {
    if ((rows <= 32 && tiles(128, GATED ? 64 : 128) < 256) || tiles(64, GATED ? 16 : 32) <= 256)
      return sk_launch<T, EPI>(p, rows, stream);
  }
  if constexpr (L == TG_NT) {
    if (rows <= 32 && p.E <= tg_most_experts(64) && static_cast<int64_t>(p.K) * TgType<T>::bytes <= 1024)
      return tg_start<T, L, EPI, 64, 128, 1, 2>(p, stream);
  }
  if constexpr (!(WEIGHT && EPI == TG_OUT_PART)) {
    if (rows >= 192 && tiles(256, GATED ? 128 : 256) >= 128) return tg_start<T, L, EPI, 256, 256, 2, 4>(p, stream);
  }
  return tg_start<T, L, EPI, 128, 128, 2, 2>(p, stream);
}

template <int T>
static hipError_t tg_launch16(const TileParams& p, int layout, int epilogue, hipStream_t stream) {
  if (layout == TG_NT)
    return epilogue == TG_OUT_GATED ? tg_launch<T, TG_NT, TG_OUT_GATED>(p, stream)
           : epilogue == TG_OUT_F32 ? tg_launch<T, TG_NT, TG_OUT_F32>(p, stream)
                                    : tg_launch<T, TG_NT, TG_OUT_16>(p, stream);
  if (layout == TG_NN)
    return epilogue == TG_OUT_PART ? tg_launch<T, TG_NN, TG_OUT_PART>(p, stream) : tg_launch<T, TG_NN, TG_OUT_16>(p, stream);
  if (layout == TG_TC)
    return epilogue == TG_OUT_PART ? tg_launch<T, TG_TC, TG_OUT_PART>(p, stream) : tg_launch<T, TG_TC, TG_OUT_16>(p, stream);
  return epilogue == TG_OUT_PART ? tg_launch<T, TG_TN, TG_OUT_PART>(p, stream) : tg_launch<T, TG_TN, TG_OUT_16>(p, stream);
}

}  // namespace nvfp4
