// Products of few rows with INT4 weights in groups along the reduction:
//   y[p, n] = sum_g s[n, g] sum_{k in g} (q[n, k] - z[n, g]) x[p, k]
// (z = 8 without zero points), rows grouped by expert, activations in 16 bits.
//
// Bound by the weights' stream (4 bits and the group's share of scale and zero
// point each), so the work on a weight has to stay under about 4 cycles of a SIMD
// a value.  A 4-bit code becomes the 16-bit float 16 + q by one shift and one
// and-or for two codes (16 + q has q in the top mantissa bits); the matrix
// instruction multiplies those with x, and what they are too large by comes off
// in the sum: a group's accumulator starts at -24 sum(x), made by the same
// instruction from a constant operand, once for all column tiles (with zero
// points: sum(x) times 16 + z comes off after the group).  Products are exact in
// float32, sums and scales are float32; the offset of 16 costs about two bits of
// the sum's 24.
//
// A wave's step is 128 codes of 16 weight rows: one 16-byte load a lane.  With
// groups of 32 or 64 the four dwords are transposed over the lane groups (two
// swaps each of 32 and 16 lanes), so that one matrix instruction takes 32
// neighbouring codes, of one group.  Within 8 codes the pairs are (i, i + 4), as
// the shifts give them; x is permuted alike in registers.
#pragma once

#include "tile_gemm.h"

namespace nvfp4 {

template <bool F16>
struct I4Type;
template <>
struct I4Type<false> {
  using TT = TgType<TG_BF16>;
  static constexpr uint32_t mask = 0x00780078u, base = 0x41804180u;     // bits of q, 16.0
  static constexpr uint32_t one = 0x3F803F80u, minus24 = 0xC1C0C1C0u;
  template <int P>
  static __device__ __forceinline__ uint32_t pair(uint32_t w) {          // codes P and P + 4
    const uint32_t s = P == 0 ? w << 3 : w >> (4 * P - 3);
    return (s & mask) | base;
  }
  static __device__ __forceinline__ float value(uint16_t b) { return bf16_to_f32(b); }
};
template <>
struct I4Type<true> {
  using TT = TgType<TG_F16>;
  static constexpr uint32_t mask = 0x03C003C0u, base = 0x4C004C00u;
  static constexpr uint32_t one = 0x3C003C00u, minus24 = 0xCE00CE00u;
  template <int P>
  static __device__ __forceinline__ uint32_t pair(uint32_t w) {
    const uint32_t s = P < 2 ? w << (6 - 4 * P) : w >> (4 * P - 6);
    return (s & mask) | base;
  }
  static __device__ __forceinline__ float value(uint16_t b) { return static_cast<float>(__builtin_bit_cast(_Float16, b)); }
};

// 8 values of x in memory order -> pairs (i, i + 4)
__device__ __forceinline__ u32x4 i4_pairs(u32x4 d) {
  u32x4 r;
  r[0] = __builtin_amdgcn_perm(d[2], d[0], 0x05040100u);
  r[1] = __builtin_amdgcn_perm(d[2], d[0], 0x07060302u);
  r[2] = __builtin_amdgcn_perm(d[3], d[1], 0x05040100u);
  r[3] = __builtin_amdgcn_perm(d[3], d[1], 0x07060302u);
  return r;
}

// dword j of lane group g  <->  dword g of lane group j
__device__ __forceinline__ u32x4 i4_transpose(u32x4 d) {
  typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
  const auto a = __builtin_amdgcn_permlane32_swap(d[0], d[2], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(d[1], d[3], false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const auto e = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return u32x4{c[0], c[1], e[0], e[1]};
}

constexpr int kI4Step = 128;               // codes of a weight row per wave and step

// Shapes of a workgroup: RT x 16 rows of an expert times WC x CT tiles of 16 weight
// rows (gated: 8 of gate and the 8 of up for the same columns), WK waves sharing
// the reduction.
struct Int4Shape {
  int rt, ct, wk, wc;
};
constexpr Int4Shape kI4Shapes[] = {{1, 1, 8, 1}, {1, 4, 1, 4}, {4, 2, 4, 1}};
#define I4_SHAPE(i) kI4Shapes[i].rt, kI4Shapes[i].ct, kI4Shapes[i].wk, kI4Shapes[i].wc

// which of them, by rows of one expert (the hint, or what m_total gives each expert
// that can have any) and the length of the reduction
static inline int i4_choice(int E, int N, int K, int64_t m_total, int64_t hint, int gated) {
  const int64_t experts = E < m_total ? E : m_total;
  const int64_t share = experts ? (m_total + experts - 1) / experts : 0;
  const int64_t rows = hint > share ? hint : share;
  if (rows > 16) return 2;
  return K <= 512 ? 1 : 0;
}
static inline int i4_tiles(const Int4Shape& s, int N, int gated) {
  const int width = gated ? N / 2 : N, per = (gated ? 8 : 16) * s.ct * s.wc;
  return (width + per - 1) / per;
}
// workgroups: at least one for each task (find_task)
static inline int64_t i4_blocks(const Int4Shape& s, int E, int N, int64_t m_total, int gated) {
  const int64_t chunks = m_total / (16 * s.rt) + (E < m_total ? E : m_total);
  return (chunks * i4_tiles(s, N, gated) + 7) / 8 * 8;
}

template <bool F16, int GROUP, bool ZEROS, int RT, int CT, int WK, int WC>
__global__ __launch_bounds__(64 * WK * WC) __attribute__((amdgpu_waves_per_eu(2))) void k_int4_gemv(const Int4Params p, int gated, int out32) {
  using I4 = I4Type<F16>;
  using TT = typename I4::TT;
  constexpr bool TR = GROUP < kI4Step;
  constexpr int GS = kI4Step / GROUP;                       // groups of a step
  constexpr int MS = 4 / GS;                                // matrix instructions of a group
  constexpr int TURNS = RT * CT <= 2 ? 4 : RT * CT <= 4 ? 2 : 1;   // steps loaded ahead
  constexpr int LD = 16 * CT + 4;                           // floats of a row of partial sums
  __shared__ float red[WK][WC][16 * RT][LD];
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
  const int cols = gated ? 8 : 16;                          // output columns of a tile
  const int width = gated ? p.N / 2 : p.N;
  const int c0 = nt * (WC * CT * cols);                     // of the task
  const int K = p.K;
  const int groups = K / GROUP;
  const uint8_t* x[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    int r = row0 + m0 + (16 * i + lr < rows ? 16 * i + lr : 0);
    if (p.a_rows) {
      r = p.a_rows[r];
      r = (r >= 0 && r < p.src_rows) ? r : 0;
    }
    x[i] = static_cast<const uint8_t*>(p.a) + static_cast<int64_t>(r) * K * 2;
  }
  const uint8_t* q[CT];
  const uint16_t* s[CT];
  const uint8_t* z[CT];
#pragma unroll
  for (int j = 0; j < CT; ++j) {
    const int at = (wc * CT + j) * cols + c0;
    const int wrow = gated ? min(at + (lr & 7), width - 1) + (lr >> 3) * width : min(at + lr, width - 1);
    const int64_t n = static_cast<int64_t>(e) * p.N + wrow;
    q[j] = p.codes + n * (K / 2) + 16 * lg;
    s[j] = static_cast<const uint16_t*>(p.scales) + n * groups;
    if constexpr (ZEROS) z[j] = p.zeros + n * groups;
  }
  float4v acc[RT][CT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < CT; ++j) acc[i][j] = float4v{0, 0, 0, 0};
  const int steps = (K + kI4Step - 1) / kI4Step;
  const int per = (steps + WK - 1) / WK;
  const int first = wk * per, last = min(first + per, steps);
  const u32x4 fixed = {ZEROS ? I4::one : I4::minus24, ZEROS ? I4::one : I4::minus24, ZEROS ? I4::one : I4::minus24,
                       ZEROS ? I4::one : I4::minus24};
  for (int t0 = first; t0 < last; t0 += TURNS) {
    u32x4 w[TURNS][CT];
    uint16_t sc[TURNS][CT][GS];
    uint8_t zp[TURNS][CT][GS];
    u32x4 xv[TURNS][RT][4];
#pragma unroll
    for (int t = 0; t < TURNS; ++t) {
      const int k0 = (t0 + t) * kI4Step;
      const bool in = t0 + t < last;
#pragma unroll
      for (int j = 0; j < CT; ++j) {
        w[t][j] = u32x4{0, 0, 0, 0};
        if (in && k0 + 32 * lg < K) {
          const u32x4* src = reinterpret_cast<const u32x4*>(q[j] + k0 / 2);
          w[t][j] = RT == 1 ? __builtin_nontemporal_load(src) : *src;
        }
#pragma unroll
        for (int g = 0; g < GS; ++g) {
          const int gi = k0 / GROUP + g;
          sc[t][j][g] = 0;
          zp[t][j][g] = 0;
          if (in && gi < groups) {
            sc[t][j][g] = s[j][gi];
            if constexpr (ZEROS) zp[t][j][g] = z[j][gi];
          }
        }
      }
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const int k = k0 + (TR ? 32 * m + 8 * lg : 32 * lg + 8 * m);
          xv[t][i][m] = u32x4{0, 0, 0, 0};
          if (in && k < K && 16 * i + lr < rows) xv[t][i][m] = *reinterpret_cast<const u32x4*>(x[i] + 2 * k);
        }
    }
#pragma unroll
    for (int t = 0; t < TURNS; ++t) {
      float4v off[RT][GS];
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          xv[t][i][m] = i4_pairs(xv[t][i][m]);
          off[i][m / MS] = TT::mfma(xv[t][i][m], fixed, m % MS ? off[i][m / MS] : float4v{0, 0, 0, 0});
        }
#pragma unroll
      for (int j = 0; j < CT; ++j) {
        const u32x4 c = TR ? i4_transpose(w[t][j]) : w[t][j];
#pragma unroll
        for (int g = 0; g < GS; ++g) {
          float4v d[RT];
#pragma unroll
          for (int i = 0; i < RT; ++i) d[i] = ZEROS ? float4v{0, 0, 0, 0} : off[i][g];
#pragma unroll
          for (int m = 0; m < MS; ++m) {
            const uint32_t v = c[g * MS + m];
            const u32x4 b = {I4::template pair<0>(v), I4::template pair<1>(v), I4::template pair<2>(v), I4::template pair<3>(v)};
#pragma unroll
            for (int i = 0; i < RT; ++i) d[i] = TT::mfma(xv[t][i][g * MS + m], b, d[i]);
          }
          const float sg = I4::value(sc[t][j][g]);
          const float zg = -16.0f - static_cast<float>(zp[t][j][g]);
#pragma unroll
          for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              float v = d[i][u];
              if constexpr (ZEROS) v = fmaf(zg, off[i][g][u], v);
              acc[i][j][u] = fmaf(sg, v, acc[i][j][u]);
            }
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < CT; ++j)
#pragma unroll
      for (int u = 0; u < 4; ++u) red[wk][wc][16 * i + 4 * lg + u][16 * j + lr] = acc[i][j][u];
  __syncthreads();

  // a thread: 8 neighbouring columns of a row, the waves' sums added in their order
  const int pieces = gated ? CT : 2 * CT;
  for (int o = threadIdx.x; o < WC * pieces * 16 * RT; o += 64 * WK * WC) {
    const int piece = o % pieces, w = o / pieces % WC, r = o / (pieces * WC);
    if (r >= rows) continue;
    const int c = c0 + (w * pieces + piece) * 8;
    if (c >= width) continue;
    const int at = gated ? 16 * piece : 8 * piece;
    float v[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float4v a = *reinterpret_cast<const float4v*>(&red[0][w][r][at + 4 * h]);
#pragma unroll
      for (int k = 1; k < WK; ++k) a += *reinterpret_cast<const float4v*>(&red[k][w][r][at + 4 * h]);
      if (gated) {
        float4v b = *reinterpret_cast<const float4v*>(&red[0][w][r][at + 8 + 4 * h]);
#pragma unroll
        for (int k = 1; k < WK; ++k) b += *reinterpret_cast<const float4v*>(&red[k][w][r][at + 8 + 4 * h]);
#pragma unroll
        for (int u = 0; u < 4; ++u) a[u] = tg_act(a[u], p.act) * b[u];
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) v[4 * h + u] = a[u];
    }
    const int64_t to = (static_cast<int64_t>(row0) + m0 + r) * width + c;
    const uint2 lo = TT::pack(float4v{v[0], v[1], v[2], v[3]}), hi = TT::pack(float4v{v[4], v[5], v[6], v[7]});
    if (width % 8 == 0) {
      if (out32) {
        float4v* dst = reinterpret_cast<float4v*>(static_cast<float*>(p.out) + to);
        dst[0] = float4v{v[0], v[1], v[2], v[3]};
        dst[1] = float4v{v[4], v[5], v[6], v[7]};
      } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + to) = make_uint4(lo.x, lo.y, hi.x, hi.y);
      }
      continue;
    }
    const uint32_t packed[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (c + u >= width) continue;
      if (out32) static_cast<float*>(p.out)[to + u] = v[u];
      else static_cast<uint16_t*>(p.out)[to + u] = static_cast<uint16_t>(packed[u / 2] >> (16 * (u % 2)));
    }
  }
}

template <bool F16, int GROUP, bool ZEROS, int RT, int CT, int WK, int WC>
static hipError_t i4_start(Int4Params p, int gated, int out32, hipStream_t stream) {
  constexpr Int4Shape shape = {RT, CT, WK, WC};
  p.n_tiles = i4_tiles(shape, p.N, gated);
  const int64_t blocks = i4_blocks(shape, p.E, p.N, p.m_total, gated);
  if (blocks == 0) return hipSuccess;
  hipLaunchKernelGGL((k_int4_gemv<F16, GROUP, ZEROS, RT, CT, WK, WC>), dim3(static_cast<unsigned>(blocks)), dim3(64 * WK * WC), 0,
                     stream, p, gated, out32);
  return hipGetLastError();
}

template <bool F16, int GROUP, bool ZEROS>
static hipError_t i4_launch(const Int4Params& p, int gated, int out32, hipStream_t stream) {
  switch (i4_choice(p.E, p.N, p.K, p.m_total, p.rows_hint, gated)) {
    case 0: return i4_start<F16, GROUP, ZEROS, I4_SHAPE(0)>(p, gated, out32, stream);
    case 1: return i4_start<F16, GROUP, ZEROS, I4_SHAPE(1)>(p, gated, out32, stream);
    default: return i4_start<F16, GROUP, ZEROS, I4_SHAPE(2)>(p, gated, out32, stream);
  }
}

template <bool F16>
static hipError_t i4_launch_type(const Int4Params& p, int group, int gated, int out32, hipStream_t stream) {
  if (p.zeros) {
    return group == 32 ? i4_launch<F16, 32, true>(p, gated, out32, stream)
         : group == 64 ? i4_launch<F16, 64, true>(p, gated, out32, stream)
                       : i4_launch<F16, 128, true>(p, gated, out32, stream);
  }
  return group == 32 ? i4_launch<F16, 32, false>(p, gated, out32, stream)
       : group == 64 ? i4_launch<F16, 64, false>(p, gated, out32, stream)
                     : i4_launch<F16, 128, false>(p, gated, out32, stream);
}

}  // namespace nvfp4
