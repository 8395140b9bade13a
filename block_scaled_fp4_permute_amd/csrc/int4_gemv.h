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
// float32, sums and scales are float32; the offset of 16 costs about three bits of
// the sum's 24 (of weights scaled by absmax / 7 the codes less 8 have an rms of 2.6,
// 16 + q one of 24), against the 8 or 11 that a 16-bit result keeps.
//
// A wave takes 256 codes (128 bytes) of 16 weight rows at a time where registers
// allow: loads of 64 bytes a row reach 3.6 TB/s from memory (non-temporal, 4 loads in
// flight), of 128 bytes 6.6, as contiguous ones do.  A step is 128 codes.  With
// groups of 32 or 64 a lane's four dwords are transposed over the lane groups (two
// swaps each of 32 and 16 lanes), so that one matrix instruction takes 32
// neighbouring codes, of one group.  Within 8 codes the pairs are (i, i + 4), as
// the shifts give them; x is permuted alike.
//
// Reached: 256 experts, 2 rows each, 6144 -> 2 x 256 (417 MB) 67 to 75 us, 5.6 to 6.2
// TB/s; 8 rows each, 256 -> 6144 (240 MB) 55 to 58, 4.2; one token (13 MB) 9.
#pragma once

#include <type_traits>

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
  static __device__ __forceinline__ uint32_t shift(uint32_t w) { return P == 0 ? w << 3 : w >> (4 * P - 3); }   // codes P and P + 4
  static __device__ __forceinline__ float value(uint16_t b) { return bf16_to_f32(b); }
};
template <>
struct I4Type<true> {
  using TT = TgType<TG_F16>;
  static constexpr uint32_t mask = 0x03C003C0u, base = 0x4C004C00u;
  static constexpr uint32_t one = 0x3C003C00u, minus24 = 0xCE00CE00u;
  template <int P>
  static __device__ __forceinline__ uint32_t shift(uint32_t w) { return P < 2 ? w << (6 - 4 * P) : w >> (4 * P - 6); }
  static __device__ __forceinline__ float value(uint16_t b) { return static_cast<float>(__builtin_bit_cast(_Float16, b)); }
};

// 8 codes -> 16 + q in pairs (i, i + 4).  mask and base are in registers that the
// compiler takes for variables: as constants they would not fit one and-or.
template <class I4>
__device__ __forceinline__ u32x4 i4_decode(uint32_t w, uint32_t mask, uint32_t base) {
  return u32x4{(I4::template shift<0>(w) & mask) | base, (I4::template shift<1>(w) & mask) | base,
               (I4::template shift<2>(w) & mask) | base, (I4::template shift<3>(w) & mask) | base};
}

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
// the reduction, in blocks of `bs` steps, `ahead` blocks of codes on their way.
struct Int4Shape {
  int rt, ct, wk, wc, bs, ahead;
};
constexpr Int4Shape kI4Shapes[] = {{1, 2, 8, 1, 2, 3}, {1, 4, 4, 1, 2, 1}, {1, 4, 1, 4, 2, 1}, {2, 2, 1, 4, 2, 1}, {1, 1, 8, 1, 2, 3}};

static inline int i4_tiles(const Int4Shape& s, int N, int gated) {
  const int width = gated ? N / 2 : N, per = (gated ? 8 : 16) * s.ct * s.wc;
  return (width + per - 1) / per;
}
// Which of them, by the length of the reduction, rows of one expert (the hint, or what
// m_total gives each expert that can have any) and tasks.
//   2  reductions of up to 512: a wave's own, over several column groups (256 experts, 8
//      rows, 256 -> 6144: 54 us; 217 in shape 1)
//   3  and two row tiles a wave above 16 rows (256 experts, 256 -> 6144: 32 rows 75 us
//      against 101, 128 rows 255 against 403); longer reductions stay with 16 rows a
//      workgroup, and the chunks of an expert read its weights at about the same time,
//      from L2 (6144 -> 2 x 256, 64 rows: 359 us; two row tiles 444, four 433)
//   1  four tiles a wave from a workgroup a CU on (64 tokens, 6144 -> 2 x 256: 67 us
//      against 128 in shape 0; 4 tokens 15 against 21)
//   0  else, twice the waves for the same columns (2 tokens: 12 us against 15; dense
//      8192 x 8192, 3 rows: 16 against 22)
//   4  and one tile a wave where even those leave CUs without a workgroup (one token:
//      9.3 us against 10.6; 2 tokens 16.0 against 11.8)
static inline int i4_choice(int E, int N, int K, int64_t m_total, int64_t hint, int gated) {
  const int64_t experts = E < m_total ? E : m_total;
  const int64_t share = experts ? (m_total + experts - 1) / experts : 0;
  if (K <= 512) return (hint > share ? hint : share) > 16 ? 3 : 2;
  if (experts * i4_tiles(kI4Shapes[1], N, gated) >= 256) return 1;
  return experts * i4_tiles(kI4Shapes[0], N, gated) >= 256 ? 0 : 4;
}
// Column groups of a wave, one after the other (short reductions): some 2048
// workgroups (256 experts, 8 rows, 256 -> 6144, before other steps: 63 us; 70 with 1024 of
// them, 80 with 8192)
static inline int i4_rounds(const Int4Shape& s, int E, int N, int64_t m_total, int gated) {
  if (s.wk > 1) return 1;
  const int64_t chunks = m_total / (16 * s.rt) + (E < m_total ? E : m_total);
  const int64_t n = chunks * i4_tiles(s, N, gated) / 2048;
  return n < 1 ? 1 : n > 16 ? 16 : static_cast<int>(n);
}
// workgroups: at least one for each task (i4_find)
static inline int64_t i4_blocks(const Int4Shape& s, int E, int N, int64_t m_total, int gated) {
  const int64_t chunks = m_total / (16 * s.rt) + (E < m_total ? E : m_total);
  const int rounds = i4_rounds(s, E, N, m_total, gated);
  return (chunks * ((i4_tiles(s, N, gated) + rounds - 1) / rounds) + 7) / 8 * 8;
}

// inclusive prefix sum over the 64 lanes
__device__ __forceinline__ int i4_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);      // row_shr:1, zeros shifted in
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);
  const int r0 = __builtin_amdgcn_readlane(v, 15), r1 = __builtin_amdgcn_readlane(v, 31), r2 = __builtin_amdgcn_readlane(v, 47);
  const int row = (threadIdx.x & 63) >> 4;
  return v + (row > 0 ? r0 : 0) + (row > 1 ? r1 : 0) + (row > 2 ? r2 : 0);
}

// The task of workgroup blockIdx.x: a chunk of MC rows of an expert and a column
// tile.  Tasks are numbered by chunk, then column tile, and each XCD (workgroups go
// round them in turn) gets a contiguous eighth, so that the tiles of a chunk share
// its rows in one L2.  Every wave finds its task on its own from the offsets, 4
// experts a lane.  row0: the chunk's first row, rows: how many.  False where the
// workgroup has none.  Offsets are clamped, so that inconsistent ones give wrong
// rows, never an access out of bounds.
template <int MC>
__device__ __forceinline__ bool i4_find(const Int4Params& p, int& e_out, int& row0, int& rows, int& nt) {
  const int lane = threadIdx.x & 63;
  int at[5], c[4], incl = 0, sum = 0;
  auto group = [&](int g0) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 5; ++i) at[i] = min(max(p.offsets[min(g0 + 4 * lane + i, p.E)], 0), p.m_total);
    sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = (max(at[i + 1] - at[i], 0) + MC - 1) / MC;
      sum += c[i];
    }
    incl = i4_scan(sum);
  };
  int64_t total = 0;
  for (int g0 = 0; g0 < p.E; g0 += 256) {
    group(g0);
    total += __builtin_amdgcn_readlane(incl, 63);
  }
  total = total * p.n_tiles;
  const int64_t per = (total + 7) >> 3;
  const int64_t id = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if ((blockIdx.x >> 3) >= per || id >= total) return false;
  int chunk = static_cast<int>(static_cast<uint32_t>(id) / static_cast<uint32_t>(p.n_tiles));
  nt = static_cast<int>(id) - chunk * p.n_tiles;
  int g0 = 0;
  if (p.E > 256) {
    for (;; g0 += 256) {
      group(g0);
      const int n = __builtin_amdgcn_readlane(incl, 63);
      if (chunk < n || g0 + 256 >= p.E) break;
      chunk -= n;
    }
  }
  const uint64_t have = __ballot(incl > chunk);
  const int who = have ? __builtin_ctzll(have) : 63;
  int m = chunk - (incl - sum), e = g0 + 4 * lane, r = at[0], end = at[1];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const bool on = e == g0 + 4 * lane + i && m >= c[i];
    m -= on ? c[i] : 0;
    e += on ? 1 : 0;
    r = on ? at[i + 1] : r;
    end = on ? at[i + 2] : end;
  }
  m = __builtin_amdgcn_readlane(m, who);
  e_out = __builtin_amdgcn_readlane(e, who);
  row0 = __builtin_amdgcn_readlane(r, who) + m * MC;
  rows = min(MC, __builtin_amdgcn_readlane(end, who) - row0);
  return e_out < p.E && m >= 0 && rows > 0;
}

// rows of 16 lanes r0 .. r3 -> four values that hold row i in every row
__device__ __forceinline__ void i4_spread(uint32_t v, uint32_t (&out)[4]) {
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);         // r0 r0 r2 r2, r1 r1 r3 r3
  const auto b = __builtin_amdgcn_permlane32_swap(a[0], a[0], false, false);
  const auto c = __builtin_amdgcn_permlane32_swap(a[1], a[1], false, false);
  out[0] = b[0];
  out[1] = c[0];
  out[2] = b[1];
  out[3] = c[1];
}

template <bool F16, int GROUP, bool ZEROS, int SHAPE>
__global__ __launch_bounds__(64 * kI4Shapes[SHAPE].wk * kI4Shapes[SHAPE].wc) __attribute__((amdgpu_waves_per_eu(2)))
void k_int4_gemv(const Int4Params p, int gated, int out32) {
  using I4 = I4Type<F16>;
  using TT = typename I4::TT;
  constexpr int RT = kI4Shapes[SHAPE].rt, CT = kI4Shapes[SHAPE].ct, WK = kI4Shapes[SHAPE].wk, WC = kI4Shapes[SHAPE].wc;
  constexpr int BS = kI4Shapes[SHAPE].bs;
  constexpr int AHEAD = kI4Shapes[SHAPE].ahead;
  constexpr bool LOOP = WK == 1;
  constexpr bool TR = GROUP < kI4Step;
  constexpr int GS = kI4Step / GROUP;                       // groups of a step
  constexpr int MS = 4 / GS;                                // matrix instructions of a group
  // A lane group holds scales of one tile and step, or of one tile and all steps of a
  // block; they are spread over the groups in registers.
  constexpr bool ALL = CT == 4;
  constexpr int PAIRS = ALL ? 4 : CT * BS, SN = ALL ? BS * GS : GS, SW = (SN + 1) / 2, ZW = (SN + 3) / 4;
  constexpr int LPR = 4 * BS, RPL = 64 / LPR;               // lanes of a row's load, rows of a load
  constexpr int LD = 16 * CT + 4;                           // floats of a row of partial sums
  static_assert(PAIRS <= 4, "four lane groups");
  static_assert(!LOOP || AHEAD == 1, "a block of the next columns");
  __shared__ float red[WK][WC][16 * RT][LD];
  __shared__ u32x4 stage[WK * WC][CT][64 * BS];
  static_assert(fits_lds(sizeof(red) + sizeof(stage), 1), "partial sums and stages exceed the LDS of a CU");
  int e, row0, rows, nt;
  if (!i4_find<16 * RT>(p, e, row0, rows, nt)) return;
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wk = wave % WK, wc = wave / WK;
  const int cols = gated ? 8 : 16;                          // output columns of a tile
  const int width = gated ? p.N / 2 : p.N;
  const int K = p.K;
  const int groups = K / GROUP;
  const int steps = (K + kI4Step - 1) / kI4Step;
  const int per = (steps + WK - 1) / WK;
  const int first = wk * per, last = min(first + per, steps);

  // Codes are read as memory has them, neighbouring lanes 64 BS bytes of a row (lanes
  // as the matrix instruction wants them would touch a line each), and change lanes
  // by way of LDS: chunk c of row r at place c ^ f(r), so that neither side meets a
  // bank twice.
  auto swizzle = [](int r) __attribute__((always_inline)) { return BS == 2 ? (r >> 1) & 7 : (r >> 2) & 3; };
  u32x4* const put = &stage[wave][0][lane];
  const u32x4* const get = &stage[wave][0][LPR * lr];
  // Weights: the wave's first row as a base, 32-bit offsets of the lane's from there
  // (gated: the caller keeps the up half's below 2^32; scales have a quarter of the
  // codes' bytes at most).
  const int pair = lg & (PAIRS - 1);
  const uint8_t *qb, *sb, *zb;
  uint32_t qo[CT][BS], so;
  auto columns = [&](int c0) __attribute__((always_inline)) {             // the wave's first column
    const int cw = min(c0, width - 1);
    const int64_t n0 = static_cast<int64_t>(e) * p.N + cw;
    qb = p.codes + n0 * (K / 2);
    sb = static_cast<const uint8_t*>(p.scales) + n0 * groups * 2;
    zb = ZEROS ? p.zeros + n0 * groups : nullptr;
    auto row_of = [&](int j, int r) __attribute__((always_inline)) {
      return static_cast<uint32_t>(min(c0 + j * cols + (gated ? r & 7 : r), width - 1) - cw + (gated ? (r >> 3) * width : 0));
    };
#pragma unroll
    for (int j = 0; j < CT; ++j)
#pragma unroll
      for (int h = 0; h < BS; ++h) {
        const int r = h * RPL + lane / LPR;
        qo[j][h] = row_of(j, r) * static_cast<uint32_t>(K / 2) + 16 * ((lane % LPR) ^ swizzle(r));
      }
    so = row_of(pair % CT, lr) * static_cast<uint32_t>(groups) + (pair / CT) * GS;
  };

  uint32_t mask = I4::mask, base = I4::base;
  asm("" : "+v"(mask));
  asm("" : "+s"(base));
  const uint32_t c24 = ZEROS ? I4::one : I4::minus24;
  const u32x4 fixed = {c24, c24, c24, c24};

  struct Block {
    u32x4 w[CT][BS];
    uint32_t s[SW], z[ZW];
  };
  // codes and scales of steps [t, t + BS); beyond the wave's last or the end of the reduction scales are 0
  auto load_codes = [&](Block& f, int t) __attribute__((always_inline)) {
    const int k0 = t * kI4Step, g0 = t * GS;
#pragma unroll
    for (int i = 0; i < ZW; ++i) f.z[i] = 0;
    if (t + BS <= last && k0 + BS * kI4Step <= K) {
#pragma unroll
      for (int j = 0; j < CT; ++j)
#pragma unroll
        for (int h = 0; h < BS; ++h) {
          const u32x4* src = reinterpret_cast<const u32x4*>(qb + k0 / 2 + qo[j][h]);
          f.w[j][h] = RT == 1 ? __builtin_nontemporal_load(src) : *src;
        }
      if constexpr (SN == 1) f.s[0] = *reinterpret_cast<const uint16_t*>(sb + 2 * g0 + 2 * so);
      else __builtin_memcpy(f.s, sb + 2 * g0 + 2 * so, 2 * SN);
      if constexpr (ZEROS) {
        if constexpr (SN == 1) f.z[0] = zb[g0 + so];
        else __builtin_memcpy(f.z, zb + g0 + so, SN);
      }
    } else {
#pragma unroll
      for (int j = 0; j < CT; ++j)
#pragma unroll
        for (int h = 0; h < BS; ++h) {
          const uint32_t chunk = (lane % LPR) ^ swizzle(h * RPL + lane / LPR);
          const bool in = k0 + 32 * static_cast<int>(chunk) < K;
          f.w[j][h] = *reinterpret_cast<const u32x4*>(qb + (in ? k0 / 2 + qo[j][h] : qo[j][h] - 16 * chunk));   // behind the end any code
        }
      const int s0 = pair / CT * GS;                        // the lane's first group of the block
#pragma unroll
      for (int g = 0; g < SN; ++g) {
        const bool in = t + (s0 + g) / GS < last && g0 + s0 + g < groups;
        const uint32_t at = in ? g0 + g + so : so - s0;
        const uint32_t v = *reinterpret_cast<const uint16_t*>(sb + 2 * at);
        f.s[g / 2] = (g % 2 ? f.s[g / 2] : 0) | (in ? v << (16 * (g % 2)) : 0);
        if constexpr (ZEROS) f.z[g / 4] |= static_cast<uint32_t>(zb[at]) << (8 * (g % 4));
      }
    }
  };
  const uint8_t* x[RT];
  u32x4 xv[BS][RT][4];
  auto load_x = [&](int t) __attribute__((always_inline)) {
    const int k0 = t * kI4Step;
    if (k0 + BS * kI4Step <= K) {
#pragma unroll
      for (int b = 0; b < BS; ++b)
#pragma unroll
        for (int i = 0; i < RT; ++i)
          if (16 * i + lr < rows)
#pragma unroll
            for (int m = 0; m < 4; ++m)
              xv[b][i][m] = *reinterpret_cast<const u32x4*>(x[i] + 2 * (k0 + b * kI4Step) + (TR ? 64 : 16) * m);
    } else {
#pragma unroll
      for (int b = 0; b < BS; ++b)
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const int k = k0 + b * kI4Step + (TR ? 32 * m + 8 * lg : 32 * lg + 8 * m);
            xv[b][i][m] = u32x4{0, 0, 0, 0};
            if (k < K && 16 * i + lr < rows)
              xv[b][i][m] = *reinterpret_cast<const u32x4*>(x[i] + 2 * (k0 + b * kI4Step) + (TR ? 64 : 16) * m);
          }
    }
  };
  constexpr bool EARLY = RT == 1;            // x is asked for a block ahead, registers allowing
  float4v acc[RT][CT];
  auto products = [&](const u32x4 (&xp)[RT][4], int b, const uint32_t (&sq)[SW][4], const uint32_t (&zq)[ZW][4])
      __attribute__((always_inline)) {
    float4v off[RT][GS];
    auto offset = [&](int m) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < RT; ++i)
        off[i][m / MS] = TT::mfma(xp[i][m], fixed, m % MS ? off[i][m / MS] : float4v{0, 0, 0, 0});
    };
    if constexpr (RT == 1)                   // for two row tiles a group at a time: registers
#pragma unroll
      for (int m = 0; m < 4; ++m) offset(m);
    u32x4 c[CT];
#pragma unroll
    for (int j = 0; j < CT; ++j) {
      c[j] = get[64 * BS * j + ((4 * b + lg) ^ swizzle(lr))];
      if constexpr (TR) c[j] = i4_transpose(c[j]);
    }
    // the tiles' products in turn: neighbouring ones do not wait for each other
#pragma unroll
    for (int g = 0; g < GS; ++g) {
      if constexpr (RT > 1)
#pragma unroll
        for (int m = 0; m < MS; ++m) offset(g * MS + m);
      float4v d[RT][CT];
#pragma unroll
      for (int m = 0; m < MS; ++m)
#pragma unroll
        for (int j = 0; j < CT; ++j) {
          const u32x4 v = i4_decode<I4>(c[j][g * MS + m], mask, base);
#pragma unroll
          for (int i = 0; i < RT; ++i)
            d[i][j] = TT::mfma(xp[i][g * MS + m], v, m ? d[i][j] : ZEROS ? float4v{0, 0, 0, 0} : off[i][g]);
        }
#pragma unroll
      for (int j = 0; j < CT; ++j) {
        const int n = ALL ? b * GS + g : g, from = ALL ? j : b * CT + j;
        const float sg = I4::value(static_cast<uint16_t>(sq[n / 2][from] >> (16 * (n % 2))));
        const float zg = ZEROS ? -16.0f - static_cast<float>((zq[n / 4][from] >> (8 * (n % 4))) & 255u) : 0.0f;
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            float v = d[i][j][u];
            if constexpr (ZEROS) v = fmaf(zg, off[i][g][u], v);
            acc[i][j][u] = fmaf(sg, v, acc[i][j][u]);
          }
      }
    }
  };
  auto unpack = [&](const Block& f, uint32_t (&sq)[SW][4], uint32_t (&zq)[ZW][4]) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < CT; ++j)
#pragma unroll
      for (int h = 0; h < BS; ++h) put[64 * (BS * j + h)] = f.w[j][h];
#pragma unroll
    for (int h = 0; h < SW; ++h) i4_spread(f.s[h], sq[h]);
    if constexpr (ZEROS)
#pragma unroll
      for (int h = 0; h < ZW; ++h) i4_spread(f.z[h], zq[h]);
  };
  // a thread: 8 neighbouring columns of a row, the waves' sums added in their order
  auto result = [&](int r, int w, int piece, int c0) __attribute__((always_inline)) {
    const int c = c0 + piece * 8;
    if (c >= width) return;
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
    const int64_t to = (static_cast<int64_t>(row0) + r) * width + c;
    const uint2 lo = TT::pack(float4v{v[0], v[1], v[2], v[3]}), hi = TT::pack(float4v{v[4], v[5], v[6], v[7]});
    if (width % 8 == 0) {
      if (out32) {
        float4v* dst = reinterpret_cast<float4v*>(static_cast<float*>(p.out) + to);
        dst[0] = float4v{v[0], v[1], v[2], v[3]};
        dst[1] = float4v{v[4], v[5], v[6], v[7]};
      } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + to) = make_uint4(lo.x, lo.y, hi.x, hi.y);
      }
      return;
    }
    const uint32_t packed[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (c + u >= width) continue;
      if (out32) static_cast<float*>(p.out)[to + u] = v[u];
      else static_cast<uint16_t*>(p.out)[to + u] = static_cast<uint16_t>(packed[u / 2] >> (16 * (u % 2)));
    }
  };
  auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < CT; ++j) acc[i][j] = float4v{0, 0, 0, 0};
  };
  auto leave = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < CT; ++j)
#pragma unroll
        for (int u = 0; u < 4; ++u) red[wk][wc][16 * i + 4 * lg + u][16 * j + lr] = acc[i][j][u];
  };
  constexpr int kLog = CT == 4 ? 2 : CT == 2 ? 1 : 0;
  const int pieces = kLog + (gated ? 0 : 1);                // log2: of 8 columns, of a wave's columns
  clear();

  // column groups of the wave: one, or (short reductions) `rounds` of them
  const int tiles = (width + WC * CT * cols - 1) / (WC * CT * cols);
  const int it0 = LOOP ? nt * p.rounds : nt, it1 = LOOP ? min(it0 + p.rounds, tiles) : nt + 1;
  const bool one = LOOP && last - first <= BS;              // x of the whole reduction stays
  Block f[AHEAD];
#pragma unroll
  for (int b = 0; b < BS; ++b)
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int m = 0; m < 4; ++m) xv[b][i][m] = u32x4{0, 0, 0, 0};
  columns((it0 * WC + wc) * CT * cols);
  // the wave's next columns; whole ones lie alike
  auto advance = [&](int it) __attribute__((always_inline)) {
    const int c1 = (it + 1) * WC * CT * cols, step = WC * CT * cols;
    if (c1 <= width) {
      qb += static_cast<int64_t>(step) * (K / 2);
      sb += static_cast<int64_t>(step) * groups * 2;
      if constexpr (ZEROS) zb += static_cast<int64_t>(step) * groups;
    } else {
      columns((it * WC + wc) * CT * cols);
    }
  };
  if (first < last) load_codes(f[0], first);
  __builtin_amdgcn_sched_barrier(0);         // the codes first: x may hang on the rows' indices
  // places past the chunk's rows hold zeros or the first row again: nothing of theirs is written
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    int r = row0 + (16 * i + lr < rows ? 16 * i + lr : 0);
    if (p.a_rows) {
      r = p.a_rows[r];
      r = (r >= 0 && r < p.src_rows) ? r : 0;
    }
    x[i] = static_cast<const uint8_t*>(p.a) + static_cast<int64_t>(r) * K * 2 + (TR ? 16 : 64) * lg;
  }
  if (EARLY && first < last) load_x(first);
#pragma unroll
  for (int d = 1; d < AHEAD; ++d)
    if (first + d * BS < last) load_codes(f[d], first + d * BS);
  u32x4 xp[BS][RT][4];
  for (int it = it0; it < it1; ++it) {
    const int c0 = (it * WC + wc) * CT * cols;
    for (int t0 = first; t0 < last; t0 += AHEAD * BS) {
#pragma unroll
      for (int d = 0; d < AHEAD; ++d) {
        const int t = t0 + d * BS;
        if (t >= last) break;
        // the block leaves the registers that the next one's loads come into
        uint32_t sq[SW][4], zq[ZW][4];
        unpack(f[d], sq, zq);
        if (!one || it == it0) {
          if constexpr (!EARLY) load_x(t);
#pragma unroll
          for (int b = 0; b < BS; ++b)
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
              for (int m = 0; m < 4; ++m) xp[b][i][m] = i4_pairs(xv[b][i][m]);
        }
        __builtin_amdgcn_sched_barrier(0);
        if (EARLY && t + BS < last) load_x(t + BS);
        if (t + AHEAD * BS < last) {
          load_codes(f[d], t + AHEAD * BS);
        } else if (LOOP && it + 1 < it1) {
          advance(it + 1);
          load_codes(f[d], first);
          if (EARLY && !one) load_x(first);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int b = 0; b < BS; ++b) products(xp[b], b, sq, zq);
      }
    }
    leave();
    if constexpr (LOOP) {
      // the sums are the wave's own
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
      for (int o = lane; o < rows << pieces; o += 64) result(o >> pieces, wc, o & ((1 << pieces) - 1), c0);
      clear();
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
    } else {
      __syncthreads();
      for (int o = threadIdx.x; o < WC * rows << pieces; o += 64 * WK * WC) {
        const int w = (o >> pieces) % WC;
        result((o >> pieces) / WC, w, o & ((1 << pieces) - 1), (it * WC + w) * CT * cols);
      }
    }
  }
}

template <bool F16, int GROUP, bool ZEROS, int SHAPE>
static hipError_t i4_start(Int4Params p, int gated, int out32, hipStream_t stream) {
  constexpr Int4Shape shape = kI4Shapes[SHAPE];
  p.rounds = i4_rounds(shape, p.E, p.N, p.m_total, gated);
  p.n_tiles = (i4_tiles(shape, p.N, gated) + p.rounds - 1) / p.rounds;
  const int64_t blocks = i4_blocks(shape, p.E, p.N, p.m_total, gated);
  if (blocks == 0) return hipSuccess;
  hipLaunchKernelGGL((k_int4_gemv<F16, GROUP, ZEROS, SHAPE>), dim3(static_cast<unsigned>(blocks)), dim3(64 * shape.wk * shape.wc), 0,
                     stream, p, gated, out32);
  return hipGetLastError();
}

template <bool F16, int GROUP, bool ZEROS>
static hipError_t i4_launch(const Int4Params& p, int gated, int out32, hipStream_t stream) {
  switch (i4_choice(p.E, p.N, p.K, p.m_total, p.rows_hint, gated)) {
    case 0: return i4_start<F16, GROUP, ZEROS, 0>(p, gated, out32, stream);
    case 1: return i4_start<F16, GROUP, ZEROS, 1>(p, gated, out32, stream);
    case 2: return i4_start<F16, GROUP, ZEROS, 2>(p, gated, out32, stream);
    case 3: return i4_start<F16, GROUP, ZEROS, 3>(p, gated, out32, stream);
    default: return i4_start<F16, GROUP, ZEROS, 4>(p, gated, out32, stream);
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
