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
  const float t = s * (1.0f - s);        // 0 far out, where the factor after it may overflow
  return t > 0.0f ? s + g * t * 1.5957691216057308f * (1.0f + 0.134145f * g2) : s;
}

constexpr int kTgStep = 128;                // a K step: 128 bytes of each K-contiguous row (64 rows of a K-major operand)

// ------------------------------------------------------------------ operand tiles in LDS
// A tile holds X rows or columns of an operand for one K step, X * 128 bytes,
// written by 16-byte direct-to-LDS loads: a wave's load fills 1024 contiguous
// bytes in lane order, so the layout's permutation is made by choosing which
// 16 bytes of memory each lane fetches.
//
// K-contiguous: row r is 128 bytes, its 16-byte chunk ch at chunk ch ^ ((r >> 1) & 7).
//   The 16 rows that a fragment read touches at one chunk cover all 64 banks.
// K-major: row k is 2 X bytes, its 32-byte unit u (16 values) at unit u ^ f(k),
//   f(k) = (k & 3) + 4 ((k >> 3) & 1): the 8 rows that half a wave's transposing
//   read touches (4 of lane groups 2q and 2q + 1 each) lie in distinct units.
typedef short s16x4 __attribute__((ext_vector_type(4)));
#define TG_LDS __attribute__((address_space(3)))

// zeros for the parts of a step behind the end of the reduction
__device__ const u32x4 tg_zero = {0, 0, 0, 0};

// The load is written as assembly because the compiler, which cannot tell
// which stage a read touches, would wait for every load in flight before each
// transposing read.  It has no register result; tg_wait waits for it.
__device__ __forceinline__ void tg_dma(const uint8_t* src, uint32_t lds_wave) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds_wave), "v"(src) : "memory");
}

// all but the N youngest loads of this wave have landed, its LDS reads are
// done, and so for every wave of the workgroup
template <int N>
__device__ __forceinline__ void tg_wait() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t tg_lds_addr(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((const TG_LDS uint8_t*)(p)));
}

// K-contiguous tile of X rows: thread t fetches chunk ch of rows t / 8 + i TH / 8
template <int X, int TH>
struct TgRows {
  static constexpr int N = X * 8 / TH;
  const uint8_t* p[N];
  int ch16;                                 // byte of the thread's chunk in the step
  template <class F>                        // row_ptr(r): first byte of tile row r (any row of the operand for a dead one)
  __device__ __forceinline__ void setup(F row_ptr) {
    const int r = threadIdx.x >> 3;
    ch16 = 16 * ((threadIdx.x & 7) ^ ((r >> 1) & 7));
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = row_ptr(r + i * (TH / 8)) + ch16;
  }
  __device__ __forceinline__ void issue(int step, int64_t kbytes, uint32_t lds_wave) {
    const int64_t o = static_cast<int64_t>(step) * kTgStep;
    const bool dead = o + ch16 >= kbytes;
#pragma unroll
    for (int i = 0; i < N; ++i)
      tg_dma(dead ? reinterpret_cast<const uint8_t*>(&tg_zero) : p[i] + o, lds_wave + i * TH * 16);
  }
};

// K-major tile of X columns of 2 bytes: thread t fetches one chunk of rows
// t / (X / 8) + i TH / (X / 8).  Columns at or behind `cols` repeat the last
// chunk (their results are not stored).
template <int X, int TH>
struct TgCols {
  static constexpr int PER = X / 8;         // chunks of a row
  static constexpr int N = 64 * PER / TH;
  static constexpr int STEP = TH / PER;     // rows between the thread's loads
  static_assert(X >= 128 && STEP % 16 == 0, "the unit permutation repeats every 16 rows and needs 8 units");
  const uint8_t* base;                      // the thread's chunk of row 0
  int64_t ld;                               // bytes of a row
  int k0;                                   // the thread's first row of a step
  int idx[N];                               // gathered: source rows of the next step
  __device__ __forceinline__ void setup(const uint8_t* mem, int64_t ld_bytes, int c0, int cols) {
    k0 = threadIdx.x / PER;
    const int f = (k0 & 3) + 4 * ((k0 >> 3) & 1);
    const int c = c0 + 8 * ((threadIdx.x % PER) ^ (2 * f));
    ld = ld_bytes;
    base = mem + 2 * static_cast<int64_t>(min(c, cols - 8));
  }
  template <class F>                        // source(k): memory row of reduction row k, any valid one where k >= kt
  __device__ __forceinline__ void fetch_rows(int step, F source) {
#pragma unroll
    for (int i = 0; i < N; ++i) idx[i] = source(step * 64 + k0 + i * STEP);
  }
  __device__ __forceinline__ void issue_gathered(int step, int kt, uint32_t lds_wave) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const bool dead = step * 64 + k0 + i * STEP >= kt;
      tg_dma(dead ? reinterpret_cast<const uint8_t*>(&tg_zero) : base + idx[i] * ld, lds_wave + i * TH * 16);
    }
  }
  __device__ __forceinline__ void issue(int step, int kt, uint32_t lds_wave) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int k = step * 64 + k0 + i * STEP;
      tg_dma(k >= kt ? reinterpret_cast<const uint8_t*>(&tg_zero) : base + k * ld, lds_wave + i * TH * 16);
    }
  }
};

// A wave's fragments of NT 16-row tiles, the first at tile t0: lane (lg, lr)
// holds row lr of the tile, 16 bytes of k from 16 lg (+ 64 with sub-step 1)
template <bool KM, int X, int NT>
__device__ __forceinline__ void tg_frags(const uint8_t* tile, int t0, int s, u32x4 (&f)[NT]) {
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  if constexpr (!KM) {
    const uint8_t* b = tile + t0 * 16 * kTgStep + lr * kTgStep + 16 * ((4 * s + lg) ^ (lr >> 1));
#pragma unroll
    for (int i = 0; i < NT; ++i) f[i] = *reinterpret_cast<const u32x4*>(b + i * 16 * kTgStep);
  } else {
    const int perm = (lr >> 2) + 4 * (lg & 1);
    const uint8_t* b = tile + (32 * s + 8 * lg + (lr >> 2)) * 2 * X + 8 * (lr & 3);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const uint8_t* q = b + 32 * ((t0 + i) ^ perm);
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((TG_LDS s16x4*)(q));
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((TG_LDS s16x4*)(q + 4 * 2 * X));
      const uint2 l = __builtin_bit_cast(uint2, lo), h = __builtin_bit_cast(uint2, hi);
      f[i] = u32x4{l.x, l.y, h.x, h.y};
    }
  }
}

// ------------------------------------------------------------------ the tile kernel
// A workgroup of WR x WC waves computes BM rows x BN columns (gated: BN / 2
// gate columns and the same BN / 2 of up); wave (wr, wc) holds BM / WR rows and
// BN / WC columns.  ST stages of both operand tiles in LDS: while step s is
// multiplied, the loads of steps s + 1 .. s + ST - 1 are in flight; one barrier
// per step.
template <int T, int L, int EPI, int BM, int BN, int WR, int WC, int ST>
__global__ __launch_bounds__(64 * WR * WC) void k_tile_gemm(const TileParams p) {
  using TT = TgType<T>;
  using acc_t = typename TT::acc_t;
  constexpr int EB = TT::bytes;
  constexpr int TH = 64 * WR * WC;
  constexpr int SK = kTgStep / EB;          // values of k per step
  constexpr bool RKM = L == TG_TN, CKM = L != TG_NT;
  constexpr bool GATED = EPI == TG_OUT_GATED;
  constexpr int RT = BM / WR / 16, CT = BN / WC / 16;     // 16-row and 16-column tiles of a wave
  constexpr int kStage = (BM + BN) * kTgStep;
  constexpr int kLoads = kStage / 16 / TH;
  static_assert(T != TG_I8 || L == TG_NT, "int8 has the forward product only");
  static_assert(!GATED || CT % 2 == 0, "a gated wave holds as many gate as up tiles");
  __shared__ __attribute__((aligned(16))) uint8_t lds[ST * kStage];
  static_assert(fits_lds(sizeof(lds), 1), "tile stages exceed the LDS of a CU");

  int e, m0, nt;
  int row0, Me;
  if constexpr (L == TG_TN) {
    // equal contiguous ranges of the tiles per XCD, as find_task gives
    const int per = p.r_tiles * p.n_tiles;
    const int n = p.E * per;
    const int share = (n + 7) >> 3;
    const int u = (blockIdx.x & 7) * share + (blockIdx.x >> 3);
    if ((blockIdx.x >> 3) >= share || u >= n) return;
    e = u / per;
    const int v = u - e * per;
    m0 = (v / p.n_tiles) * BM;
    nt = v % p.n_tiles;
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
    if (!find_task<BM / 16, false, 0>(map, e, m0, nt, narrow)) return;
    row0 = min(max(p.offsets[e], 0), p.m_total);
    Me = min(max(p.offsets[e + 1], 0), p.m_total) - row0;
    // inside an expert, groups of 4 row chunks run column tile by column tile:
    // workgroups side by side on an XCD share row chunks and weight tiles in its L2
    const int nc = (Me + BM - 1) / BM;
    const int u = (m0 / BM) * p.n_tiles + nt;
    const int grp = (m0 / BM) / 4;
    const int gq = min(4, nc - 4 * grp);
    const int w = u - 4 * grp * p.n_tiles;
    m0 = (4 * grp + w % gq) * BM;
    nt = w / gq;
  }
  const int rows = L == TG_TN ? min(BM, p.R - m0) : min(BM, Me - m0);
  const int kt = L == TG_TN ? Me : p.K;     // length of the reduction
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wave / WC, wc = wave % WC;
  const int c0 = nt * (GATED ? BN / 2 : BN);
  const int half = p.N / 2;

  const uint8_t* A = static_cast<const uint8_t*>(p.a);
  const uint8_t* B = static_cast<const uint8_t*>(p.b);
  if constexpr (L != TG_TN) B += static_cast<size_t>(e) * p.N * p.K * EB;
  // row q of the expert's rows in the operand that may be gathered; the index
  // array's entries are clamped, so that bad ones give wrong rows only
  auto src_row = [&](int q) -> int {
    int r = row0 + q;
    if (p.a_rows) {
      r = p.a_rows[r];
      r = (r >= 0 && r < p.src_rows) ? r : 0;
    }
    return r;
  };

  TgRows<BM, TH> ra;
  TgRows<BN, TH> ca;
  TgCols<(BM < 128 ? 128 : BM), TH> rk;
  TgCols<(BN < 128 ? 128 : BN), TH> ck;
  if constexpr (!RKM) {
    ra.setup([&](int r) {
      const int q = m0 + (r < rows ? r : 0);
      const int64_t sr = L == TG_NT ? src_row(q) : row0 + q;
      return A + sr * p.K * EB;
    });
  } else {
    rk.setup(A + static_cast<int64_t>(row0) * p.R * 2, static_cast<int64_t>(p.R) * 2, m0, p.R);
  }
  if constexpr (!CKM) {
    ca.setup([&](int c) {
      int col;
      if constexpr (GATED)
        col = min(c0 + (c & (BN / 2 - 1)), half - 1) + (c >= BN / 2 ? half : 0);
      else
        col = min(c0 + c, p.N - 1);
      return B + static_cast<int64_t>(col) * p.K * EB;
    });
  } else {
    ck.setup(B, static_cast<int64_t>(p.N) * 2, c0, p.N);
  }
  const uint32_t lds0 = tg_lds_addr(lds) + wave * 1024;
  auto fetch = [&](int step) {              // the gathered rows of a K-major step
    if constexpr (L == TG_TN) ck.fetch_rows(step, [&](int k) { return src_row(min(k, kt - 1)); });
  };
  auto issue = [&](int step) {
    const uint32_t l = lds0 + (step % ST) * kStage;
    if constexpr (!RKM) ra.issue(step, static_cast<int64_t>(kt) * EB, l);
    else rk.issue(step, kt, l);
    if constexpr (!CKM) ca.issue(step, static_cast<int64_t>(kt) * EB, l + BM * kTgStep);
    else if constexpr (L == TG_TN) ck.issue_gathered(step, kt, l + BM * kTgStep);
    else ck.issue(step, kt, l + BM * kTgStep);
  };

  acc_t acc[RT][CT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < CT; ++j) acc[i][j] = acc_t{0, 0, 0, 0};

  const int nsteps = (kt + SK - 1) / SK;
  if (nsteps > 0) {
    fetch(0);
#pragma unroll
    for (int s = 0; s < ST - 1; ++s)
      if (s < nsteps) {
        issue(s);
        if (s + 1 < nsteps) fetch(s + 1);
      }
  }
  const bool live = wr * (BM / WR) < rows;  // the wave has rows
  for (int step = 0; step < nsteps; ++step) {
    if (step + ST - 1 <= nsteps) tg_wait<(ST - 2) * kLoads>();
    else tg_wait<0>();
    if (step + ST - 1 < nsteps) {
      issue(step + ST - 1);
      if (step + ST < nsteps) fetch(step + ST);
    }
    const uint8_t* cur = lds + (step % ST) * kStage;
    if (live) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        u32x4 fc[CT], fr[RT];
        if constexpr (GATED) {
          u32x4 g[CT / 2], u[CT / 2];
          tg_frags<CKM, BN, CT / 2>(cur + BM * kTgStep, wc * (CT / 2), s, g);
          tg_frags<CKM, BN, CT / 2>(cur + BM * kTgStep, BN / 32 + wc * (CT / 2), s, u);
#pragma unroll
          for (int j = 0; j < CT / 2; ++j) {
            fc[j] = g[j];
            fc[CT / 2 + j] = u[j];
          }
        } else {
          tg_frags<CKM, BN, CT>(cur + BM * kTgStep, wc * CT, s, fc);
        }
        tg_frags<RKM, BM, RT>(cur, wr * RT, s, fr);
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int j = 0; j < CT; ++j) acc[i][j] = TT::mfma(fc[j], fr[i], acc[i][j]);
      }
    }
  }

  // lane: output row lr of a 16-row tile, columns 4 lg .. 4 lg + 3 of a 16-column tile
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int r = (BM / WR) * wr + 16 * i + lr;
    if (r >= rows) continue;
    const int64_t orow = L == TG_TN ? static_cast<int64_t>(e) * p.R + m0 + r : static_cast<int64_t>(row0) + m0 + r;
    float sa = 1.0f;
    if constexpr (T == TG_I8) sa = p.sa[src_row(m0 + r)];
#pragma unroll
    for (int j = 0; j < (GATED ? CT / 2 : CT); ++j) {
      const int c = c0 + (GATED ? BN / 2 : BN) / WC * wc + 16 * j + 4 * lg;
      if (c >= (GATED ? half : p.N)) continue;
      float4v v, w;
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = static_cast<float>(acc[i][j][q]);
      if constexpr (T == TG_I8) v = v * (*reinterpret_cast<const float4v*>(p.sb + static_cast<size_t>(e) * p.N + c) * sa);
      if constexpr (GATED) {
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] = static_cast<float>(acc[i][j + CT / 2][q]);
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

template <int T, int L, int EPI, int BM, int BN, int WR, int WC, int ST>
static hipError_t tg_start(TileParams p, hipStream_t stream) {
  const int cols = EPI == TG_OUT_GATED ? p.N / 2 : p.N;
  const int bn = EPI == TG_OUT_GATED ? BN / 2 : BN;
  p.n_tiles = (cols + bn - 1) / bn;
  p.r_tiles = (p.R + BM - 1) / BM;
  int64_t blocks;
  if (L == TG_TN) {
    blocks = static_cast<int64_t>(p.E) * p.r_tiles * p.n_tiles;
  } else {
    // at most min(E, m_total) experts have rows, each with one partial chunk
    const int64_t chunks = p.m_total / BM + (p.E < p.m_total ? p.E : p.m_total);
    blocks = chunks * p.n_tiles;
  }
  blocks = (blocks + 7) / 8 * 8;
  if (blocks >= (int64_t(1) << 31)) return hipErrorInvalidConfiguration;
  if (blocks == 0) return hipSuccess;
  hipLaunchKernelGGL((k_tile_gemm<T, L, EPI, BM, BN, WR, WC, ST>), dim3(static_cast<unsigned>(blocks)), dim3(64 * WR * WC), 0,
                     stream, p);
  return hipGetLastError();
}

template <int T, int L, int EPI>
static hipError_t tg_launch(const TileParams& p, hipStream_t stream) {
  const int64_t r = L == TG_TN ? p.R : p.rows_hint;
  if (r >= 192) return tg_start<T, L, EPI, 256, 256, 2, 4, 2>(p, stream);
  return tg_start<T, L, EPI, 128, 128, 2, 2, 2>(p, stream);
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
