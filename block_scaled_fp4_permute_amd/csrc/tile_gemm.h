// Grouped matrix products on plain operands (bf16, fp16, int8) for gfx950.
//
// One tile routine serves every product of the 16-bit expert FFN, its
// gradients and the INT8 product:
//   out[r, c] = sum_k R[r, k] * C[c, k]        (r, c, k as below)
//             rows r           columns c        reduction k     R          C
//   NT  y     rows of expert   N                K               [r][k]     [c][k]   y  = a B^T
//   NN  da    rows of expert   K                N               [r][k]     [k][c]   da = dy B
//   TN  dB    N                K                rows of expert  [k][r]     [k][c]   dB = dy^T a
//   TC  dB    N                K                rows of expert  [r][k]     [k][c]   the same from dy^T
// An operand stored [x][k] is K-contiguous, one stored [k][x] is K-major.
//
// The matrix instruction gets C as its first operand and R as its second, so a
// lane's four results are four neighbouring columns of one output row.
#pragma once

#include <type_traits>
#include <utility>

#include "gemm_device.h"

namespace nvfp4 {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 half4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

enum : int { TG_BF16 = 0, TG_F16 = 1, TG_I8 = 2 };            // operand type
enum : int { TG_NT = 0, TG_NN = 1, TG_TN = 2, TG_TC = 3 };    // operand layouts
enum : int { TG_OUT_16 = 0, TG_OUT_F32 = 1, TG_OUT_GATED = 2, TG_OUT_PART = 3 };  // epilogue (PART: float32 sums of one part of the reduction)

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

// f(0) .. f(N - 1) with constants
template <class F, int... I>
__device__ __forceinline__ void tg_for_each(F f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void tg_for(F f) {
  tg_for_each(f, std::make_integer_sequence<int, N>{});
}

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
// K-contiguous: row r is 128 bytes, its 16-byte chunk ch at chunk ch ^ ((r >> 1) & 7):
//   the 16 rows that a fragment read touches at one chunk cover all 64 banks.
// K-major: row k is 2 X bytes, its 32-byte unit u (16 values) at unit u ^ f(k),
//   f(k) = (k & 3) + 4 ((k >> 3) & 1): the 8 rows that half a wave's transposing
//   read touches (4 of lane groups 2q and 2q + 1 each) lie in distinct units.
typedef short s16x4 __attribute__((ext_vector_type(4)));
#define TG_LDS __attribute__((address_space(3)))

// zeros for the loads of a step behind the end of the reduction (16 bytes a lane, the same for all)
__device__ const u32x4 tg_zero = {};

// The load is written as assembly because the compiler, which cannot tell
// which stage a read touches, would wait for every load in flight before each
// transposing read.  It has no register result; tg_wait waits for it.  m0 is
// named as written, so that no m0 of the compiler's own (which it sets in front
// of an instruction that reads it, none in these kernels today) lies across it;
// the warning, that the compiler keeps no value in m0, does not matter then.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void tg_dma(const uint8_t* src, uint32_t lds_wave) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds_wave), "v"(src) : "memory", "m0");
}

// the same of 4 bytes a lane
__device__ __forceinline__ void tg_dma4(const float* src, uint32_t lds_wave) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(lds_wave), "v"(src) : "memory", "m0");
}
#pragma clang diagnostic pop

// all but the N youngest memory operations of this wave are done, its LDS
// reads too, and so for every wave of the workgroup
template <int N>
__device__ __forceinline__ void tg_wait() {
  __builtin_amdgcn_s_waitcnt(0xC07F);       // lgkmcnt(0) for the compiler to know: it does not wait for those reads again
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t tg_lds_addr(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((const TG_LDS uint8_t*)(p)));
}

// the thread's index, opaque to the compiler: what a task's start or end derives
// from it is then computed there and holds no registers during the steps
__device__ __forceinline__ int tg_thread() {
  int t = threadIdx.x;
  asm volatile("" : "+v"(t));
  return t;
}

// K-contiguous tile of X rows: thread t fetches one chunk of rows t / 8 + i TH / 8
template <int X, int TH>
struct TgRows {
  static constexpr int N = X * 8 / TH;
  static constexpr int STEP = TH / 8;       // rows between the thread's loads
  static_assert(STEP % 16 == 0, "the chunk permutation repeats every 16 rows");
  const uint8_t* p[N];                      // of the next step
  int ch16;                                 // byte of the thread's chunk in the step
  template <class F>                        // row_ptr(r): first byte of the operand row of tile row r (any row for a dead one)
  __device__ __forceinline__ void setup(F row_ptr) {
    const int t = tg_thread(), r = t >> 3;
    ch16 = 16 * ((t & 7) ^ ((r >> 1) & 7));
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = row_ptr(r + i * STEP) + ch16;
  }
  // left: bytes of the reduction from this step on
  __device__ __forceinline__ void issue(int i, int left, uint32_t lds_wave) {
    tg_dma(ch16 < left ? p[i] : reinterpret_cast<const uint8_t*>(&tg_zero), lds_wave + i * TH * 16);
    p[i] += kTgStep;
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
  static constexpr int ROWS = 64 / PER;     // rows of a wave's load
  static_assert(X >= 128 && STEP % 16 == 0, "the unit permutation repeats every 16 rows");
  const uint8_t* p[N];                      // of the next step
  int64_t ld;                               // bytes of a row
  int k0;                                   // the thread's first row of a step
  const uint8_t* base;                      // gathered: the thread's chunk in row 0 of the operand
  __device__ __forceinline__ void setup(const uint8_t* mem, int64_t ld_bytes, int c0, int cols) {
    const int t = tg_thread();
    k0 = t / PER;
    const int f = (k0 & 3) + 4 * ((k0 >> 3) & 1);
    const int c = 8 * ((t % PER) ^ (2 * f));
    ld = ld_bytes;
    base = mem + 2 * static_cast<int64_t>(c0) + 2 * min(c, cols - 8 - c0);
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = base + (k0 + i * STEP) * ld;
  }
  // left: rows of the reduction from this step on
  __device__ __forceinline__ void issue(int i, int left, uint32_t lds_wave) {
    tg_dma(k0 < left - i * STEP ? p[i] : reinterpret_cast<const uint8_t*>(&tg_zero), lds_wave + i * TH * 16);
    p[i] += 64 * ld;
  }
  // the thread's of the rows of the wave's load, which all its threads know
  __device__ __forceinline__ int own_row(const int (&rows)[ROWS]) const {
    const int w = (threadIdx.x & 63) / PER;
    int r = rows[0];
    tg_for<ROWS - 1>([&](auto ic) __attribute__((always_inline)) {
      constexpr int q = decltype(ic)::value + 1;
      // moved to a vector register here: a plain choice among the array's entries becomes a table in memory
      int a;
      asm("v_mov_b32 %0, %1" : "=v"(a) : "s"(rows[q]));
      r = w == q ? a : r;
    });
    return r;
  }
  // gathered: the thread's chunk of `row`
  __device__ __forceinline__ void issue_row(int i, int row, uint32_t ld_bytes, int left, uint32_t lds_wave) {
    const uint8_t* a = base + static_cast<uint64_t>(static_cast<uint32_t>(row)) * ld_bytes;
    tg_dma(k0 < left - i * STEP ? a : reinterpret_cast<const uint8_t*>(&tg_zero), lds_wave + i * TH * 16);
  }
};

// NT fragments (16 rows or columns each) of a tile from fragment t0 on: lane
// (lg, lr) holds entry lr of each, 16 bytes of k from 16 lg (+ 64 with sub-step 1)
template <bool KM, int X, int NT>
__device__ __forceinline__ void tg_frags(const uint8_t* tile, int t0, int s, u32x4* f) {
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

// ------------------------------------------------------------------ tasks
// A task is one output tile.  NT and NN: row chunk by row chunk, column tile by
// column tile within one, experts in order; a prefix sum of the experts'
// chunks lies in LDS, one entry for two experts.  TN and TC: every expert has the same tiles.  Each XCD gets an
// equal contiguous range of the tasks (workgroups go to XCDs round-robin), so
// that the tiles side by side in its L2 share rows and weights; a workgroup
// takes every (workgroups per XCD)th task of its XCD's range.
constexpr int kTgMaxExperts = 4096;
// Tiles of 64 rows take fewer, so that their workgroups lie three to a CU.
constexpr int tg_most_experts(int bm) { return bm == 64 ? 1024 : kTgMaxExperts; }
constexpr int tg_per_cu(int bm) { return bm == 256 ? 1 : bm == 128 ? 2 : 3; }

struct TgTask {
  int e, m0, nt;
  int row0;       // first row of the expert
  int rows;       // live rows of the tile
  int kt;         // length of the reduction
  int part, k0;   // part of the reduction and its first k
  int nsteps;     // at least 2: the loads run two steps ahead, short reductions get steps of zeros
};

// uniform reads that must not wait for the loads in flight go through scalar loads
typedef const int __attribute__((address_space(4)))* tg_const_ints;

template <int BM>
__device__ __forceinline__ int tg_chunks(const TileParams& p, int first, int end) {
  return (max(min(max(end, 0), p.m_total) - min(max(first, 0), p.m_total), 0) + BM - 1) / BM;
}

template <int BM>
__device__ __forceinline__ int tg_prefix(const TileParams& p, int* pre) {
  const int lane = threadIdx.x & 63;
  if (threadIdx.x < 64) {
    int base = 0;
    for (int g = 0; g < p.E; g += 64) {
      const int c = g + lane < p.E ? tg_chunks<BM>(p, p.offsets[g + lane], p.offsets[g + lane + 1]) : 0;
      int total;
      const int before = min(base + wave_excl_scan(c, total), 1 << 28);
      if (g + lane < p.E && !(lane & 1)) pre[(g + lane) >> 1] = before;
      base = min(base + total, 1 << 28);    // offsets that overlap: the tasks of some rows fall away
    }
    if (lane == 0) pre[0] = base;           // the place of the first expert's zero holds the total
  }
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(pre[0]);
}

// TC: the rows operand is stored transposed, [R][ld].  The columns of expert e
// start at a multiple of `align` (64: a step's 128 bytes of a row are one line;
// 8, 16 bytes, where experts have so few rows that the gaps would dominate), at
// least one element behind those of the expert before; up to the next multiple
// of 8 behind its last column they hold zeros.
__host__ __device__ __forceinline__ int64_t tg_start_col(int64_t row0, int e, int align) {
  return ((row0 + align - 1) & ~static_cast<int64_t>(align - 1)) + static_cast<int64_t>(align) * e;
}
__host__ __device__ __forceinline__ int tg_col_align(int64_t m_total, int E) { return m_total / E >= 64 ? 64 : 8; }

// task (c, nt): row chunk c of all experts' chunks (TN, TC: row tile c), column tile
// nt.  Inside an expert, groups of 4 chunks run column tile by column tile, so
// that the workgroups side by side share both operands in L2.
template <int L, int BM, int SK, bool PART>
__device__ __forceinline__ void tg_decode(const TileParams& p, const int* pre, int c, int nt, TgTask& t) {
  const tg_const_ints off = (tg_const_ints)(p.offsets);
  int q, nc;                               // chunk of its expert, chunks of the expert
  constexpr bool WEIGHT = L == TG_TN || L == TG_TC;
  if constexpr (WEIGHT) {
    t.e = c / p.r_tiles;
    q = c - t.e * p.r_tiles;
    nc = p.r_tiles;
  } else {
    const int lane = threadIdx.x & 63, pairs = (p.E + 1) >> 1;
    int i = (t.e >> 1) & ~63;              // the pairs of experts whose chunks all lie before c, counted 64 at a time
    for (;;) {
      const bool past = i + lane + 1 < pairs && pre[i + lane + 1] <= c;
      const int n = __popcll(__ballot(past));
      i += n;
      if (n < 64) break;
    }
    i = __builtin_amdgcn_readfirstlane(i);
    q = c - (i ? __builtin_amdgcn_readfirstlane(pre[i]) : 0);
    t.e = 2 * i;                           // the first of the pair, or the second
    const int of_first = tg_chunks<BM>(p, off[t.e], off[t.e + 1]);
    if (q >= of_first && t.e + 1 < p.E) {
      q -= of_first;
      ++t.e;
    }
  }
  t.row0 = min(max(off[t.e], 0), p.m_total);
  const int Me = max(min(max(off[t.e + 1], 0), p.m_total) - t.row0, 0);
  if constexpr (!WEIGHT) nc = (Me + BM - 1) / BM;
  const int w = (q & 3) * p.n_tiles + nt, left = nc - (q & ~3);
  int m = w >> 2, r = w & 3;               // w by the chunks of the group
  if (left == 1) { m = w; r = 0; }
  if (left == 2) { m = w >> 1; r = w & 1; }
  if (left == 3) { m = w / 3; r = w - 3 * m; }
  t.m0 = ((q & ~3) + r) * BM;
  t.nt = m;
  t.rows = min(BM, (WEIGHT ? p.R : Me) - t.m0);
  t.kt = WEIGHT ? Me : p.K;
  t.part = 0;
  t.k0 = 0;
  if constexpr (PART) {                    // the column tiles of part 0, then of part 1, ..
    const int per = p.n_tiles / p.parts;
    t.part = t.nt / per;
    t.nt -= t.part * per;
    const int len = WEIGHT ? ((Me + 63) / 64 + p.parts - 1) / p.parts * 64 : p.part_k;
    t.k0 = t.part * len;
    t.kt = max(min(len, t.kt - t.k0), 0);
  }
  t.nsteps = max(2, (t.kt + SK - 1) / SK);
}

// ------------------------------------------------------------------ the tile kernel
// A workgroup of WR x WC waves computes BM rows x BN columns (gated: BN / 2
// gate columns and the same BN / 2 of up) per task; wave (wr, wc) holds
// BM / WR rows and BN / WC columns.  The steps of all its tasks form one
// stream through two LDS stages.
//
// A step is four units of (half h of the wave's row tiles) x (half s of the
// step's k); while a unit is multiplied, the next unit's fragments are read
// from LDS.  The workgroup meets twice a step, before units 1 and 3:
//   before 1  the fragments of units 0 and 1 are in registers, so the parts of
//             the stage that no later unit reads are free; the loads X of step
//             + 2 go into them during units 1 and 2
//   before 3  all fragments are in registers; the loads Y of step + 2 go into
//             the rest during unit 3, and the next step's first fragments are
//             read
// With the units in the order (h, s) = 00 01 10 11 the columns operand and the
// h = 0 rows are free first (X), the h = 1 rows later (Y).  Two K-major
// operands (TN) are split by k instead: order 00 10 01 11, X the s = 0 halves.
// A load is waited for 1.25 steps or more after it went out, and never more
// than a step's loads are waited for at once.  Loads are spread over a unit's
// products: in one burst they would hold up the products behind them.  A
// finished tile is stored while the next one's loads are in flight.
//
// Tiles: 256 x 256 loads half the bytes a product that 128 x 128 does; its 128
// accumulators a lane and 128 KB of stages leave one workgroup of 8 waves a CU.
// 128 x 128 has two workgroups of 4 waves a CU, which cover each other's task
// ends: the better one where tasks are short or few.  64 x 128 has three of 2
// waves, for tasks of a few rows and steps (both sides of each are measured at
// the choice in skinny_gemm.h).
//
// Measured (MI355X, several boxes: a product's clock differs):       us   rate
//   bf16 8192^3, NT        734 - 780    1410 - 1500 TFLOP/s
//     NN, TN               750 - 785, 913 - 945    1400 - 1465, 1160 - 1200 TFLOP/s
//   int8 8192^3, NT        391 - 425    2590 - 2810 TOPS
//   256 experts, 512 rows each, bf16 6144 -> 2 x 256: forward       943 - 950   868 - 874 TFLOP/s
//     row gradient, weight gradient (TC), each in a loop of its own 995, 957    829, 862 TFLOP/s
//     the same one behind the other                                 1037, 1081  795, 763 TFLOP/s
//   256 experts, 8 rows each, bf16 6144 -> 2 x 256 / 256 -> 6144:
//                                                    284 - 291 / 160   5.5 - 5.7 / 5.2 TB/s
//   the same 256 -> 6144 in int8 (two steps a task)            89 - 90   4.9 TB/s
// Large products run at 1.9 - 2.1 GHz, the clock that the matrix cores' power
// leaves, with those busy 53 % (forward), 48 % (rows) and 38 % (weights) of the
// cycles at 512 rows an expert; LDS reads have no bank conflicts.  There the rest
// is the last chunk of each expert (512 +- 22 rows take 2.5 chunks of 256 on
// average), the task ends, and for weights the wait for gathered rows.  TN is
// bound by its LDS reads, all of 8 bytes.  Few rows: bound by the weights'
// stream from memory.
template <int T, int L, int EPI, int BM, int BN, int WR, int WC>
__global__ __launch_bounds__(64 * WR * WC) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_tile_gemm(const TileParams p) {
  using TT = TgType<T>;
  using acc_t = typename TT::acc_t;
  constexpr int EB = TT::bytes;
  constexpr int TH = 64 * WR * WC;
  constexpr int SK = kTgStep / EB;          // values of k per step
  constexpr bool RKM = L == TG_TN, CKM = L != TG_NT;
  constexpr bool GATED = EPI == TG_OUT_GATED;
  constexpr bool WEIGHT = L == TG_TN || L == TG_TC;         // a weight gradient: reduction over an expert's rows
  constexpr int RT = BM / WR / 16, CT = BN / WC / 16;     // 16-row and 16-column tiles of a wave
  constexpr int RH = RT / 2;
  constexpr int kStage = (BM + BN) * kTgStep;
  using Rows = TgRows<BM, TH>;
  using Cols = TgRows<BN, TH>;
  using RowsK = TgCols<RKM ? BM : 128, RKM ? TH : 256>;     // (the other layouts do not use it)
  using ColsK = TgCols<CKM ? BN : 128, CKM ? TH : 256>;
  constexpr int NR = Rows::N, NC = Cols::N;               // loads of a thread per step and operand
  constexpr int NX = RKM ? NR / 2 + NC / 2 : NC + NR / 2, NY = NR + NC - NX;
  static_assert(T != TG_I8 || L == TG_NT, "int8 has the forward product only");
  static_assert(CT == 4 && RT % 4 == 0, "the store's exchange takes 4 column tiles; row tiles are stored in quarters");
  static_assert((!RKM || RowsK::N == NR) && (!CKM || ColsK::N == NC) && NR % 2 == 0 && NC % 2 == 0, "halves of the loads");
  constexpr int RL = BM / WR / 2 / Rows::STEP;              // row loads of a half of a wave's rows
  static_assert(RKM || RL * Rows::STEP * WR * 2 == BM, "a load holds rows of one half");
  constexpr int kMap = WEIGHT ? 1 : tg_most_experts(BM) / 2;
  constexpr int kScales = T == TG_I8 ? BM + BN : 1;         // INT8: a tile's scales
  constexpr int SL = (kScales + TH - 1) / TH;               // a thread fetches so many
  static_assert(T != TG_I8 || kScales % 64 == 0, "whole waves fetch scales");
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * kStage];
  __shared__ int pre[kMap];
  __shared__ __attribute__((aligned(16))) float scl[2][kScales];
  static_assert(fits_lds(sizeof(lds) + sizeof(pre) + sizeof(scl), tg_per_cu(BM)), "tile stages exceed the LDS of a CU");

  int n;
  if constexpr (WEIGHT) n = p.E * p.r_tiles * p.n_tiles;
  else n = static_cast<int>(min(static_cast<int64_t>(tg_prefix<BM>(p, pre)) * p.n_tiles, int64_t(1) << 30));
  const int share = (n + 7) >> 3;
  const int lo = (blockIdx.x & 7) * share, hi = min(lo + share, n);
  const int stride = gridDim.x >> 3;
  int u = lo + (blockIdx.x >> 3);
  if (u >= hi) return;
  // task u as (chunk, column tile), and the step to the workgroup's next one
  int uc = u / p.n_tiles, un = u - uc * p.n_tiles;
  const int dc = stride / p.n_tiles, dn = stride - dc * p.n_tiles;

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wave / WC, wc = wave % WC;
  const int half = p.N / 2;
  const uint8_t* A = static_cast<const uint8_t*>(p.a);
  const uint8_t* B = static_cast<const uint8_t*>(p.b);
  // an entry of the index array, clamped, so that a bad one gives wrong rows only
  auto valid_row = [&](int r) __attribute__((always_inline)) -> int { return (r >= 0 && r < p.src_rows) ? r : 0; };

  // ---- the loads
  TgTask pt = {};                           // their task
  int ps = 0;                               // their step in it
  int pg = 0;                               // their step in the stream
  bool idle = false;                        // no task is left: zeros are loaded, which nothing reads
  Rows ra;
  Cols ca;
  RowsK rk;
  ColsK ck;
  // INT8: the task's scales, rows then columns, come with its first step's loads.
  // Two buffers in turn: a task's are read before the step in which those of the
  // task two further on go out has met.
  const float* scale[SL];                   // the thread's
  int pbuf = 0;                             // the buffer of the loads' task
  auto begin = [&]() __attribute__((always_inline)) {
    const int c0 = pt.nt * (GATED ? BN / 2 : BN);
    const uint8_t* Be = B;
    if constexpr (!WEIGHT) Be += static_cast<size_t>(pt.e) * p.N * p.K * EB;
    if constexpr (L == TG_TN) {
      rk.setup(A + (static_cast<int64_t>(pt.row0) + pt.k0) * p.R * 2, static_cast<int64_t>(p.R) * 2, pt.m0, p.R);
    } else if constexpr (L == TG_TC) {
      const uint8_t* first = A + 2 * (tg_start_col(pt.row0, pt.e, tg_col_align(p.m_total, p.E)) + pt.k0);
      ra.setup([&](int r) __attribute__((always_inline)) {
        return first + static_cast<int64_t>(pt.m0 + (r < pt.rows ? r : 0)) * p.K * 2;
      });
    } else {
      ra.setup([&](int r) __attribute__((always_inline)) {
        int q = pt.row0 + pt.m0 + (r < pt.rows ? r : 0);
        if (L == TG_NT && p.a_rows) q = valid_row(p.a_rows[q]);
        return A + (static_cast<int64_t>(q) * p.K + pt.k0) * EB;
      });
    }
    if constexpr (L == TG_NT)
      ca.setup([&](int c) __attribute__((always_inline)) {
        int col;
        if constexpr (GATED)
          col = min(c0 + (c & (BN / 2 - 1)), half - 1) + (c >= BN / 2 ? half : 0);
        else
          col = min(c0 + c, p.N - 1);
        return Be + static_cast<int64_t>(col) * p.K * EB;
      });
    else                                    // (weight gradients: every load adds its row)
      ck.setup(Be + (WEIGHT ? 0 : static_cast<int64_t>(pt.k0) * p.N * 2), static_cast<int64_t>(p.N) * 2, c0, p.N);
    if constexpr (T == TG_I8) {
      const int t = tg_thread();
#pragma unroll
      for (int i = 0; i < SL; ++i) {
        const int r = t + i * TH, c = r - BM;
        if (c < 0) {
          const int q = pt.row0 + pt.m0 + (r < pt.rows ? r : 0);
          scale[i] = p.sa + (p.a_rows ? valid_row(p.a_rows[q]) : q);
        } else {
          const int col = GATED ? min(c0 + (c & (BN / 2 - 1)), half - 1) + (c >= BN / 2 ? half : 0) : min(c0 + c, p.N - 1);
          scale[i] = p.sb + static_cast<size_t>(pt.e) * p.N + col;
        }
      }
    }
  };
  const uint32_t lds0 = tg_lds_addr(lds) + wave * 1024;
  int left = 0, left_k = 0;                 // of the reduction from the loads' step on: bytes (K-contiguous) and rows
  // Weight gradients: source rows of the wave's loads.  They are the same for half a wave, so
  // scalar loads fetch them (a vector load would wait for all loads in flight),
  // half a step before they are needed.
  constexpr int W = WEIGHT ? ColsK::ROWS : 1;
  int raw[NC][W];
  int src[NC];                              // of the thread's loads
  auto fetch = [&]() __attribute__((always_inline)) {
    if constexpr (WEIGHT) {
      const int first = pt.row0 + pt.k0, at = first + ps * 64 + wave * W, last = first + max(pt.kt - 1, 0);
#pragma unroll
      for (int j = 0; j < NC; ++j)
#pragma unroll
        for (int w = 0; w < W; ++w) {
          raw[j][w] = min(at + j * ColsK::STEP + w, last);
          if (p.a_rows && pt.kt > 0) raw[j][w] = ((tg_const_ints)(p.a_rows))[raw[j][w]];
        }
    }
  };
  auto open = [&]() __attribute__((always_inline)) {        // before a step's loads
    left_k = idle ? 0 : pt.kt - ps * 64;
    left = idle ? 0 : pt.kt * EB - ps * kTgStep;
    if constexpr (T == TG_I8) {
      if (ps == 0 && !idle) {
#pragma unroll
        for (int i = 0; i < SL; ++i)
          if (wave * 64 + i * TH < kScales) tg_dma4(scale[i], tg_lds_addr(scl) + (pbuf * kScales + wave * 64 + i * TH) * 4);
        pbuf ^= 1;
      }
    }
    if constexpr (WEIGHT) {
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        src[j] = ck.own_row(raw[j]);
        if (p.a_rows) src[j] = valid_row(src[j]);
      }
    }
  };
  auto issue_row = [&](int i, uint32_t l) __attribute__((always_inline)) {
    if constexpr (RKM) rk.issue(i, left_k, l);
    else ra.issue(i, left, l);
  };
  auto issue_col = [&](int j, uint32_t l) __attribute__((always_inline)) {
    if constexpr (L == TG_NT) {
      ca.issue(j, left, l + BM * kTgStep);
    } else if constexpr (L == TG_NN) {
      ck.issue(j, left_k, l + BM * kTgStep);
    } else {
      ck.issue_row(j, src[j], p.N * 2, left_k, l + BM * kTgStep);
    }
  };
  auto issue_x = [&](int q) __attribute__((always_inline)) {   // load q of X
    const uint32_t l = lds0 + (pg & 1) * kStage;
    if constexpr (RKM) {
      if (q < NC / 2) issue_col(q, l);
      else issue_row(q - NC / 2, l);
    } else {
      if (q < NC) issue_col(q, l);
      else issue_row((q - NC) / RL * 2 * RL + (q - NC) % RL, l);
    }
  };
  auto issue_y = [&](int q) __attribute__((always_inline)) {
    const uint32_t l = lds0 + (pg & 1) * kStage;
    if constexpr (RKM) {
      if (q < NC / 2) issue_col(NC / 2 + q, l);
      else issue_row(NR / 2 + q - NC / 2, l);
    } else {
      issue_row(q / RL * 2 * RL + q % RL + RL, l);
    }
  };
  auto advance = [&]() __attribute__((always_inline)) {     // after a step's loads
    ++pg;
    if (++ps == pt.nsteps) {
      u += stride;
      uc += dc;
      un += dn;
      if (un >= p.n_tiles) {
        un -= p.n_tiles;
        ++uc;
      }
      ps = 0;
      if (u < hi) {
        tg_decode<L, BM, SK, EPI == TG_OUT_PART>(p, pre, uc, un, pt);
        begin();
      } else {
        idle = true;
        pt.nsteps = 0;
      }
    }
    fetch();
  };

  // ---- the products
  acc_t acc[RT][CT] = {};
  auto read_rows = [&](const uint8_t* stage, int s, int h, u32x4 (&f)[RH]) __attribute__((always_inline)) {
    tg_frags<RKM, BM, RH>(stage, wr * RT + h * RH, s, f);
  };
  auto read_cols = [&](const uint8_t* stage, int s, u32x4 (&f)[CT]) __attribute__((always_inline)) {
    const uint8_t* c = stage + BM * kTgStep;
    if constexpr (GATED) {                  // the gate tiles, then the same columns of up
      tg_frags<CKM, BN, CT / 2>(c, wc * (CT / 2), s, f);
      tg_frags<CKM, BN, CT / 2>(c, BN / 32 + wc * (CT / 2), s, f + CT / 2);
    } else {
      tg_frags<CKM, BN, CT>(c, wc * CT, s, f);
    }
  };
  // the products of a unit; work(i) goes between those of row tile i and the next
  auto unit = [&](int h, bool fresh, const u32x4 (&fc)[CT], const u32x4 (&fr)[RH], auto work) __attribute__((always_inline)) {
    tg_for<RH>([&](auto ic) __attribute__((always_inline)) {
      constexpr int i = decltype(ic)::value;
#pragma unroll
      for (int j = 0; j < CT; ++j)
        acc[h * RH + i][j] = TT::mfma(fc[j], fr[i], fresh ? acc_t{0, 0, 0, 0} : acc[h * RH + i][j]);
      __builtin_amdgcn_sched_barrier(0);
      work(ic);
    });
    __builtin_amdgcn_sched_barrier(0);
  };
  TgTask ct = {};                           // their task

  // ---- the results
  // A lane holds output row lr of a 16-row tile, 4 columns from 4 lg of each column
  // tile.  Lane groups exchange 16-bit results of two tiles, so that each lane
  // has 8 neighbouring columns, and lanes lr and lr ^ 8 exchange 16 bytes, so that
  // a store instruction writes whole 128-byte lines: 8 rows of 8 pieces.
  // These stores are non-temporal: no product of the call reads them, and the
  // operands keep the caches (256 experts' weight gradients of 64 rows each 543 ->
  // 368 us, of 512 rows 1068 -> 957; other products up to 3 %).  h, which the next
  // product of a layer reads, leaves through the caches.
  constexpr int OB = EPI == TG_OUT_F32 || EPI == TG_OUT_PART ? 4 : 2;             // bytes of a result
  constexpr int PAIRB = OB == 2 ? 32 : 16;                  // columns from a lane's piece a to its piece b
  uint8_t* obase = static_cast<uint8_t*>(p.out);            // the wave's first result (gated: of h)
  float* gbase = p.gu;                      // gated: of the gate pre-activations
  uint32_t ooff = 0, goff = 0;              // bytes from there to the lane's piece of row tile 0
  int orows = 0;                            // rows from the lane's on; none where its piece lies behind the last column
  int orows2 = 0;                           // float32: the same for the second pair; gated: for the pre-activations
  constexpr int kNoRows = -BM;
  bool full = false;                        // every lane of the wave has all its results
  auto aim = [&]() __attribute__((always_inline)) {         // before the first store of task ct
    const int t = tg_thread(), lg = (t >> 4) & 3;
    const int width = GATED ? half : p.N;
    const int wave_cols = (GATED ? BN / 2 : BN) / WC;
    const int c0 = ct.nt * (GATED ? BN / 2 : BN) + wave_cols * wc;
    const int rows = ct.rows - (BM / WR) * wr;              // of the wave
    const int64_t row0 = (WEIGHT ? (static_cast<int64_t>(ct.part) * p.E + ct.e) * p.R : static_cast<int64_t>(ct.row0) + static_cast<int64_t>(ct.part) * p.m_total) + ct.m0 + (BM / WR) * wr;
    full = rows >= BM / WR && c0 + wave_cols <= width;
    const int piece = 16 * (lg & 1) + 4 * (lg & 2);         // the lane's 8 columns of a pair of tiles after the exchange
    if constexpr (GATED) {
      const int c = piece, cg = 4 * lg + (t & 8 ? 16 : 0);
      obase = static_cast<uint8_t*>(p.out) + (row0 * half + c0) * 2;
      ooff = ((t & 15) * half + c) * 2;
      orows = c0 + c < width ? rows - (t & 15) : kNoRows;
      if (p.gu) gbase = p.gu + row0 * p.N + c0;
      goff = ((t & 7) * p.N + cg) * 4;
      orows2 = c0 + cg < width ? rows - (t & 7) : kNoRows;
    } else {
      const int c = (OB == 2 ? piece : 4 * lg) + (t & 8 ? PAIRB : 0);
      obase = static_cast<uint8_t*>(p.out) + (row0 * p.N + c0) * OB;
      ooff = ((t & 7) * p.N + c) * OB;
      orows = c0 + c < width ? rows - (t & 7) : kNoRows;
      if constexpr (OB == 4) orows2 = c0 + c + 32 < width ? orows : kNoRows;
    }
  };
  auto put = [&](uint8_t* base, uint32_t off, int64_t ld, int rows, u32x4 a, u32x4 b) __attribute__((always_inline)) {
    const bool up = threadIdx.x & 8;        // the lanes that store the pieces b
    u32x4 lo, hi;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const uint32_t x = __builtin_amdgcn_update_dpp(0u, up ? a[d] : b[d], 0x128, 0xF, 0xF, false);   // from lane lr ^ 8
      lo[d] = up ? x : a[d];                // rows 0 .. 7
      hi[d] = up ? b[d] : x;                // rows 8 .. 15
    }
    if (rows > 0) __builtin_nontemporal_store(lo, reinterpret_cast<u32x4*>(base + off));
    if (rows > 8) __builtin_nontemporal_store(hi, reinterpret_cast<u32x4*>(base + 8 * ld + off));
  };
  constexpr int kStores = GATED ? 1 : 2 * CT / (OB == 2 ? 4 : 2);   // store instructions of a row tile, at least
  float row_scale[T == TG_I8 ? RT : 1];     // INT8: scales of the lane's rows and columns
  float4v col_scale[T == TG_I8 ? CT : 1];
  int cbuf = 0;
  auto scales = [&]() __attribute__((always_inline)) {
    if constexpr (T == TG_I8) {
      const int t = tg_thread();
      const float* r = scl[cbuf] + (BM / WR) * wr + (t & 15);
      const float* c = scl[cbuf] + BM + (GATED ? BN / 2 : BN) / WC * wc + 4 * ((t >> 4) & 3);
#pragma unroll
      for (int i = 0; i < RT; ++i) row_scale[i] = r[16 * i];
#pragma unroll
      for (int j = 0; j < CT; ++j)
        col_scale[j] = *reinterpret_cast<const float4v*>(c + 16 * (GATED ? j % (CT / 2) : j) + (GATED && j >= CT / 2 ? BN / 2 : 0));
      cbuf ^= 1;
    }
  };
  auto store = [&](int i) __attribute__((always_inline)) {  // row tile i
    auto value = [&](int j) __attribute__((always_inline)) {  // of column tile j, scaled
      float4v v;
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = static_cast<float>(acc[i][j][q]);
      if constexpr (T == TG_I8) v = v * (col_scale[j] * row_scale[i]);
      return v;
    };
    // 16-bit results of two column tiles as 8 neighbouring columns: lane groups 0
    // and 2 give their second tile to 1 and 3 and take those's first
    auto packed = [&](const float4v& v, const float4v& w) __attribute__((always_inline)) {
      const uint2 a = TT::pack(v), b = TT::pack(w);
      const auto x = __builtin_amdgcn_permlane16_swap(a.x, b.x, false, false);
      const auto y = __builtin_amdgcn_permlane16_swap(a.y, b.y, false, false);
      return u32x4{x[0], y[0], x[1], y[1]};
    };
    if constexpr (GATED) {
      static_assert(CT == 4, "two tiles of h");
      float4v g[2] = {value(0), value(1)}, w[2] = {value(2), value(3)};
      const int64_t ld = static_cast<int64_t>(p.N) * 4;
      if (p.gu) {
        uint8_t* o = reinterpret_cast<uint8_t*>(gbase) + 16 * i * ld;
        put(o, goff, ld, orows2 - 16 * i, __builtin_bit_cast(u32x4, g[0]), __builtin_bit_cast(u32x4, g[1]));
        put(o + 4 * static_cast<int64_t>(half), goff, ld, orows2 - 16 * i, __builtin_bit_cast(u32x4, w[0]), __builtin_bit_cast(u32x4, w[1]));
      }
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int q = 0; q < 4; ++q) g[b][q] = tg_act(g[b][q], p.act) * w[b][q];
      const u32x4 h = packed(g[0], g[1]);
      if (orows > 16 * i) *reinterpret_cast<u32x4*>(obase + 16 * i * static_cast<int64_t>(half) * 2 + ooff) = h;
    } else {
      const int64_t ld = static_cast<int64_t>(p.N) * OB;
      uint8_t* o = obase + 16 * i * ld;
      if constexpr (OB == 4) {
#pragma unroll
        for (int j = 0; j < CT; j += 2)
          put(o + 16 * j * OB, ooff, ld, (j ? orows2 : orows) - 16 * i, __builtin_bit_cast(u32x4, value(j)),
              __builtin_bit_cast(u32x4, value(j + 1)));
      } else {
        put(o, ooff, ld, orows - 16 * i, packed(value(0), value(1)), packed(value(2), value(3)));
      }
    }
  };

  // ---- the stream
  tg_decode<L, BM, SK, EPI == TG_OUT_PART>(p, pre, uc, un, pt);
  begin();
  fetch();
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    open();
#pragma unroll
    for (int q = 0; q < NX; ++q) issue_x(q);
#pragma unroll
    for (int q = 0; q < NY; ++q) issue_y(q);
    if (s == 1) ct = pt;
    advance();
  }
  tg_wait<NX + NY>();
  u32x4 c0[CT], c1[CT], ra_[RH], rb_[RH];
  read_cols(lds, 0, c0);
  read_rows(lds, 0, 0, ra_);
  __builtin_amdgcn_sched_barrier(0);

  // A meeting lets the loads of one step stay in flight, and the stores of a
  // full tile that are younger than the loads it waits for (`stores`: of so
  // many row tiles), since memory operations complete in order.
  auto meet = [&](bool may, auto stores) __attribute__((always_inline)) {
    constexpr int S = decltype(stores)::value * kStores;
    if constexpr (S > 0) {
      if (may) {
        tg_wait<NX + NY + S>();
        return;
      }
    }
    tg_wait<NX + NY>();
  };
  // INT8 results are stored at the end of the task in one go (their scales would
  // take registers during the products; gate_up of 64 rows an expert 185 us
  // among the products, 180 so).  So are TN's, whose stores among the products
  // cost more registers than there are.
  constexpr bool kSpread = T != TG_I8 && !RKM;
  // One step.  FIRST of a task: the products start from zero, and the h = 1 half
  // of the task before is stored before unit 2 overwrites it.  LAST: the h = 0
  // half, complete after unit 1, is stored.
  bool after_first = false;                 // the step follows a task's first one
  auto step = [&](int cg, auto first, auto last) __attribute__((always_inline)) {
    constexpr bool FIRST = decltype(first)::value, LAST = decltype(last)::value;
    const uint8_t* cur = lds + (cg & 1) * kStage;
    const uint8_t* nxt = lds + ((cg + 1) & 1) * kStage;
    // loads FROM .. FROM + N - 1, shared out over the row tiles of a unit
    auto part = [&](auto ic, auto nc, auto fc, auto load) __attribute__((always_inline)) {
      constexpr int i = decltype(ic)::value, n = decltype(nc)::value, from = decltype(fc)::value;
      tg_for<(i + 1) * n / RH - i * n / RH>([&](auto k) __attribute__((always_inline)) {
        load(from + i * n / RH + decltype(k)::value);
      });
    };
    const std::integral_constant<int, 0> i0;
    const std::integral_constant<int, NX / 2> nx1;
    const std::integral_constant<int, NX - NX / 2> nx2;
    const std::integral_constant<int, NY> ny;
    auto none = [](auto) __attribute__((always_inline)) {};
    // half a half's row tiles (q = 0, 1) are stored at every other row tile of a unit
    auto store_half = [&](int h, int q, auto ic) __attribute__((always_inline)) {
      constexpr int i = decltype(ic)::value;
      if constexpr (kSpread && (i & 1)) store(h * RH + q * (RH / 2) + i / 2);
    };
    constexpr int kHalf = kSpread ? RH : 0;
    if constexpr (!RKM) {
      read_cols(cur, 1, c1);
      read_rows(cur, 1, 0, rb_);
      unit(0, FIRST, c0, ra_, [&](auto i) __attribute__((always_inline)) { if constexpr (FIRST) store_half(1, 0, i); });
      if constexpr (FIRST) meet(full, std::integral_constant<int, 3 * kHalf / 2>{});
      else meet(full && after_first, std::integral_constant<int, kHalf>{});
      open();
      read_rows(cur, 0, 1, ra_);
      unit(0, false, c1, rb_, [&](auto i) __attribute__((always_inline)) {
        part(i, nx1, i0, issue_x);
        if constexpr (FIRST) store_half(1, 1, i);
      });
      if constexpr (LAST) aim();
      read_rows(cur, 1, 1, rb_);
      unit(1, FIRST, c0, ra_, [&](auto i) __attribute__((always_inline)) {
        part(i, nx2, nx1, issue_x);
        if constexpr (LAST) store_half(0, 0, i);
      });
      if constexpr (FIRST) meet(full, std::integral_constant<int, 3 * kHalf / 2>{});
      else meet(LAST && full, std::integral_constant<int, LAST ? kHalf / 2 : 0>{});
      read_cols(nxt, 0, c0);
      read_rows(nxt, 0, 0, ra_);
      unit(1, false, c1, rb_, [&](auto i) __attribute__((always_inline)) {
        part(i, ny, i0, issue_y);
        if constexpr (LAST) store_half(0, 1, i);
      });
    } else {
      read_rows(cur, 0, 1, rb_);
      unit(0, false, c0, ra_, none);
      meet(false, std::integral_constant<int, 0>{});
      open();
      read_cols(cur, 1, c1);
      read_rows(cur, 1, 0, ra_);
      unit(1, false, c0, rb_, [&](auto i) __attribute__((always_inline)) { part(i, nx1, i0, issue_x); });
      read_rows(cur, 1, 1, rb_);
      unit(0, false, c1, ra_, [&](auto i) __attribute__((always_inline)) { part(i, nx2, nx1, issue_x); });
      meet(false, std::integral_constant<int, 0>{});
      read_cols(nxt, 0, c0);
      read_rows(nxt, 0, 0, ra_);
      unit(1, false, c1, rb_, [&](auto i) __attribute__((always_inline)) { part(i, ny, i0, issue_y); });
    }
    after_first = FIRST;
  };
  const std::true_type yes;
  const std::false_type no;
  if constexpr (kSpread) {
    for (int cg = 0;;) {
      step(cg, yes, no);
      ++cg;
      advance();
      for (int cs = 2; cs < ct.nsteps; ++cs, ++cg) {
        step(cg, no, no);
        advance();
      }
      step(cg, no, yes);
      ++cg;
      if (idle) break;
      ct = pt;
      advance();
    }
#pragma unroll
    for (int i = 0; i < RH; ++i) store(RH + i);
  } else {
    int cs = 0;                             // step of the task
    for (int cg = 0;; ++cg) {
      step(cg, no, no);
      if (++cs == ct.nsteps) {
        aim();
        scales();
#pragma unroll
        for (int i = 0; i < RT; ++i) store(i);
        if (idle) break;
        ct = pt;
        cs = 0;
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int j = 0; j < CT; ++j) acc[i][j] = acc_t{0, 0, 0, 0};
      }
      advance();
    }
  }
  tg_wait<0>();                             // nothing may land in LDS after the workgroup is gone
}

// persistent workgroups: as many as are resident at once (256 CUs)
template <int T, int L, int EPI, int BM, int BN, int WR, int WC>
static hipError_t tg_start(TileParams p, hipStream_t stream) {
  const int cols = EPI == TG_OUT_GATED ? p.N / 2 : p.N;
  const int bn = EPI == TG_OUT_GATED ? BN / 2 : BN;
  p.n_tiles = (cols + bn - 1) / bn;
  if (EPI == TG_OUT_PART) p.n_tiles *= p.parts;
  p.r_tiles = (p.R + BM - 1) / BM;
  int64_t tasks;
  if (L == TG_TN || L == TG_TC) {
    tasks = static_cast<int64_t>(p.E) * p.r_tiles * p.n_tiles;
  } else {
    // at most min(E, m_total) experts have rows, each with one partial chunk
    const int64_t chunks = p.m_total / BM + (p.E < p.m_total ? p.E : p.m_total);
    tasks = chunks * p.n_tiles;
  }
  if (tasks >= (int64_t(1) << 31) - 8) return hipErrorInvalidConfiguration;
  if (tasks == 0) return hipSuccess;
  const int64_t blocks = min(int64_t(256) * tg_per_cu(BM), (tasks + 7) / 8 * 8);
  hipLaunchKernelGGL((k_tile_gemm<T, L, EPI, BM, BN, WR, WC>), dim3(static_cast<unsigned>(blocks)), dim3(64 * WR * WC), 0, stream, p);
  return hipGetLastError();
}

}  // namespace nvfp4
