// The router with scores, and the gradient of its logits.
//
//   scores    sigmoid s_e = 1 / (1 + exp(-l_e)), or softmax over the token's
//             experts whose logits are neither -inf nor NaN, whatever their bias
//   choice    by key_e = s_e + bias_e among the topk_group best of n_group groups
//             of neighbouring experts (a group's value: the sum of its group_top
//             largest keys); without a bias by the logit, which has the scores'
//             order and no saturation
//   weights   the chosen scores (without the bias), normalised to 1 or as they
//             are, times `scale`
//
// Everything that decides a choice is float64: keys that differ by less than a
// float32 step are ordered as the definition orders them, and results do not
// depend on how a float32 exponential rounds.  The kernels choose by float32 keys
// first, and take float64 ones only where two values that matter lie within the
// float32 keys' error of each other: of the candidates for their order, of one
// token's experts for its groups, of all of a token's choice where a value is not
// finite or more than 16 or 32 candidates are that close.
// Bound by latency: one chain of dependent steps a token (sort, then k rounds of
// exchanges), in one round of waves up to 16384 tokens, where neither memory (1.0 TB/s)
// nor the vector units (38 % busy; 47 with float64 scores) are full.  A launch finds
// its code in no instruction cache, and a wave that runs through 12 KB of it once waits
// some 10 us for its lines: what is rare, or long in float64, is a loop over few
// instructions.  Top-8 of 256 in 8 groups with a bias, float32: 256 tokens 7 us, 4096 9,
// 16384 15 to 17 (read at 4.86 TB/s: 3.5), with scores 26 to 27.
// An expert is closed to the choice if its logit is -inf or NaN, or its key -inf or NaN;
// closed ones are taken, by id and with weight 0, only where a token has fewer open ones
// than it needs.
#include "nvfp4_internal.h"

namespace nvfp4 {

static constexpr double kNone = -__builtin_huge_val();   // taken, behind the end, or of a group that went
static constexpr double kClosed = -1e300;                // below every open key (a float32 plus a score), above kNone

template <int DT>
__device__ __forceinline__ float rt_load(const void* base, size_t i) {
  if constexpr (DT == 0) return static_cast<const float*>(base)[i];
  if constexpr (DT == 1) return bf16_to_f32(static_cast<const uint16_t*>(base)[i]);
  return static_cast<float>(static_cast<const _Float16*>(base)[i]);
}

// NE neighbouring values from i on (those below `end`; -inf behind it).  vec: i and
// end are multiples of 4 and the row is aligned for 4 values.
template <int DT, int NE>
__device__ __forceinline__ void rt_load_row(const void* base, size_t row0, int i, int end, bool vec, float (&v)[NE]) {
  if constexpr (NE % 4 == 0) {
    if (vec) {
#pragma unroll
      for (int c = 0; c < NE; c += 4) {
        if (i + c < end) {
          if constexpr (DT == 0) {
            const float4 q = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + row0 + i + c);
            v[c] = q.x; v[c + 1] = q.y; v[c + 2] = q.z; v[c + 3] = q.w;
          } else {
            const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + row0 + i + c);
            const uint32_t u[2] = {q.x, q.y};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if constexpr (DT == 1) {
                v[c + 2 * h] = __uint_as_float(u[h] << 16);
                v[c + 2 * h + 1] = __uint_as_float(u[h] & 0xFFFF0000u);
              } else {
                const half2v f = __builtin_bit_cast(half2v, u[h]);
                v[c + 2 * h] = static_cast<float>(f[0]);
                v[c + 2 * h + 1] = static_cast<float>(f[1]);
              }
            }
          }
        } else {
          v[c] = v[c + 1] = v[c + 2] = v[c + 3] = -__builtin_huge_valf();
        }
      }
      return;
    }
  }
#pragma unroll
  for (int c = 0; c < NE; ++c) v[c] = i + c < end ? rt_load<DT>(base, row0 + i + c) : -__builtin_huge_valf();
}

// as many stores; 16 bytes at a time where rows allow
template <int NE>
__device__ __forceinline__ void rt_store_row(float* __restrict__ base, size_t row0, int i, int end, bool vec, const float (&v)[NE]) {
  if constexpr (NE % 4 == 0) {
    if (vec) {
#pragma unroll
      for (int c = 0; c < NE; c += 4)
        if (i + c < end) *reinterpret_cast<float4*>(base + row0 + i + c) = make_float4(v[c], v[c + 1], v[c + 2], v[c + 3]);
      return;
    }
  }
#pragma unroll
  for (int c = 0; c < NE; ++c)
    if (i + c < end) base[row0 + i + c] = v[c];
}

// ------------------------------------------------------------------ over the LPT (16 or 64) lanes of a token
// v of the other 16-lane row of a pair, and of the other half of the wave
__device__ __forceinline__ uint32_t rt_row_pair(uint32_t v, uint32_t& other) {
  const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  other = r[1];
  return r[0];
}
__device__ __forceinline__ uint32_t rt_half_pair(uint32_t v, uint32_t& other) {
  const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  other = r[1];
  return r[0];
}
// f over the lanes of a token, f associative and commutative (values as 32 bits)
template <int LPT, typename F>
__device__ __forceinline__ uint32_t seg_reduce(uint32_t v, F f) {
  v = f(v, dpp_u32<kDppXor1>(v));
  v = f(v, dpp_u32<kDppXor2>(v));
  v = f(v, dpp_u32<kDppHalfMirror>(v));
  v = f(v, dpp_u32<kDppMirror>(v));
  if constexpr (LPT == 64) {
    uint32_t o;
    v = rt_row_pair(v, o);
    v = f(v, o);
    v = rt_half_pair(v, o);
    v = f(v, o);
  }
  return v;
}
template <int LPT>
__device__ __forceinline__ float seg_max(float v) {
  return __uint_as_float(seg_reduce<LPT>(__float_as_uint(v), [](uint32_t a, uint32_t b) __attribute__((always_inline)) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}
template <int LPT>
__device__ __forceinline__ float seg_sum(float v) {
  return __uint_as_float(seg_reduce<LPT>(__float_as_uint(v), [](uint32_t a, uint32_t b) __attribute__((always_inline)) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}
template <int LPT>
__device__ __forceinline__ double seg_max(double v) {
#pragma unroll
  for (int d = LPT / 2; d >= 1; d >>= 1) v = fmax(v, __shfl_xor(v, d));
  return v;
}
template <int LPT>
__device__ __forceinline__ double seg_sum(double v) {
#pragma unroll
  for (int d = LPT / 2; d >= 1; d >>= 1) v += __shfl_xor(v, d);
  return v;
}
template <int LPT>
__device__ __forceinline__ uint64_t seg_ballot(bool b) {
  const uint64_t m = __ballot(b);
  if constexpr (LPT == 64) return m;
  return (m >> (threadIdx.x & 48)) & 0xFFFFull;
}

__device__ __forceinline__ float rt_finite(float l) { return fminf(l, 3.402823466e38f); }   // +inf: the largest number
__device__ __forceinline__ bool rt_open(float l) { return l > -__builtin_huge_valf(); }     // neither -inf nor NaN

// exp(x) for x <= 710 or so, without branches: 2^n times the Taylor sum of exp(r), |r| <=
// ln(2)/2, to the 12th power (the next term is below 2^-50); under- and overflow by ldexp
__device__ __forceinline__ double rt_exp(double x) {
  x = fmin(fmax(x, -800.0), 800.0);
  const double n = rint(x * 1.4426950408889634);
  double r = fma(-n, 0x1.62e42fefa39efp-1, x);
  r = fma(-n, 0x1.abc9e3b39803fp-56, r);
  double y = 1.0 / 479001600.0;
  y = fma(y, r, 1.0 / 39916800.0);
  y = fma(y, r, 1.0 / 3628800.0);
  y = fma(y, r, 1.0 / 362880.0);
  y = fma(y, r, 1.0 / 40320.0);
  y = fma(y, r, 1.0 / 5040.0);
  y = fma(y, r, 1.0 / 720.0);
  y = fma(y, r, 1.0 / 120.0);
  y = fma(y, r, 1.0 / 24.0);
  y = fma(y, r, 1.0 / 6.0);
  y = fma(y, r, 0.5);
  y = fma(y, r, 1.0);
  y = fma(y, r, 1.0);
  return ldexp(y, static_cast<int>(n));
}

// the two largest (a1 >= a2) of what two lanes hold
__device__ __forceinline__ void top2_merge(float& a1, float& a2, float b1, float b2) {
  a2 = fmaxf(fmaxf(fminf(a1, b1), a2), b2);
  a1 = fmaxf(a1, b1);
}
// ... over `s` (a power of two) neighbouring lanes
__device__ __forceinline__ void top2_lanes(float& a1, float& a2, int s) {
  auto with = [&](uint32_t b1, uint32_t b2) __attribute__((always_inline)) {
    top2_merge(a1, a2, __uint_as_float(b1), __uint_as_float(b2));
  };
  if (s > 1) with(dpp_u32<kDppXor1>(__float_as_uint(a1)), dpp_u32<kDppXor1>(__float_as_uint(a2)));
  if (s > 2) with(dpp_u32<kDppXor2>(__float_as_uint(a1)), dpp_u32<kDppXor2>(__float_as_uint(a2)));
  if (s > 4) with(dpp_u32<kDppHalfMirror>(__float_as_uint(a1)), dpp_u32<kDppHalfMirror>(__float_as_uint(a2)));
  if (s > 8) with(dpp_u32<kDppMirror>(__float_as_uint(a1)), dpp_u32<kDppMirror>(__float_as_uint(a2)));
  if (s > 16) {
    uint32_t b1, b2;
    a1 = __uint_as_float(rt_row_pair(__float_as_uint(a1), b1));
    a2 = __uint_as_float(rt_row_pair(__float_as_uint(a2), b2));
    with(b1, b2);
  }
  if (s > 32) {
    uint32_t b1, b2;
    a1 = __uint_as_float(rt_half_pair(__float_as_uint(a1), b1));
    a2 = __uint_as_float(rt_half_pair(__float_as_uint(a2), b2));
    with(b1, b2);
  }
}

__device__ __forceinline__ void rt_lds_step() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Which groups stay, by float32 keys (key(c): of the lane's expert c, -inf if there is
// none).  near: set if a group that stays and one that goes could change places: their
// values, each with the error that its own keys give it (tol + the keys' sizes, which may
// be far above that of a sum they cancel in, times 3.125 2^-24), are not clear of each
// other.  Returns a bit for each of the lane's experts that stays.  lds: E + 2 n_group
// floats of the token's own, where no lanes' borders follow the groups'.
template <int LPT, int NE, typename K>
__device__ __forceinline__ uint32_t scored_groups(const ScoredParams& p, K key, float tol, float* lds, bool& near) {
  const float none = -__builtin_huge_valf();
  const int l = threadIdx.x & (LPT - 1);
  const int e0 = l * NE;
  const int gs = p.E / p.n_group;
  auto value = [&](float a1, float a2) __attribute__((always_inline)) { return p.group_top == 2 ? a1 + a2 : a1; };
  auto error = [&](float a1, float a2) __attribute__((always_inline)) {
    return fmaf(p.group_top == 2 ? fabsf(a1) + fabsf(a2) : fabsf(a1), 0x1.9p-23f, tol);
  };
  float last = -none, next = none;          // the least that a group that stays, and the most that one that goes, may be worth
  uint32_t stays = 0;
  if (p.lanes_per_group) {
    const int s = p.lanes_per_group;
    float a1 = none, a2 = none;
#pragma unroll
    for (int c = 0; c < NE; ++c) {
      const float k = key(c);
      a2 = __builtin_amdgcn_fmed3f(a1, a2, k);
      a1 = fmaxf(a1, k);
    }
    top2_lanes(a1, a2, s);
    const float v = value(a1, a2), err = error(a1, a2);
    const int g = l / s;
    int rank = 0;
    for (int h0 = 0; h0 < p.n_group; h0 += 4) {              // four exchanges at a time
      float o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = __shfl(v, min(h0 + i, p.n_group - 1) * s, LPT);
#pragma unroll
      for (int i = 0; i < 4; ++i) rank += h0 + i < p.n_group && o[i] > v ? 1 : 0;
    }
    if (g < p.n_group) {
      if (rank < p.topk_group) {
        stays = ~0u;
        last = v - err;
      } else {
        next = v + err;
      }
      near |= !(err < -none);                // a sum beyond float32's range
    }
    // equal values at the border all stay, and are then too many
    near |= __popcll(seg_ballot<LPT>(g < p.n_group && stays != 0)) != p.topk_group * s;
  } else {
    // keys by way of LDS, a group's behind those of the one before it and a gap (no bank twice)
    float* const val = lds + p.E + p.n_group;
#pragma unroll
    for (int c = 0; c < NE; ++c) {
      const int e = e0 + c;
      if (e < p.E) lds[e + e / gs] = key(c);
    }
    rt_lds_step();
    for (int g = l; g < p.n_group; g += LPT) {
      float a1 = none, a2 = none;
      for (int i = 0; i < gs; ++i) {
        const float k = lds[g * (gs + 1) + i];
        a2 = __builtin_amdgcn_fmed3f(a1, a2, k);
        a1 = fmaxf(a1, k);
      }
      val[g] = value(a1, a2);
      lds[g * (gs + 1) + gs] = error(a1, a2);                // in the gap behind the group
    }
    rt_lds_step();
    int count = 0;
    for (int g = l; g < p.n_group; g += LPT) {
      const float v = val[g];
      int rank = 0;
      for (int h = 0; h < p.n_group; ++h) rank += val[h] > v ? 1 : 0;
      const bool in = rank < p.topk_group;
      const float err = lds[g * (gs + 1) + gs];
      count += in ? 1 : 0;
      lds[g * (gs + 1) + gs] = in ? 1.0f : 0.0f;             // the error's place, read by this lane alone
      last = in ? fminf(last, v - err) : last;
      next = in ? next : fmaxf(next, v + err);
      near |= !(err < -none);
    }
    rt_lds_step();
#pragma unroll
    for (int c = 0; c < NE; ++c) {
      const int e = e0 + c;
      if (e < p.E && lds[(e / gs) * (gs + 1) + gs] != 0.0f) stays |= 1u << c;
    }
    rt_lds_step();                          // the same words are written again
    near |= seg_sum<LPT>(static_cast<float>(count)) != static_cast<float>(p.topk_group);
  }
  last = -seg_max<LPT>(-last);
  next = seg_max<LPT>(next);
  near |= !(last > next);
  return stays;
}

// Scores of all experts in float64 by N lanes, four neighbours at a time: f(i, x, s) for
// i to i + 3, closed ones (and those past E) with score 0.  Returns the softmax's sum
// (1 for a sigmoid).  Four chains of float64 steps a lane hide their latency; all 16 of a
// row at once are 6 KB of code, which costs a cold launch more than the loop.
template <int N, int DT, typename F>
__device__ __forceinline__ double scores64(const ScoredParams& p, size_t row, int l, double top, F f) {
  double z = 1.0;
  for (int pass = p.softmax ? 0 : 1; pass < 2; ++pass) {
    double sum = 0.0;
    for (int i = 4 * l; i < p.E; i += 4 * N) {
      float x[4];
      double s[4];
      rt_load_row<DT, 4>(p.logits, row, i, p.E, p.vec, x);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const double v = static_cast<double>(rt_finite(x[c]));
        const double e = rt_exp(p.softmax ? v - top : -v);
        s[c] = rt_open(x[c]) ? (p.softmax ? e : 1.0 / (1.0 + e)) : 0.0;
        sum += s[c];
      }
      if (pass == 0) continue;
      if (p.softmax) {
#pragma unroll
        for (int c = 0; c < 4; ++c) s[c] /= z;
      }
      f(i, x, s);
    }
    if (pass == 0) {
      z = seg_sum<N>(sum);
      z = z > 0.0 ? z : 1.0;
    }
  }
  return z;
}

// Float64 keys of one token by the whole wave, expert e at lds[rt_at(p, e)] (E + 2 n_group
// doubles of the wave's own; closed experts kClosed).  Returns a bit for each group that
// stays.
__device__ __forceinline__ int rt_at(const ScoredParams& p, int e) { return p.n_group > 1 ? e + e / (p.E / p.n_group) : e; }
template <int DT>
__device__ __forceinline__ uint64_t exact_groups(const ScoredParams& p, int t, double* lds) {
  const int l = threadIdx.x & 63;
  const size_t row = static_cast<size_t>(t) * p.E;
  const int gs = p.E / p.n_group;
  double top = 0.0;
  if (p.softmax) {
    float m = -__builtin_huge_valf();
    for (int i = l; i < p.E; i += 64) {
      const float x = rt_load<DT>(p.logits, row + i);
      m = rt_open(x) ? fmaxf(m, rt_finite(x)) : m;
    }
    m = seg_max<64>(m);
    top = rt_open(m) ? m : 0.0f;
  }
  if (p.bias || p.n_group > 1) {
    scores64<64, DT>(p, row, l, top, [&](int i, const float (&x)[4], const double (&s)[4]) __attribute__((always_inline)) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (i + c >= p.E) break;
        const double v = s[c] + (p.bias ? static_cast<double>(p.bias[i + c]) : 0.0);
        lds[rt_at(p, i + c)] = rt_open(x[c]) && v > kNone ? v : kClosed;
      }
    });
  }
  rt_lds_step();
  if (p.n_group == 1) return ~0ull;
  double* const val = lds + p.E + p.n_group;
  // the lanes of a group (a power of two) take its keys in turn and join theirs
  int parts = 1;
  while (2 * parts * p.n_group <= 64) parts *= 2;
  const int g = l / parts;
  double a1 = kNone, a2 = kNone;
  auto add = [&](double b1, double b2) __attribute__((always_inline)) {
    a2 = fmax(fmin(a1, b1), fmax(a2, b2));
    a1 = fmax(a1, b1);
  };
  for (int i = l % parts; i < gs; i += parts) {
    const double k = g < p.n_group ? lds[g * (gs + 1) + i] : kNone;
    add(k > kClosed ? k : kNone, kNone);
  }
  for (int d = 1; d < parts; d *= 2) {
    const double b1 = __shfl_xor(a1, d), b2 = __shfl_xor(a2, d);
    add(b1, b2);
  }
  if (g < p.n_group && l % parts == 0) val[g] = p.group_top == 2 && a2 > kNone ? a1 + a2 : a1;
  rt_lds_step();
  const double mine = val[l < p.n_group ? l : 0];
  int rank = 0;
  for (int h = 0; h < p.n_group; ++h) rank += val[h] > mine || (val[h] == mine && h < l) ? 1 : 0;
  rt_lds_step();                            // the same words are written again
  return __ballot(l < p.n_group && rank < p.topk_group);
}

// The choice by float64 keys, one token on the whole wave: k rounds of the best that is
// left, ties to the lower id.  Lane l holds experts l, l + 64, ... in LDS.  Lanes meet on
// the float32 roundings of their best (rounding keeps the order), and only a tie there
// looks at the float64 keys and ids.  list[j] gets the j-th, with bit 30 set if it is open.
template <int DT>
__device__ __forceinline__ void choose_exact(const ScoredParams& p, int t, double* lds, int* list) {
  const int l = threadIdx.x & 63;
  const size_t row = static_cast<size_t>(t) * p.E;
  const int gs = p.E / p.n_group;
  const uint64_t stay = exact_groups<DT>(p, t, lds);
  for (int i = l; i < p.E; i += 64) {
    double* const k = lds + rt_at(p, i);
    if (!p.bias) {
      const float x = rt_load<DT>(p.logits, row + i);
      *k = rt_open(x) ? static_cast<double>(rt_finite(x)) : kClosed;
    }
    if (p.n_group > 1 && !((stay >> (i / gs)) & 1)) *k = kNone;
  }
  rt_lds_step();
  double best = kNone;
  int id = 0x7fffffff;
  auto scan = [&]() __attribute__((always_inline)) {
    best = kNone;
    id = 0x7fffffff;
    for (int i = l; i < p.E; i += 64) {
      const double k = lds[rt_at(p, i)];
      if (k > best) {
        best = k;
        id = i;
      }
    }
  };
  scan();
  for (int j = 0; j < p.k; ++j) {
    const float h = static_cast<float>(best);
    const float m = seg_max<64>(h);
    uint64_t who = __ballot(h == m);
    if (who & (who - 1)) {
      const double b = h == m ? best : kNone;
      const double most = seg_max<64>(b);    // by every lane of the wave
      const uint32_t first = seg_reduce<64>(h == m && b == most ? static_cast<uint32_t>(id) : 0xffffffffu,
                                            [](uint32_t a, uint32_t b) __attribute__((always_inline)) { return a < b ? a : b; });
      who = __ballot(h == m && b == most && static_cast<uint32_t>(id) == first);
    }
    const int w = __builtin_ctzll(who);
    if (l == w) {
      list[j] = id | (best > kClosed ? 1 << 30 : 0);
      lds[rt_at(p, id)] = kNone;
      scan();
    }
  }
  rt_lds_step();
}

// float32 bits in an order of unsigned integers (0 below all numbers)
__device__ __forceinline__ uint32_t rt_order(float f) {
  const uint32_t u = __float_as_uint(f);
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float rt_unorder(uint32_t u) {
  return __uint_as_float(u ^ (static_cast<uint32_t>(static_cast<int32_t>(~u) >> 31) | 0x80000000u));
}

// v[0 .. N) in descending order: Batcher's odd-even merge sort (two instructions an exchange)
template <int N>
__device__ __forceinline__ void rt_sort(uint32_t (&v)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            const uint32_t a = v[i + j], b = v[i + j + k];
            v[i + j] = a > b ? a : b;
            v[i + j + k] = a > b ? b : a;
          }
}

// The choice by float32 keys, of tokens whose logits (and biases) are all finite.
// list (32 ints of the token's own) gets n candidates, k or a few more, that hold the
// k chosen.  Returns n; order: the float32 keys do not settle their order; near: nor,
// with up to LPT candidates, that they are all, or which groups stay, or a value is not
// finite.
//
// An expert's key is an unsigned integer with its place in the lane in the low bits
// (so the key loses log2(NE) bits).  Each lane sorts its own, and then the lanes
// compare their first ones and one of them drops it, k times and on until a key is
// clearly smaller: 1 instruction a key and round in place of 4 for a search through
// all.
//
// Errors, in steps of 2^-24: a sigmoid from v_exp_f32 and v_rcp_f32 (1 ulp each) is off
// by s (1 - s) (|x| + 2) + 3 s < 3.2, a softmax by p (|x - max| + 35) (exp; sums of 16
// and over 6 levels; quotient), which is below 36 max p as |x - max| p <= 0.37 max p; the
// bias adds |key|, the lost bits |key| 2^5 for 16 places.  So two keys further apart than
// tol + |key| 2^-18, tol 8 steps or 128 max p, are in order (logits as keys if they differ
// at all).  A group's value, of up to two keys a with all their bits, is off by twice 3.2
// steps or 36 max p, by sum |a| for the keys' additions and, at most as much each, for
// their own and that of the bound: below tol + 3.125 sum |a| steps (the k-th largest of
// keys that are off by an error that grows with their size is off by that at its own).
// A masked group of -1e9, say, thus makes nothing near but its like.
template <int LPT, int NE, int DT>
__device__ __forceinline__ int choose_fast(const ScoredParams& p, int t, const float (&x)[NE], const float (&bias)[NE], float top,
                                           float z, double* lds, int* list, bool& order, bool& near) {
  constexpr uint32_t LOW = NE <= 4 ? 3 : 15;
  static_assert(NE <= 16, "the place takes 4 bits");
  const int l = threadIdx.x & (LPT - 1);
  const int e0 = l * NE;
  const bool full = p.E == LPT * NE;
  float key[NE];
  float big = 1.0f;                          // of a sigmoid
  float odd = 0.0f;                          // NaN if any value is not finite
#pragma unroll
  for (int c = 0; c < NE; ++c) odd = full || e0 + c < p.E ? fmaf(x[c], 0.0f, odd) : odd;
  if (p.bias || p.n_group > 1) {
    if (p.softmax) big = __builtin_amdgcn_rcpf(z);                      // the largest p
#pragma unroll
    for (int c = 0; c < NE; ++c)
      key[c] = p.softmax ? __builtin_amdgcn_exp2f((x[c] - top) * 1.44269504f) * big
                         : __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x[c] * -1.44269504f));
    if (p.bias) {
#pragma unroll
      for (int c = 0; c < NE; ++c) {
        odd = full || e0 + c < p.E ? fmaf(bias[c], 0.0f, odd) : odd;
        key[c] += bias[c];
      }
    }
  }
  near = seg_ballot<LPT>(!(odd == 0.0f)) != 0;               // NaN
  const float none = -__builtin_huge_valf();
  const float tol = p.softmax ? big * 0x1p-17f : 0x1p-21f;
  uint32_t keep = ~0u;
  if (p.n_group > 1) {
    const int base = (threadIdx.x & 63) & ~(LPT - 1);
    bool close = false;
    keep = scored_groups<LPT, NE>(p, [&](int c) __attribute__((always_inline)) { return full || e0 + c < p.E ? key[c] : none; },
                                  tol, reinterpret_cast<float*>(lds) + base / LPT * (p.E + 2 * p.n_group), close);
    close = seg_ballot<LPT>(close) != 0 && !near;
    // such tokens of the wave one after the other, on all its lanes
    for (uint64_t rest = __ballot(close && l == 0); rest; rest &= rest - 1) {
      const int at = __builtin_ctzll(rest);
      const uint64_t stay = exact_groups<DT>(p, __builtin_amdgcn_readlane(t, at), lds);
      if (base != at) continue;
      keep = 0;
      const int gs = p.E / p.n_group;
#pragma unroll 1
      for (int c = 0; c < NE; ++c) keep |= e0 + c < p.E && ((stay >> ((e0 + c) / gs)) & 1) ? 1u << c : 0u;
    }
  }
  if (!full) keep &= e0 >= p.E ? 0u : p.E - e0 >= 32 ? ~0u : (1u << (p.E - e0)) - 1;
  // by logits: the keys are exact but for the lost bits, and 16-bit ones keep theirs.  The
  // addition makes a zero of either sign the same one
  const bool exact = !p.bias && p.narrow;
  uint32_t el[NE];
#pragma unroll
  for (int c = 0; c < NE; ++c) {
    const uint32_t there = static_cast<uint32_t>(static_cast<int32_t>(keep << (31 - c)) >> 31);
    el[c] = ((rt_order((p.bias ? key[c] : x[c]) + 0.0f) & ~LOW) | (LOW - c)) & there;
  }
  rt_sort<NE>(el);
  order = false;
  float before = __builtin_huge_valf();
  int n = 0;
  bool more = true;
  for (int j = 0; __any(more); ++j) {
    const uint32_t first = el[0] & ~LOW;
    const uint32_t m = seg_reduce<LPT>(first, [](uint32_t a, uint32_t b) __attribute__((always_inline)) { return a > b ? a : b; });
    const float v = rt_unorder(m);
    const bool close = !exact && m != 0 && before - v <= (p.bias ? tol + fabsf(v) * 0x1p-18f : 0.0f);
    before = v;
    more = more && (j < p.k || close);
    if (more && j >= (LPT < 32 ? LPT : 32)) {
      near = true;
      more = false;
    }
    order |= more && close;
    n += more ? 1 : 0;
    const bool mine = l == __builtin_ctzll(seg_ballot<LPT>(first == m));
    if (mine && more) list[j] = (e0 + static_cast<int>(LOW - (el[0] & LOW))) | (1 << 30);
#pragma unroll
    for (int c = 0; c < NE - 1; ++c) el[c] = mine ? el[c + 1] : el[c];
    if (mine) el[NE - 1] = 0;
  }
  near = seg_ballot<LPT>(near) != 0;         // over the token's lanes
  return n;
}

// One token on LPT lanes, expert l * NE + c in register c of lane l (NE 0: none, the
// float64 choice at once).  Writes ids, weights and (if wanted) scores.  Returns the place
// among the k chosen of the expert and weight that the lane holds, or k.  lds: lds_wave
// doubles of the wave's own; list: 32 ints of the token's own.  Lanes of a token past T
// take part on the last token's values and write nothing.
template <int LPT, int NE, int DT>
__device__ __forceinline__ int scored_token(const ScoredParams& p, int t, bool live, double* lds, int* list, int& my_id, float& my_w) {
  const int l = threadIdx.x & (LPT - 1);
  const size_t row = static_cast<size_t>(t) * p.E;
  double top = 0.0, z = 0.0;
  int n = p.k;
  bool order = false, near = true;
  if constexpr (NE > 0) {
    const int e0 = l * NE;
    float x[NE], bias[NE];
    rt_load_row<DT, NE>(p.logits, row, e0, p.E, p.vec, x);
    if (p.bias) rt_load_row<0, NE>(p.bias, 0, e0, p.E, p.vec_bias, bias);
    float zf = 1.0f;
    if (p.softmax) {
      float m = -__builtin_huge_valf();
#pragma unroll
      for (int c = 0; c < NE; ++c) m = rt_open(x[c]) ? fmaxf(m, rt_finite(x[c])) : m;
      m = seg_max<LPT>(m);
      top = rt_open(m) ? m : 0.0f;
      if (p.bias || p.n_group > 1) {
        zf = 0.0f;
#pragma unroll
        for (int c = 0; c < NE; ++c)
          zf += rt_open(x[c]) ? __builtin_amdgcn_exp2f((rt_finite(x[c]) - static_cast<float>(top)) * 1.44269504f) : 0.0f;
        zf = seg_sum<LPT>(zf);
        zf = zf > 0.0f ? zf : 1.0f;
      }
    }
    n = choose_fast<LPT, NE, DT>(p, t, x, bias, static_cast<float>(top), zf, lds, list, order, near);
  } else if (p.softmax) {
    float m = -__builtin_huge_valf();
    for (int i = l; i < p.E; i += LPT) {
      const float x = rt_load<DT>(p.logits, row + i);
      m = rt_open(x) ? fmaxf(m, rt_finite(x)) : m;
    }
    m = seg_max<LPT>(m);
    top = rt_open(m) ? m : 0.0f;
  }
  // the tokens of the wave that are not settled, one after the other on all its lanes
  rt_lds_step();
  const int base = (threadIdx.x & 63) & ~(LPT - 1);
  for (uint64_t rest = __ballot(near && l == 0); rest; rest &= rest - 1) {
    const int at = __builtin_ctzll(rest);
    choose_exact<DT>(p, __builtin_amdgcn_readlane(t, at), lds, list + (at - base) / LPT * 32);
  }
  if (near) {
    n = p.k;
    order = false;
  }
  rt_lds_step();
  if (p.scores || (p.softmax && (!p.renormalize || (p.bias && __any(order)))))
    z = scores64<LPT, DT>(p, row, l, top, [&](int i, const float (&)[4], const double (&s)[4]) __attribute__((always_inline)) {
      if (!p.scores || !live) return;
      const float v[4] = {static_cast<float>(s[0]), static_cast<float>(s[1]), static_cast<float>(s[2]), static_cast<float>(s[3])};
      rt_store_row<4>(p.scores, row, i, p.E, p.vec_scores, v);
    });

  // the candidates' scores, one a lane.  Renormalised softmax: relative to the largest
  // chosen logit, which divides out; renormalised sigmoids of logits below -500 times
  // exp(-largest), likewise: scores that would underflow together keep their ratios.
  // (A candidate that is not chosen may have a logit hundreds above them, where keys tie.)
  const int packed = l < n ? list[l] : 0;
  my_id = packed & 0xFFFF;
  const bool open = l < n && (packed >> 30) != 0;
  const float xj = open ? rt_finite(rt_load<DT>(p.logits, row + my_id)) : 0.0f;
  const bool ratios = p.softmax && p.renormalize;
  double u = 0.0;
  if (!ratios || (p.bias && __any(order))) {
    u = rt_exp(p.softmax ? static_cast<double>(xj) - top : -static_cast<double>(xj));
    u = p.softmax ? u / z : 1.0 / (1.0 + u);
  }
  int place = l < n ? l : p.k;
  if (__any(order)) {
    // in the order of the float64 keys, ties to the lower id
    double key = p.bias ? u + static_cast<double>(p.bias[my_id]) : static_cast<double>(xj);
    if (!open) key = kClosed;
    int rank = 0;
    for (int i = 0; i < (LPT < 32 ? LPT : 32); ++i) {
      const double o = __shfl(key, i, LPT);
      const int oid = __shfl(l < n ? my_id : 0x7fffffff, i, LPT);
      rank += oid != 0x7fffffff && (o > key || (o == key && oid < my_id)) ? 1 : 0;
    }
    if (order) place = l < n ? rank : p.k;
  }
  const bool chosen = open && place < p.k;
  const float most = seg_max<LPT>(chosen ? xj : -__builtin_huge_valf());
  if (ratios) u = rt_exp(chosen ? static_cast<double>(xj) - static_cast<double>(most) : 0.0);
  else if (p.renormalize && most < -500.0f)
    u = 1.0 / (rt_exp(most) + rt_exp(chosen ? static_cast<double>(most) - static_cast<double>(xj) : 0.0));
  u = chosen ? u : 0.0;
  if (p.renormalize) {
    const double s = seg_sum<LPT>(u);
    u = s > 0.0 ? u / s : 0.0;
  }
  my_w = static_cast<float>(u * static_cast<double>(p.scale));
  if (live && place < p.k) {
    const size_t at = static_cast<size_t>(t) * p.k + place;
    p.topk_ids[at] = my_id;
    p.topk_w[at] = my_w;
  }
  return place;
}

constexpr int rt_threads(int ne) { return ne ? 256 : 64; }    // without registers a token takes up to 34 KB of LDS
template <int LPT, int NE, int DT>
__global__ __launch_bounds__(rt_threads(NE)) void k_route_scored(const ScoredParams p) {
  extern __shared__ double lds[];
  constexpr int kTokens = rt_threads(NE) / LPT;
  __shared__ int list[kTokens][32];
  const int sub = threadIdx.x / LPT;
  const int t = blockIdx.x * kTokens + sub;
  int id;
  float w;
  scored_token<LPT, NE, DT>(p, min(t, p.T - 1), t < p.T, lds + static_cast<size_t>(threadIdx.x >> 6) * p.lds_wave, list[sub], id, w);
}

// ------------------------------------------------------------------ few tokens: routing and permutation in one launch
// One workgroup: wave w routes tokens w, w + 16, ...; then every assignment counts
// the earlier ones of its expert (n <= kSmallRows: a walk over LDS), and a scan of
// the experts' counts places the rows.  Bound by latency: 7.5 us for one token, against
// 7 + 4 + 3.5 in the three launches of more.
static constexpr int kSmallRows = 256;
template <int NE, int DT>
__global__ __launch_bounds__(1024) void k_route_small(const ScoredParams p, int* __restrict__ counts, int* __restrict__ offsets,
                                                      int* __restrict__ src, int* __restrict__ row_of, float* __restrict__ row_w) {
  extern __shared__ double lds[];
  __shared__ int cnt[256];                 // E <= 256
  __shared__ int ids[kSmallRows];
  __shared__ float ws[kSmallRows];
  __shared__ int list[16][32];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n = p.T * p.k;
  for (int e = tid; e < p.E; e += 1024) cnt[e] = 0;
  for (int t = wave; t < p.T; t += 16) {
    int id;
    float w;
    const int place = scored_token<64, NE, DT>(p, t, true, lds + static_cast<size_t>(wave) * p.lds_wave, list[wave], id, w);
    if (place < p.k) {
      ids[t * p.k + place] = id;
      ws[t * p.k + place] = w;
    }
  }
  __syncthreads();
  int rank = 0;
  if (tid < n) {
    const int id = ids[tid];
    for (int i = 0; i < n; ++i) rank += (i < tid && ids[i] == id) ? 1 : 0;
    atomicAdd(&cnt[id], 1);
  }
  __syncthreads();
  // one wave, 4 neighbouring experts a lane
  if (wave == 0) {
    int c[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = 4 * lane + i;
      c[i] = e < p.E ? cnt[e] : 0;
      sum += c[i];
    }
    int incl = sum;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(incl, d);
      if (lane >= d) incl += v;
    }
    int run = incl - sum;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = 4 * lane + i;
      if (e < p.E) {
        counts[e] = c[i];
        offsets[e] = run;
        cnt[e] = run;
      }
      run += c[i];
    }
    if (lane == 0) offsets[p.E] = n;
  }
  __syncthreads();
  if (tid < n) {
    const int r = cnt[ids[tid]] + rank;
    src[r] = tid / p.k;
    row_of[tid] = r;
    if (row_w) row_w[r] = ws[tid];
  }
}

// ------------------------------------------------------------------ gradient
// With n_j the normalised chosen scores and g_j the weights' gradients, the part
// that reaches expert id_j through its weight is, as s_j dL/ds_j,
//   renormalised c_j = scale n_j (g_j - sum_i g_i n_i), else c_j = scale s_j g_j;
// the logits then get
//   sigmoid (1 - s_e) (c_e + s_e q_e),   softmax c_e - s_e sum(c) + s_e (q_e - sum(s q))
// with q the scores' own gradient.  Nothing is divided by a small score that way.
// All in float32: one read of logits (and q), one write of the gradient.  16384 tokens,
// 256 experts, float32 with q: 14 us for 50 MB (3.6 TB/s); 2051 tokens in bf16 6.
template <int LPT, int NE, int DT>
__global__ __launch_bounds__(256) void k_route_scored_grad(const ScoredGradParams p) {
  const int t0 = blockIdx.x * (256 / LPT) + threadIdx.x / LPT;
  const bool live = t0 < p.T;
  const int t = live ? t0 : p.T - 1;
  const int l = threadIdx.x & (LPT - 1);
  const int base = (threadIdx.x & 63) & ~(LPT - 1);
  const int e0 = l * NE;
  const size_t row = static_cast<size_t>(t) * p.E;
  float x[NE], s[NE], rest[NE], q[NE];
  rt_load_row<DT, NE>(p.logits, row, e0, p.E, p.vec, x);
  if (p.d_scores) {
    rt_load_row<0, NE>(p.d_scores, static_cast<size_t>(t) * p.d_scores_ld, e0, p.E, p.vec_d, q);
#pragma unroll
    for (int c = 0; c < NE; ++c) q[c] = rt_open(x[c]) ? q[c] : 0.0f;     // the score of -inf or NaN is 0 whatever the others
  } else {
#pragma unroll
    for (int c = 0; c < NE; ++c) q[c] = 0.0f;
  }
  // the chosen, one a lane.  Closed by its logit: score 0; by the bias: weight 0, told
  // by the bias alone (the score of an open logit is finite)
  int id = -1;
  float g = 0.0f;
  if (l < p.k) {
    const size_t at = static_cast<size_t>(t) * p.k + l;
    id = p.topk_ids[at];
    g = p.d_topk_w[at];
    if (id < 0 || id >= p.E) id = -1;
  }
  bool open = false;
  float xj = 0.0f;
  if (id >= 0) {
    xj = rt_load<DT>(p.logits, row + id);
    open = rt_open(xj) && (!p.bias || p.bias[id] > -__builtin_huge_valf());
    xj = rt_finite(xj);
  }
  auto e2 = [](float v) __attribute__((always_inline)) { return __builtin_amdgcn_exp2f(v * 1.44269504f); };   // exp(v): |v| + 2 half steps off
  float top = 0.0f, z = 1.0f;
  if (p.softmax) {
    float m = -__builtin_huge_valf();
#pragma unroll
    for (int c = 0; c < NE; ++c) m = rt_open(x[c]) ? fmaxf(m, rt_finite(x[c])) : m;
    m = seg_max<LPT>(m);
    top = rt_open(m) ? m : 0.0f;
    z = 0.0f;
#pragma unroll
    for (int c = 0; c < NE; ++c) {
      s[c] = rt_open(x[c]) ? e2(rt_finite(x[c]) - top) : 0.0f;
      z += s[c];
    }
    z = seg_sum<LPT>(z);
    z = __builtin_amdgcn_rcpf(z > 0.0f ? z : 1.0f);
#pragma unroll
    for (int c = 0; c < NE; ++c) s[c] *= z;
  } else {
    // 1 - s from exp(x) of its own: no cancellation
#pragma unroll
    for (int c = 0; c < NE; ++c) {
      const float a = rt_finite(x[c]), n = e2(-a), m = e2(a);
      s[c] = rt_open(x[c]) ? __builtin_amdgcn_rcpf(1.0f + n) : 0.0f;
      rest[c] = rt_open(x[c]) ? __builtin_amdgcn_rcpf(1.0f + m) : 0.0f;
    }
  }
  float u;
  if (p.softmax && p.renormalize) {
    // relative to the largest chosen logit: their own softmax, whatever the others hold
    const float m = seg_max<LPT>(open ? xj : -__builtin_huge_valf());
    u = open ? e2(xj - m) : 0.0f;
  } else if (p.softmax) {
    u = open ? e2(xj - top) * z : 0.0f;
  } else if (p.renormalize) {
    const float m = seg_max<LPT>(open ? xj : -__builtin_huge_valf());
    const float b = fminf(m, 0.0f);
    u = open ? __builtin_amdgcn_rcpf(e2(b) + e2(b - xj)) : 0.0f;
  } else {
    u = open ? __builtin_amdgcn_rcpf(1.0f + e2(-xj)) : 0.0f;
  }
  float cj;
  if (p.renormalize) {
    const float sum = seg_sum<LPT>(u);
    const float n = sum > 0.0f ? u * __builtin_amdgcn_rcpf(sum) : 0.0f;
    const float mean = seg_sum<LPT>(n > 0.0f ? n * g : 0.0f);
    cj = n > 0.0f ? p.scale * n * (g - mean) : 0.0f;
  } else {
    cj = u > 0.0f ? p.scale * u * g : 0.0f;
  }
  float less = 0.0f;                         // what every score of a softmax gets off
  if (p.softmax) {
    if (p.d_scores) {
#pragma unroll
      for (int c = 0; c < NE; ++c) less += s[c] * q[c];
      less = seg_sum<LPT>(less);
    }
    if (!p.renormalize) less += seg_sum<LPT>(cj);
  }
  // what reaches the lane's experts through the weights
  float cw[NE];
#pragma unroll
  for (int c = 0; c < NE; ++c) cw[c] = 0.0f;
  for (int j = 0; j < p.k; ++j) {
    const int ij = __shfl(id, base + j);
    const float vj = __shfl(cj, base + j);
#pragma unroll
    for (int c = 0; c < NE; ++c) cw[c] += ij == e0 + c ? vj : 0.0f;
  }
  if (!live) return;
  float d[NE];
#pragma unroll
  for (int c = 0; c < NE; ++c) {
    d[c] = p.softmax ? cw[c] + s[c] * (q[c] - less) : rest[c] * (cw[c] + s[c] * q[c]);
    if (!rt_open(x[c])) d[c] = 0.0f;
  }
  if constexpr (DT == 0) {
    rt_store_row<NE>(static_cast<float*>(p.dlogits), row, e0, p.E, p.vec_out, d);
  } else {
    if constexpr (NE % 4 == 0) {
      if (p.vec_out) {
#pragma unroll
        for (int c = 0; c < NE; c += 4) {
          if (e0 + c >= p.E) continue;
          uint2 r;
          if constexpr (DT == 1) {
            typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
            const bf16x4 v = {static_cast<__bf16>(d[c]), static_cast<__bf16>(d[c + 1]), static_cast<__bf16>(d[c + 2]), static_cast<__bf16>(d[c + 3])};
            r = __builtin_bit_cast(uint2, v);
          } else {
            typedef _Float16 half4 __attribute__((ext_vector_type(4)));
            const half4 v = {static_cast<_Float16>(d[c]), static_cast<_Float16>(d[c + 1]), static_cast<_Float16>(d[c + 2]), static_cast<_Float16>(d[c + 3])};
            r = __builtin_bit_cast(uint2, v);
          }
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.dlogits) + row + e0 + c) = r;
        }
        return;
      }
    }
#pragma unroll
    for (int c = 0; c < NE; ++c) {
      if (e0 + c >= p.E) continue;
      if constexpr (DT == 1) static_cast<__bf16*>(p.dlogits)[row + e0 + c] = static_cast<__bf16>(d[c]);
      else static_cast<_Float16*>(p.dlogits)[row + e0 + c] = static_cast<_Float16>(d[c]);
    }
  }
}

// ------------------------------------------------------------------ host side
// 16 lanes a token where its experts fit 16 registers a lane and there are tokens
// enough to fill the chip that way: the rounds then serve 4 tokens a wave (256 tokens
// 8.4 us against 7.1 on 64 lanes, 2047 9.0 against 9.6; with float64 scores of all
// experts 2051 tokens 12.4 against 11.0 and in bf16 13.0 against 9.1, 4096 13.8 against
// 14.6, 8192 16.6 against 23.7).
static bool rt_narrow(int T, int E, int k, bool scores) { return E <= 256 && k <= 16 && T >= (scores ? 4096 : 2048); }

// lanes of a group if groups end between lanes and a butterfly joins them, else 0 (by way of LDS)
static int rt_lanes_per_group(int E, int n_group, int ne) {
  const int gs = E / n_group;
  if (n_group <= 1 || gs % ne != 0) return 0;
  const int s = gs / ne;
  return (s & (s - 1)) == 0 ? s : 0;
}

// doubles of LDS a wave: the float64 choice's of one token, or the float32 one's of each of its tokens
static int rt_lds_wave(const ScoredParams& p, int lpt) {
  const int one = p.E + 2 * p.n_group;
  return p.n_group > 1 && !p.lanes_per_group && lpt < 64 ? (64 / lpt * one + 1) / 2 : one;
}

template <int LPT, int NE>
static hipError_t rt_start(ScoredParams p, int dtype, hipStream_t stream) {
  constexpr int kThreads = rt_threads(NE);
  p.lanes_per_group = NE ? rt_lanes_per_group(p.E, p.n_group, NE ? NE : 1) : 0;
  p.lds_wave = rt_lds_wave(p, LPT);
  constexpr int kTokens = kThreads / LPT;
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(p.T) + kTokens - 1) / kTokens));
  const size_t lds = static_cast<size_t>(kThreads / 64) * p.lds_wave * sizeof(double);
  if (dtype == 0) hipLaunchKernelGGL((k_route_scored<LPT, NE, 0>), grid, dim3(kThreads), lds, stream, p);
  else if (dtype == 1) hipLaunchKernelGGL((k_route_scored<LPT, NE, 1>), grid, dim3(kThreads), lds, stream, p);
  else hipLaunchKernelGGL((k_route_scored<LPT, NE, 2>), grid, dim3(kThreads), lds, stream, p);
  return hipGetLastError();
}

template <int NE>
static hipError_t rt_start_small(ScoredParams p, int dtype, int* counts, int* offsets, int* src, int* row_of, float* row_w,
                                 hipStream_t stream) {
  p.lanes_per_group = rt_lanes_per_group(p.E, p.n_group, NE);
  p.lds_wave = rt_lds_wave(p, 64);
  const size_t lds = static_cast<size_t>(16) * p.lds_wave * sizeof(double);
  if (dtype == 0)
    hipLaunchKernelGGL((k_route_small<NE, 0>), dim3(1), dim3(1024), lds, stream, p, counts, offsets, src, row_of, row_w);
  else if (dtype == 1)
    hipLaunchKernelGGL((k_route_small<NE, 1>), dim3(1), dim3(1024), lds, stream, p, counts, offsets, src, row_of, row_w);
  else
    hipLaunchKernelGGL((k_route_small<NE, 2>), dim3(1), dim3(1024), lds, stream, p, counts, offsets, src, row_of, row_w);
  return hipGetLastError();
}

hipError_t launch_route_scored(const ScoredParams& q, int dtype, int* counts, int* offsets, int* src, int* row_of, float* row_w,
                               void* ws, hipStream_t stream) {
  ScoredParams p = q;
  p.narrow = dtype != 0;
  p.vec = p.E % 4 == 0 && reinterpret_cast<uintptr_t>(p.logits) % (dtype == 0 ? 16 : 8) == 0;
  p.vec_bias = p.E % 4 == 0 && reinterpret_cast<uintptr_t>(p.bias) % 16 == 0;
  p.vec_scores = p.E % 4 == 0 && reinterpret_cast<uintptr_t>(p.scores) % 16 == 0;
  if (p.T <= 16 && p.T * p.k <= kSmallRows && p.E <= 256)
    return rt_start_small<4>(p, dtype, counts, offsets, src, row_of, row_w, stream);
  hipError_t err;
  const bool scores = p.scores || (p.softmax && !p.renormalize);
  if (rt_narrow(p.T, p.E, p.k, scores)) err = p.E <= 64 ? rt_start<16, 4>(p, dtype, stream) : rt_start<16, 16>(p, dtype, stream);
  else if (p.E <= 256) err = rt_start<64, 4>(p, dtype, stream);
  else if (p.E <= 1024) err = rt_start<64, 16>(p, dtype, stream);
  else err = rt_start<64, 0>(p, dtype, stream);
  if (err != hipSuccess) return err;
  return launch_permute(p.topk_ids, p.topk_w, p.T, p.E, p.k, counts, offsets, src, row_of, row_w, ws, stream);
}

template <int LPT, int NE>
static hipError_t rt_start_grad(const ScoredGradParams& p, int dtype, hipStream_t stream) {
  constexpr int kTokens = 256 / LPT;
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(p.T) + kTokens - 1) / kTokens));
  if (dtype == 0) hipLaunchKernelGGL((k_route_scored_grad<LPT, NE, 0>), grid, dim3(256), 0, stream, p);
  else if (dtype == 1) hipLaunchKernelGGL((k_route_scored_grad<LPT, NE, 1>), grid, dim3(256), 0, stream, p);
  else hipLaunchKernelGGL((k_route_scored_grad<LPT, NE, 2>), grid, dim3(256), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_route_scored_grad(const ScoredGradParams& q, int dtype, hipStream_t stream) {
  ScoredGradParams p = q;
  const uintptr_t four = dtype == 0 ? 16 : 8;                          // bytes of four logits
  p.vec = p.E % 4 == 0 && reinterpret_cast<uintptr_t>(p.logits) % four == 0;
  p.vec_d = p.E % 4 == 0 && reinterpret_cast<uintptr_t>(p.d_scores) % 16 == 0;
  p.vec_out = p.E % 4 == 0 && reinterpret_cast<uintptr_t>(p.dlogits) % four == 0;
  if (rt_narrow(p.T, p.E, p.k, false)) return p.E <= 64 ? rt_start_grad<16, 4>(p, dtype, stream) : rt_start_grad<16, 16>(p, dtype, stream);
  if (p.E <= 256) return rt_start_grad<64, 4>(p, dtype, stream);
  if (p.E <= 1024) return rt_start_grad<64, 16>(p, dtype, stream);
  return rt_start_grad<64, 64>(p, dtype, stream);
}

}  // namespace nvfp4
