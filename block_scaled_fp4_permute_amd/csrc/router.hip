// The router with scores, and the gradient of its logits.
//
//   scores    sigmoid s_e = 1 / (1 + exp(-l_e)), or softmax over the token's open
//             experts
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
// first, and take float64 ones for every expert only where two values that matter
// lie within the float32 keys' error of each other.  An expert is closed if its logit is
// -inf or NaN, or its key -inf or NaN; closed ones are taken, by id and with
// weight 0, only where a token has fewer open ones than it needs.
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
__device__ __forceinline__ double rt_sigmoid(float l) { return 1.0 / (1.0 + rt_exp(-static_cast<double>(l))); }

// the two largest of what two lanes hold
template <typename T>
__device__ __forceinline__ void top2_merge(T& a1, T& a2, T b1, T b2) {
  const T low = a1 < b1 ? a1 : b1;
  a1 = a1 < b1 ? b1 : a1;
  a2 = a2 < b2 ? b2 : a2;
  a2 = a2 < low ? low : a2;
}

__device__ __forceinline__ void rt_lds_step() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Which groups stay.  key(c): of the lane's expert c, above `shut` if open; T: float
// with `near` (set if two groups' values lie within tol + |value| 2^-18), or double
// (near: never).  Returns a bit for each of the lane's experts that went with its
// group.  lds: (E + 2 n_group) doubles of the token's own where no lanes' borders
// follow the groups'.
template <int LPT, int NE, typename T, typename K>
__device__ __forceinline__ uint64_t scored_groups(const ScoredParams& p, K key, T shut, T tol, double* lds_bytes, bool& near) {
  const T none = -static_cast<T>(__builtin_huge_valf());
  const int l = threadIdx.x & (LPT - 1);
  const int e0 = l * NE;
  const int gs = p.E / p.n_group;
  auto value = [&](T a1, T a2) __attribute__((always_inline)) { return p.group_top == 2 && a2 > none ? a1 + a2 : a1; };
  auto beats = [&](T o, int h, T v, int g) __attribute__((always_inline)) {
    if (h != g && fabs(o - v) <= tol + fabs(v) * static_cast<T>(0x1p-18) && o > none && v > none) near = true;
    return o > v || (o == v && h < g);
  };
  if (p.lanes_per_group) {
    const int s = p.lanes_per_group;
    T a1 = none, a2 = none;
#pragma unroll
    for (int c = 0; c < NE; ++c) {
      const T k = key(c);
      top2_merge(a1, a2, k > shut ? k : none, none);
    }
    for (int d = 1; d < s; d <<= 1) {
      const T b1 = __shfl_xor(a1, d), b2 = __shfl_xor(a2, d);
      top2_merge(a1, a2, b1, b2);
    }
    const T v = value(a1, a2);
    const int g = l / s;
    int rank = 0;
    for (int h = 0; h < p.n_group; ++h) rank += beats(__shfl(v, h * s, LPT), h, v, g) ? 1 : 0;
    if (g >= p.n_group) near = false;
    return rank < p.topk_group ? 0ull : ~0ull;
  }
  // keys by way of LDS, a group's behind those of the one before it and a gap (no bank twice)
  T* lds = reinterpret_cast<T*>(lds_bytes);
  T* val = lds + p.E + p.n_group;
#pragma unroll
  for (int c = 0; c < NE; ++c) {
    const int e = e0 + c;
    if (e < p.E) lds[e + e / gs] = key(c);
  }
  rt_lds_step();
  for (int g = l; g < p.n_group; g += LPT) {
    T a1 = none, a2 = none;
    for (int i = 0; i < gs; ++i) {
      const T o = lds[g * (gs + 1) + i];
      top2_merge(a1, a2, o > shut ? o : none, none);
    }
    val[g] = value(a1, a2);
  }
  rt_lds_step();
  for (int g = l; g < p.n_group; g += LPT) {
    const T v = val[g];
    int rank = 0;
    for (int h = 0; h < p.n_group; ++h) rank += beats(val[h], h, v, g) ? 1 : 0;
    lds[g * (gs + 1) + gs] = rank < p.topk_group ? 1 : 0;   // in the gap behind the group
  }
  rt_lds_step();
  uint64_t gone = 0;
#pragma unroll
  for (int c = 0; c < NE; ++c) {
    const int e = e0 + c;
    if (e < p.E && lds[(e / gs) * (gs + 1) + gs] == 0) gone |= 1ull << c;
  }
  rt_lds_step();                            // the same words are written again
  return gone;
}

// The choice by float64 keys: k rounds of the best that is left, ties to the lower id
// (a lane's best is its first, and lanes hold ascending ids).  Lanes meet on the
// float32 roundings (rounding keeps the order), and only a tie there looks at the
// float64 keys.  Lane j gets the j-th.
template <int LPT, int NE, typename B>
__device__ __forceinline__ void choose_exact(const ScoredParams& p, const float (&x)[NE], B bias, double top, double z, double* lds,
                                             int& my_id, bool& my_open) {
  const int l = threadIdx.x & (LPT - 1);
  const int e0 = l * NE;
  double key[NE];
#pragma unroll
  for (int c = 0; c < NE; ++c) {
    key[c] = static_cast<double>(rt_finite(x[c]));
    if (p.bias || p.n_group > 1) {
      key[c] = p.softmax ? rt_exp(key[c] - top) / z : rt_sigmoid(rt_finite(x[c]));
      if (p.bias) key[c] += static_cast<double>(bias(c));
    }
    if (!rt_open(x[c]) || !(key[c] > kNone)) key[c] = kClosed;
  }
  uint64_t gone = 0;
  if (p.n_group > 1) {
    bool near = false;
    gone = scored_groups<LPT, NE, double>(p, [&](int c) __attribute__((always_inline)) { return key[c]; }, kClosed, -1.0, lds, near);
  }
#pragma unroll
  for (int c = 0; c < NE; ++c) {
    if (!p.bias) key[c] = rt_open(x[c]) ? static_cast<double>(rt_finite(x[c])) : kClosed;
    if (((gone >> c) & 1) || e0 + c >= p.E) key[c] = kNone;
  }
  double best = kNone;
  int bid = 0;
  auto rescan = [&]() __attribute__((always_inline)) {
    best = kNone;
    bid = e0;
#pragma unroll
    for (int c = 0; c < NE; ++c) {
      const bool more = key[c] > best;
      best = more ? key[c] : best;
      bid = more ? e0 + c : bid;
    }
  };
  rescan();
  const int base = (threadIdx.x & 63) & ~(LPT - 1);
  for (int j = 0; j < p.k; ++j) {
    const float h = static_cast<float>(best);
    bool mine = h == seg_max<LPT>(h);
    uint64_t who = seg_ballot<LPT>(mine);
    if (__any((who & (who - 1)) != 0)) {
      const double b = mine ? best : kNone;
      const double m = seg_max<LPT>(b);      // by every lane of the wave
      mine = mine && b == m;
      who = seg_ballot<LPT>(mine);
    }
    const int w = __builtin_ctzll(who);
    const int packed = __shfl(bid | (best > kClosed ? 1 << 30 : 0), base + w);
    if (l == j) {
      my_id = packed & 0xFFFF;
      my_open = (packed >> 30) != 0;
    }
    if (l == w) {
#pragma unroll
      for (int c = 0; c < NE; ++c) key[c] = bid == e0 + c ? kNone : key[c];
      rescan();
    }
  }
}

// float32 bits in an order of unsigned integers
__device__ __forceinline__ uint32_t rt_order(float f) {
  const uint32_t u = __float_as_uint(f);
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float rt_unorder(uint32_t u) {
  return __uint_as_float(u ^ (static_cast<uint32_t>(static_cast<int32_t>(~u) >> 31) | 0x80000000u));
}

// The choice by float32 keys.  An expert's key is an unsigned integer, its place in
// the lane in the low bits (so the key loses log2(NE) bits): a lane's best of NE is a
// few three-way maxima.  Returns 0 (for a whole wave) where the float32 keys do not
// settle which experts or groups are chosen, 1 where they settle all, 2 where the
// order of the k chosen is open.  list: 32 ints of the token's own.
//
// Errors: a sigmoid from v_exp_f32 and v_rcp_f32 is off by at most 2^-22 (s (1 - s)
// (|x| + 2) 2^-24 + 3 s 2^-24), a softmax by p (|x - max| + 30) 2^-24 (sums of 16 and
// over 6 levels, exp, quotient), which is below 2^-18 max p (|x - max| p <= 0.37 max
// p); the bias adds 2^-24 |key|, the lost bits |key| 2^-19 for 16 places.  Two keys
// within twice that, tol + |key| 2^-18, are not settled, group values within twice
// as much.
template <int LPT, int NE>
__device__ __forceinline__ int choose_fast(const ScoredParams& p, const float (&x)[NE], const float (&bias)[NE], float top, float z,
                                           double* lds, int* list, int& my_id, bool& my_open) {
  constexpr uint32_t LOW = NE <= 4 ? 3 : 15;
  static_assert(NE <= 16, "the place takes 4 bits");
  const int l = threadIdx.x & (LPT - 1);
  const int e0 = l * NE;
  float key[NE];
  float big = 1.0f;                          // of a sigmoid
  if (p.bias || p.n_group > 1) {
    if (p.softmax) big = __builtin_amdgcn_rcpf(z);                      // the largest p
#pragma unroll
    for (int c = 0; c < NE; ++c) {
      const float a = rt_finite(x[c]);
      key[c] = p.softmax ? __builtin_amdgcn_exp2f((a - top) * 1.44269504f) * big
                         : __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(a * -1.44269504f));
      if (p.bias) key[c] += bias[c];
    }
  } else {
#pragma unroll
    for (int c = 0; c < NE; ++c) key[c] = rt_finite(x[c]);
  }
  const float none = -__builtin_huge_valf();
#pragma unroll
  for (int c = 0; c < NE; ++c) key[c] = rt_open(x[c]) && key[c] > none ? key[c] : none;
  const float tol = p.softmax ? big * 0x1p-16f : 0x1p-20f;
  bool near = false;
  uint64_t gone = 0;
  if (p.n_group > 1)
    gone = scored_groups<LPT, NE, float>(p, [&](int c) __attribute__((always_inline)) { return key[c]; }, none, 2.0f * tol, lds, near);
  // by logits: the keys are exact (and 16-bit ones keep all their bits)
  const bool exact = !p.bias && p.narrow;
  uint32_t el[NE];
#pragma unroll
  for (int c = 0; c < NE; ++c) {
    const float k = p.bias ? key[c] : rt_finite(x[c]);
    const bool open = key[c] > none;
    el[c] = ((open ? rt_order(k) & ~LOW : LOW + 1) | (LOW - c));        // closed ones below every open
    if (((gone >> c) & 1) || e0 + c >= p.E) el[c] = 0;
  }
  bool order = false;
  float before = __builtin_huge_valf();
  for (int j = 0; j <= p.k; ++j) {           // and the first that is not chosen
    uint32_t best = 0;
#pragma unroll
    for (int c = 0; c < NE; ++c) best = el[c] > best ? el[c] : best;
    const uint32_t t = best & ~LOW;
    const uint32_t m = seg_reduce<LPT>(t, [](uint32_t a, uint32_t b) __attribute__((always_inline)) { return a > b ? a : b; });
    const float v = rt_unorder(m);
    // closed and absent ones (m <= LOW + 1) are in their order already
    const bool close = !exact && m > LOW + 1 && before - v <= (p.bias ? tol : 0.0f) + fabsf(v) * 0x1p-18f;
    if (j < p.k) order |= close;
    else near |= close;
    before = m > LOW + 1 ? v : __builtin_huge_valf();
    const int w = __builtin_ctzll(seg_ballot<LPT>(t == m));
    const uint32_t gone_el = l == w ? best : 0;
    if (j < p.k && l == w) list[j] = e0 + static_cast<int>(LOW - (best & LOW)) + (m > LOW + 1 ? 1 << 30 : 0);
#pragma unroll
    for (int c = 0; c < NE; ++c) el[c] = el[c] == gone_el ? 0 : el[c];
  }
  if (__any(near)) return 0;
  rt_lds_step();
  const int packed = l < p.k ? list[l] : 0;
  my_id = packed & 0xFFFF;
  my_open = (packed >> 30) != 0;
  return __any(order) ? 2 : 1;
}

// One token on LPT lanes, expert l * NE + c in register c of lane l.  Writes ids,
// weights and (if wanted) scores; lane j < k returns the j-th choice and its weight.
// lds: of the token's own, for groups (scored_groups); list: 32 ints of its own.  Lanes
// of a token past T take part on the last token's values and write nothing.
template <int LPT, int NE, int DT>
__device__ __forceinline__ void scored_token(const ScoredParams& p, int t, bool live, double* lds, int* list, int& my_id, float& my_w) {
  const int l = threadIdx.x & (LPT - 1);
  const int e0 = l * NE;
  const size_t row = static_cast<size_t>(t) * p.E;
  float x[NE];
  rt_load_row<DT, NE>(p.logits, row, e0, p.E, p.vec, x);
  constexpr bool FAST = NE <= 16;
  float bias[FAST ? NE : 1];
  if constexpr (FAST) {
    if (p.bias) rt_load_row<0, NE>(p.bias, 0, e0, p.E, p.vec_bias, bias);
  }
  const bool by_key = p.bias || p.n_group > 1;
  double top = 0.0, z = 1.0;
  if (p.softmax) {
    float m = -__builtin_huge_valf();
#pragma unroll
    for (int c = 0; c < NE; ++c) m = rt_open(x[c]) ? fmaxf(m, rt_finite(x[c])) : m;
    m = seg_max<LPT>(m);
    top = rt_open(m) ? m : 0.0f;
  }
  auto sum64 = [&]() __attribute__((always_inline)) {
    double sum = 0.0;
#pragma unroll
    for (int c = 0; c < NE; ++c) sum += rt_open(x[c]) ? rt_exp(static_cast<double>(rt_finite(x[c])) - top) : 0.0;
    sum = seg_sum<LPT>(sum);
    z = sum > 0.0 ? sum : 1.0;
  };
  const bool have_z = p.softmax && (p.scores || !p.renormalize);
  if (have_z) sum64();
  if (p.scores && live) {
    float s[NE];
#pragma unroll
    for (int c = 0; c < NE; ++c) {
      const float a = rt_open(x[c]) ? rt_finite(x[c]) : 0.0f;
      const double v = p.softmax ? rt_exp(static_cast<double>(a) - top) / z : rt_sigmoid(a);
      s[c] = rt_open(x[c]) ? static_cast<float>(v) : 0.0f;
    }
    rt_store_row<NE>(p.scores, row, e0, p.E, p.vec_scores, s);
  }

  bool my_open = false;
  my_id = 0;
  int settled = 0;
  if constexpr (FAST) {
    float zf = static_cast<float>(z);
    if (p.softmax && by_key && !have_z) {
      zf = 0.0f;
#pragma unroll
      for (int c = 0; c < NE; ++c)
        zf += rt_open(x[c]) ? __builtin_amdgcn_exp2f((rt_finite(x[c]) - static_cast<float>(top)) * 1.44269504f) : 0.0f;
      zf = seg_sum<LPT>(zf);
      zf = zf > 0.0f ? zf : 1.0f;
    }
    settled = choose_fast<LPT, NE>(p, x, bias, static_cast<float>(top), zf, lds, list, my_id, my_open);
  }
  if (settled != 1) {
    if (p.softmax && by_key && !have_z) sum64();
    if (settled == 0) {
      choose_exact<LPT, NE>(p, x, [&](int c) __attribute__((always_inline)) {
        if constexpr (FAST) return bias[c];
        else return e0 + c < p.E ? p.bias[e0 + c] : 0.0f;
      }, top, z, lds, my_id, my_open);
    } else {
      // the chosen in the order of their float64 keys, ties to the lower id
      const float xj = rt_finite(rt_load<DT>(p.logits, row + my_id));
      double key = static_cast<double>(xj);
      if (p.bias) key = (p.softmax ? rt_exp(key - top) / z : rt_sigmoid(xj)) + static_cast<double>(p.bias[my_id]);
      if (!my_open) key = kClosed;
      int rank = 0;
      for (int i = 0; i < p.k; ++i) {
        const double o = __shfl(key, i, LPT);
        const int id = __shfl(my_id, i, LPT);
        rank += (o > key || (o == key && id < my_id)) ? 1 : 0;
      }
      rt_lds_step();
      if (l < p.k) list[rank] = my_id | (my_open ? 1 << 30 : 0);
      rt_lds_step();
      const int packed = l < p.k ? list[l] : 0;
      my_id = packed & 0xFFFF;
      my_open = (packed >> 30) != 0;
    }
  }

  // weights of the chosen: their scores again, one a lane.  Renormalised, relative to
  // the largest of the chosen logits (sigmoid: times exp(-b), b = min(largest, 0)):
  // the factor divides out, and scores that would underflow together keep their ratios
  double u = 0.0;
  my_open = my_open && l < p.k;
  const float xj = rt_finite(rt_load<DT>(p.logits, row + my_id));
  if (p.renormalize) {
    const float m = seg_max<LPT>(my_open ? xj : -__builtin_huge_valf());
    const double b = p.softmax ? m : fminf(m, 0.0f), d = my_open ? b - static_cast<double>(xj) : 0.0;
    u = my_open ? (p.softmax ? rt_exp(-d) : 1.0 / (rt_exp(b) + rt_exp(d))) : 0.0;
    const double s = seg_sum<LPT>(u);
    u = s > 0.0 ? u / s : 0.0;
  } else if (my_open) {
    u = p.softmax ? rt_exp(static_cast<double>(xj) - top) / z : rt_sigmoid(xj);
  }
  my_w = static_cast<float>(u * static_cast<double>(p.scale));
  if (live && l < p.k) {
    const size_t at = static_cast<size_t>(t) * p.k + l;
    p.topk_ids[at] = my_id;
    p.topk_w[at] = my_w;
  }
}

template <int LPT, int NE, int DT>
__global__ __launch_bounds__(256) void k_route_scored(const ScoredParams p) {
  extern __shared__ double lds[];
  __shared__ int list[256 / LPT][32];
  const int sub = threadIdx.x / LPT;
  const int t = blockIdx.x * (256 / LPT) + sub;
  int id;
  float w;
  scored_token<LPT, NE, DT>(p, min(t, p.T - 1), t < p.T, lds + static_cast<size_t>(sub) * p.lds_token, list[sub], id, w);
}

// ------------------------------------------------------------------ few tokens: routing and permutation in one launch
// One workgroup: wave w routes tokens w, w + 16, ...; then every assignment counts
// the earlier ones of its expert (n <= kSmallRows: a walk over LDS), and a scan of
// the experts' counts places the rows.  Bound by latency: four launches otherwise.
static constexpr int kSmallRows = 256;
template <int NE, int DT>
__global__ __launch_bounds__(1024) void k_route_small(const ScoredParams p, int* __restrict__ counts, int* __restrict__ offsets,
                                                      int* __restrict__ src, int* __restrict__ row_of, float* __restrict__ row_w) {
  extern __shared__ double lds[];
  __shared__ int cnt[4096];
  __shared__ int ids[kSmallRows];
  __shared__ float ws[kSmallRows];
  __shared__ int wave_sum[16];
  __shared__ int list[16][32];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n = p.T * p.k;
  for (int e = tid; e < p.E; e += 1024) cnt[e] = 0;
  for (int t = wave; t < p.T; t += 16) {
    int id;
    float w;
    scored_token<64, NE, DT>(p, t, true, lds + static_cast<size_t>(wave) * p.lds_token, list[wave], id, w);
    if (lane < p.k) {
      ids[t * p.k + lane] = id;
      ws[t * p.k + lane] = w;
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
  // thread t owns 4 neighbouring experts
  int c[4], sum = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = 4 * tid + i;
    c[i] = e < p.E ? cnt[e] : 0;
    sum += c[i];
  }
  int incl = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 63) wave_sum[wave] = incl;
  __syncthreads();
  int run = incl - sum;
  for (int w = 0; w < wave; ++w) run += wave_sum[w];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = 4 * tid + i;
    if (e < p.E) {
      counts[e] = c[i];
      offsets[e] = run;
      cnt[e] = run;
    }
    run += c[i];
  }
  if (tid == 0) offsets[p.E] = n;
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
// All in float32: one read of logits (and q), one write of the gradient.
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
    for (int c = 0; c < NE; ++c) q[c] = e0 + c < p.E ? q[c] : 0.0f;
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
// enough to fill the chip that way: the rounds then serve 4 tokens a wave.
static bool rt_narrow(int T, int E, int k) { return E <= 256 && k <= 16 && T >= 2048; }

// lanes of a group if groups end between lanes and a butterfly joins them, else 0 (by way of LDS)
static int rt_lanes_per_group(int E, int n_group, int ne) {
  const int gs = E / n_group;
  if (n_group <= 1 || gs % ne != 0) return 0;
  const int s = gs / ne;
  return (s & (s - 1)) == 0 ? s : 0;
}

template <int LPT, int NE>
static hipError_t rt_start(ScoredParams p, int dtype, hipStream_t stream) {
  p.lanes_per_group = rt_lanes_per_group(p.E, p.n_group, NE);
  p.lds_token = p.n_group > 1 && !p.lanes_per_group ? p.E + 2 * p.n_group : 0;
  constexpr int kTokens = 256 / LPT;
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(p.T) + kTokens - 1) / kTokens));
  const size_t lds = static_cast<size_t>(kTokens) * p.lds_token * sizeof(double);
  if (dtype == 0) hipLaunchKernelGGL((k_route_scored<LPT, NE, 0>), grid, dim3(256), lds, stream, p);
  else if (dtype == 1) hipLaunchKernelGGL((k_route_scored<LPT, NE, 1>), grid, dim3(256), lds, stream, p);
  else hipLaunchKernelGGL((k_route_scored<LPT, NE, 2>), grid, dim3(256), lds, stream, p);
  return hipGetLastError();
}

template <int NE>
static hipError_t rt_start_small(ScoredParams p, int dtype, int* counts, int* offsets, int* src, int* row_of, float* row_w,
                                 hipStream_t stream) {
  p.lanes_per_group = rt_lanes_per_group(p.E, p.n_group, NE);
  p.lds_token = p.n_group > 1 && !p.lanes_per_group ? p.E + 2 * p.n_group : 0;
  const size_t lds = static_cast<size_t>(16) * p.lds_token * sizeof(double);
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
  if (p.T <= 16 && p.T * p.k <= kSmallRows && p.E <= 512)
    return p.E <= 256 ? rt_start_small<4>(p, dtype, counts, offsets, src, row_of, row_w, stream)
                      : rt_start_small<8>(p, dtype, counts, offsets, src, row_of, row_w, stream);
  hipError_t err;
  if (rt_narrow(p.T, p.E, p.k)) err = p.E <= 64 ? rt_start<16, 4>(p, dtype, stream) : rt_start<16, 16>(p, dtype, stream);
  else if (p.E <= 256) err = rt_start<64, 4>(p, dtype, stream);
  else if (p.E <= 1024) err = rt_start<64, 16>(p, dtype, stream);
  else err = rt_start<64, 64>(p, dtype, stream);
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
  if (rt_narrow(p.T, p.E, p.k)) return p.E <= 64 ? rt_start_grad<16, 4>(p, dtype, stream) : rt_start_grad<16, 16>(p, dtype, stream);
  if (p.E <= 256) return rt_start_grad<64, 4>(p, dtype, stream);
  if (p.E <= 1024) return rt_start_grad<64, 16>(p, dtype, stream);
  return rt_start_grad<64, 64>(p, dtype, stream);
}

}  // namespace nvfp4
