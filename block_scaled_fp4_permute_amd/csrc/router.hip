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
// depend on how a float32 exponential rounds.  An expert is closed if its logit is
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

// ------------------------------------------------------------------ over the LPT (16 or 64) lanes of a token
template <int LPT>
__device__ __forceinline__ float seg_max(float v) {
  v = row16_max(v);
  if constexpr (LPT == 64) {
    v = fmaxf(v, __shfl_xor(v, 16));
    v = fmaxf(v, __shfl_xor(v, 32));
  }
  return v;
}
template <int LPT>
__device__ __forceinline__ double seg_max(double v) {
#pragma unroll
  for (int d = LPT / 2; d >= 1; d >>= 1) v = fmax(v, __shfl_xor(v, d));
  return v;
}
template <int LPT, typename F>
__device__ __forceinline__ F seg_sum(F v) {
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

// the two largest of what two lanes hold
__device__ __forceinline__ void top2_merge(double& a1, double& a2, double b1, double b2) {
  a2 = fmax(fmin(a1, b1), fmax(a2, b2));
  a1 = fmax(a1, b1);
}
__device__ __forceinline__ double group_value(double a1, double a2, int top) {
  return (top == 2 && a2 > kNone) ? a1 + a2 : a1;
}

// One token on LPT lanes, expert l * NE + c in register c of lane l.  Writes ids,
// weights and (if wanted) scores; my_id of lane j < k is the j-th choice.  lds: for
// groups that no lanes' borders follow, (E + 2 * 64) doubles of the token's own.
// Lanes of a token past T take part on the last token's values and write nothing.
template <int LPT, int NE, int DT>
__device__ __forceinline__ void scored_token(const ScoredParams& p, int t, bool live, double* lds, int& my_id, float& my_w) {
  const int l = threadIdx.x & (LPT - 1);
  const int e0 = l * NE;
  const size_t row = static_cast<size_t>(t) * p.E;
  double key[NE];
  double top = 0.0, z = 1.0;
  {
    float x[NE];
    rt_load_row<DT, NE>(p.logits, row, e0, p.E, p.vec, x);
    if (p.softmax && p.need_all) {
      float m = -__builtin_huge_valf();
#pragma unroll
      for (int c = 0; c < NE; ++c) m = rt_open(x[c]) ? fmaxf(m, rt_finite(x[c])) : m;
      m = seg_max<LPT>(m);
      top = rt_open(m) ? m : 0.0f;
      double sum = 0.0;
#pragma unroll
      for (int c = 0; c < NE; ++c) {
        key[c] = rt_open(x[c]) ? exp(static_cast<double>(rt_finite(x[c])) - top) : 0.0;
        sum += key[c];
      }
      z = seg_sum<LPT>(sum);
      z = z > 0.0 ? z : 1.0;
#pragma unroll
      for (int c = 0; c < NE; ++c) key[c] /= z;
    } else if (p.need_all) {
#pragma unroll
      for (int c = 0; c < NE; ++c) key[c] = rt_open(x[c]) ? 1.0 / (1.0 + exp(-static_cast<double>(rt_finite(x[c])))) : 0.0;
    }
    if (p.scores && live) {
#pragma unroll
      for (int c = 0; c < NE; ++c)
        if (e0 + c < p.E) p.scores[row + e0 + c] = static_cast<float>(key[c]);
    }
    bool stays = true;                       // the lane's experts, where groups end between lanes
    uint64_t gone = 0;                       // or which of them went with their group
    if (p.bias) {
#pragma unroll
      for (int c = 0; c < NE; ++c) {
        if (e0 + c < p.E) {
          key[c] += static_cast<double>(p.bias[e0 + c]);
          if (!rt_open(x[c]) || !(key[c] > kNone)) key[c] = kClosed;
        }
      }
    } else if (p.n_group > 1) {
#pragma unroll
      for (int c = 0; c < NE; ++c) key[c] = rt_open(x[c]) ? key[c] : kClosed;
    }
    if (p.n_group > 1) {
      const int gs = p.E / p.n_group;
      if (p.lanes_per_group) {
        const int s = p.lanes_per_group;
        double a1 = kNone, a2 = kNone;
#pragma unroll
        for (int c = 0; c < NE; ++c) top2_merge(a1, a2, key[c] > kClosed ? key[c] : kNone, kNone);
        for (int d = 1; d < s; d <<= 1) top2_merge(a1, a2, __shfl_xor(a1, d), __shfl_xor(a2, d));
        const double v = group_value(a1, a2, p.group_top);
        const int g = l / s;
        int rank = 0;
        for (int h = 0; h < p.n_group; ++h) {
          const double o = __shfl(v, h * s, LPT);
          rank += (o > v || (o == v && h < g)) ? 1 : 0;
        }
        stays = rank < p.topk_group;
      } else {
        // keys by way of LDS, a group's behind those of the one before it and a gap (no bank twice)
        double* val = lds + p.E + p.n_group;
#pragma unroll
        for (int c = 0; c < NE; ++c) {
          const int e = e0 + c;
          if (e < p.E) lds[e + e / gs] = key[c];
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        for (int g = l; g < p.n_group; g += LPT) {
          double a1 = kNone, a2 = kNone;
          for (int i = 0; i < gs; ++i) {
            const double o = lds[g * (gs + 1) + i];
            top2_merge(a1, a2, o > kClosed ? o : kNone, kNone);
          }
          val[g] = group_value(a1, a2, p.group_top);
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        for (int g = l; g < p.n_group; g += LPT) {
          const double v = val[g];
          int rank = 0;
          for (int h = 0; h < p.n_group; ++h) {
            const double o = val[h];
            rank += (o > v || (o == v && h < g)) ? 1 : 0;
          }
          lds[g * (gs + 1) + gs] = rank < p.topk_group ? 1.0 : 0.0;   // in the gap behind the group
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
        for (int c = 0; c < NE; ++c) {
          const int e = e0 + c;
          if (e < p.E && lds[(e / gs) * (gs + 1) + gs] == 0.0) gone |= 1ull << c;
        }
        // a wave's next token writes the same words
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
      }
    }
#pragma unroll
    for (int c = 0; c < NE; ++c) {
      if (!p.bias) key[c] = rt_open(x[c]) ? static_cast<double>(rt_finite(x[c])) : kClosed;
      if (!stays || ((gone >> c) & 1) || e0 + c >= p.E) key[c] = kNone;
    }
  }

  // k rounds of the best key that is left, ties to the lower id: a lane's best is
  // its first, and lanes hold ascending ids.  Lanes meet on the float32 roundings
  // (rounding keeps the order), and only a tie there looks at the float64 keys.
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
  my_id = 0;
  bool my_open = false;
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

  // weights of the chosen: their scores again, one a lane.  Renormalised, relative to
  // the largest of the chosen logits (sigmoid: times exp(-b), b = min(largest, 0)):
  // the factor divides out, and scores that would underflow together keep their ratios
  double u = 0.0;
  my_open = my_open && l < p.k;
  const float xj = rt_finite(rt_load<DT>(p.logits, row + my_id));
  if (p.renormalize) {
    const float m = seg_max<LPT>(my_open ? xj : -__builtin_huge_valf());
    const double b = p.softmax ? m : fminf(m, 0.0f), d = my_open ? b - static_cast<double>(xj) : 0.0;
    u = my_open ? (p.softmax ? exp(-d) : 1.0 / (exp(b) + exp(d))) : 0.0;
    const double s = seg_sum<LPT>(u);
    u = s > 0.0 ? u / s : 0.0;
  } else if (my_open) {
    u = p.softmax ? exp(static_cast<double>(xj) - top) / z : 1.0 / (1.0 + exp(-static_cast<double>(xj)));
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
  const int sub = threadIdx.x / LPT;
  const int t = blockIdx.x * (256 / LPT) + sub;
  int id;
  float w;
  scored_token<LPT, NE, DT>(p, min(t, p.T - 1), t < p.T, lds + static_cast<size_t>(sub) * p.lds_token, id, w);
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
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n = p.T * p.k;
  for (int e = tid; e < p.E; e += 1024) cnt[e] = 0;
  for (int t = wave; t < p.T; t += 16) {
    int id;
    float w;
    scored_token<64, NE, DT>(p, t, true, lds + static_cast<size_t>(wave) * p.lds_token, id, w);
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
  float x[NE], s[NE], q[NE];
  rt_load_row<DT, NE>(p.logits, row, e0, p.E, p.vec, x);
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
      s[c] = rt_open(x[c]) ? expf(rt_finite(x[c]) - top) : 0.0f;
      z += s[c];
    }
    z = seg_sum<LPT>(z);
    z = z > 0.0f ? z : 1.0f;
#pragma unroll
    for (int c = 0; c < NE; ++c) s[c] /= z;
  } else {
#pragma unroll
    for (int c = 0; c < NE; ++c) s[c] = rt_open(x[c]) ? 1.0f / (1.0f + expf(-rt_finite(x[c]))) : 0.0f;
  }
  // the chosen, one a lane.  Closed by its logit: score 0; by the bias: weight 0, told
  // by the bias alone (the score of an open logit is finite)
  int id = -1;
  float u = 0.0f, g = 0.0f;
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
  if (p.softmax && p.renormalize) {
    // relative to the largest chosen logit: their own softmax, whatever the others hold
    const float m = seg_max<LPT>(open ? xj : -__builtin_huge_valf());
    u = open ? expf(xj - m) : 0.0f;
  } else if (p.softmax) {
    u = open ? expf(xj - top) / z : 0.0f;
  } else if (p.renormalize) {
    const float m = seg_max<LPT>(open ? xj : -__builtin_huge_valf());
    const float b = fminf(m, 0.0f);
    u = open ? 1.0f / (expf(b) + expf(b - xj)) : 0.0f;
  } else {
    u = open ? 1.0f / (1.0f + expf(-xj)) : 0.0f;
  }
  float cj;
  if (p.renormalize) {
    const float sum = seg_sum<LPT>(u);
    const float n = sum > 0.0f ? u / sum : 0.0f;
    const float mean = seg_sum<LPT>(n > 0.0f ? n * g : 0.0f);
    cj = n > 0.0f ? p.scale * n * (g - mean) : 0.0f;
  } else {
    cj = u > 0.0f ? p.scale * u * g : 0.0f;
  }
  const float csum = p.softmax && !p.renormalize ? seg_sum<LPT>(cj) : 0.0f;
  float qs = 0.0f;
  if (p.d_scores) {
    const float* src = p.d_scores + static_cast<size_t>(t) * p.d_scores_ld;
#pragma unroll
    for (int c = 0; c < NE; ++c) {
      q[c] = e0 + c < p.E ? src[e0 + c] : 0.0f;
      if (p.softmax) qs += s[c] * q[c];
    }
    if (p.softmax) qs = seg_sum<LPT>(qs);
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
#pragma unroll
  for (int c = 0; c < NE; ++c) {
    if (e0 + c >= p.E) continue;
    const float qe = p.d_scores ? q[c] : 0.0f;
    float d;
    if (p.softmax) {
      d = cw[c] + s[c] * (qe - qs - csum);
    } else {
      const float rest = rt_open(x[c]) ? 1.0f / (1.0f + expf(rt_finite(x[c]))) : 0.0f;
      d = rest * (cw[c] + s[c] * qe);
    }
    if (!rt_open(x[c])) d = 0.0f;
    if constexpr (DT == 0) static_cast<float*>(p.dlogits)[row + e0 + c] = d;
    if constexpr (DT == 1) static_cast<__bf16*>(p.dlogits)[row + e0 + c] = static_cast<__bf16>(d);
    if constexpr (DT == 2) static_cast<_Float16*>(p.dlogits)[row + e0 + c] = static_cast<_Float16>(d);
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
  p.lds_token = p.n_group > 1 && !p.lanes_per_group ? p.E + p.n_group + 64 : 0;
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
  p.lds_token = p.n_group > 1 && !p.lanes_per_group ? p.E + p.n_group + 64 : 0;
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
  p.need_all = p.bias || p.n_group > 1 || p.scores || (p.softmax && !p.renormalize);
  p.vec = p.E % 4 == 0 && reinterpret_cast<uintptr_t>(p.logits) % (dtype == 0 ? 16 : 8) == 0;
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
  p.vec = p.E % 4 == 0 && reinterpret_cast<uintptr_t>(p.logits) % (dtype == 0 ? 16 : 8) == 0;
  if (rt_narrow(p.T, p.E, p.k)) return p.E <= 64 ? rt_start_grad<16, 4>(p, dtype, stream) : rt_start_grad<16, 16>(p, dtype, stream);
  if (p.E <= 256) return rt_start_grad<64, 4>(p, dtype, stream);
  if (p.E <= 1024) return rt_start_grad<64, 16>(p, dtype, stream);
  return rt_start_grad<64, 64>(p, dtype, stream);
}

}  // namespace nvfp4
