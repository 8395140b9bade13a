// Gradient of the gated activation between the projections and their products:
//   dg = dh * u * act'(g),  du = dh * act(g)
// from the float32 pre-activations that the forward call saved.  dg and du are
// rounded to the operands' 16-bit type: the two products that follow read them
// as matrix operands, dx row by row and dw column by column (reduction over the
// rows).  So they are written twice, row-major [m_total, 2I] and transposed
// [2I, ld]: with both operands of dw K-major, its LDS reads are all transposing
// 8-byte ones and bound it (131072 rows of 256 experts, 2 x 256 columns, in a
// training step: 3240 us with one copy, 3150 with both).  One pass, bound by
// memory: those rows, 604 MB read and written, take 113 us, 5.3 TB/s.
#include "tile_gemm.h"

namespace nvfp4 {

constexpr int kGgRows = 64, kGgCols = 64;   // a workgroup's rows of one expert and columns of h

template <int T>
__global__ __launch_bounds__(256) void k_gated_grad(const float* __restrict__ gu, const uint16_t* __restrict__ dh, int I,
                                                    int m_total, const int32_t* __restrict__ offsets, int E, int act,
                                                    uint16_t* __restrict__ dgu, uint16_t* __restrict__ dgu_t, int64_t ld) {
  // the tile transposed: dg then du columns of 64 rows; the 8-row chunk q of
  // column c lies at chunk q ^ ((c >> 2) & 7), which spreads a store's columns
  // over the banks
  __shared__ __attribute__((aligned(16))) uint16_t tr[2 * kGgCols][kGgRows];
  int e, m0, nt;
  bool narrow;
  GemmParams map{};
  map.offsets = offsets;
  map.E = E;
  map.m_total = m_total;
  map.n_tiles = (I + kGgCols - 1) / kGgCols;
  map.slots = 1 << 30;
  if (!find_task<kGgRows / 16, false, 0>(map, e, m0, nt, narrow)) return;
  const int row0 = min(max(offsets[e], 0), m_total);
  const int Me = min(max(offsets[e + 1], 0), m_total) - row0;
  const int rows = min(kGgRows, Me - m0);
  if (rows <= 0 || m0 < 0) return;          // offsets that overlap so far that the task count does not fit
  const int t = threadIdx.x;
  const int c = nt * kGgCols + 4 * (t & 15);
#pragma unroll
  for (int i = 0; i < kGgRows / 32; ++i) {
    const int r = 2 * (t >> 4) + 32 * i;    // two neighbouring rows
    uint2 pg[2], pu[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      float4v dg = {0.f, 0.f, 0.f, 0.f}, du = {0.f, 0.f, 0.f, 0.f};
      if (r + b < rows && c < I) {
        const int64_t row = static_cast<int64_t>(row0) + m0 + r + b;
        const float4v g = *reinterpret_cast<const float4v*>(gu + row * 2 * I + c);
        const float4v u = *reinterpret_cast<const float4v*>(gu + row * 2 * I + I + c);
        const uint2 d = *reinterpret_cast<const uint2*>(dh + row * I + c);
        float4v dv;
        if constexpr (T == TG_BF16) {
          dv = float4v{__uint_as_float(d.x << 16), __uint_as_float(d.x & 0xFFFF0000u), __uint_as_float(d.y << 16),
                       __uint_as_float(d.y & 0xFFFF0000u)};
        } else {
          const half4 hv = __builtin_bit_cast(half4, d);
          dv = float4v{static_cast<float>(hv[0]), static_cast<float>(hv[1]), static_cast<float>(hv[2]), static_cast<float>(hv[3])};
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float a;
          const float slope = tg_act_grad(g[q], act, a);
          dg[q] = dv[q] * u[q] * slope;
          du[q] = dv[q] * a;
        }
      }
      pg[b] = TgType<T>::pack(dg);
      pu[b] = TgType<T>::pack(du);
      if (dgu && r + b < rows && c < I) {
        uint16_t* o = dgu + (static_cast<int64_t>(row0) + m0 + r + b) * 2 * I + c;
        *reinterpret_cast<uint2*>(o) = pg[b];
        *reinterpret_cast<uint2*>(o + I) = pu[b];
      }
    }
    if (dgu_t) {
      const uint32_t w[2][4] = {{pg[0].x, pg[0].y, pu[0].x, pu[0].y}, {pg[1].x, pg[1].y, pu[1].x, pu[1].y}};
      const int at = 8 * ((r >> 3) ^ (t & 7)) + (r & 7);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int s = 16 * (q & 1);
        *reinterpret_cast<uint32_t*>(&tr[4 * (t & 15) + q][at]) =
            ((w[0][q >> 1] >> s) & 0xFFFFu) | (((w[1][q >> 1] >> s) & 0xFFFFu) << 16);
        *reinterpret_cast<uint32_t*>(&tr[kGgCols + 4 * (t & 15) + q][at]) =
            ((w[0][2 + (q >> 1)] >> s) & 0xFFFFu) | (((w[1][2 + (q >> 1)] >> s) & 0xFFFFu) << 16);
      }
    }
  }
  if (!dgu_t) return;
  __syncthreads();
  // 8 rows a lane, whole chunks of 8 up to the last row's (zeros behind it)
  const int64_t first = tg_start_col(row0, e, tg_col_align(m_total, E)) + m0;
#pragma unroll
  for (int i = 0; i < 2 * kGgCols * (kGgRows / 8) / 256; ++i) {
    const int q = t + 256 * i;
    const int col = q >> 3, r = 8 * (q & 7);
    const int h = nt * kGgCols + (col & (kGgCols - 1));
    if (r < rows && h < I)
      *reinterpret_cast<u32x4*>(dgu_t + static_cast<int64_t>(h + (col >= kGgCols ? I : 0)) * ld + first + r) =
          *reinterpret_cast<const u32x4*>(&tr[col][8 * ((q & 7) ^ ((col >> 2) & 7))]);
  }
}

int64_t gated_grad_ld(int64_t m_total, int E) {
  const int align = tg_col_align(m_total, E);
  return tg_start_col(m_total, E, align) + align;
}

int64_t gated_grad_blocks(int I, int64_t m_total, int E) {
  const int64_t chunks = m_total / kGgRows + (E < m_total ? E : m_total);
  return (chunks * ((I + kGgCols - 1) / kGgCols) + 7) / 8 * 8;
}

hipError_t launch_gated_grad(const float* gu, const void* dh, int dtype_f16, int I, int64_t m_total, const int32_t* offsets,
                             int E, int act, void* dgu, void* dgu_t, hipStream_t stream) {
  const int64_t blocks = gated_grad_blocks(I, m_total, E);
  if (blocks >= (int64_t(1) << 24)) return hipErrorInvalidConfiguration;   // 2^32 threads (the entry point refuses them)
  const dim3 grid(static_cast<unsigned>(blocks));
  const int64_t ld = gated_grad_ld(m_total, E);
  if (dtype_f16)
    hipLaunchKernelGGL((k_gated_grad<TG_F16>), grid, dim3(256), 0, stream, gu, static_cast<const uint16_t*>(dh), I,
                       static_cast<int>(m_total), offsets, E, act, static_cast<uint16_t*>(dgu), static_cast<uint16_t*>(dgu_t), ld);
  else
    hipLaunchKernelGGL((k_gated_grad<TG_BF16>), grid, dim3(256), 0, stream, gu, static_cast<const uint16_t*>(dh), I,
                       static_cast<int>(m_total), offsets, E, act, static_cast<uint16_t*>(dgu), static_cast<uint16_t*>(dgu_t), ld);
  return hipGetLastError();
}

// ------------------------------------------------------------------ joining parts
// The sums over parts of a long reduction (few output tiles), added in the order
// of the parts and rounded once.  Bound by memory (256 rows, 2048 x 5632 product's
// row gradient, parts and this together: 44 us against 108 with one part; 64 parts
// of 64 x 64: 21 us with 8 loads in flight, 40 with one).
template <int T>
__global__ __launch_bounds__(256) void k_join(const float* __restrict__ part, int parts, int64_t values, int N,
                                              const int32_t* __restrict__ offsets, int E, uint16_t* __restrict__ out) {
  const int64_t i = 4 * (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x);
  if (i >= values || (offsets && i / N >= offsets[E])) return;
  float4v v = *reinterpret_cast<const float4v*>(part + i);
#pragma unroll 8                            // as many loads in flight
  for (int s = 1; s < parts; ++s) v += *reinterpret_cast<const float4v*>(part + s * values + i);
  *reinterpret_cast<uint2*>(out + i) = TgType<T>::pack(v);
}

hipError_t launch_join(const float* part, int parts, int64_t rows, int N, const int32_t* offsets, int E, int dtype_f16,
                       void* out, hipStream_t stream) {
  const int64_t values = rows * N;
  const int64_t blocks = (values / 4 + 255) / 256;
  if (blocks >= (int64_t(1) << 24)) return hipErrorInvalidConfiguration;   // 2^32 threads (more values than the memory holds)
  const dim3 grid(static_cast<unsigned>(blocks));
  if (dtype_f16) hipLaunchKernelGGL((k_join<TG_F16>), grid, dim3(256), 0, stream, part, parts, values, N, offsets, E, static_cast<uint16_t*>(out));
  else hipLaunchKernelGGL((k_join<TG_BF16>), grid, dim3(256), 0, stream, part, parts, values, N, offsets, E, static_cast<uint16_t*>(out));
  return hipGetLastError();
}

}  // namespace nvfp4
