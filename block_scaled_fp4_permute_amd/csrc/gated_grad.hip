// Gradient of the gated activation between the projections and their products:
//   dg = dh * u * act'(g),  du = dh * act(g)
// from the float32 pre-activations that the forward call saved.  dg and du are
// rounded to the operands' 16-bit type: the two products that follow read them
// as matrix operands.  One pass, bound by memory.
#include "tile_gemm.h"

namespace nvfp4 {

template <int T>
__global__ __launch_bounds__(256) void k_gated_grad(const float* __restrict__ gu, const uint16_t* __restrict__ dh, int I,
                                                    int64_t quads, const int32_t* __restrict__ offsets, int E, int act,
                                                    uint16_t* __restrict__ dgu) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= quads) return;
  const int per = I / 4;
  const int64_t row = i / per;
  const int c = static_cast<int>(i - row * per) * 4;
  if (row >= offsets[E]) return;           // rows behind the last expert: nothing reads them
  const float4v g = *reinterpret_cast<const float4v*>(gu + row * 2 * I + c);
  const float4v u = *reinterpret_cast<const float4v*>(gu + row * 2 * I + I + c);
  const uint2 d = *reinterpret_cast<const uint2*>(dh + row * I + c);
  float4v dv, dg, du;
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
  *reinterpret_cast<uint2*>(dgu + row * 2 * I + c) = TgType<T>::pack(dg);
  *reinterpret_cast<uint2*>(dgu + row * 2 * I + I + c) = TgType<T>::pack(du);
}

hipError_t launch_gated_grad(const float* gu, const void* dh, int dtype_f16, int I, int64_t m_total, const int32_t* offsets,
                             int E, int act, void* dgu, hipStream_t stream) {
  const int64_t quads = m_total * (I / 4);
  const int64_t blocks = (quads + 255) / 256;
  if (blocks >= (int64_t(1) << 31)) return hipErrorInvalidConfiguration;
  const dim3 grid(static_cast<unsigned>(blocks));
  if (dtype_f16)
    hipLaunchKernelGGL((k_gated_grad<TG_F16>), grid, dim3(256), 0, stream, gu, static_cast<const uint16_t*>(dh), I, quads,
                       offsets, E, act, static_cast<uint16_t*>(dgu));
  else
    hipLaunchKernelGGL((k_gated_grad<TG_BF16>), grid, dim3(256), 0, stream, gu, static_cast<const uint16_t*>(dh), I, quads,
                       offsets, E, act, static_cast<uint16_t*>(dgu));
  return hipGetLastError();
}

}  // namespace nvfp4
