// INT8 products with one scale per row of each operand (tokens and output
// channels), and the quantiser that makes such operands.
#include "tile_gemm.h"

namespace nvfp4 {

// s = absmax / 127 (float32 division, 1 where that is zero), code =
// nearest-even integer of the correctly rounded float32 quotient x / s.  One
// workgroup per row, two passes over it (the second from cache).
template <int DT>
__global__ __launch_bounds__(256) void k_int8_quantize(const void* __restrict__ x, int64_t cols, int8_t* __restrict__ codes,
                                                       float* __restrict__ scales) {
  const int64_t row = blockIdx.x;
  auto at = [&](int64_t c) -> float {
    if constexpr (DT == 0) return static_cast<const float*>(x)[row * cols + c];
    return bf16_to_f32(static_cast<const uint16_t*>(x)[row * cols + c]);
  };
  float top = 0.0f;
  for (int64_t c = threadIdx.x; c < cols; c += 256) top = fmaxf(top, fabsf(at(c)));
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
  __shared__ float part[4];
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = top;
  __syncthreads();
  top = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
  float s = top / 127.0f;
  if (!(s > 0.0f)) s = 1.0f;
  if (threadIdx.x == 0) scales[row] = s;
  for (int64_t c = threadIdx.x; c < cols; c += 256)
    codes[row * cols + c] = static_cast<int8_t>(fminf(fmaxf(rintf(at(c) / s), -127.0f), 127.0f));
}

hipError_t launch_int8_quantize(const void* x, int dtype, int64_t rows, int64_t cols, int8_t* codes, float* scales,
                                hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(rows));
  if (dtype == 0) hipLaunchKernelGGL((k_int8_quantize<0>), grid, dim3(256), 0, stream, x, cols, codes, scales);
  else hipLaunchKernelGGL((k_int8_quantize<1>), grid, dim3(256), 0, stream, x, cols, codes, scales);
  return hipGetLastError();
}

hipError_t launch_tile_gemm_i8(const TileParams& p, int epilogue, hipStream_t stream) {
  return epilogue == TG_OUT_GATED ? tg_launch<TG_I8, TG_NT, TG_OUT_GATED>(p, stream)
         : epilogue == TG_OUT_F32 ? tg_launch<TG_I8, TG_NT, TG_OUT_F32>(p, stream)
                                  : tg_launch<TG_I8, TG_NT, TG_OUT_16>(p, stream);
}

}  // namespace nvfp4
