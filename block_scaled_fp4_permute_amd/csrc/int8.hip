// INT8 products with one scale per row of each operand (tokens and output
// channels), and the quantiser that makes such operands.
#include "skinny_gemm.h"

namespace nvfp4 {

// s = absmax * (1/127) (float32 product with the float32 nearest 1/127; 1 where
// that is zero), code = nearest-even integer of the correctly rounded float32
// quotient x / s.
//
// One read of x: LPR lanes hold a row in registers (NV pieces of 8 values a
// lane), reduce its maximum and write codes and scale.  Bound by memory: bf16
// 16384 x 6144 takes 50 - 55 us, 5.5 - 6.0 TB/s (164 with two reads and divisions).  The
// quotient is x * (1 / s) except where that lands within 2^-14 of a tie between
// two codes: |x / s| <= 127 (1 + 2^-22), so the product's two roundings and the
// quotient's own move it by less than 127 * 3 * 2^-24 < 2^-15, and only there
// can they decide otherwise than the divided quotient.  Below 2^-100 the
// reciprocal could leave float32's range, and the row is divided throughout.
//
// The maximum keeps a NaN (as many instructions as one that drops it): a row that
// holds one, or an infinity, gets scale NaN and codes 0.
template <int DT>
struct Q8Piece {
  u32x4 w[DT == 0 ? 2 : 1];
  __device__ __forceinline__ float at(int i) const {
    if constexpr (DT == 0) return __uint_as_float(w[i >> 2][i & 3]);
    return __uint_as_float((i & 1) ? w[0][i >> 1] & 0xFFFF0000u : w[0][i >> 1] << 16);
  }
};

template <int DT>
__device__ __forceinline__ Q8Piece<DT> q8_load(const void* __restrict__ x, int64_t first) {
  Q8Piece<DT> r;
  const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(x) + first * (DT == 0 ? 4 : 2));
  r.w[0] = p[0];
  if constexpr (DT == 0) r.w[1] = p[1];
  return r;
}

__device__ __forceinline__ int q8_code(float x, float s, float inv, bool fast) {
  float q = x * inv;
  float k = rintf(q);
  if (!fast || fabsf(fabsf(q - k) - 0.5f) < 0x1p-14f) k = rintf(x / s);
  return static_cast<int>(fminf(fmaxf(k, -127.0f), 127.0f));
}

template <int DT>
__device__ __forceinline__ void q8_store(const Q8Piece<DT>& v, float s, float inv, bool fast, uint32_t keep, int8_t* __restrict__ dst) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) r |= (static_cast<uint32_t>(q8_code(v.at(4 * h + i), s, inv, fast)) & 0xFFu) << (8 * i);
    w[h] = r & keep;
  }
  *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
}

// the maximum over the LPR lanes of a row (64: the wave, 256: the workgroup)
template <int LPR>
__device__ __forceinline__ float q8_row_max(float m) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) m = __builtin_elementwise_maximum(m, __shfl_xor(m, d));
  if constexpr (LPR == 256) {
    __shared__ float part[4];
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
    __syncthreads();
    m = __builtin_elementwise_maximum(__builtin_elementwise_maximum(part[0], part[1]), __builtin_elementwise_maximum(part[2], part[3]));
  }
  return m;
}

// NV = 0: rows of any length, read a second time (from cache) for the codes
template <int DT, int LPR, int NV>
__global__ __launch_bounds__(256) void k_int8_quantize(const void* __restrict__ x, int64_t rows, int cols,
                                                       int8_t* __restrict__ codes, float* __restrict__ scales) {
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (256 / LPR) + threadIdx.x / LPR;
  if (row >= rows) return;                  // whole waves (LPR 64) or no lane at all
  const int l = threadIdx.x % LPR;
  const int pieces = cols / 8;
  const int64_t base = row * cols;
  float top = 0.0f;
  Q8Piece<DT> v[NV > 0 ? NV : 1];
  if constexpr (NV > 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = l + i * LPR;
      v[i] = q8_load<DT>(x, base + 8 * (c < pieces ? c : 0));
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int q = 0; q < 8; ++q) top = __builtin_elementwise_maximum(top, fabsf(v[i].at(q)));
  } else {
    for (int c = l; c < pieces; c += LPR) {
      const Q8Piece<DT> w = q8_load<DT>(x, base + 8 * static_cast<int64_t>(c));
#pragma unroll
      for (int q = 0; q < 8; ++q) top = __builtin_elementwise_maximum(top, fabsf(w.at(q)));
    }
  }
  top = q8_row_max<LPR>(top);
  const bool finite = top < __builtin_inff();
  const uint32_t keep = finite ? ~0u : 0u;  // of the codes
  float s = finite ? top * (1.0f / 127.0f) : __builtin_nanf("");
  if (s == 0.0f) s = 1.0f;
  const bool fast = s > 0x1p-100f;
  const float inv = 1.0f / s;
  if (l == 0) scales[row] = s;
  if constexpr (NV > 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = l + i * LPR;
      if (c < pieces) q8_store<DT>(v[i], s, inv, fast, keep, codes + base + 8 * c);
    }
  } else {
    for (int c = l; c < pieces; c += LPR) {
      const int64_t o = base + 8 * static_cast<int64_t>(c);
      q8_store<DT>(q8_load<DT>(x, o), s, inv, fast, keep, codes + o);
    }
  }
}

template <int DT, int LPR, int NV>
static hipError_t q8_start(const void* x, int64_t rows, int cols, int8_t* codes, float* scales, hipStream_t stream) {
  // a grid has fewer than 2^32 threads
  constexpr int64_t kMost = int64_t(1) << 23;
  for (int64_t r0 = 0; r0 < rows; r0 += kMost) {
    const int64_t n = rows - r0 < kMost ? rows - r0 : kMost;
    const int64_t blocks = (n + 256 / LPR - 1) / (256 / LPR);
    hipLaunchKernelGGL((k_int8_quantize<DT, LPR, NV>), dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream,
                       static_cast<const uint8_t*>(x) + r0 * cols * (DT == 0 ? 4 : 2), n, cols, codes + r0 * cols, scales + r0);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

// a wave per row up to 1024 values (2 pieces a lane), a workgroup above, to 16384
// values in registers (8 pieces: 64 registers of float32)
template <int DT>
static hipError_t q8_launch(const void* x, int64_t rows, int cols, int8_t* codes, float* scales, hipStream_t stream) {
  if (cols <= 512) return q8_start<DT, 64, 1>(x, rows, cols, codes, scales, stream);
  if (cols <= 1024) return q8_start<DT, 64, 2>(x, rows, cols, codes, scales, stream);
  if (cols <= 2048) return q8_start<DT, 256, 1>(x, rows, cols, codes, scales, stream);
  if (cols <= 4096) return q8_start<DT, 256, 2>(x, rows, cols, codes, scales, stream);
  if (cols <= 6144) return q8_start<DT, 256, 3>(x, rows, cols, codes, scales, stream);
  if (cols <= 8192) return q8_start<DT, 256, 4>(x, rows, cols, codes, scales, stream);
  if (cols <= 16384) return q8_start<DT, 256, 8>(x, rows, cols, codes, scales, stream);
  return q8_start<DT, 256, 0>(x, rows, cols, codes, scales, stream);
}

hipError_t launch_int8_quantize(const void* x, int dtype, int64_t rows, int64_t cols, int8_t* codes, float* scales,
                                hipStream_t stream) {
  const int c = static_cast<int>(cols);
  return dtype == 0 ? q8_launch<0>(x, rows, c, codes, scales, stream) : q8_launch<1>(x, rows, c, codes, scales, stream);
}

hipError_t launch_tile_gemm_i8(const TileParams& p, int epilogue, hipStream_t stream) {
  return epilogue == TG_OUT_GATED ? tg_launch<TG_I8, TG_NT, TG_OUT_GATED>(p, stream)
         : epilogue == TG_OUT_F32 ? tg_launch<TG_I8, TG_NT, TG_OUT_F32>(p, stream)
                                  : tg_launch<TG_I8, TG_NT, TG_OUT_16>(p, stream);
}

}  // namespace nvfp4
