// INT4 weights in groups along the reduction: the quantiser and its inverse, and
// products on bfloat16 activations.
#include "int4_gemv.h"

namespace nvfp4 {

// A group of 32, 64 or 128 values along the last axis has one 16-bit scale s (and
// with zero points one z in 0..15); value = (q - z) s, z = 8 without.
//   symmetric  s = absmax * (1/7), q = clamp(rint(x / s), -8, 7) + 8
//   zeros      lo = min(x, 0), hi = max(x, 0), s = (hi - lo) * (1/15),
//              z = clamp(rint(-lo / s), 0, 15), q = clamp(rint(x / s) + z, 0, 15)
// s is a float32 product (with the float32 nearest 1/7 or 1/15), rounded to its
// 16-bit type (1 where that gives 0), and the quotients are float32 ones, correctly
// rounded, so codes are reproducible bit for bit.
// A group with a NaN or an infinity, or whose scale overflows its type, gets scale
// NaN, codes 8 (zeros: codes and z 0).
//
// One pass: 8 lanes (4 of a group of 32) hold a group, 8 values each or two times 8.
// Bound by memory where instructions are few (256 x 512 x 6144 in bf16, groups of 128: 308
// us, 6.6 TB/s; 402 with true divisions wherever x * (1 / s) lands next to a tie, which a
// group of bf16 values does often enough).  So the divisions share their reciprocal:
// with y the correctly rounded 1 / s and t = x y, t + (x - t s) y rounds to the quotient.
//   y: rcp is 1 ulp off, and one Newton step leaves 2^-46; s has at most 11 bits, so 1 / s
//   is 2^-36 at least from where its rounding changes
//   quotient: the remainder x - t s is exact, what is left 2^-46 off; a place where the
//   rounding changes is an odd number M of 25 bits, and x = S M has no solution in 24
//   bits, so x / s is 2^-36 at least from any
// Below 2^-100 the remainder could leave float32's range, and the group is divided.  The
// quotient's rounding to an integer is an addition of 1.5 * 2^23, whose low bits are the
// code after a clamp.
template <int DT>
struct I4Piece {
  u32x4 w[DT == 0 ? 2 : 1];
  __device__ __forceinline__ float at(int i) const {
    if constexpr (DT == 0) return __uint_as_float(w[i >> 2][i & 3]);
    if constexpr (DT == 1) return __uint_as_float((i & 1) ? w[0][i >> 1] & 0xFFFF0000u : w[0][i >> 1] << 16);
    const uint32_t d = w[0][i >> 1];         // a copy: a cast of the element itself reads element 0
    const half2v h = __builtin_bit_cast(half2v, d);
    return static_cast<float>(h[i & 1]);
  }
};

// over the L (4 or 8) lanes of a group
template <int L>
__device__ __forceinline__ float i4_max(float v) {
  v = __builtin_elementwise_maximum(v, __uint_as_float(dpp_u32<kDppXor1>(__float_as_uint(v))));
  v = __builtin_elementwise_maximum(v, __uint_as_float(dpp_u32<kDppXor2>(__float_as_uint(v))));
  if constexpr (L >= 8) v = __builtin_elementwise_maximum(v, __uint_as_float(dpp_u32<kDppHalfMirror>(__float_as_uint(v))));
  return v;
}

constexpr int i4_pieces(int group) { return group == 128 ? 2 : 1; }       // of 8 values a lane

template <int DT, int GROUP, bool ZEROS, bool SF16>
__global__ __launch_bounds__(256) void k_int4_quantize(const void* __restrict__ x, int64_t pieces, uint32_t* __restrict__ codes,
                                                       uint16_t* __restrict__ scales, uint8_t* __restrict__ zeros) {
  constexpr int P = i4_pieces(GROUP), L = GROUP / 8 / P;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i * P >= pieces) return;              // whole groups
  const int64_t i0 = P == 1 ? i : i / L * (P * L) + i % L;  // the lane's pieces are L apart
  I4Piece<DT> v[P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const u32x4* src = static_cast<const u32x4*>(x) + (i0 + p * L) * (DT == 0 ? 2 : 1);
    v[p].w[0] = __builtin_nontemporal_load(src);
    if constexpr (DT == 0) v[p].w[1] = __builtin_nontemporal_load(src + 1);
  }
  float hi = 0.0f, lo = 0.0f;               // lo: of -x
#pragma unroll
  for (int p = 0; p < P; ++p) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float a = v[p].at(k);
      hi = __builtin_elementwise_maximum(hi, ZEROS ? a : fabsf(a));
      if constexpr (ZEROS) lo = __builtin_elementwise_maximum(lo, -a);
    }
  }
  hi = i4_max<L>(hi);
  if constexpr (ZEROS) lo = i4_max<L>(lo);
  float raw = ZEROS ? (hi + lo) * (1.0f / 15.0f) : hi * (1.0f / 7.0f);
  asm("" : "+v"(raw));                      // a float32 product: one with the conversion to f16 in it rounds but once
  uint16_t bits;
  float s;
  if constexpr (SF16) {
    const _Float16 h = static_cast<_Float16>(raw);
    bits = __builtin_bit_cast(uint16_t, h);
    s = static_cast<float>(h);
  } else {
    const __bf16 h = static_cast<__bf16>(raw);
    bits = __builtin_bit_cast(uint16_t, h);
    s = static_cast<float>(h);
  }
  const bool finite = s < __builtin_inff();
  if (s == 0.0f) {
    s = 1.0f;
    bits = SF16 ? 0x3C00 : 0x3F80;
  }
  if (!finite) {
    s = 1.0f;
    bits = SF16 ? 0x7E00 : 0x7FC0;
  }
  constexpr float kBase = 0x1.8p23f;
  float y = __builtin_amdgcn_rcpf(s);
  y = fmaf(fmaf(-s, y, 1.0f), y, y);
  auto quotient = [&](float v) __attribute__((always_inline)) {
    const float t = v * y;
    return fmaf(fmaf(-t, s, v), y, t);
  };
  float z = 8.0f;
  if constexpr (ZEROS) z = fminf(rintf(quotient(lo)), 15.0f);
  float q[P][8];
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float t = quotient(v[p].at(k));
      q[p][k] = (ZEROS ? rintf(t) : t) + (kBase + z);        // z may be odd, and then a tie's other side even
    }
  if (s <= 0x1p-100f) {
    if constexpr (ZEROS) z = fminf(rintf(lo / s), 15.0f);
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int k = 0; k < 8; ++k) q[p][k] = rintf(v[p].at(k) / s) + (kBase + z);
  }
#pragma unroll
  for (int p = 0; p < P; ++p) {
    // kBase's own bits, shifted with the codes, reach bit 31 by the third code
    uint32_t w = 0u - (0x4B400000u + (0x4B400000u << 4) + (0x4B400000u << 8));
#pragma unroll
    for (int k = 0; k < 8; ++k) w += __float_as_uint(__builtin_amdgcn_fmed3f(q[p][k], kBase, kBase + 15.0f)) << (4 * k);
    if (!finite) w = ZEROS ? 0u : 0x88888888u;
    codes[i0 + p * L] = w;
  }
  if (threadIdx.x % L == 0) {
    scales[i / L] = bits;
    if constexpr (ZEROS) zeros[i / L] = finite ? static_cast<uint8_t>(z) : 0;
  }
}

// The inverse, 8 codes a lane: bound by memory (the same weights 387 us, 5.2 TB/s, most of it
// the values written).  16-bit values are rounded once, from an exact product.
template <int GROUP, bool ZEROS, bool SF16, bool OUT32>
__global__ __launch_bounds__(256) void k_int4_dequantize(const uint32_t* __restrict__ codes, const uint16_t* __restrict__ scales,
                                                         const uint8_t* __restrict__ zeros, int64_t pieces, void* __restrict__ out) {
  constexpr int L = GROUP / 8;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= pieces) return;
  const uint32_t w = codes[i];
  const float s = I4Type<SF16>::value(scales[i / L]);
  const float z = ZEROS ? static_cast<float>(zeros[i / L]) : 8.0f;
  float4v v[2];
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k >> 2][k & 3] = (static_cast<float>((w >> (4 * k)) & 15u) - z) * s;
  if constexpr (OUT32) {
    float4v* dst = static_cast<float4v*>(out) + 2 * i;
    __builtin_nontemporal_store(v[0], dst);
    __builtin_nontemporal_store(v[1], dst + 1);
  } else {
    const uint2 a = I4Type<SF16>::TT::pack(v[0]), b = I4Type<SF16>::TT::pack(v[1]);
    __builtin_nontemporal_store(u32x4{a.x, a.y, b.x, b.y}, static_cast<u32x4*>(out) + i);
  }
}

// a grid has fewer than 2^32 threads
static constexpr int64_t kI4Most = int64_t(1) << 31;

template <int DT, int GROUP, bool ZEROS, bool SF16>
static hipError_t i4_quantize(const void* x, int64_t pieces, uint32_t* codes, uint16_t* scales, uint8_t* zeros, hipStream_t stream) {
  for (int64_t i = 0; i < pieces; i += kI4Most) {
    const int64_t n = pieces - i < kI4Most ? pieces - i : kI4Most;
    constexpr int per = 256 * i4_pieces(GROUP);
    hipLaunchKernelGGL((k_int4_quantize<DT, GROUP, ZEROS, SF16>), dim3(static_cast<unsigned>((n + per - 1) / per)), dim3(256), 0, stream,
                       static_cast<const uint8_t*>(x) + i * (DT == 0 ? 32 : 16), n, codes + i, scales + i / (GROUP / 8),
                       ZEROS ? zeros + i / (GROUP / 8) : nullptr);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

template <int DT, int GROUP>
static hipError_t i4_quantize_group(const void* x, int64_t pieces, int sf16, uint32_t* codes, uint16_t* scales, uint8_t* zeros, hipStream_t stream) {
  if (zeros) return sf16 ? i4_quantize<DT, GROUP, true, true>(x, pieces, codes, scales, zeros, stream)
                         : i4_quantize<DT, GROUP, true, false>(x, pieces, codes, scales, zeros, stream);
  return sf16 ? i4_quantize<DT, GROUP, false, true>(x, pieces, codes, scales, zeros, stream)
              : i4_quantize<DT, GROUP, false, false>(x, pieces, codes, scales, zeros, stream);
}

template <int DT>
static hipError_t i4_quantize_type(const void* x, int64_t pieces, int group, int sf16, uint32_t* codes, uint16_t* scales, uint8_t* zeros,
                                   hipStream_t stream) {
  return group == 32 ? i4_quantize_group<DT, 32>(x, pieces, sf16, codes, scales, zeros, stream)
       : group == 64 ? i4_quantize_group<DT, 64>(x, pieces, sf16, codes, scales, zeros, stream)
                     : i4_quantize_group<DT, 128>(x, pieces, sf16, codes, scales, zeros, stream);
}

hipError_t launch_int4_quantize(const void* x, int dtype, int64_t rows, int64_t cols, int group, int scale_f16, uint8_t* codes,
                                void* scales, uint8_t* zeros, hipStream_t stream) {
  const int64_t pieces = rows * (cols / 8);
  uint32_t* c = reinterpret_cast<uint32_t*>(codes);
  uint16_t* s = static_cast<uint16_t*>(scales);
  return dtype == 0 ? i4_quantize_type<0>(x, pieces, group, scale_f16, c, s, zeros, stream)
       : dtype == 1 ? i4_quantize_type<1>(x, pieces, group, scale_f16, c, s, zeros, stream)
                    : i4_quantize_type<2>(x, pieces, group, scale_f16, c, s, zeros, stream);
}

template <int GROUP, bool ZEROS, bool SF16, bool OUT32>
static hipError_t i4_dequantize(const uint32_t* codes, const uint16_t* scales, const uint8_t* zeros, int64_t pieces, void* out,
                                hipStream_t stream) {
  for (int64_t i = 0; i < pieces; i += kI4Most) {
    const int64_t n = pieces - i < kI4Most ? pieces - i : kI4Most;
    hipLaunchKernelGGL((k_int4_dequantize<GROUP, ZEROS, SF16, OUT32>), dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0, stream,
                       codes + i, scales + i / (GROUP / 8), ZEROS ? zeros + i / (GROUP / 8) : nullptr, n,
                       static_cast<uint8_t*>(out) + i * (OUT32 ? 32 : 16));
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

template <int GROUP>
static hipError_t i4_dequantize_group(const uint32_t* codes, const uint16_t* scales, const uint8_t* zeros, int64_t pieces, int sf16,
                                      int out32, void* out, hipStream_t stream) {
  if (zeros) {
    if (sf16) return out32 ? i4_dequantize<GROUP, true, true, true>(codes, scales, zeros, pieces, out, stream)
                           : i4_dequantize<GROUP, true, true, false>(codes, scales, zeros, pieces, out, stream);
    return out32 ? i4_dequantize<GROUP, true, false, true>(codes, scales, zeros, pieces, out, stream)
                 : i4_dequantize<GROUP, true, false, false>(codes, scales, zeros, pieces, out, stream);
  }
  if (sf16) return out32 ? i4_dequantize<GROUP, false, true, true>(codes, scales, zeros, pieces, out, stream)
                         : i4_dequantize<GROUP, false, true, false>(codes, scales, zeros, pieces, out, stream);
  return out32 ? i4_dequantize<GROUP, false, false, true>(codes, scales, zeros, pieces, out, stream)
               : i4_dequantize<GROUP, false, false, false>(codes, scales, zeros, pieces, out, stream);
}

hipError_t launch_int4_dequantize(const uint8_t* codes, const void* scales, const uint8_t* zeros, int64_t rows, int64_t cols,
                                  int group, int scale_f16, int out_dtype, void* out, hipStream_t stream) {
  const int64_t pieces = rows * (cols / 8);
  const uint32_t* c = reinterpret_cast<const uint32_t*>(codes);
  const uint16_t* s = static_cast<const uint16_t*>(scales);
  const int out32 = out_dtype == 0;
  return group == 32 ? i4_dequantize_group<32>(c, s, zeros, pieces, scale_f16, out32, out, stream)
       : group == 64 ? i4_dequantize_group<64>(c, s, zeros, pieces, scale_f16, out32, out, stream)
                     : i4_dequantize_group<128>(c, s, zeros, pieces, scale_f16, out32, out, stream);
}

hipError_t launch_int4_gemv_f16(const Int4Params& p, int group, int gated, int out32, hipStream_t stream);

int64_t int4_gemv_threads(int E, int N, int K, int64_t m_total, int64_t hint, int gated) {
  const Int4Shape& s = kI4Shapes[i4_choice(E, N, K, m_total, hint, gated)];
  return i4_blocks(s, E, N, m_total, gated) * (64 * s.wk * s.wc);
}

hipError_t launch_int4_gemv(const Int4Params& p, int f16, int group, int gated, int out_f32, hipStream_t stream) {
  return f16 ? launch_int4_gemv_f16(p, group, gated, out_f32, stream) : i4_launch_type<false>(p, group, gated, out_f32, stream);
}

}  // namespace nvfp4
