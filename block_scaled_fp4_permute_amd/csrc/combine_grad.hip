// Gradients of the weighted combine out[t] = sum_j w[t, j] y[row(t, j)]:
//   dy[row(t, j)] = w[t, j] dout[t]   (rounded once to y's type)
//   dw[t, j] = <dout[t], y[row(t, j)]>   (float32 sums in a fixed order)
// in one pass: every row of y is read once, every row of dy written once, both past the
// caches.  Bound by memory: 16384 tokens, top-8, 6144 wide, bf16 (3.4 GB) 675 to 690 us, 5.0
// TB/s; in float32 (6.8 GB) 1456, 4.7 TB/s, and 4096 tokens 1024 wide 50, 5.8 TB/s.
#include "nvfp4_internal.h"

namespace nvfp4 {

typedef unsigned int u32x4g __attribute__((ext_vector_type(4)));

template <int DT>
__device__ __forceinline__ void cg_load8(const void* base, int64_t row, int H, int c, bool once, float (&v)[8]) {
  if constexpr (DT == 1) {
    const u32x4g* p = reinterpret_cast<const u32x4g*>(static_cast<const uint16_t*>(base) + row * H) + c;
    const u32x4g q = once ? __builtin_nontemporal_load(p) : *p;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      v[2 * m] = __uint_as_float(q[m] << 16);
      v[2 * m + 1] = __uint_as_float(q[m] & 0xFFFF0000u);
    }
  } else {
    const float4v* p = reinterpret_cast<const float4v*>(static_cast<const float*>(base) + row * H) + 2 * c;
    const float4v a = once ? __builtin_nontemporal_load(p) : p[0], b = once ? __builtin_nontemporal_load(p + 1) : p[1];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      v[m] = a[m];
      v[4 + m] = b[m];
    }
  }
}

typedef __bf16 bf16x2g __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t cg_pack2(float a, float b) {
  const bf16x2g r = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
  return __builtin_bit_cast(uint32_t, r);
}

template <int DT>
__device__ __forceinline__ void cg_store8(void* base, int64_t row, int H, int c, const float (&v)[8]) {
  if constexpr (DT == 1) {
    const u32x4g q = {cg_pack2(v[0], v[1]), cg_pack2(v[2], v[3]), cg_pack2(v[4], v[5]), cg_pack2(v[6], v[7])};
    __builtin_nontemporal_store(q, reinterpret_cast<u32x4g*>(static_cast<uint16_t*>(base) + row * H) + c);
  } else {
    float4v* p = reinterpret_cast<float4v*>(static_cast<float*>(base) + row * H) + 2 * c;
    __builtin_nontemporal_store(float4v{v[0], v[1], v[2], v[3]}, p);
    __builtin_nontemporal_store(float4v{v[4], v[5], v[6], v[7]}, p + 1);
  }
}

// LPT lanes (64: a wave, 256: the workgroup) for JB of a token's k rows.  A row
// outside y's is left out: nothing written, dw 0.
template <int DT, int YT, int LPT, int JB>
__global__ __launch_bounds__(256) void k_combine_grad(const CombineGradParams p, int jblocks) {
  const int64_t task = static_cast<int64_t>(blockIdx.x) * (256 / LPT) + threadIdx.x / LPT;
  if (task >= static_cast<int64_t>(p.T) * jblocks) return;     // whole waves, or no lane of the workgroup
  const int t = static_cast<int>(task / jblocks);
  const int j0 = static_cast<int>(task % jblocks) * JB;
  const int l = threadIdx.x % LPT;
  int64_t row[JB];
  float w[JB], sum[JB];
#pragma unroll
  for (int j = 0; j < JB; ++j) {
    const int64_t a = static_cast<int64_t>(t) * p.k + min(j0 + j, p.k - 1);
    row[j] = p.perm ? p.perm[a] : a;
    if (row[j] < 0 || row[j] >= p.rows || j0 + j >= p.k) row[j] = -1;
    w[j] = p.w ? p.w[a] : 1.0f;
    sum[j] = 0.0f;
  }
  for (int c = l; c < p.H / 8; c += LPT) {
    float d[8];
    cg_load8<DT>(p.dout, t, p.H, c, false, d);
    if (p.dw) {
      float v[JB][8];
#pragma unroll
      for (int j = 0; j < JB; ++j) cg_load8<YT>(p.y, row[j] < 0 ? 0 : row[j], p.H, c, true, v[j]);
#pragma unroll
      for (int j = 0; j < JB; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[j] = fmaf(d[i], v[j][i], sum[j]);
    }
    if (p.dy) {
#pragma unroll
      for (int j = 0; j < JB; ++j) {
        if (row[j] < 0) continue;
        float r[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = w[j] * d[i];
        cg_store8<YT>(p.dy, row[j], p.H, c, r);
      }
    }
  }
  if (!p.dw) return;
#pragma unroll
  for (int j = 0; j < JB; ++j)
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) sum[j] += __shfl_xor(sum[j], o);
  if constexpr (LPT == 256) {
    __shared__ float part[4][JB];
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int j = 0; j < JB; ++j) part[threadIdx.x >> 6][j] = sum[j];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < JB; ++j) sum[j] = (part[0][j] + part[1][j]) + (part[2][j] + part[3][j]);
  }
  if (l == 0)
#pragma unroll
    for (int j = 0; j < JB; ++j)
      if (j0 + j < p.k) p.dw[static_cast<int64_t>(t) * p.k + j0 + j] = row[j] < 0 ? 0.0f : sum[j];
}

template <int DT, int YT, int LPT, int JB>
static hipError_t cg_start(const CombineGradParams& p, hipStream_t stream) {
  const int jblocks = (p.k + JB - 1) / JB;
  const int64_t tasks = static_cast<int64_t>(p.T) * jblocks;
  const int64_t blocks = (tasks + 256 / LPT - 1) / (256 / LPT);
  if (blocks >= (int64_t(1) << 24)) return hipErrorInvalidConfiguration;   // refused by the caller
  hipLaunchKernelGGL((k_combine_grad<DT, YT, LPT, JB>), dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream, p, jblocks);
  return hipGetLastError();
}

// A wave for two of a token's rows up to 2048 wide, else the workgroup for four:
// top-8 in bf16, us, wave / workgroup
//   H 512, 2048 tokens 7.9 / 11.2, 16384 tokens 44 / 83;  H 1024, 16384 tokens 99 / 151
//   H 2048, 1024 tokens 12.4 / 14.5, 4096 tokens 44.7 / 46.0, 16384 tokens 245 / 231
//   H 6144, 255 tokens 12.2 / 9.8, 2048 tokens 65 / 68, 4096 tokens 193 / 174, 16384 tokens 697 / 692
// (a workgroup for one row each: 13.0, 85, 176 and 693 there)
// in float32, where rows have twice the bytes and either side of the limit is within 8 %
//   H 512, 16384 tokens 108 / 129;  H 1024, 255 tokens 4.7 / 5.2, 16384 tokens 254 / 239
//   H 2048, 255 tokens 6.3 / 7.6, 4096 tokens 114 / 105, 16384 tokens 497 / 481
//   H 4096, 255 tokens 12.7 / 15.0, 4096 tokens 259 / 249;  H 6144, 16384 tokens 1485 / 1461
template <int DT, int YT>
static hipError_t cg_launch(const CombineGradParams& p, hipStream_t stream) {
  return p.H <= 2048 ? cg_start<DT, YT, 64, 2>(p, stream) : cg_start<DT, YT, 256, 4>(p, stream);
}

hipError_t launch_combine_grad(const CombineGradParams& p, int dout_dtype, int y_dtype, hipStream_t stream) {
  if (dout_dtype == 1) return y_dtype == 1 ? cg_launch<1, 1>(p, stream) : cg_launch<1, 0>(p, stream);
  return y_dtype == 1 ? cg_launch<0, 1>(p, stream) : cg_launch<0, 0>(p, stream);
}

}  // namespace nvfp4
