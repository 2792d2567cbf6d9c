// int8_rows.cuh -- 8-bit integer rows with a scale per row, and the product of two such
// matrices:
//
//   s_r = max(max_k |x_rk| / 127, 2^-126),   q_rk = x_rk / s_r rounded to nearest, ties to even
//   out[t, n] = (sum_k q_tk w_nk) * (s_t * v_n)
//
// The division is the IEEE float32 one and |q| <= 127 by construction (max |x| / s rounds to
// at most 127 (1 + 2^-23)). The lower bound on s, the smallest normal float32, gives an
// all-zero row codes 0 without a special case. A row that holds a NaN or an infinity has no
// scale: s = NaN, codes 0, so that its products are NaN rather than finite and wrong.
// The sum is exact in 32-bit integers for K <= 131072 (127^2 K < 2^31); it is rounded once to
// float32, multiplied by the product of the scales and rounded to the output type.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "gemm_umma.cuh"
#include "route_kernels.cuh"

namespace muse {

constexpr float kInt8ScaleMin = 1.17549435e-38f;  // 2^-126

// amax (NaN or infinity: none) -> the row's scale
__device__ __forceinline__ float int8_scale(float amax) {
  return amax <= 3.402823466e38f ? fmaxf(amax / 127.0f, kInt8ScaleMin) : __int_as_float(0x7fc00000);
}
__device__ __forceinline__ int int8_code(float v, float scale) {
  return scale == scale ? __float2int_rn(v / scale) : 0;
}
// max(a, |v|) that keeps a NaN
__device__ __forceinline__ float amax_nan(float a, float v) {
  v = fabsf(v);
  return (a >= v || a != a) ? a : v;  // v NaN: the comparison fails and v is kept
}

template <typename T>
__global__ void __launch_bounds__(256) k_quant_rows_int8(const T* __restrict__ src, int64_t ld, int rows, int K,
                                                         int8_t* __restrict__ codes, float* __restrict__ scales) {
  __shared__ float part[32];
  for (int r = blockIdx.x; r < rows; r += gridDim.x) {
    const T* x = src + static_cast<int64_t>(r) * ld;
    float a = 0.0f;
    for (int i = threadIdx.x; i < K; i += blockDim.x) a = amax_nan(a, to_f32(x[i]));
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) a = amax_nan(a, __shfl_xor_sync(0xffffffffu, a, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = a;
    __syncthreads();
    for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) a = amax_nan(a, part[w]);
    const float s = int8_scale(a);
    for (int i = threadIdx.x; i < K; i += blockDim.x)
      codes[static_cast<int64_t>(r) * K + i] = static_cast<int8_t>(int8_code(to_f32(x[i]), s));
    if (threadIdx.x == 0) scales[r] = s;
  }
}

// A warp per output channel and 8 rows of x; four products per instruction.
template <typename TOut>
__global__ void __launch_bounds__(256) k_int8_matmul(const int8_t* __restrict__ x, const float* __restrict__ sx, int T,
                                                     int K, const int8_t* __restrict__ w,
                                                     const float* __restrict__ sw, int N, TOut* __restrict__ out,
                                                     int64_t ldo) {
  const int lane = threadIdx.x & 31;
  const int n = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (n >= N) return;  // warp-uniform
  for (int t0 = blockIdx.y * 8; t0 < T; t0 += 8 * gridDim.y) {
    int acc[8] = {};
    for (int k0 = lane * 16; k0 < K; k0 += 512) {
      const int4 a = *reinterpret_cast<const int4*>(w + static_cast<int64_t>(n) * K + k0);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (t0 + j < T) {
          const int4 b = *reinterpret_cast<const int4*>(x + static_cast<int64_t>(t0 + j) * K + k0);
          acc[j] = __dp4a(a.x, b.x, __dp4a(a.y, b.y, __dp4a(a.z, b.z, __dp4a(a.w, b.w, acc[j]))));
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int s = __reduce_add_sync(0xffffffffu, acc[j]);
      if (lane == j && t0 + j < T)
        out[static_cast<int64_t>(t0 + j) * ldo + n] = from_f32<TOut>(static_cast<float>(s) * (sx[t0 + j] * sw[n]));
    }
  }
}

}  // namespace muse
