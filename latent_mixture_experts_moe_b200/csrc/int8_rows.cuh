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

// The row's scale from the bits of its largest magnitude (as integers they order like the
// magnitudes, infinity and then NaN last).
__device__ __forceinline__ float int8_scale(uint32_t amax_bits) {
  return amax_bits < 0x7f800000u ? fmaxf(__uint_as_float(amax_bits) / 127.0f, kInt8ScaleMin)
                                 : __int_as_float(0x7fc00000);
}
__device__ __forceinline__ uint32_t magnitude_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

__device__ __forceinline__ uint32_t int8_pack(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040u), __byte_perm(c, d, 0x0040u), 0x5410u);
}
// (kept out of line: rare, and its registers would cost occupancy)
__device__ __noinline__ uint32_t int8_divide4(float a, float b, float c, float d, float scale) {
  return int8_pack(__float2int_rn(a / scale), __float2int_rn(b / scale), __float2int_rn(c / scale),
                   __float2int_rn(d / scale));
}
// Eight codes: v / scale rounded to nearest, ties to even; inv = 1 / scale. v * inv is within 3
// units in the last place of the quotient (at most 127: within 3 * 2^-17), so both round to the
// same integer unless the product is that near to a half; only then the eight divisions are
// done. Rounding by adding 1.5 * 2^23 leaves the integer in the sum's low bits.
__device__ __forceinline__ uint2 int8_codes8(const float (&v)[8], float scale, float inv) {
  constexpr float kRound = 12582912.0f;
  uint32_t q[8];
  float off = 0.0f;  // largest distance from an integer
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float r = v[i] * inv, t = r + kRound;
    q[i] = __float_as_uint(t);
    off = fmaxf(off, fabsf(r - (t - kRound)));
  }
  if (scale != scale) return make_uint2(0u, 0u);
  if (off > 0.4999f)
    return make_uint2(int8_divide4(v[0], v[1], v[2], v[3], scale), int8_divide4(v[4], v[5], v[6], v[7], scale));
  return make_uint2(int8_pack(q[0], q[1], q[2], q[3]), int8_pack(q[4], q[5], q[6], q[7]));
}

// eight consecutive values; ALIGNED: from a 16-byte boundary
template <typename T, bool ALIGNED>
struct Int8Load {
  T raw[8];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (ALIGNED) {
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
        reinterpret_cast<uint4*>(raw)[i] = reinterpret_cast<const uint4*>(p)[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) raw[i] = p[i];
    }
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32(raw[i]);
  }
};

// TPR threads per row (32, 128 or 256), which hold up to 32 values each, so that a row of up to 32 TPR
// values is read once, all its loads in flight together; longer rows are read again for the
// codes (from L2). Bound by reading the rows and writing the codes; five blocks an SM keep
// enough loads in flight (8192 x 8192 bf16: 83 us with two).
template <typename T, int TPR, bool ALIGNED>
__global__ void __launch_bounds__(256, 5) k_quant_rows_int8(const T* __restrict__ src, int64_t ld, int rows, int K,
                                                         int8_t* __restrict__ codes, float* __restrict__ scales) {
  constexpr int kVecs = 4;
  __shared__ uint32_t part[8];
  const int sub = threadIdx.x % TPR;
  const int r = blockIdx.x * (256 / TPR) + threadIdx.x / TPR;
  if (r >= rows) return;  // (all threads of the row)
  const T* x = src + static_cast<int64_t>(r) * ld;
  int8_t* out = codes + static_cast<int64_t>(r) * K;
  Int8Load<T, ALIGNED> hold[kVecs];
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int k = (i * TPR + sub) * 8;
    if (k < K) hold[i].load(x + k);
  }
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    if ((i * TPR + sub) * 8 < K) {
      float v[8];
      hold[i].get(v);
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = max(amax, magnitude_bits(v[j]));
    }
  }
  for (int k = (kVecs * TPR + sub) * 8; k < K; k += TPR * 8) {
    Int8Load<T, ALIGNED> more;
    more.load(x + k);
    float v[8];
    more.get(v);
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = max(amax, magnitude_bits(v[j]));
  }
  amax = __reduce_max_sync(0xffffffffu, amax);
  if constexpr (TPR > 32) {
    const int first = threadIdx.x / TPR * (TPR / 32);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = amax;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + static_cast<int>(threadIdx.x) / TPR), "n"(TPR) : "memory");
#pragma unroll
    for (int w = 0; w < TPR / 32; ++w) amax = max(amax, part[first + w]);
  }
  const float s = int8_scale(amax), inv = 1.0f / s;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int k = (i * TPR + sub) * 8;
    if (k < K) {
      float v[8];
      hold[i].get(v);
      *reinterpret_cast<uint2*>(out + k) = int8_codes8(v, s, inv);
    }
  }
  for (int k = (kVecs * TPR + sub) * 8; k < K; k += TPR * 8) {
    Int8Load<T, ALIGNED> more;
    more.load(x + k);
    float v[8];
    more.get(v);
    *reinterpret_cast<uint2*>(out + k) = int8_codes8(v, s, inv);
  }
  if (sub == 0) scales[r] = s;
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
