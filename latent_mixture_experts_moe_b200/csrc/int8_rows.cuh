// int8_rows.cuh -- 8-bit integer rows with a scale per row, and the product of two such
// matrices:
//
//   s_r = max(max_k |x_rk| / 127, 2^-126),   q_rk = x_rk / s_r rounded to nearest, ties to even
//   out[t, n] = (sum_k q_tk w_nk) * (s_t * v_n)
//
// The divisions are the IEEE float32 ones, or (MUSE_INT8_SCALE_RECIPROCAL) s_r is max |x| times the
// float32 number next to 1 / 127, which is how PyTorch evaluates `amax / 127.0` on a GPU. The two
// scales differ by a unit in the last place in 4.5 % of the rows, and that moves codes whose
// quotient lies at n + 1/2 (frequent in bf16 rows: 33 codes of 4000 x 8192). |q| <= 127 by
// construction either way (max |x| / s rounds to at most 127 (1 + 2^-22)). The lower bound on s, the smallest normal float32, gives an
// all-zero row codes 0 without a special case. A row that holds a NaN or an infinity has no
// scale: s = NaN, codes 0, so that its products are NaN rather than finite and wrong.
// The sum is exact in 32-bit integers for K <= 131072 (int8_sum); it is rounded once to
// float32, multiplied by the product of the scales and rounded to the output type.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "few_tokens.cuh"
#include "gemm_umma.cuh"
#include "route_kernels.cuh"

namespace muse {

constexpr float kInt8ScaleMin = 1.17549435e-38f;  // 2^-126

// The row's scale from the bits of its largest magnitude (as integers they order like the
// magnitudes, infinity and then NaN last); reciprocal: see above.
__device__ __forceinline__ float int8_scale(uint32_t amax_bits, bool reciprocal) {
  constexpr float kInv127 = 1.0f / 127.0f;
  const float amax = __uint_as_float(amax_bits);
  return amax_bits < 0x7f800000u ? fmaxf(reciprocal ? amax * kInv127 : amax / 127.0f, kInt8ScaleMin)
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
  alignas(16) T raw[8];
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
  // the largest magnitude's bits (see magnitude_bits), and a: bf16 two at a time
  __device__ __forceinline__ uint32_t amax(uint32_t a) const {
    if constexpr (sizeof(T) == 2) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) m = __vmaxu2(m, reinterpret_cast<const uint32_t*>(raw)[i] & 0x7fff7fffu);
      return max(a, max(m << 16, m & 0xffff0000u));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) a = max(a, magnitude_bits(to_f32(raw[i])));
      return a;
    }
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32(raw[i]);
  }
};

// TPR threads per row (32, 128 or 256), which hold up to 32 values each, so that a row of up to 32 TPR
// values is read once, all its loads in flight together; longer rows are read again for the
// codes (from L2). Float32 rows are bound by reading them (4096 x 8192: 29.9 us, 4.7 TB/s from
// DRAM). Of bf16 rows five blocks an SM keep enough loads in flight (8192 x 8192: 48-52 us, 83 with
// two); no unit is full then (issue slots, the busiest, 68 %; a row's codes wait for its maximum).
template <typename T, int TPR, bool ALIGNED>
__global__ void __launch_bounds__(256, 5) k_quant_rows_int8(const T* __restrict__ src, int64_t ld, int rows, int K,
                                                         int8_t* __restrict__ codes, float* __restrict__ scales,
                                                         bool reciprocal) {
  constexpr int kVecs = 4;
  __shared__ uint32_t part[8];
  const int sub = threadIdx.x % TPR;
  const int r = blockIdx.x * (256 / TPR) + threadIdx.x / TPR;
  if (r >= rows) return;  // (all threads of the row)
  let_dependents_start();
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
    if ((i * TPR + sub) * 8 < K) amax = hold[i].amax(amax);
  }
  for (int k = (kVecs * TPR + sub) * 8; k < K; k += TPR * 8) {
    Int8Load<T, ALIGNED> more;
    more.load(x + k);
    amax = more.amax(amax);
  }
  amax = __reduce_max_sync(0xffffffffu, amax);
  if constexpr (TPR > 32) {
    const int first = threadIdx.x / TPR * (TPR / 32);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = amax;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + static_cast<int>(threadIdx.x) / TPR), "n"(TPR) : "memory");
#pragma unroll
    for (int w = 0; w < TPR / 32; ++w) amax = max(amax, part[first + w]);
  }
  const float s = int8_scale(amax, reciprocal), inv = 1.0f / s;
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

// The product of at most 16 rows: weight rows streamed once, as in few_tokens.cuh. The channels
// are divided evenly over the CTAs (one per SM). Four producer warps fill a ring of stages, 32
// weight rows and the activation rows x KC bytes of K, by 16-byte asynchronous copies. Eight
// product warps split K and run m16n8k32 integer MMAs: weight rows as A, eight tokens as B's
// columns; lane (g, t) reads 16 consecutive bytes of rows g and g + 8 and of token g, and K's order
// is that of these bytes in both operands. Past K the activations are zeros. The warps' sums are
// added through shared memory.
// FUSED (float rows, as many as eight warps can hold in registers): every CTA quantises the rows
// itself while its ring fills, one launch less and no round trip through memory.
// Bound by reading the weights, in so short a time by the ramp of DRAM: one row through 4096 x 8192
// weights in 10.3 us (3.3 TB/s), through 8192 x 8192 in 15.3 (4.4 TB/s); 7.7 us where 4096 x 8192
// lie in L2 from the call before. From 17
// rows on the split-K kernel is faster (64 rows: 10 us, against 27 here: every SM fetches all rows).
constexpr int kInt8StreamRows = 16;
constexpr int kInt8MaxStages = kFewMaxStages;  // (the ring's barriers are laid out for as many)
template <int NT, bool FUSED>
struct Int8Stream {
  static constexpr int R = 32;                        // weight rows of a stage
  static constexpr int KC = NT == 2 ? 512 : 1024;     // bytes of K of a stage
  static constexpr uint32_t kStride = KC + 64;        // see FewGeo on bank conflicts
  static constexpr uint32_t kXOff = R * kStride;
  static constexpr uint32_t stage_bytes(int T) { return (kXOff + (FUSED ? 0 : T) * kStride + 127) / 128 * 128; }
  static constexpr uint32_t kRedBytes = 8u * 16u * 33u * 4u;
  static constexpr int kThreads = 32 * 12;
  // fused: distance of the quantised rows
  __host__ __device__ static constexpr uint32_t xstride(int K) { return static_cast<uint32_t>((K + 127) / 128 * 128 + 64); }
};
// fused: warps that share a row, and the longest row they hold (8 x 8 values a thread)
__host__ __device__ constexpr int int8_row_warps(int T) { return T == 1 ? 8 : T == 2 ? 4 : T <= 4 ? 2 : 1; }
__host__ __device__ constexpr int int8_fused_depth(int T) { return 64 * 32 * int8_row_warps(T); }

struct Int8StreamArgs {
  const void* x;            // codes [T, K], or (fused) float rows ldx apart
  int64_t ldx;
  const float* x_scale;     // of the codes
  const int8_t* w;
  const float* w_scale;
  void* out;
  int64_t ldo;
  int T, K, N, stages;
  bool after_quantiser;     // (for the host: how it is launched)
  bool reciprocal;          // (fused) how the scales are made
  uint32_t* status;
};

__device__ __forceinline__ void mma_s8_16832(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 16 bytes, or zeros
__device__ __forceinline__ void cp_async16_or_zero(bool copy, uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(copy ? 16u : 0u) : "memory");
}

template <int NT, bool FUSED, typename TX, typename TOut>
__global__ void __launch_bounds__(Int8Stream<NT, FUSED>::kThreads, 1) k_int8_stream(const Int8StreamArgs p) {
  using S = Int8Stream<NT, FUSED>;
  extern __shared__ __align__(128) uint8_t smem[];  // partial sums, quantised rows (fused), the ring
  __shared__ __align__(8) uint64_t bars[2 * kInt8MaxStages];
  __shared__ uint32_t part[8];
  __shared__ float xs[8 * NT];
  __shared__ int abort_flag;
  volatile int* abort = &abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int T = p.T, K = p.K;
  const uint32_t xq = smem_u32(smem) + S::kRedBytes;
  FewRing ring{smem_u32(bars), xq + (FUSED ? (T * S::xstride(K) + 127) / 128 * 128 : 0u), p.stages, 0, 0u,
               S::stage_bytes(T)};
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(smem_u32(bars + i), 128);
      mbar_init(smem_u32(bars + kInt8MaxStages + i), 8);
    }
    abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  FewChunks c(p.N, p.N, S::R);

  if (warp < 4) {
    // ------------------------------------------------------------------------- producers
    constexpr int kPer = S::KC / 16, kStep = 128 / kPer;  // 16-byte pieces of a row; rows per pass
    const int row = threadIdx.x / kPer, o = threadIdx.x % kPer * 16;
    const int8_t* xc = static_cast<const int8_t*>(p.x) + static_cast<int64_t>(row) * (FUSED ? 0 : K) + o;
    const int64_t step = static_cast<int64_t>(kStep) * K;
    for (; !c.done(); c.next()) {
      const int8_t* wc = p.w + static_cast<int64_t>(c.f + row) * K + o;
#pragma unroll 1
      for (int k0 = 0; k0 < K; k0 += S::KC) {
        const bool ok = few_mbar_wait(ring.empty(), ring.phase ^ 1u, abort, p.status, 0xA10u + ring.stage);
        if (__all_sync(0xffffffffu, ok)) {
          const uint32_t st = ring.addr() + row * S::kStride + o;
          const int8_t* a = wc + k0;
          const bool in = k0 + o < K;
#pragma unroll
          for (int r = 0; r < S::R; r += kStep) {
            cp_async16_if(in && r + row < c.len, st + r * S::kStride, a);
            a += step;
          }
          if constexpr (!FUSED) {
            if (k0 == 0) wait_for_predecessor();
            // (a unit of K is 64 bytes: zeros up to its end)
            const int8_t* b = xc + k0;
            const bool fill = k0 + o < ((K + 63) & ~63);
#pragma unroll 4
            for (int r = 0; r < T; r += kStep) {
              if (fill && r + row < T) cp_async16_or_zero(in, st + S::kXOff + r * S::kStride, in ? b : xc);
              b += step;
            }
          }
        }
        cp_async_arrive(ring.full());
        ring.next();
      }
    }
    cp_async_wait_all();
    return;
  }

  // ------------------------------------------------------------------------- product warps
  const int wc = warp - 4, tid = threadIdx.x - 128;
  auto sync = [] { asm volatile("bar.sync 1, 256;" ::: "memory"); };
  if constexpr (FUSED) {
    const int per = int8_row_warps(T), j = wc / per, sub = (wc % per) * 32 + lane;
    const TX* x = static_cast<const TX*>(p.x) + static_cast<int64_t>(min(j, T - 1)) * p.ldx;
    Int8Load<TX, true> hold[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int k = (i * 32 * per + sub) * 8;
      if (k < K) hold[i].load(x + k);
    }
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if ((i * 32 * per + sub) * 8 < K) amax = hold[i].amax(amax);
    }
    amax = __reduce_max_sync(0xffffffffu, amax);
    if (lane == 0) part[wc] = amax;
    sync();
    for (int w = j * per; w < (j + 1) * per; ++w) amax = max(amax, part[w]);
    const float s = int8_scale(amax, p.reciprocal), inv = 1.0f / s;
    if (j < T) {
      if (sub == 0) xs[j] = s;
      uint8_t* q = smem + S::kRedBytes + j * S::xstride(K);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int k = (i * 32 * per + sub) * 8;
        if (k < K) {
          float v[8];
          hold[i].get(v);
          *reinterpret_cast<uint2*>(q + k) = int8_codes8(v, s, inv);
        }
      }
      if (sub < 8 && K + 8 * sub < ((K + 63) & ~63)) *reinterpret_cast<uint2*>(q + K + 8 * sub) = make_uint2(0u, 0u);
    }
  } else {
    wait_for_predecessor();
    for (int j = tid; j < T; j += 256) xs[j] = p.x_scale[j];
  }
  sync();
  const int g = lane >> 2, t = lane & 3;
  int* red = reinterpret_cast<int*>(smem);
  for (; !c.done(); c.next()) {
    int acc[2][NT][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][n][i] = 0;
#pragma unroll 1
    for (int k0 = 0; k0 < K; k0 += S::KC) {
      few_mbar_wait(ring.full(), ring.phase, abort, p.status, 0xC10u + ring.stage);
      __syncwarp();
      const uint32_t st = ring.addr();
      const uint32_t w = st + g * S::kStride + t * 16u;
      const uint32_t x = (FUSED ? xq + k0 : st + S::kXOff) + t * 16u;
      const uint32_t xstride = FUSED ? S::xstride(K) : S::kStride;
      const int units = (min(S::KC, K - k0) + 63) / 64;
#pragma unroll 2
      for (int u = wc; u < units; u += 8) {
        uint4 a[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = lds128(w + 8u * i * S::kStride + 64u * u);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          // (rows past the last token are not staged, their columns not used)
          const uint4 b = lds128(x + min(8 * n + g, T - 1) * xstride + 64u * u);
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            mma_s8_16832(acc[m][n], a[2 * m].x, a[2 * m + 1].x, a[2 * m].y, a[2 * m + 1].y, b.x, b.y);
            mma_s8_16832(acc[m][n], a[2 * m].z, a[2 * m + 1].z, a[2 * m].w, a[2 * m + 1].w, b.z, b.w);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(ring.empty());
      ring.next();
    }
    // red[warp][token][row]
    int* mine = red + wc * 16 * 33;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          mine[(8 * n + 2 * t + (i & 1)) * 33 + 16 * m + 8 * (i >> 1) + g] = acc[m][n][i];
    sync();
    for (int j = wc; j < T; j += 8) {
      uint32_t v = 0;
#pragma unroll
      for (int q = 0; q < 8; ++q) v += red[(q * 16 + j) * 33 + lane];
      if (lane < c.len)
        static_cast<TOut*>(p.out)[static_cast<int64_t>(j) * p.ldo + c.f + lane] =
            from_f32<TOut>(int8_sum(v) * (xs[j] * p.w_scale[c.f + lane]));
    }
    sync();
  }
}

}  // namespace muse
