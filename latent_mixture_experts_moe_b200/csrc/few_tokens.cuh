// few_tokens.cuh -- the whole latent-MoE layer for at most 8 tokens in one kernel.
//
// With a few tokens the layer is a chain of matrix-vector products whose weights are read
// once: W_router and W_pool, the selected experts' W_gate / W_up, their W_down, W_unpool.
// One cooperative launch (one CTA per SM, all resident) runs the chain in phases separated
// by grid barriers:
//   0  xn = rmsnorm(x)                                    (only with ffn_pre_gain)
//   1  l = W_router xn, z = W_pool xn
//   1b z = rmsnorm(z)                                     (only with pre_norm_gain)
//   2  every CTA: top-k of l, the list of distinct experts and their tokens
//      h = silu(W_gate[e] z) * (W_up[e] z)
//   3  y = W_down[e] h, per-CTA partial sums of squares of y (times its gain, input-scaled)
//   4  c = sum_j g_j y_j / rms_j (1 + gamma)
//   5  out = W_unpool c
//   6  post norm and residual gate                        (only with those)
// y and the sublayer's f stay FP32; z, h and c are stored in the type the next product
// reads (bf16; f16 for NVFP4 experts, whose decoded weights are f16; float32).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <type_traits>

#include "gemm_umma_fp4.cuh"
#include "gemv_fp4.cuh"
#include "ptx.cuh"
#include "route_kernels.cuh"

namespace muse {

constexpr int kFewTokens = 8;         // most tokens of one call
constexpr int kFewAssign = 8 * 32;    // most (token, expert) pairs: top_k <= 32
constexpr int kFewGridMax = 256;      // CTAs a workspace has partial sums for
constexpr int kFewThreads = 512;

struct FewArgs {
  int T, D, L, I, E, k;
  int router_mode, norm_mode, gamma_shared;
  float eps, logit_scale, rsf, pre_norm_eps, ffn_pre_eps, ffn_post_eps, inv_temp, gate_eps;
  const void *x, *W_router, *W_pool, *W_gate, *W_up, *W_down, *gamma, *W_unpool;  // dense weights, or NVFP4 codes
  const uint8_t *s_gate, *s_up, *s_down;     // NVFP4: block scales
  const float *m_gate, *m_up, *m_down;       // NVFP4: matrix scales
  const float* router_bias;
  const void *pre_norm_gain, *ffn_pre_gain, *ffn_post_gain;
  const float* residual_gate;
  void* out;
  int *idx_out;
  float *w_out;
  // workspace
  uint32_t *status, *barrier;
  float *logits, *y, *ss, *f, *ssf;
  void *xn, *z, *h, *c;
};

// Grid barrier number i (0, 1, ...) of one launch: every CTA adds one to the counter (zeroed
// before the launch) and waits until all have. All CTAs are resident (cooperative launch), so
// the wait ends; it is bounded all the same: past the limit the status word records a timeout
// and the CTA leaves. Returns the same value on every thread of the CTA.
__device__ __forceinline__ uint32_t ld_acquire_u32(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ bool few_wait_counter(const uint32_t* counter, uint32_t target, uint32_t* status,
                                                 uint32_t detail) {
  if (ld_acquire_u32(counter) >= target) return true;
  const uint64_t t0 = globaltimer_ns();
  while (ld_acquire_u32(counter) < target) {
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      record_status(status, kStatusTimeout, detail);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool few_grid_barrier(uint32_t* counter, int i, uint32_t* status, int* flag) {
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    atomicAdd(counter, 1u);
    *flag = few_wait_counter(counter, static_cast<uint32_t>(i + 1) * gridDim.x, status, 0xF00u + i) ? 1 : 0;
    __threadfence();
  }
  __syncthreads();
  return *flag != 0;
}

// ---------------------------------------------------------------------- routing
// A float as an unsigned number of the same order (NaN and -inf lowest; -0 as +0).
__device__ __forceinline__ uint32_t order_key(float v) {
  v = (v == v) ? v + 0.0f : neg_inf();
  const uint32_t b = __float_as_uint(v);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// The k largest keys of a token by one warp, in descending order, ties to the lower expert:
// lane j < k receives the j-th. NPL keys per lane (E <= 32 NPL). Each round is one warp-wide
// maximum and one minimum over the lanes that hold it; only the lane that owned the winner
// looks for its next best.
template <int NPL>
__device__ __forceinline__ int few_topk(const float* l, const float* bias, int mode, float scale, int E, int k,
                                        int lane) {
  uint32_t key[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int e = lane + 32 * i;
    key[i] = 0;  // below every real key (-inf has 0x007fffff)
    if (e < E) {
      const float li = __ldcg(l + e);
      float kv = (mode == 0) ? li : 1.0f / (1.0f + expf(-scale * li));
      if (bias != nullptr) kv += bias[e];
      key[i] = order_key(kv);
    }
  }
  uint32_t best = 0;
  int bi = 0;
  auto rescan = [&]() {
    best = 0;
    bi = 0;
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (key[i] > best) {
        best = key[i];
        bi = i;
      }
  };
  rescan();
  int mine = 0;
  for (int j = 0; j < k; ++j) {
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    const uint32_t e = __reduce_min_sync(0xffffffffu, best == top ? static_cast<uint32_t>(lane + 32 * bi) : 0xffffffffu);
    if (best == top && static_cast<uint32_t>(lane + 32 * bi) == e) {
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (i == bi) key[i] = 0;
      rescan();
    }
    if (lane == j) mine = static_cast<int>(e);
  }
  return mine;
}

// What every CTA knows about the routing, in its shared memory. Position p numbers the T * k
// (token, slot) pairs by expert, then by pair; the pairs of distinct expert d are the
// positions first[d] .. first[d + 1] - 1.
struct FewRoute {
  int expert[kFewAssign];      // [t * k + j]
  float weight[kFewAssign];
  int pos[kFewAssign];         // pair -> position
  int pair[kFewAssign];        // position -> pair
  int rank[kFewAssign];        // pair -> number of its expert among the distinct ones
  int ids[kFewAssign];         // distinct expert -> expert
  int first[kFewAssign + 1];
  int distinct;
};

__device__ __forceinline__ void few_route(const FewArgs& p, FewRoute& r, int warp, int nwarps, int lane) {
  for (int t = warp; t < p.T; t += nwarps) {
    const float* l = p.logits + static_cast<int64_t>(t) * p.E;
    int sel;
    if (p.E <= 64) sel = few_topk<2>(l, p.router_bias, p.router_mode, p.logit_scale, p.E, p.k, lane);
    else if (p.E <= 256) sel = few_topk<8>(l, p.router_bias, p.router_mode, p.logit_scale, p.E, p.k, lane);
    else sel = few_topk<32>(l, p.router_bias, p.router_mode, p.logit_scale, p.E, p.k, lane);
    const bool mine = lane < p.k;
    const float lj = mine ? __ldcg(l + sel) : 0.0f;
    float g;
    if (p.router_mode == 0) {
      const float m = warp_max(mine ? lj : neg_inf());
      const float pj = mine ? expf(lj - m) : 0.0f;
      g = pj / warp_sum(pj);
    } else {
      const float sj = mine ? 1.0f / (1.0f + expf(-p.logit_scale * lj)) : 0.0f;
      g = p.rsf * sj / (warp_sum(sj) + 1e-15f);
    }
    if (mine) {
      const int a = t * p.k + lane;
      r.expert[a] = sel;
      r.weight[a] = g;
      if (blockIdx.x == 0) {
        if (p.idx_out != nullptr) p.idx_out[a] = sel;
        if (p.w_out != nullptr) p.w_out[a] = g;
      }
    }
  }
}

// positions, distinct experts: every thread of a group of nthreads calls it with a barrier
// over the group between the two steps (sync)
template <typename Sync>
__device__ __forceinline__ void few_lists(const FewArgs& p, FewRoute& r, int tid, int nthreads, Sync sync) {
  const int A = p.T * p.k;
  for (int a = tid; a < A; a += nthreads) {
    const int e = r.expert[a];
    int pos = 0, same = 0;
    for (int b = 0; b < A; ++b) {
      const int eb = r.expert[b];
      pos += (eb < e) || (eb == e && b < a);
      same += (eb == e && b < a);
    }
    r.pos[a] = pos;
    r.pair[pos] = a;
    r.rank[a] = same;  // 0: the first pair of its expert
  }
  sync();
  for (int a = tid; a < A; a += nthreads) {
    if (r.rank[a] != 0) continue;
    const int e = r.expert[a];
    int d = 0;
    for (int b = 0; b < A; ++b) d += (r.rank[b] == 0 && r.expert[b] < e);
    r.ids[d] = e;
    r.first[d] = r.pos[a];
  }
  if (tid == 0) {
    int n = 0;
    for (int b = 0; b < A; ++b) n += (r.rank[b] == 0);
    r.distinct = n;
    r.first[n] = A;
  }
  sync();
}

// ---------------------------------------------------------------------- products
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
// (saturating: a latent beyond f16's range does not become an infinity, as in the gather of
// the token-tiled forward)
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return f32_to_f16_sat(v); }

// One weight row against n <= 8 activation rows by a warp: lanes stride over K, eight
// elements at a time, FP32 sums, a butterfly at the end (every lane gets the sums).
template <typename TW, typename TX>
__device__ __forceinline__ void few_row_dot(const TW* w, const TX* const* x, int n, int K, int lane, float (&acc)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
  for (int k0 = lane * 8; k0 < K; k0 += 256) {
    float wv[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) wv[i] = to_f32(w[k0 + i]);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[j] = fmaf(wv[i], to_f32(x[j][k0 + i]), acc[j]);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = warp_sum(acc[j]);
}

// The same for an NVFP4 row: codes [K / 2] and block scales [K / 16] (matrix scale left out).
__device__ __forceinline__ void few_row_dot_fp4(const uint8_t* codes, const uint8_t* scales, const __half* const* x,
                                                int n, int K, int lane, float (&acc)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
  for (int k0 = lane * 8; k0 < K; k0 += 256) {
    uint32_t q[4];
    e2m1x8_to_f16x2(*reinterpret_cast<const uint32_t*>(codes + k0 / 2), q[0], q[1], q[2], q[3]);
    const uint32_t s = e4m3_bcast_f16x2(scales[k0 / 16], 0);
    float wv[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t v = f16x2_mul(q[i], s);
      const __half2 h = *reinterpret_cast<const __half2*>(&v);
      wv[2 * i] = __low2float(h);
      wv[2 * i + 1] = __high2float(h);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[j] = fmaf(wv[i], __half2float(x[j][k0 + i]), acc[j]);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = warp_sum(acc[j]);
}

// Centred RMSNorm of one row by the whole CTA: dst = src / sqrt(mean(src^2) + eps) * (1 + w).
template <typename TS, typename TG, typename TD>
__device__ __forceinline__ void few_norm_row(const TS* src, const TG* w, TD* dst, int n, float eps, float* part) {
  float s = 0.0f;
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const float v = to_f32(src[i]);
    s = fmaf(v, v, s);
  }
  const float scale = 1.0f / sqrtf(block_sum(s, part) / static_cast<float>(n) + eps);
  for (int i = threadIdx.x; i < n; i += blockDim.x) dst[i] = from_f32<TD>(to_f32(src[i]) * scale * (1.0f + to_f32(w[i])));
}

__device__ __forceinline__ float few_silu(float a) { return a / (1.0f + expf(-a)); }

// TA: activations, dense weights, gains and the output (bf16 or float). FP4: NVFP4 experts
// (TA = bf16; z and h are f16).
template <typename TA, bool FP4>
__global__ void __launch_bounds__(kFewThreads, 1) k_few_tokens(const FewArgs p) {
  using TZ = typename std::conditional<FP4, __half, TA>::type;
  __shared__ FewRoute route;
  __shared__ float part[32];
  __shared__ int flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  const int gw = blockIdx.x * nw + warp, ngw = gridDim.x * nw;
  const int T = p.T, D = p.D, L = p.L, I = p.I, E = p.E, k = p.k;
  int bar = 0;
  const TA* xin = static_cast<const TA*>(p.x);
  if (p.ffn_pre_gain != nullptr) {
    TA* xn = static_cast<TA*>(p.xn);
    for (int t = blockIdx.x; t < T; t += gridDim.x)
      few_norm_row(xin + static_cast<int64_t>(t) * D, static_cast<const TA*>(p.ffn_pre_gain),
                   xn + static_cast<int64_t>(t) * D, D, p.ffn_pre_eps, part);
    xin = xn;
    if (!few_grid_barrier(p.barrier, bar++, p.status, &flag)) return;
  }
  // phase 1
  {
    const TA* xr[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) xr[j] = xin + static_cast<int64_t>(j < T ? j : 0) * D;
    for (int r = gw; r < E + L; r += ngw) {
      const TA* w = r < E ? static_cast<const TA*>(p.W_router) + static_cast<int64_t>(r) * D
                          : static_cast<const TA*>(p.W_pool) + static_cast<int64_t>(r - E) * D;
      float acc[8];
      few_row_dot(w, xr, T, D, lane, acc);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < T && lane == j) {
          if (r < E) p.logits[static_cast<int64_t>(j) * E + r] = acc[j];
          else static_cast<TZ*>(p.z)[static_cast<int64_t>(j) * L + r - E] = from_f32<TZ>(acc[j]);
        }
    }
  }
  if (!few_grid_barrier(p.barrier, bar++, p.status, &flag)) return;
  if (p.pre_norm_gain != nullptr) {
    TZ* z = static_cast<TZ*>(p.z);
    for (int t = blockIdx.x; t < T; t += gridDim.x)
      few_norm_row(z + static_cast<int64_t>(t) * L, static_cast<const TA*>(p.pre_norm_gain),
                   z + static_cast<int64_t>(t) * L, L, p.pre_norm_eps, part);
    if (!few_grid_barrier(p.barrier, bar++, p.status, &flag)) return;
  }
  few_route(p, route, warp, nw, lane);
  __syncthreads();
  few_lists(p, route, threadIdx.x, blockDim.x, [] { __syncthreads(); });
  const int nd = route.distinct;
  // phase 2
  {
    const TZ* z = static_cast<const TZ*>(p.z);
    for (int r = gw; r < nd * I; r += ngw) {
      const int d = r / I, f = r - d * I, e = route.ids[d];
      const int64_t row = static_cast<int64_t>(e) * I + f;
      for (int p0 = route.first[d]; p0 < route.first[d + 1]; p0 += 8) {
        const int n = min(8, route.first[d + 1] - p0);
        const TZ* xr[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) xr[j] = z + static_cast<int64_t>(route.pair[p0 + (j < n ? j : 0)] / k) * L;
        float g[8], u[8];
        float mg = 1.0f, mu = 1.0f;
        if constexpr (FP4) {
          few_row_dot_fp4(static_cast<const uint8_t*>(p.W_gate) + row * (L / 2), p.s_gate + row * (L / 16), xr, n, L, lane, g);
          few_row_dot_fp4(static_cast<const uint8_t*>(p.W_up) + row * (L / 2), p.s_up + row * (L / 16), xr, n, L, lane, u);
          mg = p.m_gate[e];
          mu = p.m_up[e];
        } else {
          few_row_dot(static_cast<const TA*>(p.W_gate) + row * L, xr, n, L, lane, g);
          few_row_dot(static_cast<const TA*>(p.W_up) + row * L, xr, n, L, lane, u);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < n && lane == j)
            static_cast<TZ*>(p.h)[static_cast<int64_t>(p0 + j) * I + f] = from_f32<TZ>(few_silu(g[j] * mg) * (u[j] * mu));
      }
    }
  }
  if (!few_grid_barrier(p.barrier, bar++, p.status, &flag)) return;
  // phase 3
  {
    const TZ* h = static_cast<const TZ*>(p.h);
    for (int r = gw; r < nd * L; r += ngw) {
      const int d = r / L, f = r - d * L, e = route.ids[d];
      const int64_t row = static_cast<int64_t>(e) * L + f;
      for (int p0 = route.first[d]; p0 < route.first[d + 1]; p0 += 8) {
        const int n = min(8, route.first[d + 1] - p0);
        const TZ* xr[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) xr[j] = h + static_cast<int64_t>(p0 + (j < n ? j : 0)) * I;
        float y[8];
        float ms = 1.0f;
        if constexpr (FP4) {
          few_row_dot_fp4(static_cast<const uint8_t*>(p.W_down) + row * (I / 2), p.s_down + row * (I / 16), xr, n, I, lane, y);
          ms = p.m_down[e];
        } else {
          few_row_dot(static_cast<const TA*>(p.W_down) + row * I, xr, n, I, lane, y);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < n && lane == j) p.y[static_cast<int64_t>(p0 + j) * L + f] = y[j] * ms;
      }
    }
  }
  if (!few_grid_barrier(p.barrier, bar++, p.status, &flag)) return;
  // phase 4: token by token; every position's mean square by one warp
  {
    TA* c = static_cast<TA*>(p.c);
    const TA* gamma = static_cast<const TA*>(p.gamma);
    __shared__ float scale_s[32];
    for (int t = blockIdx.x; t < T; t += gridDim.x) {
      for (int j = warp; j < k; j += nw) {
        const int a = t * k + j;
        const float* y = p.y + static_cast<int64_t>(route.pos[a]) * L;
        const TA* gm = gamma + (p.gamma_shared ? 0 : static_cast<int64_t>(route.expert[a]) * L);
        float s = 0.0f;
        for (int i = lane; i < L; i += 32) {
          const float u = __ldcg(y + i) * (p.norm_mode == 1 ? 1.0f + to_f32(gm[i]) : 1.0f);
          s = fmaf(u, u, s);
        }
        s = warp_sum(s);
        if (lane == 0) scale_s[j] = route.weight[a] / sqrtf(s / static_cast<float>(L) + p.eps);
      }
      __syncthreads();
      for (int i = threadIdx.x; i < L; i += blockDim.x) {
        float acc = 0.0f;
        for (int j = 0; j < k; ++j) {
          const int a = t * k + j;
          const float gm = to_f32(gamma[(p.gamma_shared ? 0 : static_cast<int64_t>(route.expert[a]) * L) + i]);
          acc = fmaf(scale_s[j] * (1.0f + gm), __ldcg(p.y + static_cast<int64_t>(route.pos[a]) * L + i), acc);
        }
        c[static_cast<int64_t>(t) * L + i] = from_f32<TA>(acc);
      }
      __syncthreads();
    }
  }
  if (!few_grid_barrier(p.barrier, bar++, p.status, &flag)) return;
  // phase 5
  const bool finish = p.ffn_post_gain != nullptr || p.residual_gate != nullptr;
  {
    const TA* xr[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) xr[j] = static_cast<const TA*>(p.c) + static_cast<int64_t>(j < T ? j : 0) * L;
    for (int r = gw; r < D; r += ngw) {
      float acc[8];
      few_row_dot(static_cast<const TA*>(p.W_unpool) + static_cast<int64_t>(r) * L, xr, T, L, lane, acc);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < T && lane == j) {
          if (finish) p.f[static_cast<int64_t>(j) * D + r] = acc[j];
          else static_cast<TA*>(p.out)[static_cast<int64_t>(j) * D + r] = from_f32<TA>(acc[j]);
        }
    }
  }
  if (!finish) return;
  if (!few_grid_barrier(p.barrier, bar++, p.status, &flag)) return;
  // phase 6
  for (int t = blockIdx.x; t < T; t += gridDim.x) {
    const float* f = p.f + static_cast<int64_t>(t) * D;
    const TA* w = static_cast<const TA*>(p.ffn_post_gain);
    float scale = 1.0f;
    if (w != nullptr) {
      float s = 0.0f;
      for (int i = threadIdx.x; i < D; i += blockDim.x) {
        const float v = __ldcg(f + i) * (1.0f + to_f32(w[i]));
        s = fmaf(v, v, s);
      }
      scale = 1.0f / sqrtf(block_sum(s, part) / static_cast<float>(D) + p.ffn_post_eps);
    }
    for (int i = threadIdx.x; i < D; i += blockDim.x) {
      float v = __ldcg(f + i);
      if (w != nullptr) v *= (1.0f + to_f32(w[i])) * scale;
      if (p.residual_gate != nullptr) {
        const float wg = p.residual_gate[i] * p.inv_temp;
        const float beta = 1.0f / (1.0f + expf(-wg));
        const float alpha = sqrtf(fmaxf((1.0f / (1.0f + expf(wg))) * (1.0f + beta), p.gate_eps));
        v = alpha * to_f32(static_cast<const TA*>(p.x)[static_cast<int64_t>(t) * D + i]) + beta * v;
      }
      static_cast<TA*>(p.out)[static_cast<int64_t>(t) * D + i] = from_f32<TA>(v);
    }
  }
}

}  // namespace muse
