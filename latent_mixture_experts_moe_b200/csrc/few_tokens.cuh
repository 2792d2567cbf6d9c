// few_tokens.cuh -- the whole latent-MoE layer for at most 8 tokens in one kernel.
//
// With a few tokens the layer is a chain of matrix-vector products whose weights are read
// once: W_router and W_pool, the selected experts' W_gate / W_up, their W_down, W_unpool. It
// is bound by reading them, and by the latency of the steps between. One cooperative launch
// (one CTA per SM, all resident) runs the chain in phases separated by grid barriers:
//   0  xn = rmsnorm(x)                                    (only with ffn_pre_gain)
//   1  l = W_router xn; then z = W_pool xn, while every CTA finds the top-k of l and lists the
//      distinct experts and their tokens; z = rmsnorm(z) (only with pre_norm_gain)
//   2  h = silu(W_gate[e] z) * (W_up[e] z)
//   3  y = W_down[e] h, per-CTA partial sums of squares of y (times its gain, input-scaled)
//   4  c = sum_j g_j y_j / rms_j (1 + gamma)
//   5  out = W_unpool c
//   6  post norm and residual gate                        (only with those)
// y, the sublayer's f and a latent that a norm follows stay FP32 (raw, it may lie outside f16's
// range, from which the norm brings it back); z, h and c are stored in the type the next product
// reads (bf16; f16 for NVFP4 experts, whose decoded weights are f16; float32). bf16 products of
// intermediates carry a token as two bf16 numbers, the rounded value and what rounding took off
// (16 significant bits): up to four tokens in the MMA's eight columns, which would otherwise be
// empty, more in a second MMA. The output's error is then its own rounding (1.7e-3 of its norm
// instead of 3.7e-3; released norms 4.5e-3). The sublayer's xn is one bf16 number, as in the
// token-tiled forward. An infinite weight gives NaN where the second number is 0 or of the other
// sign.
//
// Work split: the weight rows of a phase (of all distinct experts in a row) are divided evenly
// over the CTAs by row, whatever the tile, so no SM waits for another's larger share; a row is
// always summed whole, by the same warps in the same order, so its sum does not depend on
// the split. (The norms' sums of squares of y and f are one partial per CTA, added in CTA order: their
// last bits follow the number of CTAs.)
//
// Roles (16 warps). Producers (4): three stream a CTA's weight rows through a ring of stages, up
// to 32 rows x kc elements each, by 16-byte asynchronous copies (any row count and row start;
// the row distance in shared memory is padded so that the fragment reads below are free of
// bank conflicts); the fourth adds the n <= 8 activation rows of the same K range. At a phase's
// start the ring fills with the new phase's weights while the grid barrier is still pending
// -- only the activations wait for it -- so DRAM stays busy through the barriers. (One bulk
// copy per row piece, from one producer warp, instead: one token through the full-size bf16
// layer in 331 us, against 171 with these copies. This and the other comparisons in this file
// are of two builds measured side by side, at the step where the choice was made.)
// Products (8; with 16, NVFP4 120 us against 97): they split each stage along K. 16-bit weights go to the warp-level MMA (m16n8k16:
// weight rows as A, the tokens as its 8 columns): lane (g, t) of a warp reads 16 consecutive
// bytes of rows g and g + 8 and of token g, and the MMA's K order is that of these bytes in both
// operands. NVFP4 rows are decoded in registers into the A fragment (gemv_fp4.cuh). float32 rows
// are multiplied in FP32, a lane per row, the activations broadcast. The warps' partial sums of a
// chunk of rows go to one of two buffers.
// Store (4): they add the partial sums in a fixed order, apply what follows the product and
// write the result, while the product warps go on with the next chunk. The router's rows come
// first, so that the store warps select the experts while the pooler's rows stream.
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
constexpr int kFewGridMax = 192;      // CTAs a workspace has partial sums for
constexpr int kFewProducers = 4;      // producer warps: one for activations, the others for weights
constexpr int kFewStore = 4;          // store warps
constexpr int kFewPer = 8 / kFewStore;  // tokens of each
constexpr int kFewWarps = 8;          // product warps
constexpr int kFewThreads = 32 * (kFewProducers + kFewStore + kFewWarps);
constexpr int kFewRows = 32;          // weight rows of a stage (gate/up: 16 features of each)
// More stages than 4 only lengthen the memory system's queues, and with them every barrier's
// round trips (one token, full-size bf16 layer: 165 us with 3 or 5 stages, 159 with 4).
constexpr int kFewMaxStages = 4;
constexpr int kFewBarriers = 8;       // grid barriers of a call, their counters 128 bytes apart
constexpr uint32_t kFewRedFloats = kFewWarps * 8u * 33u;      // partial sums of a chunk
constexpr uint32_t kFewRedBytes = 2u * kFewRedFloats * 4u;    // two chunks'

enum FewFormat : int { FEW_BF16 = 0, FEW_NVFP4 = 1, FEW_F32 = 2, FEW_BF16_SHORT = 3 };

// How the stages of a product with weights of a format lie in shared memory: at most kc elements
// of K per stage, so that every product warp has a share of each (its unit: 32 bf16 elements,
// 128 NVFP4, 4 float32); weight rows wstride bytes apart from offset 0, NVFP4 block scales
// sstride apart from soff, activation rows xstride apart from xoff.
// 2048 elements of NVFP4 rows are as many bytes as 512 of bf16, but each activation row would
// take 4 KB of every stage, most of a stage's time with several tokens on an expert: where they
// fit (FewArgs::x_bytes), an expert's activation rows lie whole in a buffer of their own, copied
// once for all of a CTA's rows of that expert (16 experts with four tokens each: 158 us, 390 without);
// otherwise its stages hold less of K (depth).
// FEW_BF16_SHORT: the dense products beside NVFP4 experts, whose ring is shorter by that buffer.
// The row distances keep the product warps' reads free of bank conflicts: bf16 rows 64 bytes
// past a multiple of 128 (a quarter warp reads 64 bytes of two rows), and codes too, float rows
// 16 past it (eight lanes read one row each), scales an odd multiple of 16; f16 activations
// beside codes, of which a lane reads 64 bytes in four steps, have 16 spare bytes after every
// 128 and rows 32 (or 96) past a multiple of 128.
template <int FORMAT>
struct FewGeo {
  static constexpr int kc = FORMAT == FEW_NVFP4 ? 2048 : FORMAT == FEW_BF16 ? 512 : FORMAT == FEW_BF16_SHORT ? 384 : 256;
  static constexpr int act_size = FORMAT == FEW_F32 ? 4 : 2;
  static constexpr uint32_t row_bytes = FORMAT == FEW_NVFP4 ? kc / 2 : kc * act_size;
  static constexpr uint32_t wstride = row_bytes + (FORMAT == FEW_F32 ? 16 : 64);
  static constexpr uint32_t soff = kFewRows * wstride;
  static constexpr uint32_t sstride = FORMAT == FEW_NVFP4 ? (kc / 16) | 16 : 0;
  static constexpr uint32_t xoff = soff + kFewRows * sstride;
  // elements of K per stage with n tokens; whole: the activations have their own buffer
  __host__ __device__ static constexpr int depth(int n, bool whole) {
    return FORMAT != FEW_NVFP4 || whole || n <= 2 ? kc : n <= 4 ? kc / 2 : kc / 4;
  }
  // distance of activation rows that hold k elements
  __host__ __device__ static constexpr uint32_t xstride(int k) {
    return static_cast<uint32_t>(FORMAT == FEW_NVFP4 ? k / 8 * 9 * act_size + 32
                                                     : k * act_size + (FORMAT == FEW_F32 ? 16 : 64));
  }
  // where byte a of an activation row lies
  __device__ static constexpr uint32_t xbyte(uint32_t a) { return FORMAT == FEW_NVFP4 ? a + a / 128 * 16 : a; }
  // bytes of a stage that holds up to T activation rows
  static constexpr uint32_t bytes(int T, bool whole) {
    uint32_t x = 0;
    for (int n = 1; n <= T && !(FORMAT == FEW_NVFP4 && whole); ++n)
      x = n * xstride(depth(n, false)) > x ? n * xstride(depth(n, false)) : x;
    return xoff + x;
  }
};
// Most that an expert's activation rows may take: 8 rows of 4096, what the ring can spare. With wider
// latents or hidden rows and as many tokens they go through the stages, which then hold a quarter of
// K: 29 experts of 4352 x 4352, eight tokens, 498 us (1.9 TB/s); of 4096 x 4096 233 (3.7 TB/s).
constexpr uint32_t kFewXBytes = 74 * 1024;
// The router's rows are few for a CTA (256 over 148): with at most kFewNarrow of them a stage
// holds 2 or 4 times as much of K (FewArgs::narrow), or the ring would hold next to nothing (the
// logits of the full-size layer were ready after 8.5 us, with DRAM idle, against 3).
constexpr int kFewNarrow = 4;


// whether a phase's activations are staged as two bf16 numbers each
__host__ __device__ constexpr bool few_split(int format, int phase) {
  return (format == FEW_BF16 || format == FEW_BF16_SHORT) && phase >= 2;
}
// most activation rows of a stage in a call of T tokens
__host__ __device__ constexpr int few_columns(int format, int T) { return few_split(format, 2) ? 2 * T : T; }

struct FewArgs {
  int stages;             // ring depth
  uint32_t stage_bytes;
  uint32_t x_bytes;       // NVFP4 experts: buffer of an expert's activation rows (0: in the stages)
  int narrow;             // the router's stages hold this many times as much of K (0: they are as the others)
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
  float* zraw;            // the latent before its norm (with pre_norm_gain)
  void *xn, *z, *h, *c;
};

// Grid barriers: every CTA adds one to the barrier's counter (zeroed before the launch) when
// its part is done, and waits, when it needs the others', until all have. All CTAs are resident
// (cooperative launch), so the wait ends; it is bounded all the same. Once a wait of a CTA has
// run out, *abort is set, the status word holds the timeout, and the CTA goes through the rest
// of the call without waiting or copying, so that every thread leaves.
__device__ __forceinline__ uint32_t ld_acquire_u32(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void red_release_u32(uint32_t* p, uint32_t v) {
  asm volatile("red.release.gpu.global.add.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
// mbar_wait with the wait left to the hardware (up to 20 us at a time): a warp that polls takes
// issue slots and shared-memory cycles from the warps that work.
__device__ __forceinline__ bool few_mbar_wait(uint32_t bar, uint32_t parity, volatile int* abort, uint32_t* status,
                                              uint32_t detail) {
  auto test = [&]() -> bool {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(20000u)
        : "memory");
    return ok != 0;
  };
  if (test()) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!test()) {
    if (*abort) return false;
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      *abort = 1;
      record_status(status, kStatusTimeout, detail);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ void few_poll(const uint32_t* counter, uint32_t target, volatile int* abort,
                                         uint32_t* status, uint32_t detail) {
  if (ld_acquire_u32(counter) >= target) return;
  const uint64_t t0 = globaltimer_ns();
  while (ld_acquire_u32(counter) < target) {
    if (*abort) return;
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      *abort = 1;
      record_status(status, kStatusTimeout, detail);
      return;
    }
  }
}

// ---------------------------------------------------------------------- routing
// A float as an unsigned number of the same order (NaN and -inf lowest; -0 as +0).
__device__ __forceinline__ uint32_t order_key(float v) {
  v = (v == v) ? v + 0.0f : neg_inf();
  const uint32_t b = __float_as_uint(v);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// The k largest keys of a token by one warp, in descending order, ties to the lower expert:
// lane j < k receives the j-th and its logit. NPL keys per lane (E <= 32 NPL). Each round is
// one warp-wide maximum and one minimum over the lanes that hold it; only the lane that owned
// the winner looks for its next best.
template <int NPL>
__device__ __forceinline__ int few_topk(const float* l, const float* bias, int mode, float scale, int E, int k,
                                        int lane, float& logit) {
  constexpr bool kKeep = NPL <= 8;  // the logits stay in registers (more would spill)
  uint32_t key[NPL];
  float val[kKeep ? NPL : 1];
  if constexpr (kKeep) {
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int e = lane + 32 * i;
      val[i] = e < E ? __ldcg(l + e) : 0.0f;
    }
  }
  uint32_t best = 0;
  int bi = 0;
  float bv = 0.0f;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int e = lane + 32 * i;
    key[i] = 0;  // below every real key (-inf has 0x007fffff)
    if (e < E) {
      const float li = kKeep ? val[kKeep ? i : 0] : __ldcg(l + e);
      float kv = (mode == 0) ? li : 1.0f / (1.0f + expf(-scale * li));
      if (bias != nullptr) kv += bias[e];
      key[i] = order_key(kv);
    }
  }
  auto rescan = [&]() {
    best = 0;
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (key[i] > best) {
        best = key[i];
        bi = i;
        if (kKeep) bv = val[kKeep ? i : 0];
      }
  };
  rescan();
  int mine = 0;
#pragma unroll 1
  for (int j = 0; j < k; ++j) {
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    const uint32_t e = __reduce_min_sync(0xffffffffu, best == top ? static_cast<uint32_t>(lane + 32 * bi) : 0xffffffffu);
    const float v = __shfl_sync(0xffffffffu, bv, static_cast<int>(e & 31));
    if (lane == j) {
      mine = static_cast<int>(e);
      logit = v;
    }
    if (lane == static_cast<int>(e & 31)) {
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (i == bi) key[i] = 0;
      rescan();
    }
  }
  if (!kKeep && lane < k) logit = __ldcg(l + mine);
  return mine;
}

// What every CTA knows about the routing, in its shared memory. Position p numbers the T * k
// (token, slot) pairs by expert, then by pair; the pairs of distinct expert d are the
// positions first[d] .. first[d + 1] - 1.
struct FewRoute {
  __align__(16) int expert[kFewAssign];  // [t * k + j]; past the last pair: INT_MAX
  float weight[kFewAssign];
  int pos[kFewAssign];                   // pair -> position
  int token[kFewAssign];                 // position -> token
  int distinct_of[kFewAssign];           // pair -> number of its expert among the distinct ones
  int ids[kFewAssign];                   // distinct expert -> expert
  int first[kFewAssign + 1];
  uint32_t seen[32];                     // bit e % 32 of word e / 32: expert e is selected
  int distinct;
};

// Token t's experts and weights, by one warp.
__device__ __forceinline__ void few_route(const FewArgs& p, FewRoute& r, int t, int lane) {
  const float* l = p.logits + static_cast<int64_t>(t) * p.E;
  int sel;
  float lj = 0.0f;
  if (p.E <= 64) sel = few_topk<2>(l, p.router_bias, p.router_mode, p.logit_scale, p.E, p.k, lane, lj);
  else if (p.E <= 256) sel = few_topk<8>(l, p.router_bias, p.router_mode, p.logit_scale, p.E, p.k, lane, lj);
  else sel = few_topk<32>(l, p.router_bias, p.router_mode, p.logit_scale, p.E, p.k, lane, lj);
  const bool mine = lane < p.k;
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
    atomicOr(&r.seen[sel >> 5], 1u << (sel & 31));
    if (blockIdx.x == 0) {
      if (p.idx_out != nullptr) p.idx_out[a] = sel;
      if (p.w_out != nullptr) p.w_out[a] = g;
    }
  }
}

// Positions and distinct experts, from expert[] and seen[], by a group of nthreads (all of
// whose warps call it; a barrier over the group before and after).
__device__ __forceinline__ void few_lists(const FewArgs& p, FewRoute& r, int tid, int nthreads) {
  const int A = p.T * p.k, lane = tid & 31;
  // distinct experts below word `lane` of seen
  const uint32_t word = r.seen[lane];
  int below = __popc(word);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, below, o);
    if (lane >= o) below += u;
  }
  if (tid == 31) {
    r.distinct = below;
    r.first[below] = A;
  }
  below -= __popc(word);
  for (int a0 = tid & ~31; a0 < A; a0 += nthreads) {
    const int a = a0 + lane;
    const int e = r.expert[a];
    int less = 0, same = 0;
#pragma unroll 2
    for (int b = 0; b < A; b += 4) {
      const int4 v = *reinterpret_cast<const int4*>(&r.expert[b]);
      less += (v.x < e) + (v.y < e) + (v.z < e) + (v.w < e);
      same += (v.x == e && b < a) + (v.y == e && b + 1 < a) + (v.z == e && b + 2 < a) + (v.w == e && b + 3 < a);
    }
    const int es = min(e, 1023);
    const int d = __shfl_sync(0xffffffffu, below, es >> 5) + __popc(__shfl_sync(0xffffffffu, word, es >> 5) & ((1u << (es & 31)) - 1u));
    if (a < A) {
      r.pos[a] = less + same;
      r.token[less + same] = a / p.k;
      r.distinct_of[a] = d;
      if (same == 0) {
        r.ids[d] = e;
        r.first[d] = less;
      }
    }
  }
}

// ---------------------------------------------------------------------- the row streams
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
// (saturating: a latent beyond f16's range does not become an infinity, as in the gather of
// the token-tiled forward)
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return f32_to_f16_sat(v); }

__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

enum FewPhase : int { FEW_ROUTER = 0, FEW_POOL = 1, FEW_GATE_UP = 2, FEW_DOWN = 3, FEW_OUT = 4 };

// A CTA's rows of a phase in order: units [u, u1) of U (unit: a weight row; gate/up: a feature),
// `group` units per expert (dense: all of them), cut into chunks of at most `most` units of one
// expert, the chunks of an expert's share as equal as possible. CTA c's share starts at
// floor(U c / G).
__device__ __forceinline__ int few_share(int U, int c) {
  const int G = static_cast<int>(gridDim.x), q = U / G;
  return q * c + (U - q * G) * c / G;
}
// the CTA whose share of U units holds unit u (U <= 2^24)
__device__ __forceinline__ int few_owner(int U, int u) {
  return static_cast<int>(((static_cast<uint32_t>(u) + 1u) * gridDim.x - 1u) / static_cast<uint32_t>(U));
}
struct FewChunks {
  int left, group, most;   // units left in the share; units per expert, per chunk
  int d, f, len;           // current chunk: expert number, first unit within it, units
  int base, extra;         // chunks of the current expert's share: `extra` of base + 1, then of base
  __device__ __forceinline__ FewChunks(int U, int group_, int most_) : group(group_), most(most_) {
    const int u0 = few_share(U, blockIdx.x);
    left = few_share(U, blockIdx.x + 1) - u0;
    d = u0 / group;
    f = u0 - d * group;
    begin();
  }
  __device__ __forceinline__ bool done() const { return left <= 0; }
  __device__ __forceinline__ void begin() {
    const int here = min(left, group - f);
    const int n = (here + most - 1) / most;
    base = n > 1 ? here / n : here;
    extra = here - n * base;
    len = base + (extra > 0 ? 1 : 0);
  }
  __device__ __forceinline__ void next() {
    left -= len;
    f += len;
    if (f == group) {
      ++d;
      f = 0;
      begin();
    } else {
      len = base + (--extra > 0 ? 1 : 0);
    }
  }
};

struct FewRing {
  uint32_t bar0, base;  // full barriers, then empty ones; first stage
  int stages, stage;
  uint32_t phase, stage_bytes;
  __device__ __forceinline__ uint32_t full() const { return bar0 + 8u * stage; }
  __device__ __forceinline__ uint32_t empty() const { return bar0 + 8u * (kFewMaxStages + stage); }
  __device__ __forceinline__ uint32_t addr() const { return base + stage_bytes * stage; }
  __device__ __forceinline__ void next() {
    if (++stage == stages) {
      stage = 0;
      phase ^= 1u;
    }
  }
};

template <typename TA, bool FP4>
struct FewTypes {
  using Z = typename std::conditional<FP4, __half, TA>::type;  // z and h
};

// ---- producers --------------------------------------------------------------------------
// (predicated, not branched around: a producer warp issues many in a row)
__device__ __forceinline__ void cp_async16_if(bool on, uint32_t dst, const void* src) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p cp.async.cg.shared.global [%0], [%1], 16;\n\t}" ::"r"(
                   dst),
               "l"(src), "r"(static_cast<uint32_t>(on))
               : "memory");
}
// one arrival on bar once this thread's copies so far have landed (counted in the barrier's
// expected arrivals)
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// A phase's product: its depth, and its weight rows as units (see FewChunks).
struct FewJob {
  int phase, K, U, group, most;
};
__device__ __forceinline__ FewJob few_job(const FewArgs& p, int phase, int distinct) {
  const int rows = phase == FEW_ROUTER ? p.E : phase == FEW_OUT ? p.D : phase == FEW_GATE_UP ? p.I : p.L;
  const bool experts = phase == FEW_GATE_UP || phase == FEW_DOWN;
  return {phase, phase <= FEW_POOL ? p.D : phase == FEW_DOWN ? p.I : p.L, experts ? distinct * rows : rows, rows,
          phase == FEW_GATE_UP ? kFewRows / 2 : kFewRows};
}

// A job as its producers see it: a chunk's weight rows, which follow one another in one or two
// matrices, and its activation rows.
template <typename TA, int FORMAT>
struct FewSource {
  const FewArgs& p;
  const FewRoute& r;
  const TA* xin;
  FewJob job;

  __device__ __forceinline__ bool gate_up() const { return job.phase == FEW_GATE_UP; }
  __device__ __forceinline__ bool experts() const { return job.phase == FEW_GATE_UP || job.phase == FEW_DOWN; }
  __device__ __forceinline__ int64_t row_bytes() const {
    return FORMAT == FEW_NVFP4 ? job.K / 2 : job.K * static_cast<int64_t>(sizeof(TA));
  }
  // index of the chunk's first row over all experts
  __device__ __forceinline__ int64_t first_row(const FewChunks& c) const {
    return c.f + (experts() ? static_cast<int64_t>(r.ids[c.d]) * job.group : 0);
  }
  // the chunk's first row in the phase's matrix; gate/up: of W_up if `up`
  __device__ __forceinline__ const uint8_t* row(const FewChunks& c, bool up) const {
    const void* w = job.phase == FEW_ROUTER ? p.W_router : job.phase == FEW_POOL ? p.W_pool
                  : job.phase == FEW_OUT ? p.W_unpool : job.phase == FEW_DOWN ? p.W_down : up ? p.W_up : p.W_gate;
    return static_cast<const uint8_t*>(w) + first_row(c) * row_bytes();
  }
  __device__ __forceinline__ const uint8_t* scales(const FewChunks& c, int i) const {
    const uint8_t* s = job.phase == FEW_DOWN ? p.s_down : i < 16 ? p.s_gate : p.s_up;
    return s + (first_row(c) + (gate_up() ? i & 15 : i)) * (job.K / 16);
  }
  // whether place i of a stage (gate/up: 0.. gate, 16.. up) holds a row of the chunk
  __device__ __forceinline__ bool has_row(const FewChunks& c, int i) const { return (gate_up() ? i & 15 : i) < c.len; }
  __device__ __forceinline__ int tokens(const FewChunks& c) const {
    return experts() ? r.first[c.d + 1] - r.first[c.d] : p.T;
  }
  __device__ __forceinline__ const uint8_t* activation(const FewChunks& c, int j) const {
    const void* x = job.phase <= FEW_POOL ? static_cast<const void*>(xin) : gate_up() ? p.z
                  : job.phase == FEW_DOWN ? p.h : p.c;
    // (split activations: the second numbers of all rows follow the first ones')
    const int n = tokens(c), i = j < n ? j : j - n;
    int row = gate_up() ? r.token[r.first[c.d] + i] : job.phase == FEW_DOWN ? r.first[c.d] + i : i;
    if (j >= n) row += job.phase == FEW_DOWN ? p.T * p.k : p.T;
    return static_cast<const uint8_t*>(x) + row * (job.K * static_cast<int64_t>(sizeof(TA)));
  }
};

// The buffer of an expert's activation rows: filled by producer warp 0 once the product warps are
// done with the expert before (barrier `free`); its copies precede that warp's arrival at the
// expert's first stage, which therefore also says that the rows are there.
struct FewX {
  uint32_t base, free;
  uint32_t phase;  // of the next wait on / arrival at free
};

// One producer warp's copies of a job: warp 0 the activations, once
// `ready` (the barrier before this phase; nullptr: nothing to wait for) has passed; the others
// each every third weight row (and a third of the block scales), as far ahead as the ring is free. A stage's addresses advance by
// constants from those of the chunk, so that a copy costs a few instructions.
template <typename TA, int FORMAT>
__device__ __forceinline__ void few_produce(const FewSource<TA, FORMAT>& q, FewRing& ring, FewX& xbuf,
                                            const uint32_t* ready, volatile int* abort, int pw, int lane) {
  using G = FewGeo<FORMAT>;
  constexpr int kWeightWarps = kFewProducers - 1;
  constexpr int kMine = (kFewRows + kWeightWarps - 1) / kWeightWarps;
  const FewArgs& p = q.p;
  const int K = q.job.K;
  FewChunks c(q.job.U, q.job.group, q.job.most);
  int expert = -1;  // whose rows the buffer holds
  if (pw == 0 && ready != nullptr) {
    if (lane == 0) few_poll(ready, gridDim.x, abort, p.status, 0xB00u + q.job.phase);
    __syncwarp();
  }
  for (; !c.done(); c.next()) {
    const bool whole = FORMAT == FEW_NVFP4 && p.x_bytes > 0;
    const int narrow = q.job.phase == FEW_ROUTER && FORMAT != FEW_NVFP4 ? p.narrow : 0;
    const int n = q.tokens(c), kc = narrow > 0 ? G::kc * narrow : G::depth(n, whole);
    if (pw == 0) {
      const uint32_t xstride = G::xstride(whole ? K : kc), xoff = narrow > 0 ? kFewNarrow * xstride : G::xoff;
      const int m = few_split(FORMAT, q.job.phase) ? 2 * n : n;  // activation rows
      const uint8_t* x = q.activation(c, min(lane, m - 1));         // lane j: row j
      // `bytes` of every row to dst, BATCH rows at a time: row by row this warp did not keep up with
      // the weights (eight tokens, eight bf16 experts, full size: 215 us, 393 row by row; four
      // tokens of the released sizes: 43, 49)
      auto copy = [&](uint32_t dst, int bytes, auto batch) {
        constexpr int BATCH = decltype(batch)::value;
#pragma unroll 1
        for (int j = 0; j < m; j += BATCH) {
          const uint8_t* xj[BATCH];
#pragma unroll
          for (int i = 0; i < BATCH; ++i)
            xj[i] = reinterpret_cast<const uint8_t*>(
                __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(x), j + i));
#pragma unroll (BATCH == 1 ? 2 : 1)
          for (int a = 16 * lane; a - 16 * lane < bytes; a += 512) {
#pragma unroll
            for (int i = 0; i < BATCH; ++i)
              cp_async16_if(a < bytes && j + i < m, dst + xstride * (j + i) + G::xbyte(a), xj[i] + a);
          }
        }
      };
      auto rows = [&](uint32_t dst, int bytes) {
        if (m == 1) copy(dst, bytes, std::integral_constant<int, 1>{});
        else if (m <= 4) copy(dst, bytes, std::integral_constant<int, 4>{});
        else copy(dst, bytes, std::integral_constant<int, 8>{});
      };
      if (whole && c.d != expert) {
        expert = c.d;
        if (few_mbar_wait(xbuf.free, xbuf.phase ^ 1u, abort, p.status, 0xA80u)) {
          __syncwarp();
          rows(xbuf.base, K * G::act_size);
        }
        xbuf.phase ^= 1u;
        __syncwarp();
      }
#pragma unroll 1
      for (int k0 = 0; k0 < K; k0 += kc) {
        const int kn = min(kc, K - k0);
        // (a wait that gave up: no copies; the arrivals go on so that nobody waits for them)
        const bool ok = few_mbar_wait(ring.empty(), ring.phase ^ 1u, abort, p.status, 0xA00u + ring.stage);
        if (__all_sync(0xffffffffu, ok)) {
          if (!whole) rows(ring.addr() + xoff, kn * G::act_size);
        }
        cp_async_arrive(ring.full());
        ring.next();
        x += kc * G::act_size;
      }
    } else if (FORMAT != FEW_NVFP4 && narrow > 0) {
#pragma unroll 1
      for (int k0 = 0; k0 < K; k0 += kc) {
        const int bytes = min(kc, K - k0) * G::act_size;
        const bool ok = few_mbar_wait(ring.empty(), ring.phase ^ 1u, abort, p.status, 0xA00u + ring.stage);
        if (__all_sync(0xffffffffu, ok)) {
#pragma unroll 1
          for (int i = pw - 1; i < c.len; i += kWeightWarps) {
            const uint8_t* w = q.row(c, false) + i * q.row_bytes() + k0 * static_cast<int64_t>(G::act_size);
            const uint32_t dst = ring.addr() + i * G::xstride(kc);
#pragma unroll 4
            for (int a = 16 * lane; a - 16 * lane < bytes; a += 512) cp_async16_if(a < bytes, dst + a, w + a);
          }
        }
        cp_async_arrive(ring.full());
        ring.next();
      }
    } else {
      // places i = pw - 1 + kWeightWarps * m; from 16 on (gate/up) of the other matrix
      const int64_t step = q.row_bytes();
      const uint8_t* w0 = q.row(c, false) + (pw - 1) * step + 16 * lane;
      const uint8_t* w1 = q.gate_up() ? q.row(c, true) + (pw - 1 - 16) * step + 16 * lane : w0;
      uint32_t mask = 0;
#pragma unroll
      for (int m = 0; m < kMine; ++m) {
        const int i = pw - 1 + kWeightWarps * m;
        if (i < kFewRows && q.has_row(c, i)) mask |= 1u << m;
      }
      // block scales, in 16-byte pieces (256 elements): eight a row, by all lanes of these warps
      constexpr int kSc = FORMAT == FEW_NVFP4 ? (kFewRows * 8 + 32 * kWeightWarps - 1) / (32 * kWeightWarps) : 0;
      const uint8_t* sc[kSc + 1];
      uint32_t sdst[kSc + 1];
      int sk[kSc + 1];  // first element of K a piece covers; past K: no piece
      if constexpr (FORMAT == FEW_NVFP4) {
#pragma unroll
        for (int i = 0; i < kSc; ++i) {
          const int a = (pw - 1) * 32 + lane + 32 * kWeightWarps * i, row = min(a >> 3, kFewRows - 1);
          sc[i] = q.scales(c, row) + 16 * (a & 7);
          sdst[i] = G::soff + G::sstride * row + 16 * (a & 7);
          sk[i] = a < 8 * kFewRows && q.has_row(c, row) ? 256 * (a & 7) : 0x7fffffff;
        }
      }
#pragma unroll 1
      for (int k0 = 0; k0 < K; k0 += kc) {
        const int kn = min(kc, K - k0), bytes = (FORMAT == FEW_NVFP4 ? kn / 2 : kn * G::act_size) - 16 * lane;
        const bool ok = few_mbar_wait(ring.empty(), ring.phase ^ 1u, abort, p.status, 0xA00u + ring.stage);
        if (__all_sync(0xffffffffu, ok)) {
          const uint32_t st = ring.addr() + 16 * lane + G::wstride * (pw - 1);
          const uint8_t* a0 = w0;
          const uint8_t* a1 = w1;
#pragma unroll
          for (int m = 0; m < kMine; ++m) {
            const uint8_t* a = pw - 1 + kWeightWarps * m < 16 ? a0 : a1;
#pragma unroll
            for (int o = 0; o < static_cast<int>(G::row_bytes); o += 512)
              cp_async16_if((mask >> m & 1u) && o < bytes, st + kWeightWarps * m * G::wstride + o, a + o);
            a0 += kWeightWarps * step;
            a1 += kWeightWarps * step;
          }
#pragma unroll
          for (int i = 0; i < kSc; ++i) cp_async16_if(sk[i] < kn, ring.addr() + sdst[i], sc[i]);
        }
        cp_async_arrive(ring.full());
        ring.next();
        w0 += FORMAT == FEW_NVFP4 ? kc / 2 : kc * G::act_size;
        w1 += FORMAT == FEW_NVFP4 ? kc / 2 : kc * G::act_size;
#pragma unroll
        for (int i = 0; i < kSc; ++i) sc[i] += kc / 16;
      }
    }
  }
}

// ---- products ---------------------------------------------------------------------------
// barriers over the product warps, the store warps, both with the producers
__device__ __forceinline__ void few_sync_products() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kFewWarps) : "memory"); }
__device__ __forceinline__ void few_sync_store() { asm volatile("bar.sync 2, %0;" ::"n"(32 * kFewStore) : "memory"); }
__device__ __forceinline__ void few_sync_all() { asm volatile("bar.sync 3, %0;" ::"n"(kFewThreads) : "memory"); }

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
// (zeros and no access where off)
__device__ __forceinline__ uint4 lds128_if(bool on, uint32_t a) {
  uint4 v;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\t"
      "mov.b32 %3, 0;\n\t@p ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "r"(a), "r"(static_cast<uint32_t>(on)));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ float4 as_float4(uint4 v) {
  return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
}

// The two buffers of partial sums between product and store warps: [warp][token][row], the
// tokens 33 floats apart.
struct FewRed {
  uint32_t bar0;  // full barriers, then free ones
  float* base;
  int buf;
  uint32_t phase;
  __device__ __forceinline__ uint32_t full() const { return bar0 + 8u * buf; }
  __device__ __forceinline__ uint32_t free() const { return bar0 + 16u + 8u * buf; }
  __device__ __forceinline__ float* red() const { return base + kFewRedFloats * buf; }
  __device__ __forceinline__ void next() {
    buf ^= 1;
    if (buf == 0) phase ^= 1u;
  }
};

// One chunk's products: the stages of 32 weight rows and n activation rows, this warp's share
// of K; the warp's sums go to the next buffer of partial sums.
template <int FORMAT>
__device__ __forceinline__ void few_consume(const FewArgs& p, FewRing& ring, const FewX& xbuf, int phase, int K, int n,
                                            int wc, int lane, volatile int* abort, FewRed& out) {
  using G = FewGeo<FORMAT>;
  const int g = lane >> 2, t = lane & 3;
  // token rows past n are not staged, and their columns not used; reading none for them saves up
  // to three quarters of the activations' shared-memory cycles (NVFP4, eight tokens: 425 us, 440 reading all)
  // (two numbers for each token: in columns of their own, or with more than four tokens in a second
  // MMA that adds to the first one's sums)
  const bool split = few_split(FORMAT, phase), twice = split && n > 4;
  const bool has_x = g < (split && !twice ? 2 * n : n);
  float acc[8];          // float32: this lane's row, 8 tokens
  float chain[2][2][4];  // MMA: two 16-row tiles, each in two sums, so that fewer MMAs wait for one another
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    acc[i] = 0.0f;
    chain[0][i >> 2][i & 3] = chain[1][i >> 2][i & 3] = 0.0f;
  }
  const bool whole = FORMAT == FEW_NVFP4 && p.x_bytes > 0;
  const int narrow = phase == FEW_ROUTER && FORMAT != FEW_NVFP4 ? p.narrow : 0;
  const int kc = narrow > 0 ? G::kc * narrow : G::depth(n, whole);
  const uint32_t xstride = G::xstride(whole ? K : kc);
  // a narrow stage holds kFewNarrow rows: the other rows of the MMA read these again, for nothing
  const uint32_t wstride = narrow > 0 ? xstride : G::wstride;
  const uint32_t xoff = narrow > 0 ? kFewNarrow * xstride : G::xoff;
#pragma unroll 1
  for (int k0 = 0; k0 < K; k0 += kc) {
    const int kn = min(kc, K - k0);
    few_mbar_wait(ring.full(), ring.phase, abort, p.status, 0xC00u + ring.stage);
    __syncwarp();
    const uint32_t st = ring.addr();
    if constexpr (FORMAT == FEW_BF16 || FORMAT == FEW_BF16_SHORT) {
      const uint32_t w = st + (narrow > 0 ? g & (kFewNarrow - 1) : g) * wstride + t * 16u;
      const uint32_t x = st + xoff + g * xstride + t * 16u;
      const uint32_t r8 = narrow > 0 ? 0u : 8u * wstride;
      auto products = [&](auto two) {
#pragma unroll 2
        for (int s = wc; s < kn / 32; s += kFewWarps) {  // 32 elements = 64 bytes of each row
          const uint32_t o = 64u * s;
          const uint4 b = lds128_if(has_x, x + o), a0 = lds128(w + o), a1 = lds128(w + r8 + o), a2 = lds128(w + 2 * r8 + o),
                      a3 = lds128(w + 3 * r8 + o);
          mma_bf16_16816(chain[0][0], a0.x, a1.x, a0.y, a1.y, b.x, b.y);
          mma_bf16_16816(chain[0][1], a2.x, a3.x, a2.y, a3.y, b.x, b.y);
          mma_bf16_16816(chain[1][0], a0.z, a1.z, a0.w, a1.w, b.z, b.w);
          mma_bf16_16816(chain[1][1], a2.z, a3.z, a2.w, a3.w, b.z, b.w);
          if constexpr (decltype(two)::value) {
            const uint4 c = lds128_if(has_x, x + n * xstride + o);
            mma_bf16_16816(chain[0][0], a0.x, a1.x, a0.y, a1.y, c.x, c.y);
            mma_bf16_16816(chain[0][1], a2.x, a3.x, a2.y, a3.y, c.x, c.y);
            mma_bf16_16816(chain[1][0], a0.z, a1.z, a0.w, a1.w, c.z, c.w);
            mma_bf16_16816(chain[1][1], a2.z, a3.z, a2.w, a3.w, c.z, c.w);
          }
        }
      };
      if (twice) products(std::true_type{});
      else products(std::false_type{});
    } else if constexpr (FORMAT == FEW_NVFP4) {
      const uint32_t w = st + g * G::wstride + t * 16u;
      const uint32_t x = (whole ? xbuf.base + k0 / 8 * 18 : st + G::xoff) + g * xstride + t * 64u + (t >> 1) * 16u;
      const uint32_t sc = st + G::soff + g * G::sstride + t * 2u;
#pragma unroll 1
      for (int s = wc; s < kn / 128; s += kFewWarps) {  // 128 elements; this lane's two blocks: 2 t, 2 t + 1
        uint4 cw[4];
        uint32_t sw[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          cw[i] = lds128(w + 8u * i * G::wstride + 64u * s);
          sw[i] = lds16(sc + 8u * i * G::sstride + 8u * s);
        }
        // 16 MMAs in four chains (block h, row tile m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // the lane's blocks: two code words a row each
          const uint4 x0 = lds128_if(has_x, x + 288u * s + 32u * h), x1 = lds128_if(has_x, x + 288u * s + 32u * h + 16u);
          const uint32_t xw[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            uint32_t a[2][8];            // rows g and g + 8 of the tile
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int i = 2 * m + j;
              const uint32_t b = __byte_perm(e4m3x2_to_f16x2(sw[i]), 0u, h ? 0x3232u : 0x1010u);
              e2m1x8_to_f16x2(h ? cw[i].z : cw[i].x, a[j][0], a[j][1], a[j][2], a[j][3]);
              e2m1x8_to_f16x2(h ? cw[i].w : cw[i].y, a[j][4], a[j][5], a[j][6], a[j][7]);
#pragma unroll
              for (int q = 0; q < 8; ++q) a[j][q] = f16x2_mul(a[j][q], b);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
              mma_f16_16816(chain[h][m], a[0][2 * q], a[1][2 * q], a[0][2 * q + 1], a[1][2 * q + 1], xw[2 * q],
                            xw[2 * q + 1]);
          }
        }
      }
    } else {
      const uint32_t w = st + (narrow > 0 ? lane & (kFewNarrow - 1) : lane) * wstride;
      const uint32_t x = st + xoff;
#pragma unroll 2
      for (int s = wc; s < kn / 4; s += kFewWarps) {
        const float4 a = as_float4(lds128(w + 16u * s));
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (j >= n) break;
          const float4 b = as_float4(lds128(x + j * xstride + 16u * s));
          acc[j] = fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, acc[j]))));
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(ring.empty());
    ring.next();
  }
  few_mbar_wait(out.free(), out.phase ^ 1u, abort, p.status, 0xD00u);
  __syncwarp();
  float* mine = out.red() + wc * 8 * 33;
  if constexpr (FORMAT == FEW_F32) {
#pragma unroll
    for (int j = 0; j < 8; ++j) mine[j * 33 + lane] = acc[j];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) mine[(2 * t + (i & 1)) * 33 + 16 * (i >> 2) + 8 * ((i >> 1) & 1) + g] =
        chain[0][i >> 2][i & 3] + chain[1][i >> 2][i & 3];
  }
  __syncwarp();
  if (lane == 0) mbar_arrive(out.full());
  out.next();
}

// The warps' sums of (token, row), in a fixed order.
__device__ __forceinline__ float few_sum(const float* red, int token, int row) {
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int w = 0; w < kFewWarps; ++w) v[w & 3] += red[(w * 8 + token) * 33 + row];
  return (v[0] + v[1]) + (v[2] + v[3]);
}

// An intermediate as the next product reads it: bf16 with what its rounding took off, `second`
// elements further.
template <typename T>
__device__ __forceinline__ void few_put(T* a, int64_t second, int64_t i, float v) {
  const T first = from_f32<T>(v);
  a[i] = first;
  if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    const float rest = v - to_f32(first);
    a[second + i] = from_f32<T>(fabsf(rest) < INFINITY ? rest : 0.0f);  // (infinities and NaN stay what they are)
  }
}

__device__ __forceinline__ float few_silu(float a) { return a / (1.0f + expf(-a)); }

// Sum over the product warps' threads, the same on each (part: 32 floats).
__device__ __forceinline__ float few_block_sum(float v, float* part, int wc, int lane) {
  v = warp_sum(v);
  few_sync_products();
  if (lane == 0) part[wc] = v;
  few_sync_products();
  return warp_sum(lane < kFewWarps ? part[lane] : 0.0f);
}

// Centred RMSNorm of n values by the product warps: put(i, get(i) / sqrt(mean(get^2) + eps) * (1 + w_i)).
template <typename TG, typename Get, typename Put>
__device__ __forceinline__ void few_norm_row(const TG* w, int n, float eps, float* part, int tid, Get get, Put put) {
  constexpr int kStep = 32 * kFewWarps, kKeep = 4;  // a thread's first values stay in registers
  float s = 0.0f, keep[kKeep];
#pragma unroll
  for (int j = 0; j < kKeep; ++j) keep[j] = tid + j * kStep < n ? get(tid + j * kStep) : 0.0f;
#pragma unroll
  for (int j = 0; j < kKeep; ++j) s = fmaf(keep[j], keep[j], s);
#pragma unroll 4
  for (int i = tid + kKeep * kStep; i < n; i += kStep) {
    const float v = get(i);
    s = fmaf(v, v, s);
  }
  const float scale = 1.0f / sqrtf(few_block_sum(s, part, tid >> 5, tid & 31) / static_cast<float>(n) + eps);
#pragma unroll
  for (int j = 0; j < kKeep; ++j)
    if (tid + j * kStep < n) put(tid + j * kStep, keep[j] * scale * (1.0f + to_f32(w[tid + j * kStep])));
#pragma unroll 4
  for (int i = tid + kKeep * kStep; i < n; i += kStep) put(i, get(i) * scale * (1.0f + to_f32(w[i])));
}

// c = sum_j g_j y_j / rms_j (1 + gamma) by the product warps, each CTA a slice of it. (All of it in
// every CTA, one grid barrier less, took 2 to 14 us more in small layers.)
template <typename TA>
__device__ __forceinline__ void few_combine(const FewArgs& p, const FewRoute& route, float* scale_s, int wc, int lane,
                                            int tid) {
  const int T = p.T, L = p.L, k = p.k, rows = route.distinct * L;
  const TA* gamma = static_cast<const TA*>(p.gamma);
  // every pair's weight over its root mean square, from the CTAs that hold its rows; a warp takes
  // four pairs at a time, all their loads in flight together
  for (int a0 = wc; a0 < T * k; a0 += 4 * kFewWarps) {
    float s[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int a = a0 + j * kFewWarps;
      s[j] = 0.0f;
      if (a < T * k) {
        const int pos = route.pos[a], d = route.distinct_of[a];
        const int c0 = few_owner(rows, d * L), c1 = few_owner(rows, (d + 1) * L - 1);
#pragma unroll 1
        for (int i = c0 + lane; i <= c1; i += 32)  // (with fewer rows than CTAs, some have none)
          if (rows >= static_cast<int>(gridDim.x) || few_share(rows, i) < few_share(rows, i + 1))
            s[j] += __ldcg(p.ss + static_cast<int64_t>(pos) * kFewGridMax + i);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int a = a0 + j * kFewWarps;
      const float sum = warp_sum(s[j]);
      if (lane == 0 && a < T * k) scale_s[a] = route.weight[a] / sqrtf(sum / static_cast<float>(L) + p.eps);
    }
  }
  few_sync_products();
  for (int i = blockIdx.x * (32 * kFewWarps) + tid; i < T * L; i += gridDim.x * (32 * kFewWarps)) {
    const int t = i / L, f = i - t * L;
    float acc = 0.0f;
#pragma unroll 8
    for (int j = 0; j < k; ++j) {
      const int a = t * k + j;
      const float gm = to_f32(gamma[(p.gamma_shared ? 0 : static_cast<int64_t>(route.expert[a]) * L) + f]);
      acc = fmaf(scale_s[a] * (1.0f + gm), __ldcg(p.y + static_cast<int64_t>(route.pos[a]) * L + f), acc);
    }
    few_put(static_cast<TA*>(p.c), static_cast<int64_t>(T) * L, i, acc);
  }
}

// grid barriers, by what they say is done
enum FewBarrier : int { FEW_XN = 0, FEW_LOGITS, FEW_Z, FEW_ZN, FEW_H, FEW_Y, FEW_C, FEW_F };

// TA: activations, dense weights, gains and the output (bf16 or float). FP4: NVFP4 experts
// (TA = bf16; z and h are f16).
template <typename TA, bool FP4>
__global__ void __launch_bounds__(kFewThreads, 1) k_few_tokens(const __grid_constant__ FewArgs p) {
  using TZ = typename FewTypes<TA, FP4>::Z;
  constexpr int DENSE = sizeof(TA) == 4 ? FEW_F32 : FP4 ? FEW_BF16_SHORT : FEW_BF16;
  constexpr int EXPERT = FP4 ? FEW_NVFP4 : DENSE;
  extern __shared__ __align__(128) uint8_t smem[];  // partial sums, activation rows, the ring
  __shared__ FewRoute route;
  __shared__ __align__(8) uint64_t bars[2 * kFewMaxStages + 5];
  __shared__ float part[32];
  __shared__ float scale_s[kFewAssign];
  __shared__ int abort_flag;
  volatile int* abort = &abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int T = p.T, D = p.D, L = p.L, I = p.I, E = p.E;
  FewRing ring{smem_u32(bars), smem_u32(smem) + kFewRedBytes + p.x_bytes, p.stages, 0, 0u, p.stage_bytes};
  FewX xbuf{smem_u32(smem) + kFewRedBytes, smem_u32(bars + 2 * kFewMaxStages + 4), 0u};
  FewRed red{smem_u32(bars + 2 * kFewMaxStages), reinterpret_cast<float*>(smem), 0, 0u};
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(smem_u32(bars + s), 32 * kFewProducers);
      mbar_init(smem_u32(bars + kFewMaxStages + s), kFewWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(red.bar0 + 8u * i, kFewWarps);
      mbar_init(red.bar0 + 16u + 8u * i, kFewStore);
    }
    mbar_init(xbuf.free, kFewWarps);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (threadIdx.x < 32) route.seen[threadIdx.x] = 0;
  for (int i = threadIdx.x; i < kFewAssign; i += kFewThreads) route.expert[i] = 0x7fffffff;
  __syncthreads();
  auto counter = [&](int i) { return p.barrier + 32 * i; };
  const bool pre = p.ffn_pre_gain != nullptr, zn = p.pre_norm_gain != nullptr;
  const bool finish = p.ffn_post_gain != nullptr || p.residual_gate != nullptr;
  const TA* xin = pre ? static_cast<const TA*>(p.xn) : static_cast<const TA*>(p.x);

  // ------------------------------------------------------------------------- producers
  if (warp < kFewProducers) {
#pragma unroll 1
    for (int ph = FEW_ROUTER; ph <= FEW_OUT; ++ph) {
      if (ph == FEW_GATE_UP) few_sync_all();
      const FewJob job = few_job(p, ph, route.distinct);
      const uint32_t* ready = ph <= FEW_POOL ? (pre ? counter(FEW_XN) : nullptr)
                              : counter(ph == FEW_GATE_UP ? (zn ? FEW_ZN : FEW_Z) : ph == FEW_DOWN ? FEW_H : FEW_C);
      if (FP4 && (ph == FEW_GATE_UP || ph == FEW_DOWN))
        few_produce(FewSource<TA, EXPERT>{p, route, xin, job}, ring, xbuf, ready, abort, warp, lane);
      else
        few_produce(FewSource<TA, DENSE>{p, route, xin, job}, ring, xbuf, ready, abort, warp, lane);
    }
    cp_async_wait_all();  // nothing in flight when the CTA leaves, also after a wait that gave up
    return;
  }

  const TA* gamma = static_cast<const TA*>(p.gamma);
  const TA* post = static_cast<const TA*>(p.ffn_post_gain);
  // ------------------------------------------------------------------------- store warps
  if (warp < kFewProducers + kFewStore) {
    const int ws = warp - kFewProducers, tid = threadIdx.x - 32 * kFewProducers;
    // this CTA's part of barrier i is done
    auto arrive = [&](int i) {
      few_sync_store();
      if (tid == 0) red_release_u32(counter(i), 1u);  // (cumulative: orders the warps' writes too)
    };
    // the sums of a chunk: store(chunk, token, lane's row, sum) on warp token % kFewStore
    auto chunk = [&](const FewChunks& c, int ph, int n, auto store) {
      const bool experts = ph == FEW_GATE_UP || ph == FEW_DOWN;
      const bool split = few_split(experts ? EXPERT : DENSE, ph) && n <= 4;  // (sums in two columns)
      few_mbar_wait(red.full(), red.phase, abort, p.status, 0xE00u);
      __syncwarp();
#pragma unroll 1
      for (int j = ws; j < n; j += kFewStore) {
        float v = few_sum(red.red(), j, lane);
        if (split) v += few_sum(red.red(), n + j, lane);
        store(c, j, v);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(red.free());
      red.next();
    };
    auto each = [&](int ph, auto store) {
      const FewJob job = few_job(p, ph, route.distinct);
#pragma unroll 1
      for (FewChunks c(job.U, job.group, job.most); !c.done(); c.next())
        chunk(c, ph, ph == FEW_GATE_UP || ph == FEW_DOWN ? route.first[c.d + 1] - route.first[c.d] : T, store);
    };
    each(FEW_ROUTER, [&](const FewChunks& c, int j, float v) {
      if (lane < c.len) p.logits[static_cast<int64_t>(j) * E + c.f + lane] = v;
    });
    arrive(FEW_LOGITS);
    {
      // store z and select the experts, whichever can be done first: in a large layer the logits
      // of all CTAs are there long before the pooler's rows, in a small one the rows are
      FewChunks c(L, L, kFewRows);
      bool routed = false;
#pragma unroll 1
      while (!routed || !c.done()) {
        // (votes: the lanes' reads may differ)
        if (!routed && (c.done() || __all_sync(0xffffffffu, ld_acquire_u32(counter(FEW_LOGITS)) >= gridDim.x))) {
          few_poll(counter(FEW_LOGITS), gridDim.x, abort, p.status, 0xF00u + FEW_LOGITS);
          __syncwarp();
#pragma unroll 1
          for (int t = ws; t < T; t += kFewStore) few_route(p, route, t, lane);
          routed = true;
        } else if (routed || __all_sync(0xffffffffu, *abort != 0 || mbar_try_wait(red.full(), red.phase))) {
          chunk(c, FEW_POOL, T, [&](const FewChunks& cc, int j, float v) {
            const int64_t o = static_cast<int64_t>(j) * L + cc.f + lane;
            if (lane < cc.len && zn) p.zraw[o] = v;
            else if (lane < cc.len) few_put(static_cast<TZ*>(p.z), static_cast<int64_t>(T) * L, o, v);
          });
          c.next();
        }
      }
    }
    arrive(FEW_Z);
    few_lists(p, route, tid, 32 * kFewStore);
    few_sync_all();
    each(FEW_GATE_UP, [&](const FewChunks& c, int j, float v) {
      const float u = __shfl_down_sync(0xffffffffu, v, 16);
      float mg = 1.0f, mu = 1.0f;
      if constexpr (FP4) {
        mg = p.m_gate[route.ids[c.d]];
        mu = p.m_up[route.ids[c.d]];
      }
      if (lane < c.len)
        few_put(static_cast<TZ*>(p.h), static_cast<int64_t>(T) * p.k * I,
                static_cast<int64_t>(route.first[c.d] + j) * I + c.f + lane, few_silu(v * mg) * (u * mu));
    });
    arrive(FEW_H);
    {
      // sums of squares of the rows this CTA computes of each position: tokens ws, ws + kFewStore, ...
      // of the current expert
      float ss[kFewPer] = {};
      int ss_d = -1;
      auto flush = [&]() {
        if (ss_d < 0) return;
#pragma unroll
        for (int h = 0; h < kFewPer; ++h) {
          const int pos = route.first[ss_d] + ws + kFewStore * h;
          if (lane == 0 && pos < route.first[ss_d + 1]) p.ss[static_cast<int64_t>(pos) * kFewGridMax + blockIdx.x] = ss[h];
          ss[h] = 0.0f;
        }
      };
      each(FEW_DOWN, [&](const FewChunks& c, int j, float y) {
        if (c.d != ss_d) flush();
        ss_d = c.d;
        const int e = route.ids[c.d];
        if constexpr (FP4) y *= p.m_down[e];
        float u = 0.0f;
        if (lane < c.len) {
          p.y[static_cast<int64_t>(route.first[c.d] + j) * L + c.f + lane] = y;
          u = y;
          if (p.norm_mode == 1)
            u *= 1.0f + to_f32(gamma[(p.gamma_shared ? 0 : static_cast<int64_t>(e) * L) + c.f + lane]);
        }
        const float s = warp_sum(u * u);
#pragma unroll
        for (int h = 0; h < kFewPer; ++h) ss[h] += j / kFewStore == h ? s : 0.0f;
      });
      flush();
      arrive(FEW_Y);
    }
    float ssf[kFewPer] = {};  // of this CTA's rows of tokens ws, ws + kFewStore, ...
    each(FEW_OUT, [&](const FewChunks& c, int j, float v) {
      const int64_t o = static_cast<int64_t>(j) * D + c.f + lane;
      if (!finish) {
        if (lane < c.len) static_cast<TA*>(p.out)[o] = from_f32<TA>(v);
        return;
      }
      float u = 0.0f;
      if (lane < c.len) {
        p.f[o] = v;
        if (post != nullptr) u = v * (1.0f + to_f32(post[c.f + lane]));
      }
      const float s = warp_sum(u * u);
#pragma unroll
      for (int h = 0; h < kFewPer; ++h) ssf[h] += j / kFewStore == h ? s : 0.0f;
    });
    if (finish) {
#pragma unroll
      for (int h = 0; h < kFewPer; ++h)
        if (lane == 0 && ws + kFewStore * h < T) p.ssf[(ws + kFewStore * h) * kFewGridMax + blockIdx.x] = ssf[h];
      arrive(FEW_F);
    }
    return;
  }

  // ------------------------------------------------------------------------- product warps
  const int wc = warp - kFewProducers - kFewStore, tid = threadIdx.x - 32 * (kFewProducers + kFewStore);
  constexpr int kProducts = 32 * kFewWarps;
  auto arrive = [&](int i) {
    few_sync_products();
    if (tid == 0) red_release_u32(counter(i), 1u);
  };
  auto wait = [&](int i) {
    if (tid == 0) few_poll(counter(i), gridDim.x, abort, p.status, 0xF00u + i);
    few_sync_products();
  };
  if (pre) {
    for (int t = blockIdx.x; t < T; t += gridDim.x)
      few_norm_row(
          static_cast<const TA*>(p.ffn_pre_gain), D, p.ffn_pre_eps, part, tid,
          [&](int i) { return to_f32(static_cast<const TA*>(p.x)[static_cast<int64_t>(t) * D + i]); },
          [&](int i, float v) { static_cast<TA*>(p.xn)[static_cast<int64_t>(t) * D + i] = from_f32<TA>(v); });
    arrive(FEW_XN);
  }
#pragma unroll 1
  for (int ph = FEW_ROUTER; ph <= FEW_OUT; ++ph) {
    if (ph == FEW_GATE_UP) {
      if (zn) {
        wait(FEW_Z);
        TZ* z = static_cast<TZ*>(p.z);
        for (int t = blockIdx.x; t < T; t += gridDim.x)
          few_norm_row(
              static_cast<const TA*>(p.pre_norm_gain), L, p.pre_norm_eps, part, tid,
              [&](int i) { return __ldcg(p.zraw + static_cast<int64_t>(t) * L + i); },
              [&](int i, float v) { few_put(z, static_cast<int64_t>(T) * L, static_cast<int64_t>(t) * L + i, v); });
        arrive(FEW_ZN);
      }
      few_sync_all();
    }
    if (ph == FEW_OUT) {
      wait(FEW_Y);
      few_combine<TA>(p, route, scale_s, wc, lane, tid);
      arrive(FEW_C);
    }
    const FewJob job = few_job(p, ph, route.distinct);
    const bool experts = ph == FEW_GATE_UP || ph == FEW_DOWN;
#pragma unroll 1
    for (FewChunks c(job.U, job.group, job.most); !c.done(); c.next()) {
      const int n = experts ? route.first[c.d + 1] - route.first[c.d] : T;
      if (FP4 && experts) few_consume<EXPERT>(p, ring, xbuf, ph, job.K, n, wc, lane, abort, red);
      else few_consume<DENSE>(p, ring, xbuf, ph, job.K, n, wc, lane, abort, red);
      // the last chunk of an expert: its activation rows may go
      if (FP4 && experts && p.x_bytes > 0 && lane == 0 && (c.left == c.len || c.f + c.len == c.group)) mbar_arrive(xbuf.free);
    }
  }
  if (!finish) return;
  wait(FEW_F);
  // post norm and residual gate
  for (int t = wc; t < T; t += kFewWarps) {
    float s = 0.0f;
    for (int i = lane; i < static_cast<int>(gridDim.x); i += 32) s += __ldcg(p.ssf + t * kFewGridMax + i);
    s = warp_sum(s);
    if (lane == 0) scale_s[t] = 1.0f / sqrtf(s / static_cast<float>(D) + p.ffn_post_eps);
  }
  few_sync_products();
  for (int i = blockIdx.x * kProducts + tid; i < T * D; i += gridDim.x * kProducts) {
    const int t = i / D, f = i - t * D;
    float v = __ldcg(p.f + i);
    if (post != nullptr) v *= (1.0f + to_f32(post[f])) * scale_s[t];
    if (p.residual_gate != nullptr) {
      const float wg = p.residual_gate[f] * p.inv_temp;
      const float beta = 1.0f / (1.0f + expf(-wg));
      const float alpha = sqrtf(fmaxf((1.0f / (1.0f + expf(wg))) * (1.0f + beta), p.gate_eps));
      v = alpha * to_f32(static_cast<const TA*>(p.x)[i]) + beta * v;
    }
    static_cast<TA*>(p.out)[i] = from_f32<TA>(v);
  }
}

}  // namespace muse
