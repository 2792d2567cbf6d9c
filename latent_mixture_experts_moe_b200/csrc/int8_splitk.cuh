// int8_splitk.cuh -- the int8 product (int8_rows.cuh) for a few dozen to a few hundred rows, where
// tiles of whole K would leave most SMs idle: a cluster of up to 8 CTAs shares a tile of 128
// channels x up to 256 rows, each CTA a range of K. A CTA runs as in gemm_umma.cuh (TMA ring,
// one thread issuing tcgen05 kind::i8 MMAs, weights as the A operand); then every CTA puts its
// 32-bit partial sums into its shared memory, and each adds up its share of the tile's rows from
// all of them through the cluster window: integer sums, so the result does not depend on the
// split. No workspace, one launch.
// Bound by what an SM fetches through TMA from L2 (weights once per row tile, rows once per 128
// channels); the exchange costs ~2 us. 64 rows through 8192 x 4096 weights: 13.0 us from DRAM
// (2.6 TB/s), 11.1 where they lie in L2.
#pragma once

#include <cstdint>

#include "gemm_umma.cuh"
#include "int8_rows.cuh"

namespace muse {

struct Int8SplitArgs {
  const float *x_scale, *w_scale;
  void* out;
  int64_t ldo;
  int T, N, k_blocks, m_tiles, bn;  // bn: rows per tile, a multiple of 16
  uint32_t* status;
};

template <int BN>
struct Int8SplitShape {
  static constexpr uint32_t kABytes = 128u * 128u, kBBytes = BN * 128u, kStageBytes = kABytes + kBBytes;
  static constexpr int kStagesFit = (227 * 1024 - 1024 - 1024) / static_cast<int>(kStageBytes);
  static constexpr int kStages = kStagesFit > 8 ? 8 : kStagesFit;
  static constexpr size_t kSmemBytes = 1024 + static_cast<size_t>(kStages) * kStageBytes;
  static_assert(BN * 128u * 4u <= kStages * kStageBytes, "the partial sums reuse the ring");
};

__device__ __forceinline__ uint4 ld_cluster_uint4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}

// grid: (cluster size) x tiles; cluster rank = K range
template <int BN, typename TOut>
__global__ void __launch_bounds__(192, 1) k_int8_splitk(const __grid_constant__ TmaMaps maps, const Int8SplitArgs p) {
  using S = Int8SplitShape<BN>;
  constexpr int kStages = S::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * kStages + 1];
  __shared__ uint32_t tmem_holder;
  __shared__ int abort_flag;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  volatile int* abort = &abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int splits = static_cast<int>(gridDim.x), rank = static_cast<int>(cluster_ctarank());
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (kStages + s); };
  const uint32_t done_bar = bar0 + 8u * (2 * kStages);
  const int tile = blockIdx.y, m0 = tile % p.m_tiles * 128, row0 = tile / p.m_tiles * p.bn;
  const int n = min(p.bn, p.T - row0), nb16 = (n + 15) >> 4;
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.k_blocks) * rank / splits);
  const int kb1 = static_cast<int>(static_cast<int64_t>(p.k_blocks) * (rank + 1) / splits);
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    mbar_init(done_bar, 1);
    abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&maps.a);
  }
  constexpr uint32_t kCols = BN < 32 ? 32 : BN;
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_holder), kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_holder;
  wait_for_predecessor();

  if (warp == 0) {
    if (lane == 0) {
      uint32_t issued = 0, issued_phase = 0;
      bool ok = true;
      for (int kb = kb0; ok && kb < kb1; ++kb) {
        const int i = kb - kb0, s = i % kStages;
        const uint32_t ph = static_cast<uint32_t>(i / kStages) & 1u;
        ok = mbar_wait(empty_bar(s), ph ^ 1u, abort, p.status, 0x1100u + s);
        if (!ok) break;
        mbar_arrive_expect_tx(full_bar(s), S::kABytes + static_cast<uint32_t>(nb16) * 2048u);
        const uint32_t sA = smem_u32(smem + s * S::kStageBytes);
        tma_load_2d(sA, &maps.a, full_bar(s), kb * 128, m0);
        int j16 = 0;
#pragma unroll
        for (int b = 4; b >= 0; --b)
          if ((16 << b) <= BN && (nb16 >> b) & 1) {
            tma_load_2d(sA + S::kABytes + 2048u * j16, &maps.b[b], full_bar(s), kb * 128, row0 + 16 * j16);
            j16 += 1 << b;
          }
        issued |= 1u << s;
        issued_phase = (issued_phase & ~(1u << s)) | (ph << s);
      }
      if (!ok)
        for (int s = 0; s < kStages; ++s)
          if (issued & (1u << s)) mbar_wait_drain(full_bar(s), (issued_phase >> s) & 1u);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = idesc_i8(128u, static_cast<uint32_t>(nb16) * 16u);
      for (int kb = kb0; kb < kb1; ++kb) {
        const int i = kb - kb0, s = i % kStages;
        if (!mbar_wait(full_bar(s), static_cast<uint32_t>(i / kStages) & 1u, abort, p.status, 0x1200u + s)) break;
        tc_fence_after();
        const uint32_t sA = smem_u32(smem + s * S::kStageBytes), sB = sA + S::kABytes;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_i8(tmem, sdesc_k_sw128(sA + 32u * kk), sdesc_k_sw128(sB + 32u * kk), idesc, i > 0 || kk > 0 ? 1u : 0u);
        tc_commit(empty_bar(s));
      }
      tc_commit(done_bar);  // every MMA issued has completed, also after a wait that gave up
    }
    __syncwarp();
  }
  // all warps: the accumulator is complete, and with it every read of the ring
  const bool ready = mbar_wait(done_bar, 0u, abort, p.status, 0x1300u);
  if (!ready) mbar_wait_drain(done_bar, 0u);
  __syncthreads();
  tc_fence_after();
  int* part = reinterpret_cast<int*>(smem);  // [row][128 channels]
  if (warp >= 2) {
    const int q = warp & 3;
    for (int c = 0; c * 32 < n; ++c) {
      uint32_t v[32];
      tmem_ld32(tmem + (static_cast<uint32_t>(q * 32) << 16) + 32u * c, v);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (c * 32 + i < n) part[(c * 32 + i) * 128 + q * 32 + lane] = static_cast<int>(v[i]);
    }
  }
  tc_fence_before();
  cluster_sync();
  // this CTA's share of the rows, from all ranges of K: a warp per row, four channels a lane
  const int f = m0 + 4 * lane;
  float ws[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) ws[i] = f + i < p.N ? p.w_scale[f + i] : 0.0f;
  for (int j = rank + splits * warp; j < n; j += splits * 6) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    for (int r = 0; r < splits; ++r) {
      const uint4 u = ld_cluster_uint4(mapa_shared(smem_u32(part + j * 128 + 4 * lane), static_cast<uint32_t>(r)));
      v.x += u.x;
      v.y += u.y;
      v.z += u.z;
      v.w += u.w;
    }
    const float xs = p.x_scale[row0 + j];
    const float y[4] = {int8_sum(v.x) * (xs * ws[0]), int8_sum(v.y) * (xs * ws[1]),
                        int8_sum(v.z) * (xs * ws[2]), int8_sum(v.w) * (xs * ws[3])};
    TOut* out = static_cast<TOut*>(p.out) + (static_cast<int64_t>(row0) + j) * p.ldo + f;
    // four at once where the address allows it
    if (f + 4 <= p.N && (reinterpret_cast<uintptr_t>(out) & (4 * sizeof(TOut) - 1)) == 0) {
      if constexpr (sizeof(TOut) == 4) {
        *reinterpret_cast<float4*>(out) = make_float4(y[0], y[1], y[2], y[3]);
      } else {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(y[0], y[1]), hi = __floats2bfloat162_rn(y[2], y[3]);
        *reinterpret_cast<uint2*>(out) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (f + i < p.N) out[i] = from_f32<TOut>(y[i]);
    }
  }
  cluster_sync();  // nobody leaves while another CTA still reads its sums
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
}

}  // namespace muse
