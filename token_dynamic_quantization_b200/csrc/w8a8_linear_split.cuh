// dq_w8a8_linear for 9 to 128 tokens, on the tcgen05 tensor cores
// with the operands' roles exchanged: 128 weight rows along the accumulator's
// lanes, TOK tokens along its columns. The weights are read once whatever the
// number of tokens up to TOK, and the tensor cores take them from shared memory
// as they come.
//
// n / 128 tiles are few next to 148 SMs, so K is split over the CTAs of a
// cluster; each leaves its exact int32 part in its shared memory and every CTA
// finishes a share of the tokens from all of them.
//   warp 0      TMA producer: 128 bytes of K of the weight rows and the tokens
//   warp 1      TMEM allocation; one lane issues tcgen05.mma.kind::i8
//   warps 2-5   move the accumulator to shared memory, [token][row]
//               sum the parts, epilogue, stores along the rows
// Bound by reading the weights: 48 x 7168 x 8192 reads 59 MB, 9.2 us at the copy rate,
// and takes 20; about 7 of them are the launch, the allocation of TMEM (which keeps
// the next kernel's CTAs out until this one's leave) and the clusters' joining, and
// 56 tiles of 128 rows fill 112 of the 148 SMs in clusters of two.
// Every wait is bounded. A CTA whose sum is incomplete says so beside its part,
// and the tokens that need it become NaN.
#pragma once

#include "dq_launch.cuh"
#include "tcgen05_i8.cuh"
#include "w8a8_epilogue.cuh"

namespace dq {

constexpr int kSplitThreads = 192;

template <int TOK>
struct SplitShape {
  static constexpr uint32_t kA = 128 * 128, kB = TOK * 128;  // bytes of a stage: weight rows, tokens
  static constexpr uint32_t kStage = kA + kB;
  static constexpr int kStages = 200 * 1024 / kStage;        // one CTA per SM
  static constexpr int kPitch = 132;                         // int32 parts [token][row]: 16-byte rows, no conflicts
  static constexpr uint32_t kSums = TOK * kPitch * 4;
  static constexpr uint32_t kRing = kStages * kStage > kSums ? kStages * kStage : kSums;
  static constexpr size_t kSmem = 1024 + kRing + 256 + TOK * 4;
  static constexpr uint32_t kIdesc = i8_idesc(TOK);
  static constexpr uint32_t kCols = TOK < 32 ? 32 : TOK;     // TMEM columns
};

template <int ACT, int TOK>
__global__ void __launch_bounds__(kSplitThreads) w8a8_linear_split_kernel(const __grid_constant__ CUtensorMap map_w,
                                                                          const __grid_constant__ CUtensorMap map_x,
                                                                          const LinearArgs a, const int split) {
  using Shape = SplitShape<TOK>;
  constexpr int kStages = Shape::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Shape::kRing);
  uint64_t* empty = full + kStages;
  uint64_t* ready = empty + kStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ready + 1);
  volatile uint32_t* failed = tmem_slot + 1;
  volatile uint32_t* progress = tmem_slot + 2;
  float* s_scale = reinterpret_cast<float*>(smem + Shape::kRing + 256);  // the tokens' scales

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = static_cast<int>(blockIdx.x) % split;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x / split) * 128;
  const int slices = static_cast<int>((a.k + 127) / 128);
  const int s0 = static_cast<int>(static_cast<int64_t>(slices) * part / split);
  const int s1 = static_cast<int>(static_cast<int64_t>(slices) * (part + 1) / split);

  const auto load = [&](int i) {
    const int s = i % kStages;
#ifdef DQ_TEST_SKIP_LINEAR_CHUNK
    // test builds only: leave one slice out, so that the MMA lane's bounded wait runs out
    if (n0 == 128 && part == 0 && i == DQ_TEST_SKIP_LINEAR_CHUNK) return;
#endif
    mbar_arrive_expect_tx(full + s, Shape::kStage);
    uint8_t* at = smem + s * Shape::kStage;
    tma_load_2d(at, &map_w, (s0 + i) * 128, static_cast<int>(n0), full + s);
    tma_load_2d(at + Shape::kA, &map_x, (s0 + i) * 128, 0, full + s);
  };
  if (threadIdx.x == 0) {
    prefetch_map(&map_w);
    prefetch_map(&map_x);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    mbar_init(ready, 1);
    *failed = 0u;
    *progress = 0u;
    fence_mbarrier_init();
    // the ring fills while the accumulator is being allocated
    pdl_wait_primary();
    for (int i = 0; i < kStages && i < s1 - s0; ++i) load(i);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                 "r"(Shape::kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_launch_dependents();
  pdl_wait_primary();

  // what the epilogue (warps 2-5) needs of its four columns and of the tokens,
  // asked for now
  const int tokens = static_cast<int>(a.m);
  const Columns cols(a, warp < 2 ? a.n : n0 + 4 * lane);
  for (int i = static_cast<int>(threadIdx.x) - 64; i >= 0 && i < tokens; i += 128) s_scale[i] = a.a_scale[i];

  if (warp == 0) {
    if (lane == 0) {
      int issued = s1 - s0 < kStages ? s1 - s0 : kStages;
      for (; issued < s1 - s0; ++issued) {
        if (!mbar_wait_parity(empty + issued % kStages, ((issued / kStages) & 1u) ^ 1u)) break;
        load(issued);
      }
      // nothing may still be landing when the ring is used for the parts
      for (int i = issued > kStages ? issued - kStages : 0; i < issued; ++i) {
        mbar_wait_parity(full + i % kStages, (i / kStages) & 1u);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      for (int i = 0; i < s1 - s0; ++i) {
        const int s = i % kStages;
        if (!mbar_wait_parity(full + s, (i / kStages) & 1u)) {
          *failed = 1u;
          __threadfence_block();
          break;
        }
        tc_fence_after();
        const uint64_t wd = smem_desc_k_sw128(smem + s * Shape::kStage);
        const uint64_t xd = smem_desc_k_sw128(smem + s * Shape::kStage + Shape::kA);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) tc_mma_i8(tmem, wd + 2 * kk, xd + 2 * kk, Shape::kIdesc, (i | kk) != 0 ? 1u : 0u);
        tc_commit(empty + s);
        *progress = static_cast<uint32_t>(i + 1);
      }
      tc_commit(ready);  // arrives once every MMA above has completed
      if (!wait_while_progress(ready, 0, nullptr, progress)) *failed = 1u;
    }
    __syncwarp();
  } else {
    bool ok = wait_while_progress(ready, 0, nullptr, progress);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) *failed = 1u;
  }
  tc_fence_before();
  __syncthreads();  // the ring is free: every copy has landed and every MMA has read it
  tc_fence_after();
  int* sums = reinterpret_cast<int*>(smem);
  if (warp >= 2 && *failed == 0u) {
    const int quarter = warp & 3;
    constexpr int kStep = TOK < 32 ? TOK : 32;
#pragma unroll 1
    for (int c = 0; c < TOK; c += kStep) {
      uint32_t r[32];
      tc_ld_32cols(tmem + (static_cast<uint32_t>(32 * quarter) << 16) + static_cast<uint32_t>(c), r);
#pragma unroll
      for (int j = 0; j < kStep; ++j) sums[(c + j) * Shape::kPitch + 32 * quarter + lane] = static_cast<int>(r[j]);
    }
  }
  tc_fence_before();
  if (split > 1) {
    cluster_barrier();
  } else {
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(Shape::kCols) : "memory");
  }

  // each CTA of the cluster finishes every split-th token, four rows at a time
  const int mine = (tokens - part + split - 1) / split;
  bool broken = false;
  if (split == 1) broken = *failed != 0u;
  for (int r = 0; split > 1 && r < split; ++r) broken |= load_word(smem_addr(const_cast<uint32_t*>(failed)), r) != 0u;
  // kBatch tokens at a time: their residuals and parts are all asked for before
  // the first is used
  constexpr int kBatch = 8, kWarps = 4;
  for (int i0 = warp - 2; i0 >= 0 && i0 < mine; i0 += kBatch * kWarps) {
    int4 sum[kBatch];
    uint4 res[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int i = i0 + b * kWarps, tok = i * split + part;
      sum[b] = make_int4(0, 0, 0, 0);
      if (i < mine) {
        res[b] = cols.residual(a, tok);
        const uint32_t at = smem_addr(sums) + (tok * Shape::kPitch + 4 * lane) * 4;
        for (int r = 0; r < split; ++r) {
          int4 v;
          if (split > 1) {
            uint32_t remote;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(at), "r"(r));
            asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                         : "r"(remote)
                         : "memory");
          } else {
            v = *reinterpret_cast<const int4*>(sums + tok * Shape::kPitch + 4 * lane);
          }
          sum[b].x += v.x, sum[b].y += v.y, sum[b].z += v.z, sum[b].w += v.w;
        }
      }
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int i = i0 + b * kWarps, tok = i * split + part;
      if (i < mine) cols.template finish<ACT>(a, tok, s_scale[tok], sum[b], res[b], broken);
    }
  }
  if (split > 1) cluster_barrier();  // no CTA leaves while its part is being read
}

}  // namespace dq
