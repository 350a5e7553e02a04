// tcgen05 building blocks of the int8 products: descriptors, MMA, TMA tiles,
// TMEM reads and the bounded waits around them.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "tensor_map.cuh"
#include "tma_pipeline.cuh"

namespace dq {

// Instruction descriptor of tcgen05.mma kind::i8 for an M x N tile:
// int32 accumulator (format 2), signed A and B (format 1), both K-major,
// N / 8 and M / 16.
constexpr uint32_t i8_idesc(int n, int m = 128) {
  return (2u << 4) | (1u << 7) | (1u << 10) | (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24);
}

// ---------------------------------------------------------------- clusters

// A word at the same place in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t load_word(uint32_t at, int rank) {
  uint32_t v;
  asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(at) : "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ---------------------------------------------------------------- tcgen05 helpers

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Shared-memory matrix descriptor of a K-major tile in the 128-byte swizzle
// layout: rows of 128 bytes, groups of 8 rows 1024 bytes apart (stride byte
// offset 1024; the leading byte offset is 1 for swizzled K-major tiles),
// descriptor version 1, layout type 2 (128-byte swizzle).
__device__ __forceinline__ uint64_t smem_desc_k_sw128(const void* tile) {
  const uint64_t start = (smem_addr(tile) >> 4) & 0x3FFFu;
  return start | (uint64_t(1) << 16) | (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

// The same for the 64-byte swizzle layout: rows of 64 bytes, groups of 8
// rows 512 bytes apart, layout type 4.
__device__ __forceinline__ uint64_t smem_desc_k_sw64(const void* tile) {
  const uint64_t start = (smem_addr(tile) >> 4) & 0x3FFFu;
  return start | (uint64_t(1) << 16) | (uint64_t(512 >> 4) << 32) | (uint64_t(1) << 46) | (uint64_t(4) << 61);
}

__device__ __forceinline__ void tc_mma_i8(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(tmem_d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
      ::"r"(smem_addr(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_addr(bar))
      : "memory");
}

// A kernel parameter's tensor map into the descriptor cache.
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// 32 consecutive 32-bit TMEM columns of this thread's lane.
__device__ __forceinline__ void tc_ld_32cols(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// ---------------------------------------------------------------- bounded waits

__device__ __forceinline__ bool wait_or_abort_for(uint64_t* bar, uint32_t parity, const volatile uint32_t* abort,
                                                  uint64_t limit_ns) {
  const uint32_t addr = smem_addr(bar);
  if (mbar_try_wait(addr, parity)) return true;
  const uint64_t t0 = global_ns();
  while (true) {
    if (mbar_try_wait(addr, parity)) return true;
    if (*abort != 0u || global_ns() - t0 > limit_ns) return false;
  }
}

// Wait for an accumulator that the MMA lane is still building: gives up only
// after kWaitLimitNs without the lane's stage counter `progress` moving (or
// on the abort flag), so a long K loop that keeps moving is never cut off,
// while a stuck one ends within the limit.
__device__ __forceinline__ bool wait_while_progress(uint64_t* bar, uint32_t parity, const volatile uint32_t* abort,
                                                    const volatile uint32_t* progress) {
  const uint32_t addr = smem_addr(bar);
  if (mbar_try_wait(addr, parity)) return true;
  uint64_t t0 = global_ns();
  uint32_t seen = *progress;
  while (true) {
    if (mbar_try_wait(addr, parity)) return true;
    if (abort != nullptr && *abort != 0u) return false;
    const uint32_t now_seen = *progress;
    const uint64_t now = global_ns();
    if (now_seen != seen) {
      seen = now_seen;
      t0 = now;
    } else if (now - t0 > kWaitLimitNs) {
      return false;
    }
  }
}

}  // namespace dq

namespace dq_host {

// [rows, k] int8, k contiguous: 128-byte x box_rows boxes, 128-byte swizzle.
// Boxes of box_k bytes of K (128: 128-byte swizzle, 64: 64-byte swizzle) by
// box_rows rows.
inline bool make_map(CUtensorMap* map, const void* base, int64_t rows, int64_t k, uint32_t box_rows, uint32_t box_k = 128) {
  EncodeTiledFn fn = encode_tiled();
  if (fn == nullptr) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(k), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(k)};  // bytes between rows
  const cuuint32_t box[2] = {box_k, box_rows};
  const cuuint32_t estride[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estride,
            CU_TENSOR_MAP_INTERLEAVE_NONE, box_k == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace dq_host
