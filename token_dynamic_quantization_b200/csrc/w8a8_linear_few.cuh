// dq_w8a8_linear for few tokens: the weights are read once, by all SMs, and
// everything else hides behind that.
//
// The products run with the weight rows along the matrix rows and the tokens
// along its 8 columns (m16n8k32, int32 sums): 8 tokens waste nothing. The
// contracted index may be taken in any order that both operands share, so a lane
// (g = lane / 4, t = lane % 4) loads 16-byte pieces of the rows g and g + 8 (piece t
// of every 64 bytes) straight from global memory into the A operand's registers,
// each byte used where it lands. The tokens' codes, shared by all warps of the
// CTA, are staged in shared memory, a chunk of K at a time.
//
// K is split over the CTAs of a cluster (and over the warps of a CTA when there
// are few tokens), so that short n still fills the SMs; the int32 parts are
// summed through the cluster's shared memory, exact in any order.
#pragma once

#include "dq_launch.cuh"
#include "tma_pipeline.cuh"
#include "w8a8_epilogue.cuh"

namespace dq {

#ifndef PF
#define PF 1
#endif
#ifndef RING
#define RING 100
#endif
constexpr int kFewWarps = 8, kFewThreads = kFewWarps * 32;
constexpr int kFewAhead = 4;                // K steps of 64 bytes in flight per warp

// NT: tiles of 8 tokens; KW: warps that share a 16-row set and split K.
template <int NT, int KW>
struct FewShape {
  static constexpr int kSets = kFewWarps / KW;  // 16-row sets per CTA
  static constexpr int kRows = 16 * kSets;
  static constexpr int kTokens = 8 * NT;
  static constexpr int kSteps = KW == 1 ? 8 : 4;     // K steps per warp and chunk, a multiple of kFewAhead
  static constexpr int kChunk = 64 * KW * kSteps;    // bytes of K staged at a time
  static constexpr int kPitch = kChunk + 64;         // two tokens' 64-byte pieces fall into different banks
  static constexpr int kStage = kTokens * kPitch;
  static constexpr int kSums = kTokens * (kRows + 4) * 4 * KW;  // int32 parts, rows padded
  static constexpr size_t kSmem = size_t(2 * kStage > kSums ? 2 * kStage : kSums);
};

__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// `bytes` from p on (both multiples of 16) into L2.
__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int ACT, int NT, int KW>
__global__ void __launch_bounds__(kFewThreads, 2) w8a8_linear_few_kernel(const LinearArgs a, const int split) {
  using Shape = FewShape<NT, KW>;
  constexpr int kChunk = Shape::kChunk, kPitch = Shape::kPitch, kSteps = Shape::kSteps;
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int set = warp / KW, kw = warp % KW;
  // grid.x: row blocks x cluster ranks (K parts); grid.y: token blocks
  const int part = static_cast<int>(blockIdx.x) % split;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x / split) * Shape::kRows;
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * Shape::kTokens;
  const int chunks = static_cast<int>((a.k + kChunk - 1) / kChunk);
  const int chunk0 = chunks * part / split, chunk1 = chunks * (part + 1) / split;

  pdl_launch_dependents();
  // this CTA's weights on their way into L2 while the previous kernel ends: a
  // prefetch returns nothing, and L2 is where that kernel's writes are seen
  if (PF && threadIdx.x < Shape::kRows && n0 + threadIdx.x < a.n) {
    const int64_t k0 = static_cast<int64_t>(chunk0) * kChunk;
    const int64_t k1 = static_cast<int64_t>(chunk1) * kChunk < a.k ? static_cast<int64_t>(chunk1) * kChunk : a.k;
    prefetch_l2(a.b + (n0 + threadIdx.x) * a.k + k0, static_cast<uint32_t>(k1 - k0));
  }

  // weight rows g and g + 8 of the warp's set; rows past n repeat the last one
  const int64_t last = a.n - 1;
  const int64_t row0 = n0 + 16 * set + g;
  const int8_t* w0 = a.b + (row0 < last ? row0 : last) * a.k + 16 * t;
  const int8_t* w1 = a.b + (row0 + 8 < last ? row0 + 8 : last) * a.k + 16 * t;
  // this warp's K steps: kw, kw + KW, ... of the CTA's range, 64 bytes each
  const int64_t k_end = static_cast<int64_t>(chunk1) * kChunk < a.k ? static_cast<int64_t>(chunk1) * kChunk : a.k;
  int64_t k_next = static_cast<int64_t>(chunk0) * kChunk + 64 * kw;
  uint4 wr[kFewAhead][2];
  const auto fetch = [&](uint4(&x)[2]) {
    const bool in = k_next + 16 * t < k_end;
    x[0] = in ? ld_stream_16(reinterpret_cast<const uint4*>(w0 + k_next)) : make_uint4(0u, 0u, 0u, 0u);
    x[1] = in ? ld_stream_16(reinterpret_cast<const uint4*>(w1 + k_next)) : make_uint4(0u, 0u, 0u, 0u);
    k_next += 64 * KW;
  };

  // the tokens' codes of one chunk into a stage; tokens past m repeat the last one
  const uint32_t stage0 = smem_addr(smem);
  const auto stage = [&](int chunk, int buffer) {
    if (chunk < chunk1) {
      for (int i = threadIdx.x; i < Shape::kTokens * (kChunk / 16); i += kFewThreads) {
        const int tok = i / (kChunk / 16), piece = i % (kChunk / 16);
        const int64_t m = m0 + tok < a.m ? m0 + tok : a.m - 1;
        const int64_t k = static_cast<int64_t>(chunk) * kChunk + 16 * piece;
        const int bytes = k < a.k ? 16 : 0;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(stage0 + buffer * Shape::kStage + tok * kPitch +
                                                                             16 * piece),
                     "l"(a.a + m * a.k + (bytes ? k : 0)), "r"(bytes)
                     : "memory");
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  int acc[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0;

  pdl_wait_primary();
#pragma unroll
  for (int i = 0; i < kFewAhead; ++i) fetch(wr[i]);
  stage(chunk0, 0);
  for (int chunk = chunk0; chunk < chunk1; ++chunk) {
    const int buffer = (chunk - chunk0) & 1;
    stage(chunk + 1, buffer ^ 1);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncthreads();
    const uint32_t base = stage0 + buffer * Shape::kStage + g * kPitch + 16 * t + 64 * kw;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      uint4(&w)[2] = wr[s % kFewAhead];
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        uint32_t x0, x1, x2, x3;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(x0), "=r"(x1), "=r"(x2), "=r"(x3)
                     : "r"(base + i * 8 * kPitch + s * 64 * KW));
        mma_s8(acc[i], w[0].x, w[1].x, w[0].y, w[1].y, x0, x1);
        mma_s8(acc[i], w[0].z, w[1].z, w[0].w, w[1].w, x2, x3);
      }
      fetch(w);
    }
    __syncthreads();  // the stage is read; the next but one chunk goes there
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();

  // int32 parts to shared memory: [kw][token][row]
  int* sums = reinterpret_cast<int*>(smem);
  constexpr int kRowPitch = Shape::kRows + 4;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      sums[(kw * Shape::kTokens + 8 * i + 2 * t + (c & 1)) * kRowPitch + 16 * set + g + 8 * (c >> 1)] = acc[i][c];
  }
  if (split > 1) {
    cluster_barrier();
  } else {
    __syncthreads();
  }
  // each CTA of the cluster finishes every split-th token
  const int rank = part;
  const int mine = Shape::kTokens / split > 0 ? (Shape::kTokens + split - 1 - rank) / split : (rank < Shape::kTokens ? 1 : 0);
  const bool has_bias = a.bias != nullptr;
  for (int i = threadIdx.x; i < mine * Shape::kRows; i += kFewThreads) {
    const int tok = (i / Shape::kRows) * split + rank, row = i % Shape::kRows;
    const int64_t m = m0 + tok, n = n0 + row;
    if (m >= a.m || n >= a.n) continue;
    int sum = 0;
    const uint32_t at = smem_addr(sums) + (tok * kRowPitch + row) * 4;
    for (int r = 0; r < split; ++r) {
      uint32_t remote = at;
      if (split > 1) asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(at), "r"(r));
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        int v;
        if (split > 1) {
          asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(remote + w * Shape::kTokens * kRowPitch * 4) : "memory");
        } else {
          v = sums[(w * Shape::kTokens + tok) * kRowPitch + row];
        }
        sum += v;
      }
    }
    float x = linear_value<ACT>(sum, a.a_scale[m], a.b_scale[n], has_bias ? load_param(a.bias, a.bias_dtype, n) : 0.0f,
                                has_bias);
    const int64_t e = m * a.n + n;
    if (a.residual != nullptr) x = __fadd_rn(x, load_out(a.residual, a.out_kind, e));
    store_one(a.out, a.out_kind, e, x);
  }
  if (split > 1) cluster_barrier();  // no CTA leaves while its parts are being read
}

}  // namespace dq
