// dq_w8a8_linear for few tokens: the weights are read once, by all SMs, and
// everything else hides behind that.
//
// The products run with the weight rows along the matrix rows and the tokens
// along its 8 columns (m16n8k32, int32 sums): 8 tokens waste nothing. A warp
// keeps a ring of its own weight rows, copied row by row in runs of kRun bytes
// (one bulk copy each: memory serves long runs at almost twice the rate of
// 64-byte pieces loaded straight into registers). The contracted index may be
// taken in any order that both operands share, so a lane (g = lane / 4,
// t = lane % 4) reads 16-byte pieces of the rows g and g + 8 (piece t of every 64
// bytes) as its A operand, every byte where it lands. The tokens' codes, shared
// by all warps of the CTA, are staged beside it, a chunk of K at a time.
//
// KW warps share their rows and split K, as do the CTAs of a cluster where the
// rows are few; the int32 parts are exact in any order.
// Every wait is bounded; a sum that misses a copy becomes NaN.
#pragma once

#include "dq_launch.cuh"
#include "tma_pipeline.cuh"
#include "w8a8_epilogue.cuh"

namespace dq {

#ifndef FEW_STAGES
#define FEW_STAGES 2
#endif
#ifndef FEW_RUN1
#define FEW_RUN1 512
#endif
#ifndef FEW_RUN2
#define FEW_RUN2 256
#endif
#ifndef FEW_RS2
#define FEW_RS2 2
#endif
#ifndef FEW_KW2
#define FEW_KW2 4
#endif
constexpr int kFewWarps = 4, kFewThreads = kFewWarps * 32;
constexpr int kFewStages = FEW_STAGES;

// NT: tiles of 8 tokens; RS: sets of 16 weight rows per warp (a token piece read
// from shared memory serves them all); KW: warps that share their rows and split K.
template <int NT, int RS, int KW>
struct FewShape {
  static constexpr int kRows = 16 * RS * (kFewWarps / KW);  // per CTA
  static constexpr int kTokens = 8 * NT;
  static constexpr int kRun = RS == 1 ? FEW_RUN1 : FEW_RUN2;  // bytes of K per weight row and stage
  static constexpr int kRowPitch = kRun + 64;               // two rows' 64-byte pieces fall into different banks
  static constexpr int kStage = 16 * RS * kRowPitch;        // one warp's stage
  static constexpr int kChunk = kRun * KW;                  // bytes of K per token and stage, all warps
  static constexpr int kPitch = kChunk + 64;
  static constexpr int kTokenStage = kTokens * kPitch;
  static constexpr int kSumPitch = kRows + 4;
  static constexpr int kSums = kTokens * kSumPitch * 4 * KW;  // int32 parts [kw][token][row]
  static constexpr int kRings = kFewWarps * kFewStages * kStage + 2 * kTokenStage;
  static constexpr int kBody = kRings > kSums ? kRings : kSums;
  static constexpr size_t kSmem = size_t(kBody) + kTokens * 4 + kFewWarps * kFewStages * 8 + 16;
};

__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four int32 parts, of another CTA of the cluster or of this one.
__device__ __forceinline__ int4 load_part(uint32_t at, bool remote) {
  int4 v;
  if (remote) {
    asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  } else {
    asm volatile("ld.shared.v4.s32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  }
  return v;
}

// A word at the same place in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t load_word(uint32_t at, int rank) {
  uint32_t v;
  asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(at) : "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

__device__ __forceinline__ uint4 load_piece16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int ACT, int NT, int RS, int KW>
__global__ void __launch_bounds__(kFewThreads) w8a8_linear_few_kernel(const LinearArgs a, const int split) {
  using Shape = FewShape<NT, RS, KW>;
  constexpr int kRun = Shape::kRun, kChunk = Shape::kChunk, kPitch = Shape::kPitch;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* rings = smem;  // weights [warp][stage][row], then tokens [2][token]; later the sums
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Shape::kBody);
  float* s_scale = reinterpret_cast<float*>(bars + kFewWarps * kFewStages);
  volatile uint32_t* failed = reinterpret_cast<uint32_t*>(s_scale + Shape::kTokens);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int kw = warp % KW, set = warp / KW * RS;  // the warp's K share and first row set
  // grid.x: row blocks x cluster ranks (K parts); grid.y: token blocks
  const int part = static_cast<int>(blockIdx.x) % split;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x / split) * Shape::kRows;
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * Shape::kTokens;
  const int chunks = static_cast<int>((a.k + kChunk - 1) / kChunk);
  const int chunk0 = chunks * part / split, chunk1 = chunks * (part + 1) / split;

  uint64_t* bar = bars + warp * kFewStages;
  if (lane < kFewStages) mbar_init(bar + lane, 1);
  if (threadIdx.x == 0) *failed = 0u;
  fence_mbarrier_init();
  __syncwarp();
  pdl_launch_dependents();
  pdl_wait_primary();

  // The warp's runs of one chunk: one row per lane (rows past n repeat the last
  // one). Past k nothing is copied: the tokens are zero there.
  const int64_t row = n0 + 16 * set + lane;
  const int8_t* mine_row = a.b + (row < a.n ? row : a.n - 1) * a.k;
  const uint32_t ring = smem_addr(rings) + warp * kFewStages * Shape::kStage;
  const uint64_t policy = l2_evict_first_policy();
  const auto run_bytes = [&](int chunk) -> int {
    const int64_t left = a.k - (static_cast<int64_t>(chunk) * kChunk + kw * kRun);
    return chunk >= chunk1 || left <= 0 ? 0 : (left < kRun ? static_cast<int>(left) : kRun);
  };
  const auto issue = [&](int chunk, int st) {
    const int bytes = run_bytes(chunk);
    if (bytes == 0) return;
    if (lane == 0) mbar_arrive_expect_tx(bar + st, 16 * RS * bytes);
    __syncwarp();
    if (lane < 16 * RS)
      bulk_copy_g2s(rings + (warp * kFewStages + st) * Shape::kStage + lane * Shape::kRowPitch,
                    mine_row + static_cast<int64_t>(chunk) * kChunk + kw * kRun, bytes, bar + st, policy);
  };
  // the tokens' codes of one chunk, zeros past m and past k
  const uint32_t tokens0 = smem_addr(rings) + kFewWarps * kFewStages * Shape::kStage;
  const auto stage = [&](int chunk, int buffer) {
    if (chunk < chunk1) {
      for (int i = threadIdx.x; i < Shape::kTokens * (kChunk / 16); i += kFewThreads) {
        const int tok = i / (kChunk / 16), piece = i % (kChunk / 16);
        const int64_t k = static_cast<int64_t>(chunk) * kChunk + 16 * piece;
        const int bytes = m0 + tok < a.m && k < a.k ? 16 : 0;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tokens0 + buffer * Shape::kTokenStage + tok * kPitch +
                                                                             16 * piece),
                     "l"(a.a + (bytes ? (m0 + tok) * a.k + k : 0)), "r"(bytes)
                     : "memory");
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kFewStages; ++i) issue(chunk0 + i, i);
  stage(chunk0, 0);
  constexpr int kQuads = Shape::kRows / 4, kLines = kFewThreads / kQuads;
  const int quad = threadIdx.x % kQuads, line = threadIdx.x / kQuads;
  const Columns cols(a, n0 + 4 * quad);
  if (threadIdx.x < Shape::kTokens && m0 + threadIdx.x < a.m) s_scale[threadIdx.x] = a.a_scale[m0 + threadIdx.x];

  int acc[RS][NT][4];
#pragma unroll
  for (int r = 0; r < RS; ++r) {
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[r][i][0] = acc[r][i][1] = acc[r][i][2] = acc[r][i][3] = 0;
  }
  int st = 0;
  uint32_t filled = 0u;  // bit st: parity of stage st's next completion
  for (int chunk = chunk0; chunk < chunk1; ++chunk) {
    const int buffer = (chunk - chunk0) & 1;
    stage(chunk + 1, buffer ^ 1);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncthreads();
    const int bytes = run_bytes(chunk);
    if (bytes > 0) {
      if (!mbar_wait_parity(bar + st, (filled >> st) & 1u)) *failed = 1u;
      filled ^= 1u << st;
      const uint32_t wx = ring + st * Shape::kStage + g * Shape::kRowPitch + 16 * t;
      const uint32_t tx = tokens0 + buffer * Shape::kTokenStage + g * kPitch + kw * kRun + 16 * t;
#pragma unroll
      for (int s = 0; s < kRun / 64; ++s) {
        if (64 * s < bytes) {
          uint4 x[RS][2];
#pragma unroll
          for (int r = 0; r < RS; ++r) {
#pragma unroll
            for (int h = 0; h < 2; ++h) x[r][h] = load_piece16(wx + (16 * r + 8 * h) * Shape::kRowPitch + 64 * s);
          }
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            const uint4 y = load_piece16(tx + i * 8 * kPitch + 64 * s);
#pragma unroll
            for (int r = 0; r < RS; ++r) {
              mma_s8(acc[r][i], x[r][0].x, x[r][1].x, x[r][0].y, x[r][1].y, y.x, y.y);
              mma_s8(acc[r][i], x[r][0].z, x[r][1].z, x[r][0].w, x[r][1].w, y.z, y.w);
            }
          }
        }
      }
      __syncwarp();
      issue(chunk + kFewStages, st);
      st = st + 1 == kFewStages ? 0 : st + 1;
    }
    __syncthreads();  // the tokens are read; the next but one chunk goes there
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();

  // int32 parts to shared memory: [kw][token][row]
  int* sums = reinterpret_cast<int*>(rings);
#pragma unroll
  for (int r = 0; r < RS; ++r) {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        sums[(kw * Shape::kTokens + 8 * i + 2 * t + (c & 1)) * Shape::kSumPitch + 16 * (set + r) + g + 8 * (c >> 1)] = acc[r][i][c];
    }
  }
  // each CTA of the cluster finishes every split-th token, a thread four rows
  const int tokens = static_cast<int>(a.m - m0 < Shape::kTokens ? a.m - m0 : Shape::kTokens);
  const int mine = (tokens - part + split - 1) / split;
  if (split > 1) {
    cluster_barrier();
  } else {
    __syncthreads();
  }
  bool broken = *failed != 0u;
  for (int r = 0; split > 1 && r < split; ++r) broken |= load_word(smem_addr(const_cast<uint32_t*>(failed)), r) != 0u;
  for (int i = line; i < mine; i += kLines) {
    const int tok = i * split + part;
    const uint4 res = cols.residual(a, m0 + tok);
    int4 sum = make_int4(0, 0, 0, 0);
    const uint32_t at = smem_addr(sums) + (tok * Shape::kSumPitch + 4 * quad) * 4;
    for (int r = 0; r < split; ++r) {
      uint32_t remote = at;
      if (split > 1) asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(at), "r"(r));
#pragma unroll
      for (int x = 0; x < KW; ++x) {
        const int4 v = load_part(remote + x * Shape::kTokens * Shape::kSumPitch * 4, split > 1);
        sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
      }
    }
    cols.template finish<ACT>(a, m0 + tok, s_scale[tok], sum, res, broken);
  }
  if (split > 1) cluster_barrier();  // no CTA leaves while its parts are being read
}

}  // namespace dq
