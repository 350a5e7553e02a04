// dq_w8a8_linear for up to 8 tokens: the weights are read once, by all SMs, and
// everything else hides behind that.
//
// The products run with 16 weight rows along the matrix rows and the 8 tokens
// along its columns (m16n8k32, int32 sums), so a single token wastes no weight
// traffic. Each of the CTA's four warps keeps a ring of those rows, copied in runs
// of kFewRun bytes (one bulk copy per row and stage: memory serves long runs at
// almost twice the rate of 64-byte pieces loaded straight into registers), and
// takes every fourth run of K. The contracted index may be taken in any order that
// both operands share, so a lane (g = lane / 4, t = lane % 4) reads 16-byte pieces of
// the rows g and g + 8 (piece t of every 64 bytes) as its A operand, every byte
// where it lands. The tokens' codes are staged beside it, a chunk of K at a time.
// The warps' int32 parts are exact in any order.
// 1 x 4096 x 4096 takes 5.7 us (2.6 us to read the weights, about 2.2 for a launch);
// 5.8 with runs of 512 bytes, 7.8 with 1024, 7.2 with four stages of 256, 8.9 with
// three stages of 512. Every wait is bounded; a sum that misses a copy becomes NaN.
#pragma once

#include "decoder_device.cuh"
#include "dq_launch.cuh"
#include "tma_pipeline.cuh"
#include "w8a8_epilogue.cuh"

namespace dq {

constexpr int kFewWarps = 4, kFewThreads = kFewWarps * 32;
constexpr int kFewStages = 2;
constexpr int kFewTokens = 8, kFewRows = 16;
constexpr int kFewRun = 512;                              // bytes of K per weight row and stage
constexpr int kFewRowPitch = kFewRun + 64;                // two rows' 64-byte pieces fall into different banks
constexpr int kFewStage = kFewRows * kFewRowPitch;        // one warp's stage
constexpr int kFewChunk = kFewRun * kFewWarps;            // bytes of K per token and stage, all warps
constexpr int kFewTokenPitch = kFewChunk + 64;
constexpr int kFewTokenStage = kFewTokens * kFewTokenPitch;
constexpr int kFewSumPitch = kFewRows + 4;                // int32 parts [warp][token][row]
constexpr int kFewBody = kFewWarps * kFewStages * kFewStage + 2 * kFewTokenStage;
constexpr size_t kFewSmem = size_t(kFewBody) + kFewTokens * 4 + kFewWarps * kFewStages * 8 + 16;

template <int ACT>
__global__ void __launch_bounds__(kFewThreads) w8a8_linear_few_kernel(const LinearArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* rings = smem;  // weights [warp][stage][row], then tokens [2][token]; later the sums
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kFewBody);
  float* s_scale = reinterpret_cast<float*>(bars + kFewWarps * kFewStages);
  volatile uint32_t* failed = reinterpret_cast<uint32_t*>(s_scale + kFewTokens);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * kFewRows;
  const int tokens = static_cast<int>(a.m);
  const int chunks = static_cast<int>((a.k + kFewChunk - 1) / kFewChunk);

  uint64_t* bar = bars + warp * kFewStages;
  if (lane < kFewStages) mbar_init(bar + lane, 1);
  if (threadIdx.x == 0) *failed = 0u;
  fence_mbarrier_init();
  __syncwarp();
  pdl_launch_dependents();
  pdl_wait_primary();

  // The warp's runs of one chunk: one row per lane (rows past n repeat the last
  // one). Past k nothing is copied: the tokens are zero there.
  const int64_t row = n0 + lane;
  const int8_t* lane_row = a.b + (row < a.n ? row : a.n - 1) * a.k;
  const uint32_t ring = smem_addr(rings) + warp * kFewStages * kFewStage;
  const uint64_t policy = l2_evict_first_policy();
  const auto run_bytes = [&](int chunk) -> int {
    const int64_t left = a.k - (static_cast<int64_t>(chunk) * kFewChunk + warp * kFewRun);
    return chunk >= chunks || left <= 0 ? 0 : (left < kFewRun ? static_cast<int>(left) : kFewRun);
  };
  int issued = 0;     // chunks whose copies have been issued
  bool alive = true;  // no copy has failed to come
  const auto issue = [&](int chunk, int st) {
    const int bytes = run_bytes(chunk);
    if (bytes == 0 || !alive) return;
    issued = chunk + 1;
#ifdef DQ_TEST_SKIP_LINEAR_CHUNK
    // test builds only: leave one warp's run out, so that the bounded wait runs out
    if (blockIdx.x == 1 && warp == 2 && chunk == DQ_TEST_SKIP_LINEAR_CHUNK) return;
#endif
    if (lane == 0) mbar_arrive_expect_tx(bar + st, kFewRows * bytes);
    __syncwarp();
    if (lane < kFewRows)
      bulk_copy_g2s(rings + (warp * kFewStages + st) * kFewStage + lane * kFewRowPitch,
                    lane_row + static_cast<int64_t>(chunk) * kFewChunk + warp * kFewRun, bytes, bar + st, policy);
  };
  // the tokens' codes of one chunk, zeros past m and past k
  const uint32_t tokens0 = smem_addr(rings) + kFewWarps * kFewStages * kFewStage;
  const auto stage = [&](int chunk, int buffer) {
    if (chunk < chunks) {
      for (int i = threadIdx.x; i < kFewTokens * (kFewChunk / 16); i += kFewThreads) {
        const int tok = i / (kFewChunk / 16), piece = i % (kFewChunk / 16);
        const int64_t k = static_cast<int64_t>(chunk) * kFewChunk + 16 * piece;
        const int bytes = tok < tokens && k < a.k ? 16 : 0;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tokens0 + buffer * kFewTokenStage +
                                                                             tok * kFewTokenPitch + 16 * piece),
                     "l"(a.a + (bytes ? tok * a.k + k : 0)), "r"(bytes)
                     : "memory");
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kFewStages; ++i) issue(i, i);
  stage(0, 0);
  const int quad = threadIdx.x % 4, line = threadIdx.x / 4;  // the epilogue's columns and token
  const Columns cols(a, line < tokens ? n0 + 4 * quad : a.n);
  if (threadIdx.x < tokens) s_scale[threadIdx.x] = a.a_scale[threadIdx.x];

  int acc[4] = {0, 0, 0, 0};
  int st = 0;
  uint32_t filled = 0u;  // bit st: parity of stage st's next completion
  for (int chunk = 0; chunk < chunks; ++chunk) {
    const int buffer = chunk & 1;
    stage(chunk + 1, buffer ^ 1);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncthreads();
    const int bytes = run_bytes(chunk);
    if (bytes > 0) {
      if (chunk >= issued || !__all_sync(0xffffffffu, mbar_wait_parity(bar + st, (filled >> st) & 1u))) {
        *failed = 1u;
        alive = false;
      }
      filled ^= 1u << st;
      const uint32_t wx = ring + st * kFewStage + g * kFewRowPitch + 16 * t;
      const uint32_t tx = tokens0 + buffer * kFewTokenStage + g * kFewTokenPitch + warp * kFewRun + 16 * t;
#pragma unroll
      for (int s = 0; s < kFewRun / 64; ++s) {
        if (64 * s < bytes) {
          uint32_t x0[4], x1[4], y[4];
          load_piece<16>(x0, wx + 64 * s);
          load_piece<16>(x1, wx + 8 * kFewRowPitch + 64 * s);
          load_piece<16>(y, tx + 64 * s);
          mma_s8(acc, x0[0], x1[0], x0[1], x1[1], y[0], y[1]);
          mma_s8(acc, x0[2], x1[2], x0[3], x1[3], y[2], y[3]);
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

  int* sums = reinterpret_cast<int*>(rings);
#pragma unroll
  for (int c = 0; c < 4; ++c)
    sums[(warp * kFewTokens + 2 * t + (c & 1)) * kFewSumPitch + g + 8 * (c >> 1)] = acc[c];
  __syncthreads();
  if (line < tokens) {
    const uint4 res = cols.residual(a, line);
    int4 sum = make_int4(0, 0, 0, 0);
#pragma unroll
    for (int x = 0; x < kFewWarps; ++x) {
      const int4 v = *reinterpret_cast<const int4*>(sums + (x * kFewTokens + line) * kFewSumPitch + 4 * quad);
      sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
    }
    cols.template finish<ACT>(a, line, s_scale[line], sum, res, *failed != 0u);
  }
}

}  // namespace dq
