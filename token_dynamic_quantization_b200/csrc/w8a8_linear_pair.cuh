// dq_w8a8_linear for many tokens: tiles of 256 tokens by 256 weight rows, each
// by a pair of SMs (tcgen05 with cta_group::2).
//
// A single SM's 128 x 256 tile writes and reads 48 KB of operands per K slice
// of 128 bytes, more than shared memory moves while the tensor core works on
// it. A pair shares the weights: each SM holds its own 128 tokens and half of the
// weight rows, 32 KB a slice, and the tensor cores read the other half from the
// peer.
//
// Persistent: clusters of two CTAs walk a list of tiles; the last ones are halved
// (256 x 128) when that evens out the last wave. Roles per CTA:
//   warp 0      TMA producer: the CTA's tokens and its half of the weight rows;
//               the copies complete on the leader's barrier
//   warp 1      TMEM allocation; in the leader, one lane issues the MMAs for both
//               SMs and frees both SMs' stages with multicast commits
//   warps 2-9   epilogue of the CTA's 128 rows, two warps to a TMEM quarter; the
//               int32 accumulator is double-buffered in TMEM (2 x 256 columns), so
//               it overlaps the next tile's MMAs
// 4096^3 with bias, GELU and residual takes 66 us, 41 of them the products at twice the
// bf16 rate (the tensor pipe is active for half of a launch by itself, DRAM at 12 % of its
// peak), about 8 the residual, and the rest the
// start (7) and the last tiles' epilogue; without any of the three it takes 56, and
// 9472 x 4096 x 8192 runs at 3.2 POP/s.
// Every wait is bounded; after one has run out the CTA's remaining tiles become NaN.
#pragma once

#include "dq_launch.cuh"
#include "tcgen05_i8.cuh"
#include "w8a8_epilogue.cuh"

namespace dq {

constexpr int kPairEpilogueWarps = 8;
constexpr int kPairThreads = 64 + 32 * kPairEpilogueWarps;
constexpr uint32_t kPairA = 128 * 128, kPairB = 128 * 128;  // bytes of a stage in one CTA
constexpr uint32_t kPairStage = kPairA + kPairB;
constexpr uint32_t kPairCols = 512;
constexpr uint32_t kPairIdescWide = i8_idesc(256, 256), kPairIdescNarrow = i8_idesc(128, 256);
// Two epilogues. Where rows of the output (and residual) lie in 16-byte pieces and
// n is a multiple of 32, a lane finishes its own row, 32 columns at a time.
// Elsewhere (n odd, unaligned rows) each warp first turns 32 x 32 accumulator words in shared memory, at the
// price of one stage of the ring, and works along the rows: 1000 x 2051 x 1040 to
// binary32 takes 12.3 us that way and 17.5 with a row per lane, whose 4-byte stores
// scatter; but 4096^3 with everything takes 88 us against 67, for the extra
// instructions.
constexpr int kPairPitch = 34;
constexpr uint32_t kPairTurn = kPairEpilogueWarps * 32 * (kPairPitch + 1) * 4;  // the words, and the rows' scales
template <bool TURN>
struct PairShape {
  static constexpr int kStages = TURN ? 5 : 6;
  // ring, two buffers of 256 column scales and biases, the turned words, barriers
  static constexpr size_t kSmem = 1024 + kStages * kPairStage + 2 * 2 * 256 * 4 + (TURN ? kPairTurn : 0) + 256;
};

struct PairSched {
  int64_t n_tiles;  // 256-wide column tiles
  int64_t wide;     // list items that are whole tiles
  int64_t items;    // wide + 2 * (tiles split in two)
};

__device__ __forceinline__ void pair_item(const PairSched& ps, int64_t item, int64_t& m0, int64_t& n0, bool& wide) {
  wide = item < ps.wide;
  const int64_t t = wide ? item : ps.wide + (item - ps.wide) / 2, half = wide ? 0 : (item - ps.wide) & 1;
  m0 = t / ps.n_tiles * 256;
  n0 = t % ps.n_tiles * 256 + half * 128;
}

// A box into this CTA's shared memory, completing on a barrier of either CTA of
// the pair (`bar`: its address in the cluster's window).
__device__ __forceinline__ void tma_load_pair(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
      ::"r"(smem_addr(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void tc_mma_i8_pair(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(tmem_d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Arrives on the barrier at this place in both CTAs once every MMA issued so far
// has completed.
__device__ __forceinline__ void tc_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_addr(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr(p)), "r"(rank));
  return r;
}

// 32 columns of one output row from the accumulator's words, 16-byte rows.
template <int ACT>
__device__ __forceinline__ void finish_row32(const LinearArgs& a, int64_t row, int64_t c0, const uint32_t (&r)[32],
                                             const uint4 (&raw)[4], float sa, const float* scale, const float* bias) {
  const bool has_bias = a.bias != nullptr;
  const int64_t e = row * a.n + c0;
  const bool narrow = a.out_kind != kOutF32;
#pragma unroll
  for (int q = 0; q < 8; ++q) {  // four columns, two to an instruction
    const float4 sb = *reinterpret_cast<const float4*>(scale + 4 * q);
    float2 lo = make_float2(__int2float_rn(static_cast<int>(r[4 * q])), __int2float_rn(static_cast<int>(r[4 * q + 1])));
    float2 hi = make_float2(__int2float_rn(static_cast<int>(r[4 * q + 2])), __int2float_rn(static_cast<int>(r[4 * q + 3])));
    lo = __fmul2_rn(lo, __fmul2_rn(f2(sa), make_float2(sb.x, sb.y)));
    hi = __fmul2_rn(hi, __fmul2_rn(f2(sa), make_float2(sb.z, sb.w)));
    if (has_bias) {
      const float4 bb = *reinterpret_cast<const float4*>(bias + 4 * q);
      lo = __fadd2_rn(lo, make_float2(bb.x, bb.y));
      hi = __fadd2_rn(hi, make_float2(bb.z, bb.w));
    }
    float x[4] = {activate<ACT>(lo.x), activate<ACT>(lo.y), activate<ACT>(hi.x), activate<ACT>(hi.y)};
    if (narrow) {
      if (a.residual != nullptr) {
        const uint4 w = raw[q / 2];
        const float2 r0 = unpack2(q & 1 ? w.z : w.x, a.out_kind), r1 = unpack2(q & 1 ? w.w : w.y, a.out_kind);
        x[0] = __fadd_rn(x[0], r0.x), x[1] = __fadd_rn(x[1], r0.y), x[2] = __fadd_rn(x[2], r1.x), x[3] = __fadd_rn(x[3], r1.y);
      }
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + e + 4 * q) =
          make_uint2(pack2(x[0], x[1], a.out_kind), pack2(x[2], x[3], a.out_kind));
    } else {
      float* o = static_cast<float*>(a.out) + e + 4 * q;
      if (a.residual != nullptr) {
        const float4 w = *reinterpret_cast<const float4*>(static_cast<const float*>(a.residual) + e + 4 * q);
        x[0] = __fadd_rn(x[0], w.x), x[1] = __fadd_rn(x[1], w.y), x[2] = __fadd_rn(x[2], w.z), x[3] = __fadd_rn(x[3], w.w);
      }
      *reinterpret_cast<float4*>(o) = make_float4(x[0], x[1], x[2], x[3]);
    }
  }
}

// The two neighbouring columns of a lane in 16 rows of a chunk (rows 2i + lane / 16,
// columns 2 (lane % 16) and the next), as words of the residual.
struct PairResidual {
  uint32_t w[32];
};

// Where the lane's first element lies, how far its rows are apart, and what of it exists.
struct PairSpan {
  int64_t e;      // element of row lane / 16
  int rows;       // of the 16, how many lie before the end of out
  int columns;    // 0, 1 or 2
  bool paired;    // both columns in one access
};

__device__ __forceinline__ PairSpan pair_span(const LinearArgs& a, int64_t row0, int64_t c0, int lane) {
  PairSpan x;
  const int64_t row = row0 + (lane >> 4), col = c0 + 2 * (lane & 15);
  x.e = row * a.n + col;
  const int64_t left = a.m - row;
  x.rows = left <= 0 ? 0 : (left >= 32 ? 16 : static_cast<int>((left + 1) / 2));
  x.columns = col >= a.n ? 0 : (col + 2 <= a.n ? 2 : 1);
  x.paired = x.columns == 2 && a.pair_out;
  return x;
}

__device__ __forceinline__ void ask_residual(const LinearArgs& a, const PairSpan& x, PairResidual& r) {
  if (a.residual == nullptr || x.columns == 0) return;
  const int64_t step = 2 * a.n;
  if (a.out_kind == kOutF32) {
    const uint32_t* p = static_cast<const uint32_t*>(a.residual) + x.e;
#pragma unroll
    for (int i = 0; i < 16; ++i, p += step) {
      if (i < x.rows) {
        if (x.paired) {
          const uint2 v = *reinterpret_cast<const uint2*>(p);
          r.w[2 * i] = v.x;
          r.w[2 * i + 1] = v.y;
        } else {
          r.w[2 * i] = p[0];
          r.w[2 * i + 1] = x.columns == 2 ? p[1] : 0u;
        }
      }
    }
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(a.residual) + x.e;
#pragma unroll
    for (int i = 0; i < 16; ++i, p += step) {
      if (i < x.rows) {
        if (x.paired) {
          r.w[i] = *reinterpret_cast<const uint32_t*>(p);
        } else {
          r.w[i] = p[0] | (x.columns == 2 ? static_cast<uint32_t>(p[1]) << 16 : 0u);
        }
      }
    }
  }
}

// The lane's 16 x 2 outputs of a chunk whose words lie in `turn`, rows' scales behind them.
template <int ACT>
__device__ __forceinline__ void finish_chunk(const LinearArgs& a, const PairSpan& x, const PairResidual& r, const int* turn,
                                             float2 scale, float2 bias, int lane) {
  if (x.columns == 0) return;
  const float* row_scale = reinterpret_cast<const float*>(turn + 32 * kPairPitch);
  const bool has_bias = a.bias != nullptr, has_residual = a.residual != nullptr;
  int64_t e = x.e;
#pragma unroll
  for (int i = 0; i < 16; ++i, e += 2 * a.n) {
    const int row = 2 * i + (lane >> 4);
    const int2 acc = *reinterpret_cast<const int2*>(turn + row * kPairPitch + 2 * (lane & 15));
    float2 v = __fmul2_rn(make_float2(__int2float_rn(acc.x), __int2float_rn(acc.y)), __fmul2_rn(f2(row_scale[row]), scale));
    if (has_bias) v = __fadd2_rn(v, bias);
    v = make_float2(activate<ACT>(v.x), activate<ACT>(v.y));
    if (a.out_kind == kOutF32) {
      if (has_residual) v = __fadd2_rn(v, make_float2(__uint_as_float(r.w[2 * i]), __uint_as_float(r.w[2 * i + 1])));
      if (i < x.rows) {
        float* o = static_cast<float*>(a.out) + e;
        if (x.paired) {
          *reinterpret_cast<float2*>(o) = v;
        } else {
          o[0] = v.x;
          if (x.columns == 2) o[1] = v.y;
        }
      }
    } else {
      if (has_residual) v = __fadd2_rn(v, unpack2(r.w[i], a.out_kind));
      const uint32_t w = pack2(v.x, v.y, a.out_kind);
      if (i < x.rows) {
        uint16_t* o = static_cast<uint16_t*>(a.out) + e;
        if (x.paired) {
          *reinterpret_cast<uint32_t*>(o) = w;
        } else {
          o[0] = static_cast<uint16_t>(w);
          if (x.columns == 2) o[1] = static_cast<uint16_t>(w >> 16);
        }
      }
    }
  }
}

template <int ACT, bool TURN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    w8a8_linear_pair_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b128,
                            const __grid_constant__ CUtensorMap map_b64, const LinearArgs a, const PairSched ps) {
  constexpr int kPairStages = PairShape<TURN>::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* col_scale = reinterpret_cast<float*>(smem + kPairStages * kPairStage);  // [2][256]
  float* col_bias = col_scale + 2 * 256;                                         // [2][256]
  int* turns = reinterpret_cast<int*>(col_bias + 2 * 256);                       // [warps][32 * (kPairPitch + 1)]
  uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(turns) + (TURN ? kPairTurn : 0));  // the leader's are used
  uint64_t* empty = full + kPairStages;
  uint64_t* acc_full = empty + kPairStages;  // [2]
  uint64_t* acc_empty = acc_full + 2;        // [2], the leader's are used
  uint64_t* mma_done = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile uint32_t* abort_flag = tmem_slot + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t rank;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const int64_t first_item = blockIdx.x / 2, step = gridDim.x / 2;
  const int slices = static_cast<int>((a.k + 127) / 128);

  if (threadIdx.x == 0) {
    prefetch_map(&map_a);
    prefetch_map(&map_b128);
    prefetch_map(&map_b64);
    for (int s = 0; s < kPairStages; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full + b, 1);
      mbar_init(acc_empty + b, 2 * kPairEpilogueWarps);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0u;
    fence_mbarrier_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                 "r"(kPairCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_barrier();  // both CTAs' barriers exist before either touches the other's
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_launch_dependents();
  pdl_wait_primary();

  if (warp == 0) {
    if (lane == 0) {
      uint32_t slice = 0;
      bool ok = true;
      for (int64_t item = first_item; ok && item < ps.items; item += step) {
        int64_t m0, n0;
        bool wide;
        pair_item(ps, item, m0, n0, wide);
        const int rows_b = wide ? 128 : 64;  // this CTA's half of the weight rows
        const CUtensorMap* map_b = wide ? &map_b128 : &map_b64;
        for (int kt = 0; kt < slices; ++kt, ++slice) {
          const uint32_t s = slice % kPairStages;
          if (!wait_or_abort_for(empty + s, ((slice / kPairStages) & 1u) ^ 1u, abort_flag, kWaitLimitNs)) {
            *abort_flag = 1u;
            ok = false;
            break;
          }
#ifdef DQ_TEST_SKIP_LINEAR_CHUNK
          // test builds only: leave one slice out, so that the MMA lane's bounded wait runs out
          if (m0 == 256 && n0 == 0 && kt == DQ_TEST_SKIP_LINEAR_CHUNK) continue;
#endif
          if (rank == 0) mbar_arrive_expect_tx(full + s, 2 * (kPairA + rows_b * 128));
          const uint32_t bar = cluster_addr(full + s, 0);
          uint8_t* at = smem + s * kPairStage;
          tma_load_pair(at, &map_a, kt * 128, static_cast<int>(m0 + 128 * rank), bar);
          tma_load_pair(at + kPairA, map_b, kt * 128, static_cast<int>(n0 + rows_b * rank), bar);
        }
      }
      // no copy of either CTA may still be landing when the pair exits
      if (rank == 0) {
        for (uint32_t j = slice > kPairStages ? slice - kPairStages : 0; j < slice; ++j)
          mbar_wait_parity(full + j % kPairStages, (j / kPairStages) & 1u);
      }
      // nor an arrival of the leader's commits that frees a stage
      for (uint32_t j = slice > kPairStages ? slice - kPairStages : 0; ok && j < slice; ++j)
        ok = wait_or_abort_for(empty + j % kPairStages, (j / kPairStages) & 1u, abort_flag, kWaitLimitNs);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      uint32_t slice = 0;
      bool ok = true;
      int i = 0;
      for (int64_t item = first_item; ok && item < ps.items; item += step, ++i) {
        int64_t m0, n0;
        bool wide;
        pair_item(ps, item, m0, n0, wide);
        const int acc = i & 1;
        if (!wait_or_abort_for(acc_empty + acc, ((i >> 1) & 1) ^ 1u, abort_flag, kWaitLimitNs)) {
          *abort_flag = 1u;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + static_cast<uint32_t>(acc * 256);
        const uint32_t idesc = wide ? kPairIdescWide : kPairIdescNarrow;
        for (int kt = 0; kt < slices; ++kt, ++slice) {
          const uint32_t s = slice % kPairStages;
          if (!wait_or_abort_for(full + s, (slice / kPairStages) & 1u, abort_flag, kWaitLimitNs)) {
            *abort_flag = 1u;
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t ad = smem_desc_k_sw128(smem + s * kPairStage);
          const uint64_t bd = smem_desc_k_sw128(smem + s * kPairStage + kPairA);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) tc_mma_i8_pair(d, ad + 2 * kk, bd + 2 * kk, idesc, (kt | kk) != 0 ? 1u : 0u);
          tc_commit_pair(empty + s);
        }
        if (ok) tc_commit_pair(acc_full + acc);
      }
      // both CTAs wait for it below: the TMEM is freed, and a CTA's barriers go, only after
      // every MMA issued has completed
      tc_commit_pair(mma_done);
    }
    __syncwarp();
  } else {
    const int ew = warp - 2, quarter = warp & 3, half = ew >> 2;  // two warps per quarter, each half of the columns
    const int et = threadIdx.x - 64;
    bool dead = false;
    int i = 0;
    for (int64_t item = first_item; item < ps.items; item += step, ++i) {
      int64_t m0, n0;
      bool wide;
      pair_item(ps, item, m0, n0, wide);
      const int bn = wide ? 256 : 128;
      const int acc = i & 1;
      float* scale = col_scale + acc * 256;
      float* bias = col_bias + acc * 256;
      for (int j = et; j < bn; j += 32 * kPairEpilogueWarps) {
        const bool in = n0 + j < a.n;
        scale[j] = in ? a.b_scale[n0 + j] : 0.0f;
        bias[j] = in && a.bias != nullptr ? load_param(a.bias, a.bias_dtype, n0 + j) : 0.0f;
      }
      if constexpr (TURN) {
        const int64_t row0 = m0 + 128 * rank + 32 * quarter;  // the warp's rows
        int* turn = turns + ew * 32 * (kPairPitch + 1);
        __syncwarp();  // the previous tile's row scales are read
        turn[32 * kPairPitch + lane] = __float_as_int(row0 + lane < a.m ? a.a_scale[row0 + lane] : 0.0f);
        // the residual of a chunk is asked for one chunk ahead, the first before the wait
        const int c_end = (half + 1) * (bn / 64);
        PairResidual next;
        ask_residual(a, pair_span(a, row0, n0 + 32 * half * (bn / 64), lane), next);
        asm volatile("bar.sync 1, %0;" ::"n"(32 * kPairEpilogueWarps) : "memory");
        if (!dead) dead = !wait_or_abort_for(acc_full + acc, (i >> 1) & 1, abort_flag, kWaitLimitNs);
        dead = __any_sync(0xffffffffu, dead);  // the warp agrees: the TMEM loads below are collective
        tc_fence_after();
        for (int c = half * (bn / 64); c < c_end; ++c) {
          const int64_t c0 = n0 + 32 * c;
          if (c0 >= a.n) break;  // the same for every lane
          const PairSpan span = pair_span(a, row0, c0, lane);
          if (dead) {
            for (int y = 0; y < span.rows; ++y) {
              for (int z = 0; z < span.columns; ++z) store_one(a.out, a.out_kind, span.e + 2 * y * a.n + z, __int_as_float(0x7fc00000));
            }
            continue;
          }
          const PairResidual now = next;
          if (c + 1 < c_end) ask_residual(a, pair_span(a, row0, c0 + 32, lane), next);
          uint32_t r[32];
          tc_ld_32cols(tmem + (static_cast<uint32_t>(32 * quarter) << 16) + static_cast<uint32_t>(acc * 256 + 32 * c), r);
          __syncwarp();  // the previous chunk's words are read
  #pragma unroll
          for (int q = 0; q < 16; ++q)
            *reinterpret_cast<int2*>(turn + lane * kPairPitch + 2 * q) = make_int2(static_cast<int>(r[2 * q]), static_cast<int>(r[2 * q + 1]));
          __syncwarp();
          const int col = 32 * c + 2 * (lane & 15);
          finish_chunk<ACT>(a, span, now, turn, *reinterpret_cast<const float2*>(scale + col), *reinterpret_cast<const float2*>(bias + col), lane);
        }
      } else {
        const int64_t row = m0 + 128 * rank + 32 * quarter + lane;
        const bool row_ok = row < a.m;
        const float sa = row_ok ? a.a_scale[row] : 0.0f;
        // the residual of a chunk is asked for one chunk ahead, the first before the wait
        const auto ask = [&](int c, uint4(&raw)[4]) {
          const int64_t c0 = n0 + 32 * c;
          if (a.residual != nullptr && a.out_kind != kOutF32 && row_ok && c0 < a.n && c < (half + 1) * (bn / 64)) {
            const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.residual) + row * a.n + c0);
  #pragma unroll
            for (int q = 0; q < 4; ++q) raw[q] = p[q];
          }
        };
        uint4 next[4];
        ask(half * (bn / 64), next);
        asm volatile("bar.sync 1, %0;" ::"n"(32 * kPairEpilogueWarps) : "memory");
        if (!dead) dead = !wait_or_abort_for(acc_full + acc, (i >> 1) & 1, abort_flag, kWaitLimitNs);
        dead = __any_sync(0xffffffffu, dead);  // the warp agrees: the TMEM loads below are collective
        tc_fence_after();
        for (int c = half * (bn / 64); c < (half + 1) * (bn / 64); ++c) {
          const int64_t c0 = n0 + 32 * c;
          if (c0 >= a.n) break;  // the same for every lane
          if (dead) {
            if (row_ok) {
              for (int j = 0; j < 32 && c0 + j < a.n; ++j) store_one(a.out, a.out_kind, row * a.n + c0 + j, __int_as_float(0x7fc00000));
            }
            continue;
          }
          uint4 raw[4];
  #pragma unroll
          for (int q = 0; q < 4; ++q) raw[q] = next[q];
          ask(c + 1, next);
          uint32_t r[32];
          tc_ld_32cols(tmem + (static_cast<uint32_t>(32 * quarter) << 16) + static_cast<uint32_t>(acc * 256 + 32 * c), r);
          if (row_ok) finish_row32<ACT>(a, row, c0, r, raw, sa, scale + 32 * c, bias + 32 * c);
        }
      }
      if (dead) *abort_flag = 1u;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr(acc_empty + acc, 0)) : "memory");
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  // the last commit arrives in both CTAs; every accumulator it stands for has been read by now
  if (threadIdx.x == 32) mbar_wait_parity(mma_done, 0);
  __syncwarp();
  cluster_barrier();  // no CTA leaves (or frees TMEM) while its peer still uses it
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kPairCols) : "memory");
  }
}

}  // namespace dq
