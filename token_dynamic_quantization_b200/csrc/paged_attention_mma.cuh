// Paged decode attention on the tensor cores: one pass over the visible rows
// of the cache with the softmax's running maximum and sum.
//
// One product serves up to 8 * HT query heads of a key head at once, the
// tokens along the matrix rows so that few heads waste nothing:
//   S^T[token, head] = K[token, :] . Q[head, :]          K as the A operand
//   O^T[dim, head]  += V^T[dim, token] . P[token, head]  V^T as the A operand
// The order of the contracted index is free as long as both operands share
// it, and so is the order of the rows of O^T. A lane (g = lane / 4, t = lane % 4)
// therefore takes 16-byte pieces of the K rows g and g + 8 (pieces t of every 4)
// and of the V rows of its tokens (pieces g of every 8), each used whole.
// movmatrix turns P from the accumulator's layout into the B operand's.
//
// Rows come through shared memory: each warp has a ring of its own, filled by
// TMA with 16 rows to a box where pages hold whole groups of 16 tokens, else with
// four rows of any pages to a gather (64 x 8192, INT8: 108 us with pages of 16, 120
// with pages of 20; 97 with pages of 64, whose boxes lie side by side), so that no
// warp waits for another inside an item and tens of kilobytes per SM are on their
// way; loads of 64-byte pieces into registers reach 3 TB/s, the copies close to 6.
//
// INT8 caches keep their codes as operands. S: Q as two signed 8-bit digits of
// a 16-bit integer (m16n8k32, exact int32 sums). O: a code's bits plus 128 in the low
// byte of an f16 are a subnormal, (code + 128) * 2^-24, exact in the products; an
// operand of 128s beside the same weights collects what the 128s add up to, and
// it is taken off every other tile, while it is small. Value scales are folded into the
// weights, relative to the power of two of a head's largest weight times scale so far (not
// of the largest scale: its token may have no weight), so the products that count
// keep f16's bits whatever the scales' size.
//
// A weight is rounded to 16 bits for its product, and what that cuts off goes into a
// second one: alone, a bf16 would be off by 2^-9 beside bf16 outputs, an f16 by 2^-12 beside f16
// outputs, as much as the output's own rounding (f16 caches: 2.8e-4 of the result in
// norm against 2.1e-4). Beside codes with bf16 outputs one f16 is enough, an eighth of the
// output's half step; there the second would cost 3 % with up to 8 query heads to a
// key head (64 x 8192: 112 us from 108.4) and 10 % with more (64 x 4000, 16 heads: 97.6 us
// from 88.8). Beside f16 it costs 1 to 5 % (window 48 x 6000: 30.4 us from 28.9).
//
// The running maximum moves only when a score exceeds it by 8 (in log2), or beside
// codes a weight times its scale may exceed f16's range: weights then stay below 2^(8 +
// kLift) and the rescaling of O is rare. In f16 kLift raises the weights so that
// those down to 2^-30 of the largest count.
//
// What a warp or a CTA leaves for others to join is its own quotient O / sum beside
// (max, sum): no larger than the values, so that a join of large ones does not overflow.
//
// Work: all (sequence, key head, head set) items' tiles of TT tokens, laid end
// to end, are cut into equal ranges, one per CTA, whatever the lengths; a CTA's
// warps take its tiles in turn. Items inside one range are finished by their
// CTA. Of an item that ranges cut, each CTA leaves (max, sum, O / sum) in the
// workspace, and a second kernel joins them. Short items (the host's rule) get a
// CTA each and need no second kernel. Where there are many items (the host's
// rule), a CTA is a single warp: no warp waits for another when an item ends.
//
// Bound by reading the cache: one sequence of 131072 tokens, bf16, 8 key heads takes
// 88 us against 82 at the copy rate (6.1 TB/s); 64 ragged sequences of up to 8192,
// INT8, 108.5 against 81 (opening the next item costs a CTA about 2 us each time,
// and the start 5; DRAM at 59 % of its peak, issue slots at 38 %, tensor pipe at 16 %); 200
// of up to 8000, INT8, 301 against 259; one of 127 tokens takes 5, nearly all of it latency.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "decoder_device.cuh"
#include "dq_device.cuh"
#include "paged_attention_args.cuh"
#include "tma_pipeline.cuh"

namespace dq {

constexpr float kSlack = 8.0f;  // log2 by which a score may exceed the running maximum
// log2 of the weight at the running maximum: in f16 it raises the small ones above the type's
// smallest steps; in bf16, whose range is that of the sums, it keeps those of values up to the
// type's largest from overflowing before they are divided.
constexpr int kLiftF16 = 6, kLiftBf16 = -16;
template <typename T, typename C>
constexpr float kLift = sizeof(C) == 2 && __is_same(T, __nv_bfloat16) ? kLiftBf16 : kLiftF16;
// log2 of a sum of such weights, without the lift (which is exact as a factor)
template <typename T, typename C>
__device__ __forceinline__ float log2_weights(float sum) {
  return log2f(sum * (sizeof(C) == 2 && __is_same(T, __nv_bfloat16) ? 0x1p16f : 0x1p-6f));
}
constexpr uint32_t kRowHidden = 0xFFFFFFFFu, kRowBad = 0xFFFFFFFEu;  // row numbers outside every cache

// W: warps of a CTA, which share an item's tiles.
template <typename C, int D, int HT, int W>
struct PagedShape {
  static constexpr int kThreads = 32 * W;
  static constexpr bool kCodes = sizeof(C) == 1;
  static constexpr int kTokens = kCodes && D <= 128 ? 32 : 16;
  static constexpr int kHeads = 8 * HT;
  // one CTA's parts: O / sum [kHeads][D], then (max, sum) [kHeads]
  static constexpr int kPartFloats = kHeads * D + 2 * kHeads;
  // CTAs per SM: three, and two where their rings would be too short (codes of 128
  // channels: 109 us with two, 115 with three) or the registers do not allow more
  static constexpr int kCtas = (HT * D > 128 || (kCodes && D == 128) ? 2 : 3) * 4 / W;
  // rows lie in shared memory in boxes of 128 bytes (64 for 64 codes), swizzled
  static constexpr int kBox = D * int(sizeof(C)) < 128 ? D * int(sizeof(C)) : 128;
  static constexpr int kBoxes = D * int(sizeof(C)) / kBox;
  // a warp's ring: K and V boxes of kStages tiles, then the tiles' scales
  static constexpr int kRowBytes = kTokens * D * int(sizeof(C));
  static constexpr int kScaleBytes = kCodes ? 2 * 4 * kTokens : 0;
  static constexpr int kStageBytes = 2 * kRowBytes;
  static constexpr int kPitch = D + 4;                      // of a head's row there, against bank conflicts
  static constexpr int kJoin = W * (kHeads * kPitch + 2 * kHeads) * 4;
  static constexpr int kFit = (227 * 1024 / kCtas - 2048 - 256 - kJoin) / W / (kStageBytes + kScaleBytes);
  static constexpr int kStages = kFit < 2 ? 2 : (kFit > 8 ? 8 : kFit);
  static constexpr int kRings = W * kStages * kStageBytes;
  static constexpr int kScales = W * kStages * kScaleBytes;
  static constexpr int kBarriers = W * kStages * 8;
  static constexpr int kBody = kRings + kScales + kJoin;
  static constexpr size_t kSmem = 1024 + size_t(kBody) + kBarriers;  // 1024: alignment of the swizzle pattern
};

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) { return __byte_perm(a, b, sel); }

// Transpose of an 8x8 matrix of 16-bit values held two to a lane.
__device__ __forceinline__ uint32_t movmatrix(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

template <bool kBf16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if constexpr (kBf16) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  } else {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
}

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Four neighbouring outputs, times r.
template <typename T>
__device__ __forceinline__ void store_row4(T* out, const float4& v, float r) {
  if constexpr (__is_same(T, __nv_bfloat16)) {
    *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16(v.x * r, v.y * r), pack_bf16(v.z * r, v.w * r));
  } else {
    *reinterpret_cast<uint2*>(out) = make_uint2(pack_f16(v.x * r, v.y * r), pack_f16(v.z * r, v.w * r));
  }
}

// The value of 16 bits of type T.
template <typename T>
__device__ __forceinline__ float half_bits(uint32_t b) {
  if constexpr (__is_same(T, __nv_bfloat16)) return __uint_as_float(b << 16);
  return __half2float(__ushort_as_half(static_cast<unsigned short>(b)));
}

// Two bytes of w as f16: a byte in the low bits of an f16 is the subnormal byte *
// 2^-24, exact in the products.
__device__ __forceinline__ uint32_t bytes_f16(uint32_t w, uint32_t sel) { return prmt(w, 0u, sel); }

// 1 / x of a sum of weights (0 for none): between 2^-126 and 2^126 a unit in the last place
// off, and a sum of fewer than 2^31 weights stays there.
__device__ __forceinline__ float inverse(float x) {
  return x == 0.0f ? 0.0f : rcp_approx(x);
}

// A box of a tensor map, from element `x` of row `row` on, to `dst`.
__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap* map, int x, int row, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(row), "r"(bar)
      : "memory");
}

// Four rows of a tensor map, `x` elements into each, one after the other to
// `dst`; a row outside the map is filled with zeros.
__device__ __forceinline__ void gather_rows(uint32_t dst, const CUtensorMap* map, int x, int r0, int r1, int r2, int r3,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, "
      "%6}], [%7];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(r0), "r"(r1), "r"(r2), "r"(r3), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void copy_async4(uint32_t dst, const void* src, int from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(from) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Offset of 16-byte piece `piece` of row `row` in a stage's boxes, as the
// copies' swizzle lays them: within 128-byte rows the piece's number is XORed
// with the row's low three bits, within 64-byte rows with bits 1 and 2.
template <typename Shape, int TT>
__device__ __forceinline__ uint32_t box_offset(int row, int piece) {
  if constexpr (Shape::kBox == 128) {
    return (piece >> 3) * TT * 128 + row * 128 + (((piece & 7) ^ (row & 7)) << 4);
  } else {
    return row * 64 + ((piece ^ ((row >> 1) & 3)) << 4);
  }
}

// Which of 8 tokens stands at place i of the products. In 128-byte rows, 8
// lanes of a 16-byte K load hold places 2j and 2j + 1, pieces 0-3: tokens whose
// numbers differ in bit 2 put them into different halves of the banks. The V
// load's 8 lanes hold places 0, 2, 4, 6 (or the odd ones), two pieces each:
// tokens that differ in bits 1 and 2.
template <int BOX>
__device__ __forceinline__ int token_order(int i) {
  return BOX == 128 ? (0x37156240u >> (4 * i)) & 7 : i;
}

// ---------------------------------------------------------------- the schedule

// The visible tokens of one sequence as groups of 16 that start at multiples of
// 16: first those that hold the first tokens [0, first), then those from the
// one with token `start` on. A length that the page table cannot hold is one
// token past the table, which makes the rows NaN.
struct Groups {
  int len, first, start;
  int first_groups, count;
};

__device__ __forceinline__ Groups visible_groups(const PagedArgs& a, int len) {
  const int64_t room = a.max_pages * a.page_size;
  Groups v{len, 0, 0, 0, 0};
  if (len <= 0) {
    v.len = 0;
    return v;
  }
  if (len > room) {
    v.start = static_cast<int>(room);
    v.len = v.start + 1;
    v.count = 1;
    return v;
  }
  if (a.window != 0 && len > a.window) {
    v.start = len - static_cast<int>(a.window);
    v.first = a.sinks < v.start ? static_cast<int>(a.sinks) : v.start;
    v.first_groups = (v.first + 15) >> 4;
  }
  v.count = v.first_groups + (((len - 1) >> 4) - (v.start >> 4) + 1);
  return v;
}

// Opening and joining an item takes a CTA as long as several tiles (3.4 us against
// 0.6 us a tile on 64 sequences of up to 8192 tokens, four warps): ranges are cut
// in units of which an item has kItemCost more than tiles, the first ones empty. On
// those sequences, INT8, 137 us with 0, 119 with 4, 115 with 6 and 10. A warp by itself
// takes longer for a tile: 444 sequences of up to 600 tokens take 87 us with 1, 79
// with 2, 81 with 4.
template <int W>
constexpr int kItemCost = W == 4 ? 8 : 2;

// Tiles of one sequence's item; a sequence without tokens still has one, whose
// CTA writes its zeros.
template <int TT>
__device__ __forceinline__ int tiles_of(const Groups& v) {
  constexpr int kGroups = TT / 16;
  return v.count == 0 ? 1 : (v.count + kGroups - 1) / kGroups;
}
template <int TT, int W>
__device__ __forceinline__ int64_t item_units(const PagedArgs& a, int64_t b) {
  return tiles_of<TT>(visible_groups(a, a.lengths[b])) + kItemCost<W>;
}

__device__ __forceinline__ int64_t warp_sum_i64(int64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// All units of the call (every lane of the warp gets the sum).
template <int TT, int W>
__device__ int64_t total_units(const PagedArgs& a) {
  int64_t sum = 0;
  const int lane = threadIdx.x & 31;
  for (int64_t b = lane; b < a.batch; b += 32) sum += item_units<TT, W>(a, b);
  return warp_sum_i64(sum) * a.kv_heads * a.head_sets;
}

// The sequence that unit `x` belongs to, and the number of its first unit.
template <int TT, int W>
__device__ void find_sequence(const PagedArgs& a, int64_t x, int64_t& seq, int64_t& base) {
  const int lane = threadIdx.x & 31;
  const int64_t per = static_cast<int64_t>(a.kv_heads) * a.head_sets;
  int64_t before = 0;
  for (int64_t b0 = 0;; b0 += 32) {
    const int64_t b = b0 + lane;
    int64_t end = b < a.batch ? item_units<TT, W>(a, b) * per : 0;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int64_t up = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += up;
    }
    end += before;
    const uint32_t hit = __ballot_sync(0xffffffffu, b < a.batch && end > x);
    if (hit != 0u || b0 + 32 >= a.batch) {
      const int first = hit != 0u ? __ffs(hit) - 1 : 0;
      const int64_t prev = __shfl_up_sync(0xffffffffu, end, 1);
      seq = b0 + first;
      base = first == 0 ? before : __shfl_sync(0xffffffffu, prev, first);
      return;
    }
    before = __shfl_sync(0xffffffffu, end, 31);
  }
}

// Units per CTA: equal shares, and at least a short item for each.
template <int W>
__device__ __forceinline__ int64_t units_per_cta(int64_t total, int64_t ctas) {
  const int64_t per = (total + ctas - 1) / ctas;
  return per < kItemCost<W> + W ? kItemCost<W> + W : per;
}

// ---------------------------------------------------------------- main kernel

template <typename T, typename C, int D, int HT, bool RUN, int W>
__global__ void __launch_bounds__(32 * W, (PagedShape<C, D, HT, W>::kCtas))
    paged_attention_mma_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                               const PagedArgs a) {
  using Shape = PagedShape<C, D, HT, W>;
  constexpr int kItemCost = dq::kItemCost<W>;
  constexpr bool kCodes = Shape::kCodes;
  constexpr bool kBf16 = !kCodes && sizeof(T) == 2 && __is_same(T, __nv_bfloat16);
  // a weight as two operands of 16 bits; one of f16 does beside codes where the output is bf16
  constexpr float kLift = dq::kLift<T, C>;
  constexpr bool kTwoParts = !kCodes || __is_same(T, __half);
  constexpr int TT = Shape::kTokens, MT = TT / 16, kHeads = Shape::kHeads;
  constexpr int kElem = sizeof(C);
  constexpr int kPiece = 16 / kElem;         // elements of a 16-byte piece
  constexpr int KP = D / (4 * kPiece);       // K pieces per lane and row
  constexpr int kVBytes = D * kElem / 8 >= 16 ? 16 : D * kElem / 8;
  constexpr int kVPiece = kVBytes / kElem;   // elements of a V piece
  constexpr int VP = D / (8 * kVPiece);      // V pieces per lane and row
  constexpr int KS = D / 16;                 // k-steps of S, and row tiles of O^T
  constexpr int kStages = Shape::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  // the warps' rings and scales; what they leave of an item, [warps][kHeads][D] and [warps][kHeads][2]
  float* s_o = reinterpret_cast<float*>(smem + Shape::kRings + Shape::kScales);
  float* s_stat = s_o + W * kHeads * Shape::kPitch;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t ring = smem_addr(smem) + warp * kStages * Shape::kStageBytes;
  const uint32_t scales = smem_addr(smem) + Shape::kRings + warp * kStages * Shape::kScaleBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Shape::kBody) + warp * kStages;
  if (lane < kStages) mbar_init(bars + lane, 1);
  fence_mbarrier_init();
  __syncwarp();
  uint32_t filled = 0u;  // bit st: parity of stage st's next completion

  pdl_launch_dependents();
  pdl_wait_primary();

  // this CTA's units [unit, unit_end); `base` is the first one of sequence seq
  int64_t seq, base, unit, unit_end;
  const int items_per_seq = a.kv_heads * a.head_sets;
  if (a.whole) {
    seq = blockIdx.x / items_per_seq;
    const int64_t n = item_units<TT, W>(a, seq);
    base = 0;
    unit = (blockIdx.x - seq * items_per_seq) * n;
    unit_end = unit + n;
  } else {
    const int64_t total = total_units<TT, W>(a);
    const int64_t per = units_per_cta<W>(total, gridDim.x);
    unit = per * blockIdx.x;
    unit_end = unit + per < total ? unit + per : total;
    if (unit >= total) {
      if (threadIdx.x == 0) a.cuts[blockIdx.x].seq = -1;
      return;
    }
    find_sequence<TT, W>(a, unit, seq, base);
  }
  const int64_t range_begin = unit, range = unit_end - unit;
  // tokens of a tile in the order that spreads them over the banks: lane g's K
  // row, and the rows of a lane's V tokens
  const int order = token_order<Shape::kBox>(g), order_even = token_order<Shape::kBox>(2 * t);
  const int order_odd = token_order<Shape::kBox>(2 * t + 1);

  // ---- the item at hand: its tokens, heads and rows of the page table; this CTA
  // has its tiles [t0, t1)
  int len = a.lengths[seq], len_next = seq + 1 < a.batch ? a.lengths[seq + 1] : 0;
  Groups vis = visible_groups(a, len);
  int n = tiles_of<TT>(vis);
  int item = static_cast<int>((unit - base) / (n + kItemCost));
  int64_t item_begin = base + static_cast<int64_t>(item) * (n + kItemCost);
  int kvh = item / a.head_sets, set = item - kvh * a.head_sets;
  int t0 = 0, t1 = 0, head0 = 0, heads = 0;
  const int32_t* table = a.page_table + seq * a.max_pages;
  const auto enter = [&]() {
    const int64_t first = unit - item_begin - kItemCost, last = unit_end - item_begin - kItemCost;
    t0 = first < 0 ? 0 : static_cast<int>(first);
    t1 = last < n ? static_cast<int>(last) : n;  // <= 0: the range ends in the item's empty units
    head0 = kvh * a.group + set * kHeads;        // first query head
    heads = a.group - set * kHeads < kHeads ? a.group - set * kHeads : kHeads;
  };
  // the item behind the one at hand
  const auto advance = [&]() {
    item_begin += n + kItemCost;
    unit = item_begin;
    ++item;
    if (++set == a.head_sets) {
      set = 0;
      if (++kvh == a.kv_heads) {
        kvh = item = 0;
        ++seq;
        len = len_next;
        len_next = seq + 1 < a.batch ? a.lengths[seq + 1] : 0;
        vis = visible_groups(a, len);
        n = tiles_of<TT>(vis);
        table += a.max_pages;
      }
    }
  };
  // Token at place r of tile tl, and whether it is visible.
  const auto token_of = [&](int tl, int r, bool& seen) -> uint32_t {
    const int group = tl * MT + (r >> 4);
    if (group < vis.first_groups) {
      const uint32_t j = 16u * group + (r & 15);
      seen = j < static_cast<uint32_t>(vis.first);
      return j;
    }
    // unsigned: the last tile may reach past token 2^31 - 1
    const uint32_t j = 16u * (group - vis.first_groups) + (vis.start & ~15) + (r & 15);
    seen = j >= static_cast<uint32_t>(vis.start) && j < static_cast<uint32_t>(vis.len);
    return j;
  };
  // Cache row numbers of a tile, in two steps so that the page table's latency
  // is off the path (the page, one tile ahead of the row): of its groups' first
  // tokens in lanes 0 .. MT - 1 where pages hold whole groups, else of token r in
  // lane r. -2: nothing there, -1: no such page.
  const auto find_page = [&](int tl, uint32_t& in_page) -> int32_t {
    bool seen;
    const uint32_t j = token_of(tl, RUN ? 16 * lane : lane, seen);
    if constexpr (RUN) {
      seen = tl * MT + lane < vis.count && lane < MT;
    }
    if (tl >= t1 || !seen || lane >= TT) return -2;
    const uint32_t p = (__umulhi(j, a.page_mul) + j) >> a.page_shift;
    in_page = j - p * static_cast<uint32_t>(a.page_size);
    return p < a.max_pages ? max(__ldg(table + p), -1) : -1;
  };
  const auto row_of = [&](int32_t page, uint32_t in_page) -> uint32_t {
    if (page == -2) return kRowHidden;
    if (page < 0 || page >= a.num_pages) return kRowBad;
    return (static_cast<uint32_t>(page) * static_cast<uint32_t>(a.kv_heads) + static_cast<uint32_t>(kvh)) *
               static_cast<uint32_t>(a.page_size) + in_page;
  };

  bool broken = false;  // a page outside the cache, or a copy that never came: the rows become NaN
  bool dead = false;    // a copy never came: the warp copies nothing any more, its items become NaN
  const auto issue = [&](int st, uint32_t row) {
    broken |= row == kRowBad;
#ifdef DQ_TEST_SKIP_ATTENTION_SEQ
    // test builds only: leave one tile of one sequence's first key head out, so
    // that the bounded wait for it runs out
    if (seq == DQ_TEST_SKIP_ATTENTION_SEQ && kvh == 0 && st == 1 && warp == 0) {
      if constexpr (kCodes) copies_commit();
      return;
    }
#endif
    const uint32_t bar = smem_addr(bars + st), dst = ring + st * Shape::kStageBytes;
    if (lane == 0) mbar_arrive_expect_tx(bars + st, Shape::kStageBytes);
    if constexpr (RUN) {
      uint32_t r[MT];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) r[mt] = __shfl_sync(0xffffffffu, row, mt);
      if (lane == 0) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
          for (int x = 0; x < Shape::kBoxes; ++x) {
            const uint32_t to = dst + (x * TT + 16 * mt) * Shape::kBox;
            copy_box(to, &k_map, x * (Shape::kBox / kElem), r[mt], bar);
            copy_box(to + Shape::kRowBytes, &v_map, x * (Shape::kBox / kElem), r[mt], bar);
          }
        }
      }
      // from here on lane r's row is token r's
      const uint32_t mine = lane < 16 ? r[0] : r[MT - 1];
      row = mine < kRowBad ? mine + (lane & 15) : mine;
    } else {
      const uint32_t r0 = __shfl_sync(0xffffffffu, row, (4 * lane) & 31), r1 = __shfl_sync(0xffffffffu, row, (4 * lane + 1) & 31);
      const uint32_t r2 = __shfl_sync(0xffffffffu, row, (4 * lane + 2) & 31), r3 = __shfl_sync(0xffffffffu, row, (4 * lane + 3) & 31);
      if (lane < TT / 4) {
#pragma unroll
        for (int x = 0; x < Shape::kBoxes; ++x) {
          const uint32_t to = dst + (x * TT + 4 * lane) * Shape::kBox;
          gather_rows(to, &k_map, x * (Shape::kBox / kElem), r0, r1, r2, r3, bar);
          gather_rows(to + Shape::kRowBytes, &v_map, x * (Shape::kBox / kElem), r0, r1, r2, r3, bar);
        }
      }
    }
    if constexpr (kCodes) {
      if (lane < TT) {
        const uint32_t dst = scales + st * Shape::kScaleBytes + lane * 8;
        const uint32_t r = row < kRowBad ? row : 0u;
        copy_async4(dst, a.k_scale + r, row < kRowBad ? 4 : 0);
        copy_async4(dst + 4, a.v_scale + r, row < kRowBad ? 4 : 0);
      }
      copies_commit();
    }
  };

  // The warp's first tiles of the item into its ring, and the item's queries as
  // they lie in memory: asked for before the previous item is joined.
  uint32_t in_page_next = 0u;
  int32_t page_next = -2;
  int st = 0;
  bool opened = false;  // copies of the item's tiles have been issued
  uint2 qw[HT][KS];
#pragma unroll
  for (int ht = 0; ht < HT; ++ht) {
#pragma unroll
    for (int s = 0; s < KS; ++s) qw[ht][s] = make_uint2(0u, 0u);
  }
  const auto open = [&]() {
    enter();
    broken = false;
    opened = !dead;
    if (dead) return;
    const int first = t0 + warp;
    int32_t page[kStages];
    uint32_t in_page[kStages];
#pragma unroll
    for (int i = 0; i < kStages; ++i) page[i] = find_page(first + i * W, in_page[i]);
#pragma unroll
    for (int ht = 0; ht < HT; ++ht) {
      const bool on = 8 * ht + g < heads;
      const T* q = static_cast<const T*>(a.q) + seq * a.q_stride + static_cast<int64_t>(head0 + 8 * ht + g) * D;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const int c = kCodes ? (s / 4) * 64 + 16 * t + 4 * (s % 4) : (s / 2) * 32 + 8 * t + 4 * (s % 2);
        qw[ht][s] = on ? *reinterpret_cast<const uint2*>(q + c) : make_uint2(0u, 0u);
      }
    }
#pragma unroll
    for (int i = 0; i < kStages; ++i) {
      if (first + i * W < t1) {
        issue(i, row_of(page[i], in_page[i]));
      } else if constexpr (kCodes) {
        copies_commit();
      }
    }
    page_next = find_page(first + kStages * W, in_page_next);
  };

  // The item at hand goes on in the next CTA: its first and last tile's CTAs, for
  // the second kernel. Every range that ends before the last one is `range` long.
  const auto record_cut = [&]() {
    if (t1 >= n || threadIdx.x != 0) return;
    const int64_t first = t0 == 0 ? static_cast<int64_t>(blockIdx.x) : (item_begin + kItemCost) / range;
    a.cuts[blockIdx.x] = {seq, item, static_cast<int>(first), static_cast<int>((item_begin + kItemCost + n - 1) / range)};
  };

  enter();
  if (t1 <= t0) {  // the range is nothing but empty units: they end with it, or its item is the next CTA's
    if (threadIdx.x == 0) a.cuts[blockIdx.x].seq = -1;
    return;
  }
  open();
  record_cut();
  while (true) {
    // Q as the B operand, head g. Beside a 16-bit cache as it is, four channels
    // per k-step. Beside codes as two signed 8-bit digits, 256 q1 + q0, of a
    // power of two times it, |.| <= 32639: channels down to 2^-7 (bf16; f16:
    // 2^-4) of the head's largest are exact, the others off by at most
    // half a unit, 0.5 / 16319 of it: a 64th (f16: an 8th) of what the type's own rounding
    // has moved that largest one by. The results' error in norm is 2.05e-4 beside f16 outputs, whose
    // rounding alone is 2.04e-4; a third digit would add half to the products of S.
    uint32_t qf[HT][KS][2];
    float q_mul[HT][2];  // scores' factor of heads 2t and 2t + 1, log2(e) included
#pragma unroll
    for (int ht = 0; ht < HT; ++ht) {
      float mul = fabsf(a.softmax_scale) * kLog2e;  // its sign goes into Q: the largest product has the largest score
      if constexpr (kCodes) {
        uint32_t top = 0u;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const uint2 w = qw[ht][s];
          top = max(top, max(max(w.x & 0x7FFFu, (w.x >> 16) & 0x7FFFu), max(w.y & 0x7FFFu, (w.y >> 16) & 0x7FFFu)));
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float largest = half_bits<T>(top);
        int e = 0;
        if (!isfinite(largest)) {
          mul = NAN;
        } else if (largest > 0.0f) {
          e = 14 - ilogbf(largest);
          if (scalbnf(largest, e) > 32639.0f) --e;
          if (e > 126) e = 126;
          mul = scalbnf(mul, -e);
        }
        const float f = a.softmax_scale < 0.0f ? -scalbnf(1.0f, e) : scalbnf(1.0f, e);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const uint2 w = qw[ht][s];
          int x[4] = {__float2int_rn(half_bits<T>(w.x & 0xFFFFu) * f), __float2int_rn(half_bits<T>(w.x >> 16) * f),
                      __float2int_rn(half_bits<T>(w.y & 0xFFFFu) * f), __float2int_rn(half_bits<T>(w.y >> 16) * f)};
          uint32_t hi = 0u, lo = 0u;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int q1 = (x[i] + 128) >> 8;
            hi |= (static_cast<uint32_t>(q1) & 255u) << (8 * i);
            lo |= (static_cast<uint32_t>(x[i] - (q1 << 8)) & 255u) << (8 * i);
          }
          qf[ht][s][0] = hi;
          qf[ht][s][1] = lo;
        }
      } else {
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const uint2 w = qw[ht][s];
          const uint32_t sign = a.softmax_scale < 0.0f ? 0x80008000u : 0u;
          qf[ht][s][0] = w.x ^ sign;
          qf[ht][s][1] = w.y ^ sign;
        }
      }
      q_mul[ht][0] = __shfl_sync(0xffffffffu, mul, 8 * t);
      q_mul[ht][1] = __shfl_sync(0xffffffffu, mul, 8 * t + 4);
    }

    float o[HT][KS][4], m[HT][2], l[HT][2];
    float o_bias[HT][4];  // what the codes' bias of 128 has added to every channel of O
    // the power of two that takes the head's largest weight times value scale so far
    // into [1, 2)
    float v_mul[HT][2];
#pragma unroll
    for (int ht = 0; ht < HT; ++ht) {
      v_mul[ht][0] = v_mul[ht][1] = 0x1p126f;
      m[ht][0] = m[ht][1] = -INFINITY;
      l[ht][0] = l[ht][1] = 0.0f;
      o_bias[ht][0] = o_bias[ht][1] = o_bias[ht][2] = o_bias[ht][3] = 0.0f;
#pragma unroll
      for (int i = 0; i < KS; ++i) o[ht][i][0] = o[ht][i][1] = o[ht][i][2] = o[ht][i][3] = 0.0f;
    }

    // v_mul's reciprocal, a power of two as well
    const auto v_size = [&](int ht, int c) { return __uint_as_float((254u << 23) - __float_as_uint(v_mul[ht][c])); };

    // groups whose tokens are all visible
    const int inside_first = vis.first_groups == 0 && (vis.start & 15) == 0 ? 0 : vis.first_groups + ((vis.start & 15) != 0 ? 1 : 0);
    const int inside_last = vis.first_groups + (vis.len >> 4) - (vis.start >> 4);
    bool biased = false;  // O still holds the last tile's bias
    const auto remove_bias = [&]() {
#pragma unroll
      for (int ht = 0; ht < HT; ++ht) {
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          o[ht][i][0] -= o_bias[ht][0];
          o[ht][i][1] -= o_bias[ht][1];
          o[ht][i][2] -= o_bias[ht][0];
          o[ht][i][3] -= o_bias[ht][1];
        }
        o_bias[ht][0] = o_bias[ht][1] = o_bias[ht][2] = o_bias[ht][3] = 0.0f;
      }
    };
    int tl = t0 + warp;
    st = 0;
    for (; tl < t1; tl += W) {
      const uint32_t stage = ring + st * Shape::kStageBytes;
      dead = __any_sync(0xffffffffu, dead || !mbar_wait_parity(bars + st, (filled >> st) & 1u));
      if constexpr (kCodes) copies_wait<kStages - 1>();
      __syncwarp();
      if (__any_sync(0xffffffffu, broken || dead)) break;
      filled ^= 1u << st;
      // ---- S^T = K Q^T
      float s[HT][MT][4];
      if constexpr (kCodes) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          uint32_t k0[KP][4], k1[KP][4];  // rows g and g + 8
#pragma unroll
          for (int i = 0; i < KP; ++i) {
            const uint32_t at = stage + box_offset<Shape, TT>(16 * mt + order, 4 * i + t);
            load_piece<16>(k0[i], at);
            load_piece<16>(k1[i], at + 8 * Shape::kBox);
          }
#pragma unroll
          for (int ht = 0; ht < HT; ++ht) {
            int d[4] = {0, 0, 0, 0};
#pragma unroll
            for (int digit = 0; digit < 2; ++digit) {
              if (digit == 1) d[0] <<= 8, d[1] <<= 8, d[2] <<= 8, d[3] <<= 8;
#pragma unroll
              for (int i = 0; i < KP; ++i) {
#pragma unroll
                for (int u = 0; u < 4; u += 2)
                  mma_s8(d, k0[i][u], k1[i][u], k0[i][u + 1], k1[i][u + 1], qf[ht][4 * i + u][digit],
                              qf[ht][4 * i + u + 1][digit]);
              }
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) s[ht][mt][x] = __int2float_rn(d[x]);
          }
        }
      } else {
#pragma unroll
        for (int ht = 0; ht < HT; ++ht) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) s[ht][mt][0] = s[ht][mt][1] = s[ht][mt][2] = s[ht][mt][3] = 0.0f;
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
          for (int i = 0; i < KP; ++i) {
            uint32_t k0[4], k1[4];  // rows g and g + 8
            const uint32_t at = stage + box_offset<Shape, TT>(16 * mt + order, 4 * i + t);
            load_piece<16>(k0, at);
            load_piece<16>(k1, at + 8 * Shape::kBox);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
#pragma unroll
              for (int ht = 0; ht < HT; ++ht)
                mma16816<kBf16>(s[ht][mt], k0[2 * u], k1[2 * u], k0[2 * u + 1], k1[2 * u + 1], qf[ht][2 * i + u][0],
                                qf[ht][2 * i + u][1]);
            }
          }
        }
      }
      // ---- scores up to the heads' factors q_mul, hidden tokens out
      const bool inside = tl * MT >= inside_first && tl * MT + MT <= inside_last;  // no token of the tile is hidden
      float vw[MT][2];
      bool move = false;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int tok = 16 * mt + 8 * h + order;
          vw[mt][h] = 1.0f;
          if constexpr (kCodes) {
            float k_mul;
            asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];"
                         : "=f"(k_mul), "=f"(vw[mt][h])
                         : "r"(scales + st * Shape::kScaleBytes + tok * 8));
            // NaN where a scale is not finite: such a token spoils the row whatever its weight
            const float spoil = fmaf(k_mul, 0.0f, vw[mt][h] * 0.0f);
#pragma unroll
            for (int ht = 0; ht < HT; ++ht) {
              s[ht][mt][2 * h] = fmaf(s[ht][mt][2 * h], k_mul, spoil);
              s[ht][mt][2 * h + 1] = fmaf(s[ht][mt][2 * h + 1], k_mul, spoil);
            }
          }
          if (!inside) {
            bool seen;
            token_of(tl, tok, seen);
            if (!seen) {
              vw[mt][h] = 0.0f;
#pragma unroll
              for (int ht = 0; ht < HT; ++ht) s[ht][mt][2 * h] = s[ht][mt][2 * h + 1] = -INFINITY;
            }
          }
        }
      }
      float v_top = 0.0f;
      if constexpr (kCodes) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) v_top = max3(v_top, fabsf(vw[mt][0]), fabsf(vw[mt][1]));
      }
#pragma unroll
      for (int ht = 0; ht < HT; ++ht) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float top = fmaxf(s[ht][0][c], s[ht][0][2 + c]);
#pragma unroll
          for (int mt = 1; mt < MT; ++mt) top = max3(top, s[ht][mt][c], s[ht][mt][2 + c]);
          move |= top * q_mul[ht][c] > m[ht][c] + kSlack;
          // none of the lane's operands below is larger than this
          if constexpr (kCodes) move |= !(exp2_approx(fmaf(top, q_mul[ht][c], kLift - m[ht][c])) * v_top * v_mul[ht][c] <= 0x1p15f);
        }
      }
      // hidden tokens of a group that was copied whole may hold anything: their
      // values have to be finite beside weights of zero (codes always are)
      if constexpr (RUN && !kCodes) {
        if (!inside) {
          bool seen;
          token_of(tl, lane, seen);
          if (lane < TT && !seen) {
#pragma unroll
            for (int x = 0; x < Shape::kBoxes; ++x) {
#pragma unroll
              for (int i = 0; i < Shape::kBox; i += 16)
                asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(stage + Shape::kRowBytes + (x * TT + lane) * Shape::kBox + i), "r"(0u)
                             : "memory");
            }
          }
          fence_proxy_async_smem();  // before the next copy into these rows
          __syncwarp();
        }
      }
      // ---- the running maximum and the largest weight times scale, when they have to move
      if (__any_sync(0xffffffffu, move)) {
#pragma unroll
        for (int ht = 0; ht < HT; ++ht) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float top = -INFINITY;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) top = fmaxf(top, fmaxf(s[ht][mt][c], s[ht][mt][2 + c]));
#pragma unroll
            for (int x = 4; x < 32; x *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
            top *= q_mul[ht][c];
            float fall = 0.0f;  // log2 of what the weights so far are multiplied by
            if (top > m[ht][c]) {
              fall = m[ht][c] - top;
              m[ht][c] = top;
              l[ht][c] *= exp2f(fall);
            }
            if constexpr (kCodes) {
              float x = 0.0f;
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                  x = fmaxf(x, exp2_approx(fmaf(s[ht][mt][2 * h + c], q_mul[ht][c], -m[ht][c])) * fabsf(vw[mt][h]));
              }
#pragma unroll
              for (int y = 4; y < 32; y *= 2) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, y));
              x = fmaxf(x, exp2f(fall) * v_size(ht, c));
              const uint32_t e = __float_as_uint(x) >> 23;  // 2^(127 - e) takes x into [1, 2)
              const uint32_t next = 254u - (e < 1u ? 1u : (e > 253u ? 253u : e));
              fall += static_cast<float>(static_cast<int>(next) - static_cast<int>(__float_as_uint(v_mul[ht][c]) >> 23));
              v_mul[ht][c] = __uint_as_float(next << 23);
            }
            const float keep = exp2f(fall);
            o_bias[ht][c] *= keep;
#pragma unroll
            for (int i = 0; i < KS; ++i) {
              o[ht][i][c] *= keep;
              o[ht][i][2 + c] *= keep;
            }
          }
        }
      }
      // ---- weights, as the B operand
      uint32_t p[HT][MT][2], p_lo[HT][MT][2];
#pragma unroll
      for (int ht = 0; ht < HT; ++ht) {
        const float z0 = (m[ht][0] == -INFINITY ? 0.0f : m[ht][0]) - kLift;
        const float z1 = (m[ht][1] == -INFINITY ? 0.0f : m[ht][1]) - kLift;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float w0 = exp2_approx(fmaf(s[ht][mt][2 * h], q_mul[ht][0], -z0)), w1 = exp2_approx(fmaf(s[ht][mt][2 * h + 1], q_mul[ht][1], -z1));
            if (!inside) {  // a factor of zero takes a hidden token's -infinity to NaN
              bool seen;
              token_of(tl, 16 * mt + 8 * h + order, seen);
              w0 = seen ? w0 : 0.0f;
              w1 = seen ? w1 : 0.0f;
            }
            l[ht][0] += w0;
            l[ht][1] += w1;
            if constexpr (kCodes) {
              w0 = w0 * vw[mt][h] * v_mul[ht][0];
              w1 = w1 * vw[mt][h] * v_mul[ht][1];
            }
            // what 16 bits cut off, kept in a second operand
            if constexpr (kBf16) {
              const uint32_t hi = pack_bf16(w0, w1);
              p[ht][mt][h] = movmatrix(hi);
              p_lo[ht][mt][h] = movmatrix(pack_bf16(w0 - __uint_as_float(hi << 16), w1 - __uint_as_float(hi & 0xFFFF0000u)));
            } else {
              const uint32_t hi = pack_f16(w0, w1);
              p[ht][mt][h] = movmatrix(hi);
              if constexpr (kTwoParts) {
                const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&hi));
                p_lo[ht][mt][h] = movmatrix(pack_f16(w0 - back.x, w1 - back.y));
              }
            }
          }
        }
      }
      // ---- O^T += V^T P
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int i = 0; i < VP; ++i) {
          uint32_t vr[4][kVBytes / 4];  // tokens 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int r = 16 * mt + 8 * (k >> 1) + ((k & 1) ? order_odd : order_even);
            load_piece<kVBytes>(vr[k], stage + Shape::kRowBytes + (kVBytes == 16 ? box_offset<Shape, TT>(r, 8 * i + g)
                                                                                : box_offset<Shape, TT>(r, g >> 1) + 8 * (g & 1)));
          }
#pragma unroll
          for (int w = 0; w < kVBytes / 4; ++w) {
            const uint32_t va = vr[0][w], vb = vr[1][w], vc = vr[2][w], vd = vr[3][w];
            if constexpr (kCodes) {  // four channels of two tokens pairs: two row tiles
              const int tile0 = (i * (kVBytes / 4) + w) * 2;
              const uint32_t ab01 = prmt(va, vb, 0x5140u) ^ 0x80808080u, ab23 = prmt(va, vb, 0x7362u) ^ 0x80808080u;
              const uint32_t cd01 = prmt(vc, vd, 0x5140u) ^ 0x80808080u, cd23 = prmt(vc, vd, 0x7362u) ^ 0x80808080u;
#pragma unroll
              for (int ht = 0; ht < HT; ++ht) {
                mma16816<false>(o[ht][tile0], bytes_f16(ab01, 0x4140u), bytes_f16(ab01, 0x4342u),
                                bytes_f16(cd01, 0x4140u), bytes_f16(cd01, 0x4342u), p[ht][mt][0], p[ht][mt][1]);
                mma16816<false>(o[ht][tile0 + 1], bytes_f16(ab23, 0x4140u), bytes_f16(ab23, 0x4342u),
                                bytes_f16(cd23, 0x4140u), bytes_f16(cd23, 0x4342u), p[ht][mt][0], p[ht][mt][1]);
                if constexpr (kTwoParts) {
                  mma16816<false>(o[ht][tile0], bytes_f16(ab01, 0x4140u), bytes_f16(ab01, 0x4342u),
                                  bytes_f16(cd01, 0x4140u), bytes_f16(cd01, 0x4342u), p_lo[ht][mt][0], p_lo[ht][mt][1]);
                  mma16816<false>(o[ht][tile0 + 1], bytes_f16(ab23, 0x4140u), bytes_f16(ab23, 0x4342u),
                                  bytes_f16(cd23, 0x4140u), bytes_f16(cd23, 0x4342u), p_lo[ht][mt][0], p_lo[ht][mt][1]);
                }
              }
            } else {  // two channels of two token pairs: one row tile
              const int tile0 = i * (kVBytes / 4) + w;
              const uint32_t a0 = prmt(va, vb, 0x5410u), a1 = prmt(va, vb, 0x7632u);
              const uint32_t a2 = prmt(vc, vd, 0x5410u), a3 = prmt(vc, vd, 0x7632u);
#pragma unroll
              for (int ht = 0; ht < HT; ++ht) {
                mma16816<kBf16>(o[ht][tile0], a0, a1, a2, a3, p[ht][mt][0], p[ht][mt][1]);
                if constexpr (kTwoParts)
                  mma16816<kBf16>(o[ht][tile0], a0, a1, a2, a3, p_lo[ht][mt][0], p_lo[ht][mt][1]);
              }
            }
          }
        }
      }
      if constexpr (kCodes) {
        // the bias is a sum of weights that an operand of 128s collects; it leaves O
        // every other tile, before it grows large beside it
#pragma unroll
        for (int ht = 0; ht < HT; ++ht) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            mma16816<false>(o_bias[ht], 0x00800080u, 0x00800080u, 0x00800080u, 0x00800080u, p[ht][mt][0], p[ht][mt][1]);
            if constexpr (kTwoParts)
              mma16816<false>(o_bias[ht], 0x00800080u, 0x00800080u, 0x00800080u, 0x00800080u, p_lo[ht][mt][0], p_lo[ht][mt][1]);
          }
        }
        biased = !biased;
        if (!biased) remove_bias();
      }
      // ---- refill the stage; its table entries were asked for one tile ago
      __syncwarp();
      if (tl + kStages * W < t1) {
        issue(st, row_of(page_next, in_page_next));
      } else if constexpr (kCodes) {
        copies_commit();
      }
      page_next = find_page(tl + (kStages + 1) * W, in_page_next);
      st = st + 1 == kStages ? 0 : st + 1;
    }
    if constexpr (kCodes) copies_wait<0>();
    if (__any_sync(0xffffffffu, broken || (dead && t0 + warp < t1))) {
      // copies still on their way are waited for (each wait bounded) before the
      // ring is used again, which it is not once a copy has failed to come
      for (int i = 0; i < kStages && tl + i * W < t1 && opened; ++i) {
        const int at = st + i < kStages ? st + i : st + i - kStages;
        if (!__all_sync(0xffffffffu, mbar_wait_parity(bars + at, (filled >> at) & 1u))) dead = true;
        filled ^= 1u << at;
      }
      __syncwarp();
#pragma unroll
      for (int ht = 0; ht < HT; ++ht) l[ht][0] = l[ht][1] = NAN;
    }

    if (kCodes && biased) remove_bias();
    // ---- join the warps
#pragma unroll
    for (int ht = 0; ht < HT; ++ht) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float sum = l[ht][c];
#pragma unroll
        for (int x = 4; x < 32; x *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        const int h = 8 * ht + 2 * t + c;
        if (g == 0) {
          s_stat[(warp * kHeads + h) * 2] = m[ht][c];
          s_stat[(warp * kHeads + h) * 2 + 1] = sum;
        }
        // codes: 2^24 / v_mul in two factors, either of which is finite
        const float inv = (kCodes ? 0x1p24f : 1.0f) * inverse(sum), size = kCodes ? v_size(ht, c) : 1.0f;
        // row tile i holds the lane's channels 2i and 2i + 1, counted over its V pieces
        float* dst = s_o + (warp * kHeads + h) * Shape::kPitch + kVPiece * g;
#pragma unroll
        for (int i = 0; i < KS; i += 2) {
          const int ch = (2 * i / kVPiece) * 8 * kVPiece + 2 * i % kVPiece;
          *reinterpret_cast<float4*>(dst + ch) = make_float4(o[ht][i][c] * inv * size, o[ht][i][2 + c] * inv * size,
                                                             o[ht][i + 1][c] * inv * size, o[ht][i + 1][2 + c] * inv * size);
        }
      }
    }
    // on to the next item: its first copies are on their way while this one is joined
    const bool complete = t0 == 0 && t1 == n, empty = vis.len == 0;
    const int done_head0 = head0, done_heads = heads;
    const int64_t done_seq = seq, done_begin = item_begin;
    const bool cut = t1 < n;  // the range ends inside the item
    advance();
    const bool more = unit + kItemCost < unit_end;  // a tile of it is this CTA's
    if (!cut && !more && !a.whole && threadIdx.x == 0) a.cuts[blockIdx.x].seq = -1;
    if (more) {
      open();
      record_cut();
    }
    __syncthreads();  // every warp has left its part
    float* part = a.parts + (static_cast<int64_t>(blockIdx.x) * 2 + (done_begin + kItemCost < range_begin ? 0 : 1)) *
                                static_cast<int64_t>(Shape::kPartFloats);
    for (int x = threadIdx.x; x < done_heads * (D / 4); x += 32 * W) {
      const int h = x / (D / 4), c = (x - h * (D / 4)) * 4;
      float top = -INFINITY, total = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) top = fmaxf(top, s_stat[(w * kHeads + h) * 2]);
      float share[W];
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float mw = s_stat[(w * kHeads + h) * 2];
        share[w] = s_stat[(w * kHeads + h) * 2 + 1] * (mw == top ? 1.0f : exp2f(mw - top));
        total += share[w];
      }
      const float inv = inverse(total);
      float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float f = share[w] * inv;
        const float4 v = *reinterpret_cast<const float4*>(s_o + (w * kHeads + h) * Shape::kPitch + c);
        sum.x = fmaf(v.x, f, sum.x);
        sum.y = fmaf(v.y, f, sum.y);
        sum.z = fmaf(v.z, f, sum.z);
        sum.w = fmaf(v.w, f, sum.w);
      }
      if (complete) {
        const int64_t at = done_seq * a.q_heads + done_head0 + h;
        // no weight at all, though tokens are visible: 0 / 0
        store_row4(static_cast<T*>(a.out) + at * D + c, sum, total == 0.0f && !empty ? NAN : 1.0f);
        if (a.lse != nullptr && c == 0)
          a.lse[at] = empty ? -INFINITY : ((top == -INFINITY ? 0.0f : top) + log2_weights<T, C>(total)) * kLn2;
      } else {
        *reinterpret_cast<float4*>(part + h * D + c) = sum;
        if (c == 0) {
          part[kHeads * D + 2 * h] = top;
          part[kHeads * D + 2 * h + 1] = total;
        }
      }
    }
    if (!more) break;
    __syncthreads();  // the parts are read; the next item's go there
  }
}

// ---------------------------------------------------------------- joining kernel

constexpr int kPagedJoinThreads = 512;

// Joins what CTAs have left of the items that their ranges cut. There is one CTA
// per border between two ranges, and those inside an item share its heads. A head
// takes D / 4 threads, each up to kBatch parts whose loads are all on their way
// at once; of an item with more parts, several such rows, joined through shared memory.
// It adds 3 us to the main kernel, most of them two trips to L2 (1 x 131072 bf16: 88 us
// in all, 84 without it; 91 with one border doing all heads, a part after the
// other; 89 with kBatch 2, and 88 with 8, whose registers delay the CTAs' start).
template <typename T, typename C, int D, int HT>
__global__ void __launch_bounds__(kPagedJoinThreads) paged_attention_join_kernel(const PagedArgs a) {
  using Shape = PagedShape<C, D, HT, 4>;
  constexpr int kHeads = Shape::kHeads, kVec = D / 4, kRows = kPagedJoinThreads / kVec, kBatch = 4;
  static_assert(kRows >= kHeads, "a row per head");
  __shared__ __align__(16) float s_o[kRows][D];
  __shared__ float s_m[kRows], s_l[kRows];
  pdl_launch_dependents();
  pdl_wait_primary();
  const PagedCut cut = a.cuts[blockIdx.x];
  if (cut.seq < 0) return;
  const int kvh = cut.item / a.head_sets, set = cut.item - kvh * a.head_sets;
  const int heads = a.group - set * kHeads < kHeads ? a.group - set * kHeads : kHeads;
  const int parts = cut.last - cut.first + 1;
  // this border has heads share, share + sharers, ...
  const int share = static_cast<int>(blockIdx.x) - cut.first, sharers = parts - 1 < heads ? parts - 1 : heads;
  if (share >= sharers) return;
  const int mine = (heads - share + sharers - 1) / sharers;
  const int want = (parts + kBatch - 1) / kBatch, splits = want * mine <= kRows ? want : kRows / mine;
  const int vec = threadIdx.x % kVec, row = threadIdx.x / kVec, split = row / mine;
  const int h = share + (row - split * mine) * sharers;

  float top = -INFINITY, sum_l = 0.0f;
  float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (split < splits) {
    for (int c0 = cut.first + split; c0 <= cut.last; c0 += kBatch * splits) {
      float2 st[kBatch];
      float4 v[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int64_t c = c0 + i * splits;
        st[i] = make_float2(-INFINITY, 0.0f);
        v[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (c <= cut.last) {
          const float* part = a.parts + (c * 2 + (c == cut.first ? 1 : 0)) * static_cast<int64_t>(Shape::kPartFloats);
          st[i] = *reinterpret_cast<const float2*>(part + kHeads * D + 2 * h);
          v[i] = *reinterpret_cast<const float4*>(part + h * D + 4 * vec);
        }
      }
      float next = top;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) next = fmaxf(next, st[i].x);
      const float before = sum_l * (top == next ? 1.0f : exp2f(top - next));
      float share[kBatch];
      sum_l = before;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        share[i] = st[i].y * (st[i].x == next ? 1.0f : exp2f(st[i].x - next));
        sum_l += share[i];
      }
      const float inv = inverse(sum_l), keep = before * inv;
      sum.x *= keep, sum.y *= keep, sum.z *= keep, sum.w *= keep;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const float f = share[i] * inv;
        sum.x = fmaf(v[i].x, f, sum.x);
        sum.y = fmaf(v[i].y, f, sum.y);
        sum.z = fmaf(v[i].z, f, sum.z);
        sum.w = fmaf(v[i].w, f, sum.w);
      }
      top = next;
    }
  }
  if (splits > 1) {
    *reinterpret_cast<float4*>(&s_o[row][4 * vec]) = sum;
    if (vec == 0) {
      s_m[row] = top;
      s_l[row] = sum_l;
    }
    __syncthreads();
    if (split == 0) {
      for (int p = row + mine; p < splits * mine; p += mine) top = fmaxf(top, s_m[p]);
      sum_l = 0.0f;
      for (int p = row; p < splits * mine; p += mine) sum_l = fmaf(s_l[p], s_m[p] == top ? 1.0f : exp2f(s_m[p] - top), sum_l);
      const float inv = inverse(sum_l);
      sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int p = row; p < splits * mine; p += mine) {
        const float f = s_l[p] * (s_m[p] == top ? 1.0f : exp2f(s_m[p] - top)) * inv;
        const float4 v = *reinterpret_cast<const float4*>(&s_o[p][4 * vec]);
        sum.x = fmaf(v.x, f, sum.x);
        sum.y = fmaf(v.y, f, sum.y);
        sum.z = fmaf(v.z, f, sum.z);
        sum.w = fmaf(v.w, f, sum.w);
      }
    }
  }
  if (split == 0) {
    const int64_t at = cut.seq * a.q_heads + kvh * a.group + set * kHeads + h;
    store_row4(static_cast<T*>(a.out) + at * D + 4 * vec, sum, sum_l == 0.0f ? NAN : 1.0f);
    if (vec == 0 && a.lse != nullptr) a.lse[at] = ((top == -INFINITY ? 0.0f : top) + log2_weights<T, C>(sum_l)) * kLn2;
  }
}

}  // namespace dq
