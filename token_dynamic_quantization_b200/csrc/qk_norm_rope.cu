// RMS norm of every query and key head with the position rotation in the same
// pass, keys and values optionally written into a paged 16-bit or INT8 cache
// (dq_qk_norm_rope, dq_qk_norm_rope_cache).
//
// For a head row x of D values with weight w:
//   y = x * rsqrt(mean(x^2) + epsilon) * w
//   (y[a], y[b]) <- (y[a] cos - y[b] sin, y[b] cos + y[a] sin)
// The angle is reduced in integers (a binary32 product of inv_freq with a
// position of 100000 is off by up to 2^-8 of a radian).
#include <cmath>

#include "dq.h"
#include "dq_device.cuh"
#include "dq_launch.cuh"

namespace dq {

struct NormRopeArgs {
  const void* q;
  const void* k;
  const void* v;  // cache calls only
  int64_t q_stride, k_stride, v_stride;
  int64_t tokens;
  int q_heads, kv_heads, head_dim;
  const void* q_weight;
  const void* k_weight;
  int weight_dtype;
  float epsilon;
  float inv_dim;
  const int32_t* positions;
  const float* inv_freq;
  int rope_dim;
  int interleaved;
  void* q_out;
  void* k_out;  // nullptr for cache calls
  int64_t q_out_stride, k_out_stride;
  void* k_cache;
  void* v_cache;
  float* k_scale;
  float* v_scale;
  const int64_t* slots;
  int64_t num_slots;
  int page_size;
  int parts;       // vector kernel: warps that share a token's rows
  int lane_shift;  // vector kernel: log2 of the lanes per row
};

enum : int { kCacheNone = 0, kCacheSame = 1, kCacheInt8 = 2 };

// An angle pos * inv_freq is pos * (inv_freq / 2 pi) turns, of which only the
// fraction counts: with inv_freq / 2 pi as a 64-bit fraction of a turn (from its
// binary64 value), the integer product with the position is exact modulo one
// turn, and its upper half is the angle to 2^-32 of a turn.
__device__ __forceinline__ void rope_angle(int32_t pos, float inv_freq, float& c, float& s) {
  const double t = static_cast<double>(inv_freq) * 0.15915494309189533577;  // 1 / (2 pi)
  const uint64_t turns = static_cast<uint64_t>((t - floor(t)) * 0x1p63) << 1;
  const uint64_t part = static_cast<uint64_t>(static_cast<int64_t>(pos)) * turns;
  sincospif(static_cast<float>(static_cast<int32_t>(part >> 32)) * 0x1p-31f, &s, &c);
}

__device__ __forceinline__ float warp_sum_f32(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Maxima that a NaN passes through, for the magnitudes of a row that becomes codes:
// the scale absmax / 127 of a row with a NaN is NaN (and so is that of a row with an
// infinity), which the attention over the cache turns into NaN where it is visible.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float warp_max_nan(float v) {
  float r;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

template <typename T>
__device__ __forceinline__ T narrow(float v);
template <>
__device__ __forceinline__ __half narrow<__half>(float v) {
  return __float2half_rn(v);
}
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

constexpr int kNormRopeBlock = 128;
// CTAs per SM of the vector kernel, which bounds its registers (102): 8192 tokens of
// 32 and 8 heads of 128 channels take 35 us with 5, 35 with 4 and 40 with 6; INT8
// pages 88, 94 and 106 us.
constexpr int kNormRopeCtas = 5;
// Few tokens: warps per SM that the rows of the tokens are spread over. 1003 tokens
// of 12 and 4 heads take 5.5 us with 16, 6.8 with 8 and 7.8 with 32 (each warp
// computes its token's angles anew).
constexpr int kNormRopeWarps = 16;

// Any head dimension, stride and alignment: one warp per (token, head row),
// the row in registers (rotation pairs lane, lane + 32, ..., then the channels
// that are only normed), so an output may overwrite its own input.
template <typename T, int CACHE>
__global__ void __launch_bounds__(kNormRopeBlock) norm_rope_generic_kernel(const NormRopeArgs a) {
  pdl_launch_dependents();
  pdl_wait_primary();
  const int lane = threadIdx.x & 31;
  const int rows_per_token = a.q_heads + a.kv_heads * (CACHE == kCacheNone ? 1 : 2);
  const int64_t rows = a.tokens * rows_per_token;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kNormRopeBlock / 32);
  const int pairs = a.rope_dim / 2;
  constexpr int kPairs = DQ_MAX_HEAD_DIM / 64, kRest = DQ_MAX_HEAD_DIM / 32;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * (kNormRopeBlock / 32) + (threadIdx.x >> 5); row < rows;
       row += warps) {
    const int64_t t = row / rows_per_token;
    int h = static_cast<int>(row - t * rows_per_token);
    const int which = h < a.q_heads ? 0 : (h < a.q_heads + a.kv_heads ? 1 : 2);
    h -= which == 0 ? 0 : (which == 1 ? a.q_heads : a.q_heads + a.kv_heads);
    const T* x = static_cast<const T*>(which == 0 ? a.q : (which == 1 ? a.k : a.v)) +
                 t * (which == 0 ? a.q_stride : (which == 1 ? a.k_stride : a.v_stride)) +
                 static_cast<int64_t>(h) * a.head_dim;
    int64_t slot = 0;
    if (CACHE != kCacheNone && which != 0) {
      slot = a.slots[t];
      if (slot < 0 || slot >= a.num_slots) continue;
    }
    float first[kPairs], second[kPairs], rest[kRest];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const int p = lane + 32 * i;
      const bool in = p < pairs;
      first[i] = in ? static_cast<float>(x[a.interleaved ? 2 * p : p]) : 0.0f;
      second[i] = in ? static_cast<float>(x[a.interleaved ? 2 * p + 1 : p + pairs]) : 0.0f;
      sum = fmaf(first[i], first[i], fmaf(second[i], second[i], sum));
    }
#pragma unroll
    for (int i = 0; i < kRest; ++i) {
      const int c = a.rope_dim + lane + 32 * i;
      rest[i] = c < a.head_dim ? static_cast<float>(x[c]) : 0.0f;
      sum = fmaf(rest[i], rest[i], sum);
    }
    if (which != 2) {
      const float r = rsqrtf(fmaf(warp_sum_f32(sum), a.inv_dim, a.epsilon));
      const void* w = which == 0 ? a.q_weight : a.k_weight;
      const int32_t pos = a.positions[t];
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const int p = lane + 32 * i;
        if (p < pairs) {
          const int e0 = a.interleaved ? 2 * p : p, e1 = a.interleaved ? 2 * p + 1 : p + pairs;
          const float y0 = first[i] * r * (w ? load_param(w, a.weight_dtype, e0) : 1.0f);
          const float y1 = second[i] * r * (w ? load_param(w, a.weight_dtype, e1) : 1.0f);
          float c, s;
          rope_angle(pos, a.inv_freq[p], c, s);
          first[i] = y0 * c - y1 * s;
          second[i] = y1 * c + y0 * s;
        }
      }
#pragma unroll
      for (int i = 0; i < kRest; ++i) {
        const int c = a.rope_dim + lane + 32 * i;
        if (c < a.head_dim) rest[i] = rest[i] * r * (w ? load_param(w, a.weight_dtype, c) : 1.0f);
      }
    }
    if (CACHE == kCacheInt8 && which != 0) {
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < kPairs; ++i) top = max_nan(top, fabsf(first[i]), fabsf(second[i]));
#pragma unroll
      for (int i = 0; i < kRest; ++i) top = max_nan(top, fabsf(rest[i]));
      const RowQuant rq = make_sym<127>(warp_max_nan(top));
      const int64_t page = slot / a.page_size;
      const int64_t at = (page * a.kv_heads + h) * a.page_size + (slot - page * a.page_size);
      int8_t* y = static_cast<int8_t*>(which == 1 ? a.k_cache : a.v_cache) + at * a.head_dim;
      const auto code = [&](float v) {
        return static_cast<int8_t>(rq.zero_scale ? 0 : code_exact<false>(v, rq, -127.0f, 127.0f));
      };
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const int p = lane + 32 * i;
        if (p < pairs) {
          y[a.interleaved ? 2 * p : p] = code(first[i]);
          y[a.interleaved ? 2 * p + 1 : p + pairs] = code(second[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < kRest; ++i) {
        const int c = a.rope_dim + lane + 32 * i;
        if (c < a.head_dim) y[c] = code(rest[i]);
      }
      if (lane == 0) (which == 1 ? a.k_scale : a.v_scale)[at] = rq.scale;
      continue;
    }
    T* y;
    if (which == 0) {
      y = static_cast<T*>(a.q_out) + t * a.q_out_stride + static_cast<int64_t>(h) * a.head_dim;
    } else if (CACHE == kCacheNone) {
      y = static_cast<T*>(a.k_out) + t * a.k_out_stride + static_cast<int64_t>(h) * a.head_dim;
    } else {
      const int64_t page = slot / a.page_size;
      y = static_cast<T*>(which == 1 ? a.k_cache : a.v_cache) +
          ((page * a.kv_heads + h) * a.page_size + (slot - page * a.page_size)) * a.head_dim;
    }
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const int p = lane + 32 * i;
      if (p < pairs) {
        y[a.interleaved ? 2 * p : p] = narrow<T>(first[i]);
        y[a.interleaved ? 2 * p + 1 : p + pairs] = narrow<T>(second[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < kRest; ++i) {
      const int c = a.rope_dim + lane + 32 * i;
      if (c < a.head_dim) y[c] = narrow<T>(rest[i]);
    }
  }
}

// ---- vector kernel

// VEC values of one chunk (8: 16 bytes, 4: 8 bytes).
template <typename T, int VEC>
struct Chunk {
  uint32_t w[VEC / 2];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (VEC == 8) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x, w[1] = v.y;
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (VEC == 8) {
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ void widen(float2 (&f)[VEC / 2]) const {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      if constexpr (__is_same(T, __nv_bfloat16)) {
        f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
      } else {
        f[i] = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      }
    }
  }
  __device__ __forceinline__ void narrow(const float2 (&f)[VEC / 2]) {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      if constexpr (__is_same(T, __nv_bfloat16)) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[i].x, f[i].y);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __half2 h = __floats2half2_rn(f[i].x, f[i].y);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
  }
};

// VEC weights from channel c on, as binary32.
template <int VEC>
__device__ __forceinline__ void load_weights(const void* p, int dtype, int c, float2 (&w)[VEC / 2]) {
  if (p == nullptr) {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) w[i] = make_float2(1.0f, 1.0f);
  } else if (dtype == kF32) {
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + c) + i);
      w[2 * i] = make_float2(v.x, v.y);
      w[2 * i + 1] = make_float2(v.z, v.w);
    }
  } else if (dtype == kF16) {
    Chunk<__half, VEC> x;
    x.load(static_cast<const __half*>(p) + c);
    x.widen(w);
  } else {
    Chunk<__nv_bfloat16, VEC> x;
    x.load(static_cast<const __nv_bfloat16*>(p) + c);
    x.widen(w);
  }
}

// A warp takes one token and loops over its head rows, 32 / L rows at a time,
// L the power of two that covers head_dim / (2 VEC) lanes: each lane holds two
// chunks of VEC channels, those that rotate with each other (i and i +
// rope_dim / 2) or two neighbouring ones (interleaved pairs, channels past
// rope_dim), so the rotation needs no exchange. A token's angles are computed
// once, each by one lane, and handed round. The next rows are loaded before the
// current ones are worked on. Few tokens: `parts` warps share one token's rows.
//
// Bound by memory in the limit: 8192 tokens read and write 168 MB, 25.6 us at the
// copy rate, and take 35 (4.8 TB/s, half of the written rows still in L2 when the kernel
// ends; issue slots at 49 %, waiting for loads most of the rest); into 16-bit pages 42 us
// against 30.7, into INT8 pages (16384 tokens) 88 against 56.5, and of 4 and 1 heads a token,
// whose angles weigh more, 14.8 against 3.9. The same kernel without the angles takes 31
// and as a bare copy 27. Loading two or three groups of rows ahead costs more
// registers than it hides (36 and 38 us), and so does folding the weights into the
// sines and cosines (36); warps that stay and walk over tokens take 40.
template <typename T, int VEC, int CACHE, int LANES>
__global__ void __launch_bounds__(kNormRopeBlock, kNormRopeCtas) norm_rope_kernel(const NormRopeArgs a) {
  constexpr int H = VEC / 2;
  __shared__ __align__(16) float s_cos[kNormRopeBlock / 32][DQ_MAX_HEAD_DIM / 2];
  __shared__ __align__(16) float s_sin[kNormRopeBlock / 32][DQ_MAX_HEAD_DIM / 2];
  pdl_launch_dependents();
  pdl_wait_primary();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int lanes = LANES ? LANES : 1 << a.lane_shift, rows_at_once = 32 / lanes, l = lane & (lanes - 1);
  const int normed_rows = a.q_heads + a.kv_heads;
  const int heads = normed_rows + (CACHE == kCacheNone ? 0 : a.kv_heads);

  // the lane's chunks
  const int half = a.rope_dim / 2, pair_chunks = a.interleaved ? 0 : half / VEC;
  const bool split = l < pair_chunks;
  const int c0 = (split ? l : pair_chunks + 2 * (l - pair_chunks) + pair_chunks) * VEC;
  const int c1 = split ? c0 + half : c0 + VEC;
  const bool in = c1 < a.head_dim;
  const int apart = c1 - c0;
  const int step = rows_at_once * a.parts;

  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kNormRopeBlock / 32) + warp;
  const int64_t token = unit / a.parts;
  if (token >= a.tokens) return;
  const int begin = static_cast<int>(unit - token * a.parts) * rows_at_once;

  // Rows 0 .. heads - 1 of the token are its queries, keys and values. A place
  // walks over them `step` rows at a time; only where a kind ends is it looked up.
  struct Place {
    int row, which, end;
    const T* p;
  };
  const auto find = [&](Place& x) {
    x.which = x.row < a.q_heads ? 0 : (x.row < normed_rows ? 1 : 2);
    x.end = x.which == 0 ? a.q_heads : (x.which == 1 ? normed_rows : heads);
    const int at = x.row - (x.which == 0 ? 0 : (x.which == 1 ? a.q_heads : normed_rows));
    const T* base = static_cast<const T*>(x.which == 0 ? a.q : (x.which == 1 ? a.k : a.v));
    x.p = base + token * (x.which == 0 ? a.q_stride : (x.which == 1 ? a.k_stride : a.v_stride)) + at * a.head_dim + c0;
  };
  Place from;
  from.row = begin + (lane / lanes);
  find(from);
  Chunk<T, VEC> x0, x1;
  const auto fetch = [&]() {
    if (from.row < heads && in) {
      x0.load(from.p);
      x1.load(from.p + apart);
    } else {
      x0.clear();
      x1.clear();
    }
    from.row += step;
    from.p += step * a.head_dim;
    if (from.row >= from.end && from.row < heads) find(from);
  };
  fetch();

  // Angles: angle i turns channels (i, i + rope_dim / 2), or (2i, 2i + 1). The
  // lanes compute them once for the token's rows, then each picks its own VEC.
  float2 cs[H], sn[H], ns[H];
  // chunks whose channels turn; the others are left out below, not turned by an angle of
  // zero: an infinity would make its partner NaN
  const bool turn0 = a.interleaved ? c0 < a.rope_dim : split, turn1 = a.interleaved ? c1 < a.rope_dim : split;
  if (half > 0) {
    const int32_t pos = a.positions[token];
    for (int i = lane; i < half; i += 32) rope_angle(pos, a.inv_freq[i], s_cos[warp][i], s_sin[warp][i]);
    __syncwarp();
  }
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    // split: c0 + i; interleaved: c0 / 2 ... of the first chunk, then c1 / 2 ... of the second
    const int want = a.interleaved ? (i < H ? c0 / 2 + i : c1 / 2 + i - H) : c0 + i;
    const bool turned = i < H ? turn0 : turn1;
    const float c = turned ? s_cos[warp][want] : 1.0f, z = turned ? s_sin[warp][want] : 0.0f;
    if (i & 1) {
      cs[i / 2].y = c, sn[i / 2].y = z, ns[i / 2].y = -z;
    } else {
      cs[i / 2].x = c, sn[i / 2].x = z, ns[i / 2].x = -z;
    }
  }
  int64_t slot = -1, page_row = 0;
  if (CACHE != kCacheNone) {
    slot = a.slots[token];
    if (slot >= a.num_slots) slot = -1;
    if (slot >= 0) {
      const int64_t page = slot / a.page_size;
      page_row = page * a.kv_heads * a.page_size + (slot - page * a.page_size);
    }
  }

  // where the rows go: elements (codes: bytes) of q_out, k_out or a cache
  Place to;
  to.row = begin + (lane / lanes);
  char* out = nullptr;
  int64_t out_step = 0, cache_row = 0;
  float2 w0[H], w1[H];
#pragma unroll
  for (int i = 0; i < H; ++i) w0[i] = w1[i] = f2(0.0f);  // lanes past the row: their zeros stay zeros
  const auto aim = [&]() {
    find(to);
    const int at = to.row - (to.which == 0 ? 0 : (to.which == 1 ? a.q_heads : normed_rows));
    if (to.which == 0) {
      out = static_cast<char*>(a.q_out) + (token * a.q_out_stride + at * a.head_dim + c0) * sizeof(T);
      out_step = static_cast<int64_t>(step) * a.head_dim * sizeof(T);
    } else if (CACHE == kCacheNone) {
      out = static_cast<char*>(a.k_out) + (token * a.k_out_stride + at * a.head_dim + c0) * sizeof(T);
      out_step = static_cast<int64_t>(step) * a.head_dim * sizeof(T);
    } else {
      constexpr int kElem = CACHE == kCacheInt8 ? 1 : sizeof(T);
      cache_row = page_row + static_cast<int64_t>(at) * a.page_size;
      out = static_cast<char*>(to.which == 1 ? a.k_cache : a.v_cache) + (cache_row * a.head_dim + c0) * kElem;
      out_step = static_cast<int64_t>(step) * a.page_size * a.head_dim * kElem;
    }
    if (to.which != 2 && in) {
      const void* w = to.which == 0 ? a.q_weight : a.k_weight;
      load_weights<VEC>(w, a.weight_dtype, c0, w0);
      load_weights<VEC>(w, a.weight_dtype, c1, w1);
    }
  };
  aim();

  const auto work_on = [&](int first, const Chunk<T, VEC>& r0, const Chunk<T, VEC>& r1) {
    float2 f0[H], f1[H];
    r0.widen(f0);
    r1.widen(f1);
    if (first < normed_rows) {  // some row of the warp is normed
      float2 sum2 = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int i = 0; i < H; ++i) sum2 = __ffma2_rn(f0[i], f0[i], __ffma2_rn(f1[i], f1[i], sum2));
      float sum = sum2.x + sum2.y;
#pragma unroll
      for (int o = 1; o < (LANES ? LANES : 32); o *= 2) {
        if (o < lanes) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      }
      if (to.which != 2) {
        const float r = rsqrtf(fmaf(sum, a.inv_dim, a.epsilon));
#pragma unroll
        for (int i = 0; i < H; ++i) {
          f0[i] = __fmul2_rn(__fmul2_rn(f0[i], f2(r)), w0[i]);
          f1[i] = __fmul2_rn(__fmul2_rn(f1[i], f2(r)), w1[i]);
        }
        if (a.interleaved) {
#pragma unroll
          for (int i = 0; i < H; ++i) {
            const float ca = i & 1 ? cs[i / 2].y : cs[i / 2].x, sa = i & 1 ? sn[i / 2].y : sn[i / 2].x;
            const float cb = i & 1 ? cs[(H + i) / 2].y : cs[(H + i) / 2].x, sb = i & 1 ? sn[(H + i) / 2].y : sn[(H + i) / 2].x;
            if (turn0) f0[i] = make_float2(f0[i].x * ca - f0[i].y * sa, f0[i].y * ca + f0[i].x * sa);
            if (turn1) f1[i] = make_float2(f1[i].x * cb - f1[i].y * sb, f1[i].y * cb + f1[i].x * sb);
          }
        } else if (turn0) {
#pragma unroll
          for (int i = 0; i < H; ++i) {
            const float2 y0 = f0[i], y1 = f1[i];
            f0[i] = __ffma2_rn(y0, cs[i], __fmul2_rn(y1, ns[i]));
            f1[i] = __ffma2_rn(y1, cs[i], __fmul2_rn(y0, sn[i]));
          }
        }
      }
    }
    const bool live = to.row < heads && in && (CACHE == kCacheNone || to.which == 0 || slot >= 0);
    if constexpr (CACHE == kCacheInt8) {
      if (first + rows_at_once > a.q_heads) {  // some row of the warp becomes codes
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < H; ++i)
          top = max_nan(top, max_nan(fabsf(f0[i].x), fabsf(f0[i].y)), max_nan(fabsf(f1[i].x), fabsf(f1[i].y)));
#pragma unroll
        for (int o = 1; o < (LANES ? LANES : 32); o *= 2) {
          if (o < lanes) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
        }
        if (to.which != 0) {
          if (live) {
            const RowQuant rq = make_sym<127>(top);
            uint32_t bits[8];
            const auto codes = [&](const float(&f)[8]) -> uint2 {
              if (rq.zero_scale) return make_uint2(0u, 0u);
              if (rq.exact_row) {
                quant8_exact<false>(f, rq, -127.0f, 127.0f, bits);
              } else {
                quant8<false, false>(f, rq, -127.0f, 127.0f, bits);
              }
              return pack8_int8(bits);
            };
            if constexpr (VEC == 8) {
              const float a0[8] = {f0[0].x, f0[0].y, f0[1].x, f0[1].y, f0[2].x, f0[2].y, f0[3].x, f0[3].y};
              const float a1[8] = {f1[0].x, f1[0].y, f1[1].x, f1[1].y, f1[2].x, f1[2].y, f1[3].x, f1[3].y};
              *reinterpret_cast<uint2*>(out) = codes(a0);
              *reinterpret_cast<uint2*>(out + apart) = codes(a1);
            } else {
              const float f[8] = {f0[0].x, f0[0].y, f0[1].x, f0[1].y, f1[0].x, f1[0].y, f1[1].x, f1[1].y};
              const uint2 b = codes(f);
              *reinterpret_cast<uint32_t*>(out) = b.x;
              *reinterpret_cast<uint32_t*>(out + apart) = b.y;
            }
            if (l == 0) (to.which == 1 ? a.k_scale : a.v_scale)[cache_row] = rq.scale;
          }
          return;
        }
      }
    }
    if (!live) return;
    Chunk<T, VEC> o0, o1;
    o0.narrow(f0);
    o1.narrow(f1);
    o0.store(reinterpret_cast<T*>(out));
    o1.store(reinterpret_cast<T*>(out) + apart);
  };

  // the bounds are the same for the whole warp: its lanes meet in the reductions
  for (int first = begin; first < heads; first += step) {
    const Chunk<T, VEC> r0 = x0, r1 = x1;
    fetch();
    work_on(first, r0, r1);
    to.row += step;
    out += out_step;
    cache_row += static_cast<int64_t>(step) * a.page_size;
    if (to.row >= to.end && to.row < heads) aim();
  }
}

}  // namespace dq

namespace {

using dq_host::aligned;

template <typename T, int CACHE>
dq_status launch_generic(const dq::NormRopeArgs& a, cudaStream_t stream) {
  void (*fn)(const dq::NormRopeArgs) = dq::norm_rope_generic_kernel<T, CACHE>;
  const int device = dq_host::current_device();
  const int64_t rows = a.tokens * (a.q_heads + a.kv_heads * (CACHE == dq::kCacheNone ? 1 : 2));
  const int64_t want = (rows + dq::kNormRopeBlock / 32 - 1) / (dq::kNormRopeBlock / 32);
  const int64_t most = static_cast<int64_t>(dq_host::sm_count(device)) * 8;
  return dq_host::launch_programmatic(fn, a, static_cast<int>(want < most ? want : most), dq::kNormRopeBlock, 0,
                                      stream);
}

// Whether every row splits into aligned chunks of `vec` values, two to a lane:
// pairs (i, i + rope_dim / 2) lie in two chunks, the rest in pairs of chunks.
bool vector_ok(const dq::NormRopeArgs& a, int cache, int vec) {
  const int bytes = 2 * vec, codes = vec;
  const int weight_bytes = a.weight_dtype == dq::kF32 ? 16 : bytes;
  if (!aligned(a.q_weight, weight_bytes) || !aligned(a.k_weight, weight_bytes)) return false;
  if (a.head_dim % (2 * vec) != 0) return false;
  if (a.interleaved ? a.rope_dim % vec != 0 : a.rope_dim / 2 % vec != 0) return false;
  const auto rows = [&](const void* p, int64_t stride) { return aligned(p, bytes) && stride % vec == 0; };
  if (!rows(a.q, a.q_stride) || !rows(a.k, a.k_stride) || !rows(a.q_out, a.q_out_stride)) return false;
  if (cache == dq::kCacheNone) return rows(a.k_out, a.k_out_stride);
  const int at = cache == dq::kCacheInt8 ? codes : bytes;
  return rows(a.v, a.v_stride) && aligned(a.k_cache, at) && aligned(a.v_cache, at);
}

template <typename T, int VEC, int CACHE, int LANES>
dq_status launch_vector(dq::NormRopeArgs a, cudaStream_t stream) {
  void (*fn)(const dq::NormRopeArgs) = dq::norm_rope_kernel<T, VEC, CACHE, LANES>;
  const int heads = a.q_heads + a.kv_heads * (CACHE == dq::kCacheNone ? 1 : 2);
  a.lane_shift = 0;
  while ((1 << a.lane_shift) * 2 * VEC < a.head_dim) ++a.lane_shift;
  // warps per token: one row each while the warps leave the device empty
  const int groups = (heads + (32 >> a.lane_shift) - 1) / (32 >> a.lane_shift);
  const int64_t room = static_cast<int64_t>(dq_host::sm_count(dq_host::current_device())) * dq::kNormRopeWarps;
  int64_t parts = room / a.tokens;
  a.parts = static_cast<int>(parts < 1 ? 1 : (parts > groups ? groups : parts));
  const int64_t warps = a.tokens * a.parts;
  const int64_t grid = (warps + dq::kNormRopeBlock / 32 - 1) / (dq::kNormRopeBlock / 32);
  return dq_host::launch_programmatic(fn, a, static_cast<int>(grid), dq::kNormRopeBlock, 0, stream);
}

template <typename T, int VEC, int CACHE>
dq_status by_lanes(const dq::NormRopeArgs& a, cudaStream_t stream) {
  if (VEC == 8 && a.head_dim > 32 && a.head_dim <= 64) return launch_vector<T, 8, CACHE, 4>(a, stream);
  if (VEC == 8 && a.head_dim > 64 && a.head_dim <= 128) return launch_vector<T, 8, CACHE, 8>(a, stream);
  return launch_vector<T, VEC, CACHE, 0>(a, stream);
}

template <typename T, int CACHE>
dq_status launch(const dq::NormRopeArgs& a, cudaStream_t stream) {
  if (vector_ok(a, CACHE, 8)) return by_lanes<T, 8, CACHE>(a, stream);
  if (vector_ok(a, CACHE, 4)) return by_lanes<T, 4, CACHE>(a, stream);
  return launch_generic<T, CACHE>(a, stream);
}

template <typename T>
dq_status dispatch(const dq::NormRopeArgs& a, int cache, cudaStream_t stream) {
  if (cache == dq::kCacheNone) return launch<T, dq::kCacheNone>(a, stream);
  if (cache == dq::kCacheSame) return launch<T, dq::kCacheSame>(a, stream);
  return launch<T, dq::kCacheInt8>(a, stream);
}

bool is_param_float(dq_dtype t) { return t == DQ_F32 || t == DQ_F16 || t == DQ_BF16; }
size_t float_size(dq_dtype t) { return t == DQ_F32 ? 4 : 2; }

// Checks shared by both entry points; *done is set when there is nothing to do.
dq_status check(const dq::NormRopeArgs& a, dq_dtype dtype, dq_dtype weight_dtype) {
  if (a.tokens < 0 || a.tokens >= (int64_t(1) << 31) || a.q_heads < 1 || a.q_heads > DQ_MAX_HEADS || a.kv_heads < 1 ||
      a.kv_heads > DQ_MAX_HEADS || a.head_dim < 1 || a.head_dim > DQ_MAX_HEAD_DIM)
    return DQ_ERR_BAD_SHAPE;
  if (a.rope_dim < 0 || a.rope_dim > a.head_dim || a.rope_dim % 2 != 0) return DQ_ERR_BAD_SHAPE;
  if (a.q_stride < static_cast<int64_t>(a.q_heads) * a.head_dim || a.q_out_stride < static_cast<int64_t>(a.q_heads) * a.head_dim ||
      a.k_stride < static_cast<int64_t>(a.kv_heads) * a.head_dim)
    return DQ_ERR_BAD_SHAPE;
  if (a.q_stride > (int64_t(1) << 31) || a.q_out_stride > (int64_t(1) << 31) || a.k_stride > (int64_t(1) << 31))
    return DQ_ERR_BAD_SHAPE;
  if (dtype != DQ_F16 && dtype != DQ_BF16) return DQ_ERR_BAD_DTYPE;
  if ((a.q_weight != nullptr || a.k_weight != nullptr) && !is_param_float(weight_dtype)) return DQ_ERR_BAD_DTYPE;
  if (!std::isfinite(a.epsilon) || a.epsilon < 0.0f) return DQ_ERR_BAD_ARGUMENT;
  if (a.interleaved != 0 && a.interleaved != 1) return DQ_ERR_BAD_ARGUMENT;
  return DQ_OK;
}

dq_status check_pointers(const dq::NormRopeArgs& a, dq_dtype weight_dtype) {
  if (a.q == nullptr || a.k == nullptr || a.q_out == nullptr || a.positions == nullptr ||
      (a.inv_freq == nullptr && a.rope_dim > 0))
    return DQ_ERR_NULL_POINTER;
  const size_t ws = float_size(weight_dtype);
  if (!aligned(a.q, 2) || !aligned(a.k, 2) || !aligned(a.q_out, 2) || !aligned(a.positions, 4) ||
      !aligned(a.inv_freq, 4) || (a.q_weight && !aligned(a.q_weight, ws)) || (a.k_weight && !aligned(a.k_weight, ws)))
    return DQ_ERR_MISALIGNED;
  return DQ_OK;
}

dq::NormRopeArgs common_args(const void* q, int64_t q_stride, const void* k, int64_t k_stride, int64_t tokens,
                             int32_t q_heads, int32_t kv_heads, int32_t head_dim, const void* q_weight,
                             const void* k_weight, dq_dtype weight_dtype, float epsilon, const int32_t* positions,
                             const float* inv_freq, int32_t rope_dim, int32_t interleaved, void* q_out,
                             int64_t q_out_stride) {
  dq::NormRopeArgs a{};
  a.q = q;
  a.k = k;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.tokens = tokens;
  a.q_heads = q_heads;
  a.kv_heads = kv_heads;
  a.head_dim = head_dim;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.weight_dtype = static_cast<int>(weight_dtype);
  a.epsilon = epsilon;
  a.inv_dim = head_dim > 0 ? 1.0f / static_cast<float>(head_dim) : 0.0f;
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.rope_dim = rope_dim;
  a.interleaved = interleaved;
  a.q_out = q_out;
  a.q_out_stride = q_out_stride;
  return a;
}

}  // namespace

extern "C" dq_status dq_qk_norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride, dq_dtype dtype,
                                     int64_t tokens, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                     const void* q_weight, const void* k_weight, dq_dtype weight_dtype, float epsilon,
                                     const int32_t* positions, const float* inv_freq, int32_t rope_dim,
                                     int32_t interleaved, void* q_out, int64_t q_out_stride, void* k_out,
                                     int64_t k_out_stride, cudaStream_t stream) {
  dq::NormRopeArgs a = common_args(q, q_stride, k, k_stride, tokens, q_heads, kv_heads, head_dim, q_weight, k_weight,
                                   weight_dtype, epsilon, positions, inv_freq, rope_dim, interleaved, q_out,
                                   q_out_stride);
  a.k_out = k_out;
  a.k_out_stride = k_out_stride;
  dq_status st = check(a, dtype, weight_dtype);
  if (st != DQ_OK) return st;
  if (k_out_stride < static_cast<int64_t>(kv_heads) * head_dim || k_out_stride > (int64_t(1) << 31))
    return DQ_ERR_BAD_SHAPE;
  if (tokens == 0) return DQ_OK;
  if (k_out == nullptr) return DQ_ERR_NULL_POINTER;
  st = check_pointers(a, weight_dtype);
  if (st != DQ_OK) return st;
  if (!aligned(k_out, 2)) return DQ_ERR_MISALIGNED;
  return dtype == DQ_F16 ? dispatch<__half>(a, dq::kCacheNone, stream)
                         : dispatch<__nv_bfloat16>(a, dq::kCacheNone, stream);
}

extern "C" dq_status dq_qk_norm_rope_cache(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                           const void* v, int64_t v_stride, dq_dtype dtype, int64_t tokens,
                                           int32_t q_heads, int32_t kv_heads, int32_t head_dim, const void* q_weight,
                                           const void* k_weight, dq_dtype weight_dtype, float epsilon,
                                           const int32_t* positions, const float* inv_freq, int32_t rope_dim,
                                           int32_t interleaved, void* q_out, int64_t q_out_stride, void* k_cache,
                                           void* v_cache, dq_dtype cache_dtype, float* k_scale, float* v_scale,
                                           const int64_t* slots, int64_t num_pages, int32_t page_size,
                                           cudaStream_t stream) {
  dq::NormRopeArgs a = common_args(q, q_stride, k, k_stride, tokens, q_heads, kv_heads, head_dim, q_weight, k_weight,
                                   weight_dtype, epsilon, positions, inv_freq, rope_dim, interleaved, q_out,
                                   q_out_stride);
  dq_status st = check(a, dtype, weight_dtype);
  if (st != DQ_OK) return st;
  if (v_stride < static_cast<int64_t>(kv_heads) * head_dim || v_stride > (int64_t(1) << 31)) return DQ_ERR_BAD_SHAPE;
  if (num_pages < 1 || num_pages >= (int64_t(1) << 31) || page_size < 1) return DQ_ERR_BAD_SHAPE;
  if (cache_dtype != dtype && cache_dtype != DQ_INT8) return DQ_ERR_BAD_DTYPE;
  const bool codes = cache_dtype == DQ_INT8;
  if (tokens == 0) return DQ_OK;
  if (v == nullptr || k_cache == nullptr || v_cache == nullptr || slots == nullptr ||
      (codes && (k_scale == nullptr || v_scale == nullptr)))
    return DQ_ERR_NULL_POINTER;
  st = check_pointers(a, weight_dtype);
  if (st != DQ_OK) return st;
  const size_t cs = codes ? 1 : 2;
  if (!aligned(v, 2) || !aligned(k_cache, cs) || !aligned(v_cache, cs) || !aligned(slots, 8) ||
      (codes && (!aligned(k_scale, 4) || !aligned(v_scale, 4))))
    return DQ_ERR_MISALIGNED;
  a.v = v;
  a.v_stride = v_stride;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_scale = codes ? k_scale : nullptr;
  a.v_scale = codes ? v_scale : nullptr;
  a.slots = slots;
  a.num_slots = num_pages * page_size;
  a.page_size = page_size;
  const int cache = codes ? dq::kCacheInt8 : dq::kCacheSame;
  return dtype == DQ_F16 ? dispatch<__half>(a, cache, stream) : dispatch<__nv_bfloat16>(a, cache, stream);
}
