// RMS norm of every query and key head with the position rotation in the same
// pass, keys and values optionally written into a paged 16-bit or INT8 cache
// (dq_qk_norm_rope, dq_qk_norm_rope_cache).
//
// For a head row x of D values with weight w:
//   y = x * rsqrt(mean(x^2) + epsilon) * w
//   (y[a], y[b]) <- (y[a] cos - y[b] sin, y[b] cos + y[a] sin)
// The angle pos * inv_freq is formed and reduced in binary64 (a binary32
// product of a position of 100000 is off by up to 2^-8 of a radian), then
// sincospi is taken of the remainder in [-1, 1], in units of pi.
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
};

enum : int { kCacheNone = 0, kCacheSame = 1, kCacheInt8 = 2 };

// cos and sin of pos * inv_freq: t is the angle in units of pi, reduced
// exactly to [-1, 1] before the rounding to binary32.
__device__ __forceinline__ void rope_angle(int32_t pos, float inv_freq, float& c, float& s) {
  const double t = static_cast<double>(pos) * static_cast<double>(inv_freq) * 0.31830988618379067154;
  sincospif(static_cast<float>(t - 2.0 * rint(0.5 * t)), &s, &c);
}

__device__ __forceinline__ float warp_sum_f32(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
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

constexpr int kNormRopeBlock = 256;

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
      for (int i = 0; i < kPairs; ++i) top = fmaxf(top, fmaxf(fabsf(first[i]), fabsf(second[i])));
#pragma unroll
      for (int i = 0; i < kRest; ++i) top = fmaxf(top, fabsf(rest[i]));
      const RowQuant rq = make_sym<127>(warp_max(top));
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

template <typename T>
dq_status dispatch(const dq::NormRopeArgs& a, int cache, cudaStream_t stream) {
  if (cache == dq::kCacheNone) return launch_generic<T, dq::kCacheNone>(a, stream);
  if (cache == dq::kCacheSame) return launch_generic<T, dq::kCacheSame>(a, stream);
  return launch_generic<T, dq::kCacheInt8>(a, stream);
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
