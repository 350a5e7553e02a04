// Attention of one new token per sequence over a paged key-value cache
// (dq_paged_attention): 16-bit caches, or INT8 codes with a scale per token
// and head as dq_qk_norm_rope_cache writes them.
//
// With a running maximum m over the tokens seen so far,
//   l <- l * exp(m_old - m) + sum_j exp(s_j - m)
//   o <- o * exp(m_old - m) + sum_j exp(s_j - m) V_j
// so the cache is read once, and parts of a sequence that were computed apart
// join by the same rule. The visible tokens of a sequence are numbered 0, 1,
// ... without the gap that a window leaves behind the first tokens, so no tile
// holds masked tokens except the last.
#include <cmath>

#include "dq.h"
#include "dq_device.cuh"
#include "dq_launch.cuh"

namespace dq {

struct PagedArgs {
  const void* q;
  int64_t q_stride;
  const void* k_cache;
  const void* v_cache;
  const float* k_scale;
  const float* v_scale;
  const int32_t* page_table;
  const int32_t* lengths;
  int64_t batch;
  int q_heads, kv_heads, head_dim, group;  // group: query heads per key head
  int64_t num_pages;
  int page_size;
  int64_t max_pages;
  int64_t window, sinks;
  float softmax_scale;
  void* out;
  float* lse;
};

// The visible tokens of one sequence: `count` of them, number i being token
// i (i < first) or i + skip. A length that the page table cannot hold is one
// visible token past the table, which makes the rows NaN.
struct Visible {
  int64_t count, first, skip;
};

__device__ __forceinline__ Visible visible_tokens(const PagedArgs& a, int64_t b) {
  const int64_t len = a.lengths[b];
  const int64_t room = a.max_pages * a.page_size;
  if (len <= 0) return {0, 0, 0};
  if (len > room) return {1, 0, room};
  if (a.window == 0 || len <= a.window) return {len, len, 0};
  const int64_t start = len - a.window;
  const int64_t first = a.sinks < start ? a.sinks : start;
  return {first + a.window, first, start - first};
}

constexpr int kPagedGenericWarps = 4;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ float load_row(const __half* p, int64_t i) { return __half2float(p[i]); }
__device__ __forceinline__ float load_row(const __nv_bfloat16* p, int64_t i) { return __bfloat162float(p[i]); }
__device__ __forceinline__ float load_row(const int8_t* p, int64_t i) { return static_cast<float>(p[i]); }

// Any head dimension and alignment: one CTA per (sequence, query head), its
// warps taking the visible tokens in turn, lanes over the channels.
template <typename T, typename C>
__global__ void __launch_bounds__(kPagedGenericWarps * 32) paged_attention_generic_kernel(const PagedArgs a) {
  constexpr bool kCodes = sizeof(C) == 1;
  constexpr int kChan = DQ_MAX_HEAD_DIM / 32;
  __shared__ float s_m[kPagedGenericWarps], s_l[kPagedGenericWarps];
  __shared__ float s_o[kPagedGenericWarps][DQ_MAX_HEAD_DIM];
  pdl_launch_dependents();
  pdl_wait_primary();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t b = blockIdx.x / a.q_heads;
  const int h = static_cast<int>(blockIdx.x - b * a.q_heads);
  const int kvh = h / a.group;
  const Visible vis = visible_tokens(a, b);
  const T* q = static_cast<const T*>(a.q) + b * a.q_stride + static_cast<int64_t>(h) * a.head_dim;
  const float to_log2 = a.softmax_scale * kLog2e;
  float qv[kChan], o[kChan];
#pragma unroll
  for (int i = 0; i < kChan; ++i) {
    const int c = lane + 32 * i;
    qv[i] = c < a.head_dim ? load_row(q, c) : 0.0f;
    o[i] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  for (int64_t i = warp; i < vis.count; i += kPagedGenericWarps) {
    const int64_t j = i < vis.first ? i : i + vis.skip;
    const int64_t p = j / a.page_size;
    const int64_t page = p < a.max_pages ? a.page_table[b * a.max_pages + p] : -1;
    if (page < 0 || page >= a.num_pages) {  // no such page: the rows become NaN
      m = l = NAN;
#pragma unroll
      for (int e = 0; e < kChan; ++e) o[e] = NAN;
      break;
    }
    const int64_t row = (page * a.kv_heads + kvh) * a.page_size + (j - p * a.page_size);
    const C* k = static_cast<const C*>(a.k_cache) + row * a.head_dim;
    const C* v = static_cast<const C*>(a.v_cache) + row * a.head_dim;
    float dot = 0.0f;
#pragma unroll
    for (int e = 0; e < kChan; ++e) {
      const int c = lane + 32 * e;
      if (c < a.head_dim) dot = fmaf(qv[e], load_row(k, c), dot);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
    float s = dot * to_log2;
    if (kCodes) s *= a.k_scale[row];
    const float next = fmaxf(m, s);
    const float keep = m == next ? 1.0f : exp2f(m - next);
    const float w = s == -INFINITY ? 0.0f : exp2f(s - next);
    l = fmaf(l, keep, w);
    const float wv = kCodes ? w * a.v_scale[row] : w;
#pragma unroll
    for (int e = 0; e < kChan; ++e) {
      const int c = lane + 32 * e;
      if (c < a.head_dim) o[e] = fmaf(o[e], keep, wv * load_row(v, c));
    }
    m = next;
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int i = 0; i < kChan; ++i) s_o[warp][lane + 32 * i] = o[i];
  __syncthreads();
  float top = -INFINITY, total = 0.0f, f[kPagedGenericWarps];
  for (int w = 0; w < kPagedGenericWarps; ++w) top = s_m[w] != s_m[w] ? s_m[w] : (top != top ? top : fmaxf(top, s_m[w]));
  for (int w = 0; w < kPagedGenericWarps; ++w) {
    f[w] = s_m[w] == -INFINITY && top != -INFINITY ? 0.0f : exp2f(s_m[w] - top);
    total = fmaf(s_l[w], f[w], total);
  }
  const int64_t at = b * a.q_heads + h;
  const bool empty = vis.count == 0;
  for (int c = threadIdx.x; c < a.head_dim; c += kPagedGenericWarps * 32) {
    float sum = 0.0f;
    for (int w = 0; w < kPagedGenericWarps; ++w) sum = fmaf(s_o[w][c], f[w], sum);
    const float r = empty ? 0.0f : sum / total;
    static_cast<T*>(a.out)[at * a.head_dim + c] = static_cast<T>(r);
  }
  if (threadIdx.x == 0 && a.lse != nullptr) a.lse[at] = empty ? -INFINITY : (top + log2f(total)) * kLn2;
}

}  // namespace dq

namespace {

using dq_host::aligned;

template <typename T, typename C>
dq_status launch_generic(const dq::PagedArgs& a, cudaStream_t stream) {
  void (*fn)(const dq::PagedArgs) = dq::paged_attention_generic_kernel<T, C>;
  return dq_host::launch_programmatic(fn, a, static_cast<int>(a.batch * a.q_heads), dq::kPagedGenericWarps * 32, 0,
                                      stream);
}

dq_status check_heads(int64_t batch, int32_t q_heads, int32_t kv_heads, int32_t head_dim) {
  if (batch < 0 || batch > 65535 * 16 || q_heads < 1 || q_heads > DQ_MAX_HEADS || kv_heads < 1 ||
      kv_heads > DQ_MAX_HEADS || q_heads % kv_heads != 0 || head_dim < 1 || head_dim > DQ_MAX_HEAD_DIM)
    return DQ_ERR_BAD_SHAPE;
  return DQ_OK;
}

bool is_cache(dq_dtype t) { return t == DQ_F16 || t == DQ_BF16 || t == DQ_INT8; }

}  // namespace

extern "C" dq_status dq_paged_attention_get_workspace_size(int64_t batch, int32_t q_heads, int32_t kv_heads,
                                                           int32_t head_dim, dq_dtype cache_dtype,
                                                           size_t* workspace_bytes) {
  if (workspace_bytes == nullptr) return DQ_ERR_NULL_POINTER;
  const dq_status st = check_heads(batch, q_heads, kv_heads, head_dim);
  if (st != DQ_OK) return st;
  if (!is_cache(cache_dtype)) return DQ_ERR_BAD_DTYPE;
  *workspace_bytes = 0;
  return DQ_OK;
}

extern "C" dq_status dq_paged_attention(const void* q, dq_dtype q_dtype, int64_t q_stride, const void* k_cache,
                                        const void* v_cache, dq_dtype cache_dtype, const float* k_scale,
                                        const float* v_scale, const int32_t* page_table, const int32_t* lengths,
                                        int64_t batch, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                        int64_t num_pages, int32_t page_size, int64_t max_pages, int64_t window,
                                        int64_t sinks, float softmax_scale, void* out, float* lse, void* workspace,
                                        size_t workspace_bytes, cudaStream_t stream) {
  const dq_status st = check_heads(batch, q_heads, kv_heads, head_dim);
  if (st != DQ_OK) return st;
  if (q_stride < static_cast<int64_t>(q_heads) * head_dim || q_stride > (int64_t(1) << 31)) return DQ_ERR_BAD_SHAPE;
  if (num_pages < 1 || num_pages >= (int64_t(1) << 31) || page_size < 1 || max_pages < 1 ||
      max_pages >= (int64_t(1) << 31))
    return DQ_ERR_BAD_SHAPE;
  if (q_dtype != DQ_F16 && q_dtype != DQ_BF16) return DQ_ERR_BAD_DTYPE;
  if (cache_dtype != q_dtype && cache_dtype != DQ_INT8) return DQ_ERR_BAD_DTYPE;
  if (window < 0 || sinks < 0 || !std::isfinite(softmax_scale)) return DQ_ERR_BAD_ARGUMENT;
  if (batch == 0) return DQ_OK;
  const bool codes = cache_dtype == DQ_INT8;
  if (q == nullptr || k_cache == nullptr || v_cache == nullptr || page_table == nullptr || lengths == nullptr ||
      out == nullptr || (codes && (k_scale == nullptr || v_scale == nullptr)))
    return DQ_ERR_NULL_POINTER;
  const size_t cs = codes ? 1 : 2;
  if (!aligned(q, 2) || !aligned(k_cache, cs) || !aligned(v_cache, cs) || !aligned(page_table, 4) ||
      !aligned(lengths, 4) || !aligned(out, 2) || (lse && !aligned(lse, 4)) ||
      (codes && (!aligned(k_scale, 4) || !aligned(v_scale, 4))))
    return DQ_ERR_MISALIGNED;
  size_t needed = 0;
  dq_paged_attention_get_workspace_size(batch, q_heads, kv_heads, head_dim, cache_dtype, &needed);
  if (needed > 0 && (workspace == nullptr || workspace_bytes < needed)) return DQ_ERR_WORKSPACE_TOO_SMALL;
  if (needed > 0 && !aligned(workspace, 16)) return DQ_ERR_MISALIGNED;

  dq::PagedArgs a{};
  a.q = q;
  a.q_stride = q_stride;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.page_table = page_table;
  a.lengths = lengths;
  a.batch = batch;
  a.q_heads = q_heads;
  a.kv_heads = kv_heads;
  a.head_dim = head_dim;
  a.group = q_heads / kv_heads;
  a.num_pages = num_pages;
  a.page_size = page_size;
  a.max_pages = max_pages;
  a.window = window;
  a.sinks = sinks;
  a.softmax_scale = softmax_scale;
  a.out = out;
  a.lse = lse;
  if (q_dtype == DQ_F16) {
    return codes ? launch_generic<__half, int8_t>(a, stream) : launch_generic<__half, __half>(a, stream);
  }
  return codes ? launch_generic<__nv_bfloat16, int8_t>(a, stream)
               : launch_generic<__nv_bfloat16, __nv_bfloat16>(a, stream);
}
