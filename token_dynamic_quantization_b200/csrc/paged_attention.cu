// Attention of one new token per sequence over a paged key-value cache
// (dq_paged_attention): 16-bit caches, or INT8 codes with a scale per token
// and head as dq_qk_norm_rope_cache writes them.
//
// With a running maximum m over the tokens seen so far,
//   l <- l * exp(m_old - m) + sum_j exp(s_j - m)
//   o <- o * exp(m_old - m) + sum_j exp(s_j - m) V_j
// so the cache is read once, and parts of a sequence that were computed apart
// join by the same rule. Head dimensions of 64, 128 and 256 run on the tensor
// cores (paged_attention_mma.cuh); what follows here serves all others, and
// unaligned tensors, at the price that one CTA reads a query head's whole sequence (64
// sequences of up to 4000 tokens, INT8, 32 query and 8 key heads: 2.0 ms with 80 or 96
// channels against 64 us with 128 on the tensor cores). It numbers the visible tokens 0, 1, ... without the gap that a
// window leaves behind the first tokens.
#include <cmath>

#include "decoder_launch.cuh"
#include "dq.h"
#include "dq_device.cuh"
#include "dq_launch.cuh"
#include "paged_attention_args.cuh"
#include "paged_attention_mma.cuh"
#include "tensor_map.cuh"

namespace dq {

constexpr int kPagedGenericWarps = 4;
__device__ __forceinline__ float load_row(const __half* p, int64_t i) { return __half2float(p[i]); }
__device__ __forceinline__ float load_row(const __nv_bfloat16* p, int64_t i) { return __bfloat162float(p[i]); }
__device__ __forceinline__ float load_row(const int8_t* p, int64_t i) { return static_cast<float>(p[i]); }

// Any head dimension and alignment: one CTA per (sequence, query head), its
// warps taking the visible tokens in turn, lanes over the channels.
template <typename T, typename C>
__global__ void __launch_bounds__(kPagedGenericWarps * 32) paged_attention_generic_kernel(const PagedArgs a) {
  constexpr bool kCodes = sizeof(C) == 1;
  constexpr int kChan = DQ_MAX_HEAD_DIM / 32;
  __shared__ float s_m[kPagedGenericWarps], s_l[kPagedGenericWarps], s_size[kPagedGenericWarps];
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
  float shrink = 1.0f;  // o is this much smaller: beside value scales past 2^64 it could overflow where the result does not
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
    if (kCodes) s = fmaf(s, a.k_scale[row], fmaf(a.k_scale[row], 0.0f, a.v_scale[row] * 0.0f));  // not finite: NaN
    const float next = fmaxf(m, s);
    const float keep = m == next ? 1.0f : exp2f(m - next);
    const float w = s == -INFINITY ? 0.0f : exp2f(s - next);
    l = fmaf(l, keep, w);
    float wv = w;
    if (kCodes) {
      wv = w * a.v_scale[row] * shrink;
      if (fabsf(wv) > 0x1p64f) {
        shrink = 0x1p-64f;
        wv *= 0x1p-64f;
#pragma unroll
        for (int e = 0; e < kChan; ++e) o[e] *= 0x1p-64f;
      }
    }
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
    s_size[warp] = 1.0f / shrink;
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
    for (int w = 0; w < kPagedGenericWarps; ++w) sum = fmaf(s_o[w][c] * (f[w] / total), s_size[w], sum);
    const float r = empty ? 0.0f : sum;
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

// ---- tensor-core path

// Query heads of one item: two sets of 8 where a key head serves more than 8
// and the accumulators fit (16 heads of 256 channels do not).
constexpr int head_tiles(int group, int dim) { return group > 8 && dim <= 128 ? 2 : 1; }

// CTAs that share the tiles at most: what fits the device at once, eight to an SM.
int64_t most_ctas() { return static_cast<int64_t>(dq_host::sm_count(dq_host::current_device())) * 8; }

bool mma_dim(int dim) { return dim == 64 || dim == 128 || dim == 256; }

size_t parts_bytes(int group, int dim) {
  const int heads = 8 * head_tiles(group, dim);
  return static_cast<size_t>(most_ctas()) * (2 * (heads * dim + 2 * heads) * sizeof(float) + sizeof(dq::PagedCut));
}

// A cache as a list of rows, copied in boxes of 128 bytes (64 for 64 codes) by
// box_rows with the swizzle of that width (box_rows 1: gathered row by row).
template <typename C, int BOX>
bool rows_map(CUtensorMap* map, const void* base, int64_t rows, int dim, int box_rows) {
  dq_host::EncodeTiledFn fn = dq_host::encode_tiled();
  if (fn == nullptr) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(dim), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(dim) * sizeof(C)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(BOX / sizeof(C)), static_cast<cuuint32_t>(box_rows)}, estride[2] = {1, 1};
  return fn(map, sizeof(C) == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 2,
            const_cast<void*>(base), dims, strides, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
            BOX == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, typename C, int D, int HT, bool RUN, int W>
dq_status launch_mma(dq::PagedArgs a, cudaStream_t stream) {
  using Shape = dq::PagedShape<C, D, HT, W>;
  auto fn = dq::paged_attention_mma_kernel<T, C, D, HT, RUN, W>;
  CUtensorMap k_map, v_map;
  const int64_t rows = a.num_pages * a.kv_heads * a.page_size;
  if (!rows_map<C, Shape::kBox>(&k_map, a.k_cache, rows, D, RUN ? 16 : 1) ||
      !rows_map<C, Shape::kBox>(&v_map, a.v_cache, rows, D, RUN ? 16 : 1))
    return dq_host::kNotLaunchable;
  const int device = dq_host::current_device();
  if (!dq_host::allow_smem_bytes(reinterpret_cast<const void*>(fn), device, Shape::kSmem)) return dq_host::kNotLaunchable;
  int64_t ctas = static_cast<int64_t>(dq_host::sm_count(device)) *
                 dq_host::blocks_per_sm(reinterpret_cast<const void*>(fn), Shape::kThreads, Shape::kSmem, device);
  if (ctas > most_ctas()) ctas = most_ctas();
  if (a.whole) {
    const dim3 items(static_cast<unsigned>(a.batch * a.kv_heads * a.head_sets));
    return dq_host::launch_dependent(fn, items, Shape::kThreads, Shape::kSmem, 1, stream, k_map, v_map, a);
  }
  a.cuts = reinterpret_cast<dq::PagedCut*>(a.parts + most_ctas() * 2 * Shape::kPartFloats);
  const dim3 grid(static_cast<unsigned>(ctas));
  const dq_status st = dq_host::launch_dependent(fn, grid, Shape::kThreads, Shape::kSmem, 1, stream, k_map, v_map, a);
  if (st != DQ_OK) return st;
  return dq_host::launch_dependent(dq::paged_attention_join_kernel<T, C, D, HT>, dim3(static_cast<unsigned>(ctas - 1)),
                                   dq::kPagedJoinThreads, 0, 1, stream, a);
}

// How the work is cut, from the number of items (sequence, key head, head set)
// and the most tiles that one can have.
//   up to 16 tiles: an item is a CTA's, whole, and there is nothing to join (1
// sequence of 127 tokens, INT8: 5.0 us against 7.0 in ranges; 444 x 100: 28 against 39);
// longer ones are cut into ranges.
//   six items per SM or more, whole: a CTA is one warp, else four that share the
// item. 444 sequences of up to 100 tokens, 8 key heads, take 27 us (bf16) and 28 (INT8)
// with one warp, 54 and 60 with four; 32 to 128 sequences have too few items.
//   six items per SM or more, cut into ranges: one warp for INT8 caches of 128 or
// 256 channels (444 x 600 tokens 79 us against 101, 128 x 600 33 against 36, 256 x 1000 of 256
// channels 119 against 133, but with fewer items 64 x 4160 66 against 65 and 32 x 600
// 18 against 15), four for 16-bit caches (256 x 1000: 94 us, one warp 101) and 64
// channels (256 x 1000 INT8: 56 us, one warp 64).
template <typename T, typename C, int D, int HT>
dq_status by_pages(dq::PagedArgs a, cudaStream_t stream) {
  using Shape = dq::PagedShape<C, D, HT, 4>;
  a.head_sets = (a.group + Shape::kHeads - 1) / Shape::kHeads;
  const int64_t room = a.max_pages * a.page_size;
  const int64_t most_seen = a.window != 0 && a.window + a.sinks < room ? a.window + a.sinks + 32 : room;
  a.whole = most_seen <= 16 * Shape::kTokens ? 1 : 0;
  const int64_t items = a.batch * a.kv_heads * a.head_sets;
  const bool many = items >= int64_t(6) * dq_host::sm_count(dq_host::current_device());
  const bool run = a.page_size % 16 == 0;
  if (many && (a.whole || (Shape::kCodes && D >= 128)))
    return run ? launch_mma<T, C, D, HT, true, 1>(a, stream) : launch_mma<T, C, D, HT, false, 1>(a, stream);
  return run ? launch_mma<T, C, D, HT, true, 4>(a, stream) : launch_mma<T, C, D, HT, false, 4>(a, stream);
}

template <typename T, typename C>
dq_status dispatch_mma(const dq::PagedArgs& a, cudaStream_t stream) {
  const int ht = head_tiles(a.group, a.head_dim);
  if (a.head_dim == 64) return ht == 2 ? by_pages<T, C, 64, 2>(a, stream) : by_pages<T, C, 64, 1>(a, stream);
  if (a.head_dim == 128) return ht == 2 ? by_pages<T, C, 128, 2>(a, stream) : by_pages<T, C, 128, 1>(a, stream);
  return by_pages<T, C, 256, 1>(a, stream);
}

template <typename T, typename C>
dq_status dispatch(const dq::PagedArgs& a, bool mma, cudaStream_t stream) {
  if (mma) {
    const dq_status st = dispatch_mma<T, C>(a, stream);
    if (st != dq_host::kNotLaunchable) return st;
  }
  return launch_generic<T, C>(a, stream);
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
  *workspace_bytes = batch > 0 && mma_dim(head_dim) ? parts_bytes(q_heads / kv_heads, head_dim) : 0;
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
  // lengths stay below 2^31: larger numbers mean the same, and their sum cannot overflow
  a.window = window < (int64_t(1) << 31) ? window : int64_t(1) << 31;
  a.sinks = sinks < (int64_t(1) << 31) ? sinks : int64_t(1) << 31;
  a.softmax_scale = softmax_scale;
  a.out = out;
  a.lse = lse;
  // token / page_size for tokens below 2^31: shift = ceil(log2 d), mul = 2^32 (2^shift - d) / d + 1
  uint32_t shift = 0;
  while ((int64_t(1) << shift) < page_size) ++shift;
  a.page_shift = shift;
  a.page_mul = static_cast<uint32_t>(((uint64_t(1) << 32) * ((uint64_t(1) << shift) - page_size)) / page_size + 1);
  a.parts = static_cast<float*>(workspace);
  // 16-byte pieces of cache rows, 8-byte pieces of q and out rows, row numbers below 2^31
  const bool mma = mma_dim(head_dim) && aligned(k_cache, 16) && aligned(v_cache, 16) && aligned(q, 8) &&
                   q_stride % 4 == 0 && aligned(out, 8) &&
                   num_pages <= int64_t(0x7FFFFFFF) / page_size / kv_heads;
  if (q_dtype == DQ_F16) {
    return codes ? dispatch<__half, int8_t>(a, mma, stream) : dispatch<__half, __half>(a, mma, stream);
  }
  return codes ? dispatch<__nv_bfloat16, int8_t>(a, mma, stream)
               : dispatch<__nv_bfloat16, __nv_bfloat16>(a, mma, stream);
}
