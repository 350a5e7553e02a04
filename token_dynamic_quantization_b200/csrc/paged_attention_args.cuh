// Arguments and the token numbering shared by the paged attention kernels.
#pragma once

#include <math.h>
#include <stdint.h>

namespace dq {

// The item inside which a CTA's range of work units ends (seq < 0: it ends with one).
struct PagedCut {
  int64_t seq;           // -1: no item is cut here
  int item, first, last; // the item of that sequence, and the CTAs of its first and last tile
};

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
  // tensor-core kernels only
  uint32_t page_mul, page_shift;  // token / page_size = (mulhi(token, mul) + token) >> shift
  int head_sets;                  // sets of 8 * HT query heads that share a key head
  float* parts;                   // workspace: what CTAs leave of items that they share
  PagedCut* cuts;                 // workspace, one per CTA
  int whole;                      // 1: a CTA per item, nothing shared
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

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

}  // namespace dq
