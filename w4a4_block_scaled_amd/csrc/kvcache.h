// Shared by the paged key-value cache's kernels (kvcache.hip) and the
// attention that reads it (attn_decode.hip, attn_prefill.hip): the device
// view of a cache and of its sequences, the division by the page size, page
// lookups that never leave the table, and the host launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "w4a4.h"

namespace w4a4 {

// n / d for 0 <= n < 2^31 and a fixed 1 <= d < 2^31, as a product with
// m = floor(2^(31+s) / d) + 1, s = ceil(log2 d): the error n e / (d 2^(31+s)),
// 0 < e <= d, stays below 1 / d.
struct FastDiv {
  uint32_t d;
  uint64_t m;
  int shift;
#ifdef __HIPCC__
  __device__ __forceinline__ int div(int n) const { return int((uint64_t(uint32_t(n)) * m) >> shift); }
#endif
};
inline FastDiv fast_div(uint32_t d) {
  int s = 0;
  while ((uint64_t(1) << s) < d) ++s;
  return {d, (uint64_t(1) << (31 + s)) / d + 1, 31 + s};
}

// Device view of w4a4_kv_cache + w4a4_kv_seqs.  Strides in elements.
struct KvView {
  const void* k;
  const void* v;
  const float* k_scale;
  const float* v_scale;
  int64_t page_stride, token_stride, head_stride;
  const int32_t* tables;
  const int32_t* lens;
  int64_t table_stride;
  int32_t pages, heads, seqs, max_pages;
  FastDiv page;
};

struct AttnArgs {
  KvView kv;
  const void* q;
  void* out;
  float* lse;                     // [rows, q_heads] or NULL
  int64_t q_row, q_head, o_row, o_head;   // strides in elements
  int32_t q_heads, group;         // group = q_heads / heads
  int32_t window, sinks;          // window 0: none
  float scale_log2;               // scale * log2(e)
};

#ifdef __HIPCC__
// Page of token `t` (t >= 0) of the table row `row`; -1 where the table has
// no valid page for it (past its end, or an entry outside 0..pages-1).
__device__ __forceinline__ int kv_page(const KvView& kv, const int32_t* row, int t, int* slot) {
  const int i = kv.page.div(t);
  *slot = t - i * int(kv.page.d);
  if (i >= kv.max_pages) return -1;
  const int p = row[i];
  return (p >= 0 && p < kv.pages) ? p : -1;
}
#endif

hipError_t launch_kv_append(const KvView& kv, int dtype, int head_dim, const int32_t* cu, int64_t tokens, int in_dtype,
                            const void* k, int64_t k_row, int64_t k_head, const void* v, int64_t v_row, int64_t v_head,
                            hipStream_t stream);

size_t attn_decode_workspace(int q_heads, int heads, int head_dim);
hipError_t launch_attn_decode(const AttnArgs& a, int cache_dtype, int dtype, int head_dim, void* workspace,
                              hipStream_t stream);

// The same kernel for several queries per sequence, where there are few of them.
bool attn_few_serves(int64_t seqs, int64_t tokens, int group, int page_size);
size_t attn_few_workspace(int head_dim);
hipError_t launch_attn_few(const AttnArgs& a, const int32_t* cu, int64_t tokens, int cache_dtype, int dtype,
                           int head_dim, void* workspace, hipStream_t stream);

size_t attn_prefill_workspace(int64_t seqs, int64_t tokens, int q_heads, int heads, int head_dim, int page_size);
int64_t attn_prefill_workgroups(int64_t seqs, int64_t tokens, int q_heads, int heads, int page_size);
hipError_t launch_attn_prefill(const AttnArgs& a, const int32_t* cu, int64_t tokens, int cache_dtype, int dtype,
                               int head_dim, void* workspace, hipStream_t stream);

// Page bookkeeping.  `refs` holds the number of sequences on each page (0: free).
struct PageMove {
  void* const* arrays;          // host array of n device base pointers
  int n;
  int64_t stride_bytes, page_bytes;
};
hipError_t launch_kv_copy_pages(const PageMove& mv, int pages, const int32_t* src, const int32_t* dst, int64_t pairs,
                                hipStream_t stream);
size_t kv_reserve_workspace(int64_t seqs, int64_t pages);
hipError_t launch_kv_reserve(int32_t* tables, int64_t table_stride, const int32_t* lens, int seqs, int max_pages,
                             int32_t* refs, int pages, int page_size, int32_t* lacking, void* workspace,
                             hipStream_t stream);
size_t kv_fork_workspace(int64_t children, int64_t pages);
hipError_t launch_kv_fork(const PageMove& mv, int32_t* tables, int64_t table_stride, int32_t* lens, int seqs,
                          int max_pages, int32_t* refs, int pages, int page_size, const int32_t* parents,
                          const int32_t* children, int n, int32_t* lacking, void* workspace, hipStream_t stream);
hipError_t launch_kv_free(int32_t* tables, int64_t table_stride, int32_t* lens, int seqs, int max_pages, int32_t* refs,
                          int pages, int page_size, const int32_t* ids, int n, bool trim, int window, int sinks,
                          hipStream_t stream);
size_t kv_compact_workspace(int64_t pages);
hipError_t launch_kv_compact(const PageMove& mv, int32_t* tables, int64_t table_stride, int seqs, int max_pages,
                             int32_t* refs, int pages, int32_t* remap, void* workspace, hipStream_t stream);

}  // namespace w4a4
