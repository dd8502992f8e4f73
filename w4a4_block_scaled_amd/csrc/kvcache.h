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
// (E2M1: in bytes; a page's scale bytes begin scale_at bytes into it, head by head,
// scale_head bytes each: [head_dim / 32, page_size].)
struct KvView {
  const void* k;
  const void* v;
  const float* k_scale;
  const float* v_scale;
  int64_t page_stride, token_stride, head_stride;
  int64_t scale_at, scale_head;
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

// Row of `cu` that holds token i: the last s with cu[s] <= i < cu[s + 1].
__device__ __forceinline__ int find_seq(const int32_t* cu, int seqs, int i) {
  int lo = 0, hi = seqs;          // cu[lo] <= i < cu[hi] if the token belongs to any
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= i) lo = mid; else hi = mid;
  }
  return lo;
}
#endif

hipError_t launch_kv_append(const KvView& kv, int dtype, int head_dim, const int32_t* cu, int64_t tokens, int in_dtype,
                            const void* k, int64_t k_row, int64_t k_head, const void* v, int64_t v_row, int64_t v_head,
                            hipStream_t stream);

// Rotation of rows, alone (kv.heads == 0) or on the way into a cache.
struct RowsIn {
  KvView kv;
  const int32_t* cu;              // NULL: one row per sequence
  const int32_t* positions;       // NULL: the tokens' places in their sequences
  const float* freqs;
  const void *q, *k, *v;
  void* out;                      // of the rotated q
  int64_t q_row, q_head, k_row, k_head, v_row, v_head, o_row, o_head;    // elements
  int64_t tokens;
  int32_t q_heads, dim;
  int32_t rot;                    // 0: no rotation
  int32_t interleaved, inverse;
  float factor;
};
// cache_dtype: of kv, if it has heads; dtype: of the rows
int64_t rows_workgroups(int64_t tokens, int64_t q_heads, int64_t kv_heads, int dim);      // of launch_rows_in (and _out: more)
hipError_t launch_rows_in(const RowsIn& a, int cache_dtype, int dtype, hipStream_t stream);

// Rows of the cache in 16 bits.
struct RowsOut {
  KvView kv;
  const int32_t* cu;
  void *k, *v;
  int64_t k_row, k_head, v_row, v_head;
  int64_t tokens;
  int32_t dim;
};
hipError_t launch_rows_out(const RowsOut& a, int cache_dtype, int dtype, hipStream_t stream);

size_t attn_decode_workspace(int q_heads, int heads, int head_dim);
hipError_t launch_attn_decode(const AttnArgs& a, int cache_dtype, int dtype, int head_dim, void* workspace,
                              hipStream_t stream);

// The same kernel for several queries per sequence, where there are few of them.
bool attn_few_serves(int64_t seqs, int64_t tokens, int group, int page_size, int cache_dtype, int head_dim);
size_t attn_few_workspace(int64_t seqs, int64_t tokens, int group, int cache_dtype, int head_dim);
hipError_t launch_attn_few(const AttnArgs& a, const int32_t* cu, int64_t tokens, int cache_dtype, int dtype,
                           int head_dim, void* workspace, hipStream_t stream);

// Over a 4-bit cache: one query per sequence (cu NULL), or a few (pages of a multiple of 8).
// attn_fp4_blocks: blocks of 16 rows that a kv head of a sequence has on average, 0 where
// they are too many.
int attn_fp4_blocks(int64_t seqs, int64_t tokens, int group, int head_dim);
size_t attn_fp4_workspace(int rows, int head_dim);
hipError_t launch_attn_fp4(const AttnArgs& a, const int32_t* cu, int64_t tokens, int dtype, int head_dim,
                           void* workspace, hipStream_t stream);

size_t attn_prefill_workspace(int64_t seqs, int64_t tokens, int q_heads, int heads, int head_dim, int page_size,
                              int cache_dtype);
int64_t attn_prefill_workgroups(int64_t seqs, int64_t tokens, int q_heads, int heads, int head_dim, int page_size,
                                int cache_dtype);
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
