// C ABI of the paged key-value cache and its attention (declared in
// include/w4a4.h): argument validation and dispatch.  Contents of device
// arrays are never read here; the kernels keep every access inside the buffers
// whatever the arrays hold.
#include <math.h>

#include <algorithm>

#include "kvcache.h"
#include "status.h"

namespace {

using w4a4::aligned;
using w4a4::fail;
using w4a4::hip_status;
using w4a4::ok;

// The kernels count in int32: rows in tiles of up to 128 (kMaxRows leaves room for
// the last one), sequences and list entries in steps of up to 1024, and a launch
// has fewer than 2^32 threads.
const int64_t kMaxIndex = int64_t(1) << 31, kMaxRows = kMaxIndex - 256, kMaxCount = int64_t(1) << 30;
const int64_t kMaxGrid = int64_t(1) << 24;      // workgroups of 256

w4a4_status check_cache(const char* what, const w4a4_kv_cache* c) {
  if (!c) return fail(W4A4_ERR_NULL, "%s: cache must be non-NULL", what);
  if (c->dtype != W4A4_BF16 && c->dtype != W4A4_F16 && c->dtype != W4A4_E4M3)
    return fail(W4A4_ERR_FORMAT, "%s: unknown cache type %d", what, int(c->dtype));
  if (c->pages < 1 || c->page_size < 1 || c->page_size > 65536 || c->heads < 1 ||
      (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256))
    return fail(W4A4_ERR_SHAPE,
                "%s: cache of pages=%d page_size=%d heads=%d head_dim=%d (need pages, heads >= 1, 1 <= page_size <= "
                "65536, head_dim 64, 128 or 256)",
                what, int(c->pages), int(c->page_size), int(c->heads), int(c->head_dim));
  if (!c->k || !c->v) return fail(W4A4_ERR_NULL, "%s: cache k and v must be non-NULL", what);
  const int64_t unit = c->dtype == W4A4_E4M3 ? 16 : 8;
  if (c->page_stride < 0 || c->token_stride < 0 || c->head_stride < 0)
    return fail(W4A4_ERR_SHAPE, "%s: cache strides must not be negative", what);
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || c->page_stride % unit || c->token_stride % unit ||
      c->head_stride % unit || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
    return fail(W4A4_ERR_ALIGN,
                "%s: cache k and v need 16-byte alignment, strides in multiples of 16 bytes, scales 4-byte alignment", what);
  return W4A4_OK;
}

w4a4_status check_seqs(const char* what, const w4a4_kv_seqs* s, bool lens) {
  if (!s) return fail(W4A4_ERR_NULL, "%s: seqs must be non-NULL", what);
  if (s->seqs < 0 || s->seqs > kMaxCount || s->max_pages < 1 || s->table_stride < s->max_pages)
    return fail(W4A4_ERR_SHAPE,
                "%s: seqs=%d max_pages=%d table_stride=%lld (need 0 <= seqs <= 2^30, 1 <= max_pages <= table_stride)",
                what, int(s->seqs), int(s->max_pages), (long long)s->table_stride);
  if (s->seqs > 0 && (!s->tables || (lens && !s->lens)))
    return fail(W4A4_ERR_NULL, "%s: tables and lens must be non-NULL", what);
  if (!aligned(s->tables, 4) || !aligned(s->lens, 4))
    return fail(W4A4_ERR_ALIGN, "%s: tables and lens need 4-byte alignment", what);
  return W4A4_OK;
}

w4a4_status check_type(const char* what, const w4a4_kv_cache* c, w4a4_dtype t) {
  if (t != W4A4_BF16 && t != W4A4_F16) return fail(W4A4_ERR_FORMAT, "%s: type %d (need BF16 or FP16)", what, int(t));
  if (c->dtype != W4A4_E4M3 && c->dtype != int(t))
    return fail(W4A4_ERR_FORMAT, "%s: type %d with a cache of type %d", what, int(t), int(c->dtype));
  return W4A4_OK;
}

w4a4_status check_rows(const char* what, const char* name, const void* p, int64_t row, int64_t head) {
  if (!p) return fail(W4A4_ERR_NULL, "%s: %s must be non-NULL", what, name);
  if (row < 0 || head < 0) return fail(W4A4_ERR_SHAPE, "%s: %s strides must not be negative", what, name);
  if (!aligned(p, 16) || row % 8 || head % 8)
    return fail(W4A4_ERR_ALIGN, "%s: %s needs 16-byte alignment and strides in multiples of 8 elements", what, name);
  return W4A4_OK;
}

w4a4::KvView view(const w4a4_kv_cache* c, const w4a4_kv_seqs* s) {
  w4a4::KvView v;
  v.k = c->k;
  v.v = c->v;
  v.k_scale = c->dtype == W4A4_E4M3 ? c->k_scale : nullptr;
  v.v_scale = c->dtype == W4A4_E4M3 ? c->v_scale : nullptr;
  v.page_stride = c->page_stride;
  v.token_stride = c->token_stride;
  v.head_stride = c->head_stride;
  v.tables = s->tables;
  v.lens = s->lens;
  v.table_stride = s->table_stride;
  v.pages = c->pages;
  v.heads = c->heads;
  v.seqs = s->seqs;
  v.max_pages = s->max_pages;
  v.page = w4a4::fast_div(uint32_t(c->page_size));
  return v;
}

bool heads_ok(const w4a4_kv_cache* c, int q_heads) {
  return q_heads >= 1 && q_heads <= 65536 && q_heads % c->heads == 0;
}

// What both attention entry points ask of their arguments.
w4a4_status check_attn(const char* what, const w4a4_kv_cache* c, const w4a4_kv_seqs* s, w4a4_dtype dtype, int q_heads,
                       int64_t rows, const void* q, int64_t q_row, int64_t q_head, float scale, int window, int sinks,
                       const void* out, int64_t o_row, int64_t o_head, const float* lse, const void* ws,
                       size_t ws_bytes, size_t need) {
  w4a4_status st = check_type(what, c, dtype);
  if (st != W4A4_OK) return st;
  if (!heads_ok(c, q_heads) || rows * q_heads >= kMaxRows)
    return fail(W4A4_ERR_SHAPE, "%s: %d query heads for %d kv heads, %lld rows", what, q_heads, int(c->heads),
                (long long)rows);
  if (window < 0 || sinks < 0)
    return fail(W4A4_ERR_SHAPE, "%s: window=%d sinks=%d must not be negative", what, window, sinks);
  if (!(scale > 0.0f) || !isfinite(scale))
    return fail(W4A4_ERR_SHAPE, "%s: scale=%g must be positive and finite", what, double(scale));
  if (rows == 0 || s->seqs == 0) return W4A4_OK;
  st = check_rows(what, "q", q, q_row, q_head);
  if (st == W4A4_OK) st = check_rows(what, "out", out, o_row, o_head);
  if (st != W4A4_OK) return st;
  if (!aligned(lse, 4)) return fail(W4A4_ERR_ALIGN, "%s: lse needs 4-byte alignment", what);
  if (need && (!ws || ws_bytes < need))
    return fail(W4A4_ERR_WORKSPACE, "%s: needs %zu workspace bytes, got %zu", what, need, ws ? ws_bytes : size_t(0));
  if (need && !aligned(ws, 16)) return fail(W4A4_ERR_ALIGN, "%s: workspace needs 16-byte alignment", what);
  return W4A4_OK;
}

w4a4::AttnArgs attn_args(const w4a4_kv_cache* c, const w4a4_kv_seqs* s, int q_heads, const void* q, int64_t q_row,
                         int64_t q_head, float scale, int window, int sinks, void* out, int64_t o_row, int64_t o_head,
                         float* lse) {
  w4a4::AttnArgs a;
  a.kv = view(c, s);
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.q_row = q_row;
  a.q_head = q_head;
  a.o_row = o_row;
  a.o_head = o_head;
  a.q_heads = q_heads;
  a.group = q_heads / c->heads;
  a.window = std::min(window, 1 << 30);     // no sequence is longer
  a.sinks = sinks;
  a.scale_log2 = float(double(scale) * 1.4426950408889634);
  return a;
}

w4a4_status check_arrays(const char* what, int n, void* const* arrays, int64_t stride, int64_t bytes, int pages) {
  if (n < 0 || pages < 1 || bytes < 1 || stride < bytes)
    return fail(W4A4_ERR_SHAPE, "%s: %d arrays of %d pages of %lld bytes, stride %lld", what, n, pages, (long long)bytes,
                (long long)stride);
  if (n > 0 && !arrays) return fail(W4A4_ERR_NULL, "%s: arrays must be non-NULL", what);
  for (int i = 0; i < n; ++i) {
    if (!arrays[i]) return fail(W4A4_ERR_NULL, "%s: array %d is NULL", what, i);
    if (!aligned(arrays[i], 16)) return fail(W4A4_ERR_ALIGN, "%s: array %d needs 16-byte alignment", what, i);
  }
  return W4A4_OK;
}

w4a4_status check_refs(const char* what, const int32_t* refs, int pages, int page_size) {
  if (pages < 1 || page_size < 1 || page_size > 65536)
    return fail(W4A4_ERR_SHAPE, "%s: pages=%d page_size=%d", what, pages, page_size);
  if (!refs) return fail(W4A4_ERR_NULL, "%s: refs must be non-NULL", what);
  if (!aligned(refs, 4)) return fail(W4A4_ERR_ALIGN, "%s: refs needs 4-byte alignment", what);
  return W4A4_OK;
}

w4a4_status check_ws(const char* what, const void* ws, size_t bytes, size_t need) {
  if (!ws || bytes < need)
    return fail(W4A4_ERR_WORKSPACE, "%s: needs %zu workspace bytes, got %zu", what, need, ws ? bytes : size_t(0));
  if (!aligned(ws, 16)) return fail(W4A4_ERR_ALIGN, "%s: workspace needs 16-byte alignment", what);
  return W4A4_OK;
}

w4a4_status check_list(const char* what, const void* a, const void* b, int64_t n) {
  if (n < 0 || n > kMaxCount) return fail(W4A4_ERR_SHAPE, "%s: %lld entries", what, (long long)n);
  if (n > 0 && (!a || !b)) return fail(W4A4_ERR_NULL, "%s: the index lists must be non-NULL", what);
  if (!aligned(a, 4) || !aligned(b, 4)) return fail(W4A4_ERR_ALIGN, "%s: index lists need 4-byte alignment", what);
  return W4A4_OK;
}

}  // namespace

extern "C" {

w4a4_status w4a4_kv_append(const w4a4_kv_cache* cache, const w4a4_kv_seqs* seqs, const int32_t* cu, int64_t tokens,
                           w4a4_dtype dtype, const void* k, int64_t k_row, int64_t k_head, const void* v,
                           int64_t v_row, int64_t v_head, void* stream) {
  const char* what = "kv_append";
  w4a4_status st = check_cache(what, cache);
  if (st == W4A4_OK) st = check_seqs(what, seqs, true);
  if (st == W4A4_OK) st = check_type(what, cache, dtype);
  if (st != W4A4_OK) return st;
  if (tokens < 0 || tokens >= kMaxIndex || (!cu && tokens != seqs->seqs))
    return fail(W4A4_ERR_SHAPE, "%s: %lld tokens for %d sequences", what, (long long)tokens, int(seqs->seqs));
  if (!aligned(cu, 4)) return fail(W4A4_ERR_ALIGN, "%s: cu needs 4-byte alignment", what);
  if (tokens == 0 || seqs->seqs == 0) return ok();
  st = check_rows(what, "k", k, k_row, k_head);
  if (st == W4A4_OK) st = check_rows(what, "v", v, v_row, v_head);
  if (st != W4A4_OK) return st;
  return hip_status(w4a4::launch_kv_append(view(cache, seqs), cache->dtype, cache->head_dim, cu, tokens, dtype, k, k_row,
                                           k_head, v, v_row, v_head, static_cast<hipStream_t>(stream)),
                    "kv_append launch");
}

size_t w4a4_attn_decode_workspace_bytes(const w4a4_kv_cache* cache, int64_t seqs, int q_heads) {
  if (check_cache("attn_decode_workspace_bytes", cache) != W4A4_OK || !heads_ok(cache, q_heads) || seqs <= 0) return 0;
  return w4a4::attn_decode_workspace(q_heads, cache->heads, cache->head_dim);
}

w4a4_status w4a4_attn_decode(const w4a4_kv_cache* cache, const w4a4_kv_seqs* seqs, w4a4_dtype dtype, int q_heads,
                             const void* q, int64_t q_row, int64_t q_head, float scale, int window, int sinks,
                             void* out, int64_t o_row, int64_t o_head, float* lse, void* workspace, size_t ws_bytes,
                             void* stream) {
  const char* what = "attn_decode";
  w4a4_status st = check_cache(what, cache);
  if (st == W4A4_OK) st = check_seqs(what, seqs, true);
  if (st != W4A4_OK) return st;
  const size_t need = seqs->seqs > 0 && heads_ok(cache, q_heads)
                          ? w4a4::attn_decode_workspace(q_heads, cache->heads, cache->head_dim) : 0;
  st = check_attn(what, cache, seqs, dtype, q_heads, seqs->seqs, q, q_row, q_head, scale, window, sinks, out, o_row,
                  o_head, lse, workspace, ws_bytes, need);
  if (st != W4A4_OK) return st;
  if (seqs->seqs == 0) return ok();
  return hip_status(w4a4::launch_attn_decode(attn_args(cache, seqs, q_heads, q, q_row, q_head, scale, window, sinks,
                                                       out, o_row, o_head, lse),
                                             cache->dtype, dtype, cache->head_dim, workspace,
                                             static_cast<hipStream_t>(stream)),
                    "attn_decode launch");
}

size_t w4a4_attn_prefill_workspace_bytes(const w4a4_kv_cache* cache, int64_t seqs, int64_t tokens, int q_heads) {
  if (check_cache("attn_prefill_workspace_bytes", cache) != W4A4_OK || !heads_ok(cache, q_heads) || seqs <= 0 ||
      tokens <= 0 || tokens * q_heads >= kMaxRows)
    return 0;
  return w4a4::attn_prefill_workspace(seqs, tokens, q_heads, cache->heads, cache->head_dim, cache->page_size);
}

w4a4_status w4a4_attn_prefill(const w4a4_kv_cache* cache, const w4a4_kv_seqs* seqs, const int32_t* cu, int64_t tokens,
                              w4a4_dtype dtype, int q_heads, const void* q, int64_t q_row, int64_t q_head, float scale,
                              int window, int sinks, void* out, int64_t o_row, int64_t o_head, float* lse,
                              void* workspace, size_t ws_bytes, void* stream) {
  const char* what = "attn_prefill";
  w4a4_status st = check_cache(what, cache);
  if (st == W4A4_OK) st = check_seqs(what, seqs, true);
  if (st != W4A4_OK) return st;
  if (tokens < 0 || tokens >= kMaxIndex || (tokens > 0 && seqs->seqs == 0))
    return fail(W4A4_ERR_SHAPE, "%s: %lld tokens for %d sequences", what, (long long)tokens, int(seqs->seqs));
  const size_t need = w4a4_attn_prefill_workspace_bytes(cache, seqs->seqs, tokens, q_heads);
  st = check_attn(what, cache, seqs, dtype, q_heads, tokens, q, q_row, q_head, scale, window, sinks, out, o_row, o_head,
                  lse, workspace, ws_bytes, need);
  if (st != W4A4_OK) return st;
  if (tokens == 0) return ok();
  if (w4a4::attn_prefill_workgroups(seqs->seqs, tokens, q_heads, cache->heads, cache->page_size) >= kMaxGrid)
    return fail(W4A4_ERR_SHAPE, "%s: %lld tokens of %d sequences are too many for one call", what, (long long)tokens,
                int(seqs->seqs));
  if (!cu) return fail(W4A4_ERR_NULL, "%s: cu must be non-NULL", what);
  if (!aligned(cu, 4)) return fail(W4A4_ERR_ALIGN, "%s: cu needs 4-byte alignment", what);
  return hip_status(w4a4::launch_attn_prefill(attn_args(cache, seqs, q_heads, q, q_row, q_head, scale, window, sinks,
                                                        out, o_row, o_head, lse),
                                              cu, tokens, cache->dtype, dtype, cache->head_dim, workspace,
                                              static_cast<hipStream_t>(stream)),
                    "attn_prefill launch");
}

w4a4_status w4a4_kv_copy_pages(int n, void* const* arrays, int64_t page_stride_bytes, int64_t page_bytes, int pages,
                               const int32_t* src, const int32_t* dst, int64_t pairs, void* stream) {
  const char* what = "kv_copy_pages";
  w4a4_status st = check_arrays(what, n, arrays, page_stride_bytes, page_bytes, pages);
  if (st == W4A4_OK) st = check_list(what, src, dst, pairs);
  if (st != W4A4_OK) return st;
  if (n == 0 || pairs == 0) return ok();
  return hip_status(w4a4::launch_kv_copy_pages({arrays, n, page_stride_bytes, page_bytes}, pages, src, dst, pairs,
                                               static_cast<hipStream_t>(stream)),
                    "kv_copy_pages launch");
}

size_t w4a4_kv_workspace_bytes(int64_t rows, int64_t pages) {
  if (rows < 0 || pages < 1 || rows >= kMaxIndex || pages >= kMaxIndex) return 0;
  return std::max({w4a4::kv_reserve_workspace(rows, pages), w4a4::kv_fork_workspace(rows, pages),
                   w4a4::kv_compact_workspace(pages)});
}

w4a4_status w4a4_kv_reserve(const w4a4_kv_seqs* seqs, int page_size, int32_t* refs, int pages, int32_t* lacking,
                            void* workspace, size_t ws_bytes, void* stream) {
  const char* what = "kv_reserve";
  w4a4_status st = check_seqs(what, seqs, true);
  if (st == W4A4_OK) st = check_refs(what, refs, pages, page_size);
  if (st == W4A4_OK && !aligned(lacking, 4)) st = fail(W4A4_ERR_ALIGN, "%s: lacking needs 4-byte alignment", what);
  if (st == W4A4_OK) st = check_ws(what, workspace, ws_bytes, w4a4::kv_reserve_workspace(seqs->seqs, pages));
  if (st != W4A4_OK) return st;
  return hip_status(w4a4::launch_kv_reserve(seqs->tables, seqs->table_stride, seqs->lens, seqs->seqs, seqs->max_pages,
                                            refs, pages, page_size, lacking, workspace,
                                            static_cast<hipStream_t>(stream)),
                    "kv_reserve launch");
}

w4a4_status w4a4_kv_fork(int n_arrays, void* const* arrays, int64_t page_stride_bytes, int64_t page_bytes,
                         const w4a4_kv_seqs* seqs, int page_size, int32_t* refs, int pages, const int32_t* parents,
                         const int32_t* children, int n, int32_t* lacking, void* workspace, size_t ws_bytes,
                         void* stream) {
  const char* what = "kv_fork";
  w4a4_status st = check_arrays(what, n_arrays, arrays, page_stride_bytes, page_bytes, pages);
  if (st == W4A4_OK) st = check_seqs(what, seqs, true);
  if (st == W4A4_OK) st = check_refs(what, refs, pages, page_size);
  if (st == W4A4_OK) st = check_list(what, parents, children, n);
  if (st == W4A4_OK && !aligned(lacking, 4)) st = fail(W4A4_ERR_ALIGN, "%s: lacking needs 4-byte alignment", what);
  if (st == W4A4_OK) st = check_ws(what, workspace, ws_bytes, w4a4::kv_fork_workspace(n, pages));
  if (st != W4A4_OK) return st;
  return hip_status(w4a4::launch_kv_fork({arrays, n_arrays, page_stride_bytes, page_bytes}, seqs->tables,
                                         seqs->table_stride, seqs->lens, seqs->seqs, seqs->max_pages, refs, pages,
                                         page_size, parents, children, n, lacking, workspace,
                                         static_cast<hipStream_t>(stream)),
                    "kv_fork launch");
}

static w4a4_status free_pages(const char* what, const w4a4_kv_seqs* seqs, int page_size, int32_t* refs, int pages,
                              const int32_t* ids, int n, bool trim, int window, int sinks, void* stream) {
  w4a4_status st = check_seqs(what, seqs, true);
  if (st == W4A4_OK) st = check_refs(what, refs, pages, page_size);
  if (st != W4A4_OK) return st;
  if (n < 0 || (!ids && n != 0 && n != seqs->seqs))
    return fail(W4A4_ERR_SHAPE, "%s: %d ids (without a list: all %d sequences)", what, n, int(seqs->seqs));
  if (!aligned(ids, 4)) return fail(W4A4_ERR_ALIGN, "%s: ids needs 4-byte alignment", what);
  if (n == 0 || seqs->seqs == 0) return ok();
  return hip_status(w4a4::launch_kv_free(seqs->tables, seqs->table_stride, seqs->lens, seqs->seqs, seqs->max_pages,
                                         refs, pages, page_size, ids, n, trim, window, sinks,
                                         static_cast<hipStream_t>(stream)),
                    what);
}

w4a4_status w4a4_kv_free(const w4a4_kv_seqs* seqs, int32_t* refs, int pages, const int32_t* ids, int n, void* stream) {
  return free_pages("kv_free", seqs, 1, refs, pages, ids, n, false, 0, 0, stream);
}

w4a4_status w4a4_kv_trim(const w4a4_kv_seqs* seqs, int page_size, int32_t* refs, int pages, const int32_t* ids, int n,
                         int window, int sinks, void* stream) {
  if (window < 1 || sinks < 0)
    return fail(W4A4_ERR_SHAPE, "kv_trim: window=%d sinks=%d (need window >= 1, sinks >= 0)", window, sinks);
  return free_pages("kv_trim", seqs, page_size, refs, pages, ids, n, true, window, sinks, stream);
}

w4a4_status w4a4_kv_compact(int n_arrays, void* const* arrays, int64_t page_stride_bytes, int64_t page_bytes,
                            const w4a4_kv_seqs* seqs, int32_t* refs, int pages, int32_t* remap, void* workspace,
                            size_t ws_bytes, void* stream) {
  const char* what = "kv_compact";
  w4a4_status st = check_arrays(what, n_arrays, arrays, page_stride_bytes, page_bytes, pages);
  if (st == W4A4_OK) st = check_seqs(what, seqs, false);
  if (st == W4A4_OK) st = check_refs(what, refs, pages, 1);
  if (st == W4A4_OK && !remap) st = fail(W4A4_ERR_NULL, "%s: remap must be non-NULL", what);
  if (st == W4A4_OK && !aligned(remap, 4)) st = fail(W4A4_ERR_ALIGN, "%s: remap needs 4-byte alignment", what);
  if (st == W4A4_OK) st = check_ws(what, workspace, ws_bytes, w4a4::kv_compact_workspace(pages));
  if (st != W4A4_OK) return st;
  return hip_status(w4a4::launch_kv_compact({arrays, n_arrays, page_stride_bytes, page_bytes}, seqs->tables,
                                            seqs->table_stride, seqs->seqs, seqs->max_pages, refs, pages, remap,
                                            workspace, static_cast<hipStream_t>(stream)),
                    "kv_compact launch");
}

}  // extern "C"
