// The paged key-value cache: storing new tokens, and the bookkeeping of its
// pages (room for tokens, copies, forks, letting go, closing holes).  The
// sequences' tables, lengths and the pages' reference counts live on the
// device and are only read there, so that a serving step needs no host round
// trip and can be captured in a graph.  All of it moves bytes: the bound is
// HBM bandwidth, and for small calls the launches.
#include "kvcache.h"

#include <algorithm>

namespace w4a4 {
namespace {

typedef uint32_t kv_u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t kv_u32x2 __attribute__((ext_vector_type(2)));

// ------------------------------------------------------------------ append --

struct AppendArgs {
  KvView kv;
  const int32_t* cu;
  const void* src[2];
  int64_t row[2], head[2];
  int64_t tokens;
  int head_chunks;    // head_dim / 8
};

// Row of `cu` that holds token i: the last s with cu[s] <= i < cu[s + 1].
__device__ __forceinline__ int find_seq(const int32_t* cu, int seqs, int i) {
  int lo = 0, hi = seqs;          // cu[lo] <= i < cu[hi] if the token belongs to any
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= i) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ float bits_to_f32(uint16_t b, bool f16) {
  if (f16) return float(__builtin_bit_cast(_Float16, b));
  return __builtin_bit_cast(float, uint32_t(b) << 16);
}

// fp32 -> the value an E4M3 conversion takes: saturated, NaN kept
__device__ __forceinline__ float e4m3_range(float x) {
  return x != x ? x : fminf(fmaxf(x, -448.0f), 448.0f);
}

// A workgroup takes `per_wg` tokens: their cache rows are looked up by its first
// threads, then `lanes` threads copy a token's 16-byte chunks (8 elements) of K
// and V, consecutive threads on consecutive chunks of a head, 256 / lanes tokens
// at a time and kFlight of them in flight per thread.  MODE 0 copies 16-bit
// elements, 1 / 2 convert BF16 / FP16 to E4M3 (one IEEE division by the head's
// scale, one RNE conversion per element).
//
// One token each of 16 sequences (0.13 MB): 3.7 us of GPU time, 8.3 with the
// call: latency of the lookups and the copy behind them.  14400 tokens to E4M3, 44 MB: 14.2 us, 3.1 TB/s.
constexpr int kMaxTok = 32, kFlight = 4;

template <int MODE>
__global__ void __launch_bounds__(256) append_kernel(AppendArgs a, int lanes, int per_wg) {
  __shared__ int64_t base[kMaxTok];
  const int64_t first = int64_t(blockIdx.x) * per_wg;
  if (int(threadIdx.x) < per_wg) {
    const int64_t i = first + threadIdx.x;
    int64_t b = -1;
    if (i < a.tokens) {
      int s = int(i), back = 1;     // back: tokens from this one to the sequence's last, inclusive
      bool in = i < a.kv.seqs;
      if (a.cu) {
        s = find_seq(a.cu, a.kv.seqs, int(i));
        back = a.cu[s + 1] - int(i);
        in = back > 0 && a.cu[s] <= int(i);
      }
      if (in) {
        const int64_t pos = int64_t(a.kv.lens[s]) - back;
        if (pos >= 0) {
          int slot;
          const int p = kv_page(a.kv, a.kv.tables + s * a.kv.table_stride, int(pos), &slot);
          if (p >= 0) b = p * a.kv.page_stride + slot * a.kv.token_stride;
        }
      }
    }
    base[threadIdx.x] = b;
  }
  __syncthreads();
  const int per_side = a.kv.heads * a.head_chunks;
  const int t0 = threadIdx.x / lanes, step = 256 / lanes;
  for (int c = threadIdx.x % lanes; c < 2 * per_side; c += lanes) {
    const int side = c >= per_side, r = c - side * per_side;
    const int h = r / a.head_chunks, d = 8 * (r - h * a.head_chunks);
    const uint16_t* src = static_cast<const uint16_t*>(a.src[side]) + first * a.row[side] + h * a.head[side] + d;
    const int64_t at = h * a.kv.head_stride + d;
    void* dst = const_cast<void*>(side ? a.kv.v : a.kv.k);
    float sc = 1.0f;
    if (MODE) {
      const float* scales = side ? a.kv.v_scale : a.kv.k_scale;
      if (scales) sc = scales[h];
    }
    for (int tt = t0; tt < per_wg; tt += kFlight * step) {
      kv_u32x4 x[kFlight];
#pragma unroll
      for (int j = 0; j < kFlight; ++j) {
        const int t = tt + j * step;
        if (t < per_wg && base[t] >= 0) x[j] = *reinterpret_cast<const kv_u32x4*>(src + t * a.row[side]);
      }
#pragma unroll
      for (int j = 0; j < kFlight; ++j) {
        const int t = tt + j * step;
        if (t >= per_wg || base[t] < 0) continue;
        if (MODE == 0) {
          *reinterpret_cast<kv_u32x4*>(static_cast<uint16_t*>(dst) + base[t] + at) = x[j];
        } else {
          kv_u32x2 o;
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            float f[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t u = x[j][2 * w + k / 2];
              f[k] = e4m3_range(bits_to_f32(uint16_t(k & 1 ? u >> 16 : u), MODE == 2) / sc);
            }
            int p = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
            p = __builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], p, true);
            o[w] = uint32_t(p);
          }
          *reinterpret_cast<kv_u32x2*>(static_cast<uint8_t*>(dst) + base[t] + at) = o;
        }
      }
    }
  }
}

// --------------------------------------------------------------- page data --

constexpr int kMaxArrays = 128;     // pointers passed by value: 1 KiB of kernel arguments
struct Arrays {
  uint8_t* p[kMaxArrays];
};

// The tables' share of an operation that moves pages: its first `blocks`
// workgroups, so that it takes no launch of its own.
struct NoBook {
  int blocks = 0;
  __device__ void operator()() const {}
};
// The children's tables, one workgroup each; whole pages get one more reference.
struct ForkBook {
  int32_t* tables;
  int64_t table_stride;
  const int32_t* lens;
  int seqs, max_pages;
  int32_t* refs;
  int pages, page_size;
  const int32_t *parents, *children, *own;
  int blocks;
  __device__ void operator()() const {
    const int p = parents[blockIdx.x], c = children[blockIdx.x];
    if (p < 0 || p >= seqs || c < 0 || c >= seqs || p == c) return;
    const int full = max(lens[p], 0) / page_size;
    const int last = own[blockIdx.x];
    for (int j = threadIdx.x; j < max_pages; j += 256) {
      int e = -1;
      if (j < full) {
        e = tables[p * table_stride + j];
        if (e >= 0 && e < pages) atomicAdd(&refs[e], 1);
        else e = -1;
      } else if (j == full) {
        e = last;
      }
      tables[c * table_stride + j] = e;
    }
  }
};
// Every table entry to its page's new place; the references move along.
struct CompactBook {
  int32_t* tables;
  int64_t table_stride, entries;
  int max_pages;
  int32_t* refs;
  int pages;
  const int32_t *remap, *src, *dst, *count;
  int blocks;
  __device__ void operator()() const {
    const int64_t stride = int64_t(blocks) * 256, at = int64_t(blockIdx.x) * 256 + threadIdx.x;
    for (int64_t i = at; i < entries; i += stride) {
      int32_t* e = tables + (i / max_pages) * table_stride + i % max_pages;
      const int32_t p = *e;
      if (p >= 0) *e = p < pages ? remap[p] : -1;
    }
    const int n = *count;
    for (int64_t i = at; i < n; i += stride) {
      refs[dst[i]] = refs[src[i]];
      refs[src[i]] = 0;
    }
  }
};

// Moves page src[i] to dst[i], i < pairs (or *count if given), in n arrays.
// Work items are 16 KiB pieces of a page (4 units of 16 bytes per thread, all
// loaded before the first store), handed out in a grid-stride loop, since the
// number of pairs may only be known on the device.  1.07 GB (read and written)
// in 212 to 219 us, 4.9 TB/s: a large copy's rate.  The copies of a fork of 4
// sequences into 32 over 16 layers, 67 MB of which 4 MB are read from HBM: 8.5 to
// 10 us.
template <typename UNIT, class BOOK>
__global__ void __launch_bounds__(256) copy_pages_kernel(Arrays arrays, int n, int64_t stride, int64_t units, int pages,
                                                         const int32_t* __restrict__ src,
                                                         const int32_t* __restrict__ dst, int64_t pairs,
                                                         const int32_t* __restrict__ count, BOOK book) {
  if (int(blockIdx.x) < book.blocks) {
    book();
    return;
  }
  if (count) pairs = min(pairs, int64_t(*count));
  const int64_t pieces = (units + 1023) / 1024;
  const int64_t items = pairs * n * pieces;
  for (int64_t it = blockIdx.x - book.blocks; it < items; it += gridDim.x - book.blocks) {
    const int64_t piece = it % pieces, rest = it / pieces;
    const int64_t i = rest / n;
    const int s = src[i], d = dst[i];
    if (s < 0 || s >= pages || d < 0 || d >= pages) continue;
    uint8_t* base = arrays.p[rest - i * n];
    const UNIT* from = reinterpret_cast<const UNIT*>(base + s * stride);
    UNIT* to = reinterpret_cast<UNIT*>(base + d * stride);
    const int64_t u = piece * 1024 + threadIdx.x;
    UNIT x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (u + 256 * j < units) x[j] = from[u + 256 * j];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (u + 256 * j < units) to[u + 256 * j] = x[j];
  }
}

template <class BOOK>
hipError_t copy_pairs(const PageMove& mv, int pages, const int32_t* src, const int32_t* dst, int64_t pairs,
                      const int32_t* count, BOOK book, hipStream_t stream) {
  const bool wide = mv.page_bytes % 16 == 0 && mv.stride_bytes % 16 == 0;   // array bases are 16-byte aligned
  const int64_t units = wide ? mv.page_bytes / 16 : mv.page_bytes;
  for (int at = 0; at < std::max(mv.n, 1); at += kMaxArrays) {
    const int n = std::min(mv.n - at, kMaxArrays);
    Arrays a;
    for (int i = 0; i < kMaxArrays; ++i) a.p[i] = i < n ? static_cast<uint8_t*>(mv.arrays[at + i]) : nullptr;
    if (at) book.blocks = 0;
    const int64_t items = pairs * n * ((units + 1023) / 1024);
    const unsigned grid = unsigned(std::min<int64_t>(items, 4096) + book.blocks);
    if (grid == 0) continue;
    if (wide)
      copy_pages_kernel<kv_u32x4><<<grid, 256, 0, stream>>>(a, n, mv.stride_bytes, units, pages, src, dst, pairs, count, book);
    else
      copy_pages_kernel<uint8_t><<<grid, 256, 0, stream>>>(a, n, mv.stride_bytes, units, pages, src, dst, pairs, count, book);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// --------------------------------------------------------------- page plans --

constexpr int kPlan = 1024;         // threads of the one workgroup that plans

// Exclusive sum of x over the workgroup's threads in order; *total gets the sum.
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t* wave_sums, int64_t* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t in = x;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t y = __shfl_up(in, d);
    if (lane >= d) in += y;
  }
  __syncthreads();                  // wave_sums may still be read from the scan before
  if (lane == 63) wave_sums[wave] = in;
  __syncthreads();
  int64_t before = 0, all = 0;
  for (int w = 0; w < kPlan / 64; ++w) {
    const int64_t y = wave_sums[w];
    if (w < wave) before += y;
    all += y;
  }
  *total = all;
  return before + in - x;
}

// Writes the lowest `want` free pages (refs == 0) in ascending order to list;
// returns how many there were (at most `want`).
__device__ int64_t lowest_free(const int32_t* refs, int pages, int64_t want, int32_t* list, int64_t* wave_sums) {
  int64_t found = 0;
  for (int64_t base = 0; base < pages && found < want; base += 8 * kPlan) {
    const int64_t p0 = base + 8 * threadIdx.x;
    int32_t r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = p0 + j < pages ? refs[p0 + j] : 1;
    int mine = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) mine += r[j] == 0;
    int64_t total;
    int64_t rank = found + block_scan(mine, wave_sums, &total);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (r[j] == 0) {
        if (rank < want) list[rank] = int32_t(p0 + j);
        ++rank;
      }
    found += total;
  }
  __syncthreads();
  return found < want ? found : want;
}

// One workgroup: rows are looked at 1024 at a time (a thread walks back from
// the last entry its row needs; a row whose walk is long, as a new sequence's,
// is searched by its wave together), then the free pages are listed and dealt
// out.  first[s] and off[s] (the row's first missing entry and its place among
// all missing ones) live in the workspace.  The order of pages is part of the
// result, so one workgroup counts; its chain of reads and barriers bounds it:
// 3.5 us at 32 sequences.
__global__ void __launch_bounds__(kPlan) reserve_kernel(int32_t* tables, int64_t table_stride,
                                                        const int32_t* __restrict__ lens, int seqs, int max_pages,
                                                        int32_t* refs, int pages, int page_size,
                                                        int32_t* __restrict__ lacking, int64_t* off, int32_t* first,
                                                        int32_t* list) {
  __shared__ int64_t sums[kPlan / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t want = 0, beyond = 0;
  for (int base = 0; base < seqs; base += kPlan) {
    const int s = base + threadIdx.x;
    int64_t over = 0;
    int j = 0, end = 0;
    if (s < seqs) {
      const int64_t need = (int64_t(max(lens[s], 0)) + page_size - 1) / page_size;
      end = int(min(need, int64_t(max_pages)));
      over = need - end;
      j = end;
      const int32_t* row = tables + s * table_stride;
      for (int k = 0; k < 2 && j > 0 && row[j - 1] < 0; ++k) --j;
    }
    const bool more = s < seqs && j > 0 && end - j == 2;
    for (uint64_t todo = __ballot(more); todo; todo &= todo - 1) {
      const int l = __ffsll((unsigned long long)todo) - 1;
      const int32_t* row = tables + int64_t(__shfl(s, l)) * table_stride;
      int at = __shfl(j, l);
      while (at > 0) {
        const bool held = at - 1 - lane >= 0 && row[at - 1 - lane] >= 0;
        const uint64_t m = __ballot(held);
        if (m) {
          at -= __ffsll((unsigned long long)m) - 1;
          break;
        }
        at = max(at - 64, 0);
      }
      if (lane == l) j = at;
    }
    int64_t total;
    const int64_t before = block_scan(end - j, sums, &total);
    if (s < seqs) {
      off[s] = want + before;
      first[s] = j;
    }
    want += total;
    block_scan(over, sums, &total);
    beyond += total;
  }
  if (threadIdx.x == 0) off[seqs] = want;
  const int64_t got = want ? lowest_free(refs, pages, min(want, int64_t(pages)), list, sums) : 0;
  __syncthreads();
  if (want)
    for (int s = wave; s < seqs; s += kPlan / 64) {
      const int64_t from = off[s], to = off[s + 1];
      for (int64_t r = from + lane; r < to && r < got; r += 64) {
        const int32_t p = list[r];
        tables[s * table_stride + first[s] + (r - from)] = p;
        refs[p] = 1;
      }
    }
  if (lacking && threadIdx.x == 0) *lacking = int32_t(min(want - got + beyond, int64_t(INT32_MAX)));
}

// One workgroup: which children need a page of their own for the parent's last
// tokens, and which one.  src / dst get the pages to copy (-1: none).  6 us, as
// reserve_kernel a chain of reads and barriers.
__global__ void __launch_bounds__(kPlan) fork_plan_kernel(const int32_t* __restrict__ tables, int64_t table_stride,
                                                          int32_t* lens, int seqs, int max_pages, int32_t* refs,
                                                          int pages, int page_size,
                                                          const int32_t* __restrict__ parents,
                                                          const int32_t* __restrict__ children, int n,
                                                          int32_t* __restrict__ lacking, int32_t* src, int32_t* dst,
                                                          int32_t* list) {
  __shared__ int64_t sums[kPlan / 64];
  int64_t want = 0;
  for (int base = 0; base < n; base += kPlan) {
    const int i = base + threadIdx.x;
    int page = -1;
    if (i < n) {
      const int p = parents[i], c = children[i];
      if (p >= 0 && p < seqs && c >= 0 && c < seqs && p != c) {
        const int len = max(lens[p], 0), full = len / page_size;
        if (len % page_size && full < max_pages) {
          page = tables[p * table_stride + full];
          if (page >= pages) page = -1;
        }
        lens[c] = len;
      }
      src[i] = page;
    }
    int64_t total;
    const int64_t rank = want + block_scan(page >= 0, sums, &total);
    if (i < n) dst[i] = page >= 0 ? int32_t(rank) : -1;     // its place in the list, until that is known
    want += total;
  }
  const int64_t got = want ? lowest_free(refs, pages, min(want, int64_t(pages)), list, sums) : 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlan) {
    const int rank = dst[i];
    const int p = rank >= 0 && rank < got ? list[rank] : -1;
    dst[i] = p;
    if (p >= 0) refs[p] = 1;
  }
  if (lacking && threadIdx.x == 0) *lacking = int32_t(want - got);
}

// One workgroup per sequence.  An entry is taken out of the table with an
// atomic exchange, and only who got it drops the reference, so an id that is
// listed twice is freed once.  3.1 us for 32 sequences, of which launching is most.
__global__ void __launch_bounds__(256) free_kernel(int32_t* tables, int64_t table_stride, int32_t* lens, int seqs,
                                                   int max_pages, int32_t* refs, int pages, int page_size,
                                                   const int32_t* __restrict__ ids, int trim, int window, int sinks) {
  const int s = ids ? ids[blockIdx.x] : int(blockIdx.x);
  if (s < 0 || s >= seqs) return;
  int from = 0, to = max_pages, keep = -1;
  if (trim) {
    const int64_t len = lens[s], last = len - window;            // tokens after `last` stay visible
    from = int(min((int64_t(sinks) + page_size - 1) / page_size, int64_t(max_pages)));
    to = last < 0 ? 0 : int(min((last + 1) / page_size, int64_t(max_pages)));
    keep = len > 0 ? int((len - 1) / page_size) : -1;
  }
  int32_t* row = tables + s * table_stride;
  for (int j = from + int(threadIdx.x); j < to; j += 256) {
    if (j == keep || row[j] < 0) continue;
    const int e = atomicExch(&row[j], -1);
    if (e >= 0 && e < pages) atomicSub(&refs[e], 1);
  }
  if (!trim && threadIdx.x == 0) lens[s] = 0;
}

// One workgroup: counts the pages in use, then lists the free pages below that
// count and the used ones from there on (equally many), in ascending order.
// 6.9 us beside the copies' 212.
__global__ void __launch_bounds__(kPlan) compact_plan_kernel(const int32_t* __restrict__ refs, int pages,
                                                             int32_t* remap, int32_t* src, int32_t* dst,
                                                             int32_t* count) {
  __shared__ int64_t sums[kPlan / 64];
  int64_t live = 0;
  for (int64_t p = threadIdx.x; p < pages; p += kPlan) live += refs[p] != 0;
  int64_t total;
  block_scan(live, sums, &total);
  live = total;
  int64_t holes = 0, movers = 0;
  for (int64_t base = 0; base < pages; base += 8 * kPlan) {
    const int64_t p0 = base + 8 * threadIdx.x;
    bool hole[8], mover[8];
    int nh = 0, nm = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t p = p0 + j;
      const bool in = p < pages, used = in && refs[p] != 0;
      hole[j] = in && !used && p < live;
      mover[j] = used && p >= live;
      nh += hole[j];
      nm += mover[j];
      if (in) remap[p] = used ? int32_t(p) : -1;
    }
    // both counts in one scan: fewer than 2^31 of each
    const int64_t before = block_scan(int64_t(nh) | (int64_t(nm) << 32), sums, &total);
    int64_t h = holes + (before & 0xffffffff), m = movers + (before >> 32);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (hole[j]) dst[h++] = int32_t(p0 + j);
      if (mover[j]) src[m++] = int32_t(p0 + j);
    }
    holes += total & 0xffffffff;
    movers += total >> 32;
  }
  __syncthreads();
  for (int64_t i = threadIdx.x; i < movers; i += kPlan) remap[src[i]] = dst[i];
  if (threadIdx.x == 0) *count = int32_t(movers);
}

size_t round16(size_t n) { return (n + 15) / 16 * 16; }

}  // namespace

template <int MODE>
static void append_mode(const AppendArgs& a, hipStream_t stream) {
  int lanes = 16;                                      // a power of two that holds a token's chunks, at most 256
  while (lanes < 256 && lanes < 2 * a.kv.heads * a.head_chunks) lanes *= 2;
  // as many passes as a thread has loads in flight (14400 tokens to E4M3: one
  // pass 19.2 us, four 15.7; 16 tokens 8.4 and 8.3)
  const int per_wg = std::min(kMaxTok, 256 / lanes * kFlight);
  append_kernel<MODE><<<unsigned((a.tokens + per_wg - 1) / per_wg), 256, 0, stream>>>(a, lanes, per_wg);
}

hipError_t launch_kv_append(const KvView& kv, int dtype, int head_dim, const int32_t* cu, int64_t tokens, int in_dtype,
                            const void* k, int64_t k_row, int64_t k_head, const void* v, int64_t v_row, int64_t v_head,
                            hipStream_t stream) {
  AppendArgs a{kv, cu, {k, v}, {k_row, v_row}, {k_head, v_head}, tokens, head_dim / 8};
  if (dtype != W4A4_E4M3) append_mode<0>(a, stream);
  else if (in_dtype == W4A4_BF16) append_mode<1>(a, stream);
  else append_mode<2>(a, stream);
  return hipGetLastError();
}

hipError_t launch_kv_copy_pages(const PageMove& mv, int pages, const int32_t* src, const int32_t* dst, int64_t pairs,
                                hipStream_t stream) {
  return copy_pairs(mv, pages, src, dst, pairs, nullptr, NoBook(), stream);
}

// [off int64 x (seqs + 1)] [first int32 x seqs] [list int32 x pages]
size_t kv_reserve_workspace(int64_t seqs, int64_t pages) {
  return round16(size_t(seqs + 1) * 8) + round16(size_t(seqs) * 4) + round16(size_t(pages) * 4);
}

hipError_t launch_kv_reserve(int32_t* tables, int64_t table_stride, const int32_t* lens, int seqs, int max_pages,
                             int32_t* refs, int pages, int page_size, int32_t* lacking, void* workspace,
                             hipStream_t stream) {
  char* w = static_cast<char*>(workspace);
  int64_t* off = reinterpret_cast<int64_t*>(w);
  w += round16(size_t(seqs + 1) * 8);
  int32_t* first = reinterpret_cast<int32_t*>(w);
  w += round16(size_t(seqs) * 4);
  reserve_kernel<<<1, kPlan, 0, stream>>>(tables, table_stride, lens, seqs, max_pages, refs, pages, page_size, lacking,
                                          off, first, reinterpret_cast<int32_t*>(w));
  return hipGetLastError();
}

// [src int32 x n] [dst int32 x n] [list int32 x pages]
size_t kv_fork_workspace(int64_t n, int64_t pages) { return 2 * round16(size_t(n) * 4) + round16(size_t(pages) * 4); }

hipError_t launch_kv_fork(const PageMove& mv, int32_t* tables, int64_t table_stride, int32_t* lens, int seqs,
                          int max_pages, int32_t* refs, int pages, int page_size, const int32_t* parents,
                          const int32_t* children, int n, int32_t* lacking, void* workspace, hipStream_t stream) {
  char* w = static_cast<char*>(workspace);
  int32_t* src = reinterpret_cast<int32_t*>(w);
  w += round16(size_t(n) * 4);
  int32_t* dst = reinterpret_cast<int32_t*>(w);
  w += round16(size_t(n) * 4);
  fork_plan_kernel<<<1, kPlan, 0, stream>>>(tables, table_stride, lens, seqs, max_pages, refs, pages, page_size,
                                            parents, children, n, lacking, src, dst, reinterpret_cast<int32_t*>(w));
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || n == 0) return e;
  return copy_pairs(mv, pages, src, dst, n, nullptr,
                    ForkBook{tables, table_stride, lens, seqs, max_pages, refs, pages, page_size, parents, children, dst, n},
                    stream);
}

hipError_t launch_kv_free(int32_t* tables, int64_t table_stride, int32_t* lens, int seqs, int max_pages, int32_t* refs,
                          int pages, int page_size, const int32_t* ids, int n, bool trim, int window, int sinks,
                          hipStream_t stream) {
  free_kernel<<<unsigned(n), 256, 0, stream>>>(tables, table_stride, lens, seqs, max_pages, refs, pages, page_size, ids,
                                               trim, window, sinks);
  return hipGetLastError();
}

// [src int32 x pages] [dst int32 x pages] [count]
size_t kv_compact_workspace(int64_t pages) { return 2 * round16(size_t(pages) * 4) + 16; }

hipError_t launch_kv_compact(const PageMove& mv, int32_t* tables, int64_t table_stride, int seqs, int max_pages,
                             int32_t* refs, int pages, int32_t* remap, void* workspace, hipStream_t stream) {
  char* w = static_cast<char*>(workspace);
  int32_t* src = reinterpret_cast<int32_t*>(w);
  w += round16(size_t(pages) * 4);
  int32_t* dst = reinterpret_cast<int32_t*>(w);
  w += round16(size_t(pages) * 4);
  int32_t* count = reinterpret_cast<int32_t*>(w);
  compact_plan_kernel<<<1, kPlan, 0, stream>>>(refs, pages, remap, src, dst, count);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // at most half of the pages move: as many holes lie below them
  const int64_t entries = int64_t(seqs) * max_pages;
  const int blocks = int(std::min<int64_t>(256, (std::max<int64_t>(entries, pages / 2 + 1) + 255) / 256));
  return copy_pairs(mv, pages, src, dst, pages / 2 + 1, count,
                    CompactBook{tables, table_stride, entries, max_pages, refs, pages, remap, src, dst, count, blocks},
                    stream);
}

}  // namespace w4a4
