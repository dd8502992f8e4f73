// The list of work that the decoding kernels share: units (a kv head's query rows
// of one sequence), cut into tiles of visible tokens, one list over all sequences, of
// which every workgroup takes an equal piece; partial results of units that are cut,
// and the kernel that joins them.
#pragma once

#include <algorithm>
#include <type_traits>

#include "attn_common.h"

namespace w4a4 {
namespace {

constexpr int kTile = 128;       // tokens per workgroup step: 4 waves x 32
constexpr int kRows = 16;        // of a unit

// The list of work: per sequence, tiles over [0, sink_end) and [start, len).
// A length beyond the table's capacity is cut to it and marked (`over`).
struct SeqSpan {
  int len, low, start, sink_end, sink_tiles, tiles;
  bool over;
};

// `count`: the sequence's queries, its last tokens.
__device__ __forceinline__ SeqSpan seq_span(const AttnArgs& a, int length, int count) {
  SeqSpan z;
  const int cap = int(min(int64_t(a.kv.max_pages) * a.kv.page.d, int64_t(1) << 30));
  const int len = max(length, 0);
  z.over = len > cap;
  z.len = min(len, cap);
  z.low = a.window ? max(z.len - count + 1 - a.window, 0) : 0;   // first token of the first query's window
  z.start = z.low & ~7;
  z.sink_end = min(a.sinks, z.start);
  z.sink_tiles = (z.sink_end + kTile - 1) / kTile;
  // at least one: a sequence without tokens still has outputs to write
  z.tiles = max(z.sink_tiles + (z.len - z.start + kTile - 1) / kTile, 1);
  return z;
}

// Results of a unit's piece: unnormalised sums o [rows x D], references m of the
// weights and sums of weights l [rows], in the log2 domain.
struct Partial {
  float *o, *m, *l;
};

// A cut unit: written by the workgroup that begins it.
struct Cut {
  int32_t seq, unit, count, unused;      // count: workgroups that hold parts of it
};

struct Work {
  float* parts;       // [workgroups x 2] partial results
  Cut* cuts;          // [workgroups]
  int rows;           // of a partial result
  const int32_t* cu;  // FEW: rows of q
  int tokens;
  FastDiv group;
};

__host__ __device__ constexpr int partial_floats(int rows, int D) { return (rows * (D + 2) + 3) / 4 * 4; }

// A workgroup has at most two pieces of cut units: one that goes on from the
// workgroup before (slot 0) and one that it begins (slot 1).
__device__ __forceinline__ Partial partial_at(const Work& w, int D, int64_t wg, int slot) {
  float* p = w.parts + (wg * 2 + slot) * partial_floats(w.rows, D);
  return {p, p + w.rows * D, p + w.rows * (D + 1)};
}

// A sequence's queries: the rows of one kv head are count * group, token by token.
struct Queries {
  int count, first;
};
template <bool FEW>
__device__ __forceinline__ Queries queries_of(const Work& w, int s) {
  if (!FEW) return {1, s};
  const int first = w.cu[s];
  return {min(max(w.cu[s + 1] - first, 0), w.tokens), first};
}

__device__ __forceinline__ int readlane(int x, int l) { return __builtin_amdgcn_readlane(x, l); }
__device__ __forceinline__ int64_t readlane(int64_t x, int l) {
  return int64_t(uint32_t(__builtin_amdgcn_readlane(int(x), l))) | int64_t(__builtin_amdgcn_readlane(int(x >> 32), l)) << 32;
}

// Output columns d .. d + 3 of row `row` of a kv head from its reference, sum of
// weights and unnormalised sum.
template <class T, int D, int E, bool FEW>
__device__ __forceinline__ void finish(const AttnArgs& a, const Work& w, int head, const Queries& qs, const SeqSpan& sp,
                                       int row, int d, float M, float L, at_f32x4 O) {
  const int tok = FEW ? w.group.div(row) : 0, h = head * a.group + row - tok * a.group;
  const int64_t at = int64_t(qs.first) + tok;
  if (FEW && (at < 0 || at >= w.tokens)) return;
  const bool none = sp.len - qs.count + tok < 0 && !sp.over;       // a query before position 0
  const float inv = (E == 1 && a.kv.v_scale ? a.kv.v_scale[head] : 1.0f) / L;
  at_u32x2 y = {T::pack(O[0] * inv, O[1] * inv), T::pack(O[2] * inv, O[3] * inv)};
  if (none) y = (at_u32x2){0, 0};
  *reinterpret_cast<at_u32x2*>(static_cast<uint16_t*>(a.out) + at * a.o_row + h * a.o_head + d) = y;
  if (a.lse && d == 0) a.lse[at * a.q_heads + h] = none ? kNegInf : (M + __log2f(L)) * 0.693147180559945f;
}

// Tiles that beginning a unit counts as, where a workgroup has 8 tiles or more:
// with 0 the pieces of short sequences, of many units each, end last.  0 / 1 / 2
// on 32 sequences of 100 to 6000 tokens: E4M3, D=128 66.5 / 53.1 / 53.4 us,
// bf16, D=256 157.9 / 147.2 / 148.7; on equal lengths of 3050, 53.6 / 54.8 for
// 0 / 2; the ragged batch 158.9 / 157.5 / 160.1.
constexpr int kStart = 1;
// A workgroup's piece of the list of work, and the place in it where that begins.
struct Piece {
  int64_t item, end, total, wgs, seq_begin;
  int seq, extra, len0;
};

// False where there is none.  unit_rows: rows of a unit.
template <bool FEW>
__device__ __forceinline__ bool find_piece(const AttnArgs& a, const Work& work, int unit_rows, int lane, Piece* out) {
  typedef std::conditional_t<FEW, int64_t, int> Sum;     // of tiles (FEW: times units) of 64 sequences
  const int64_t wg = blockIdx.x;
  // This workgroup's piece [item, end) of the list of (sequence, unit, tile),
  // and the sequence that `item` falls in, with the place where that begins.
  // Lane l looks after the sequences l, l + 64, ...; up to 64 sequences take one
  // load of the lengths.
  auto units_of = [&](int count) { return a.kv.heads * ((count * a.group + unit_rows - 1) / unit_rows); };
  const int64_t units1 = FEW ? 1 : units_of(1);
  auto length = [&](int s) { return s < a.kv.seqs ? a.kv.lens[s] : 0; };
  auto share_of = [&](int s, int len) -> Sum {
    if (s >= a.kv.seqs) return 0;
    const int count = queries_of<FEW>(work, s).count;
    const Sum tiles = seq_span(a, len, count).tiles;
    return FEW ? tiles * units_of(count) : tiles;
  };
  auto scan = [&](Sum t) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const Sum y = __shfl_up(t, d);
      if (lane >= d) t += y;
    }
    return t;
  };
  const int len0 = length(lane);
  const Sum mine0 = share_of(lane, len0), in0 = scan(mine0);
  int64_t total = readlane(in0, 63);
  for (int base = 64; base < a.kv.seqs; base += 64) total += readlane(scan(share_of(base + lane, length(base + lane))), 63);
  // a unit's first tiles stand for the cost of beginning it, and hold no tokens
  const int extra = !FEW && total * units1 >= 8 * int64_t(gridDim.x) ? kStart : 0;
  total = (total + int64_t(extra) * (FEW ? 0 : a.kv.seqs)) * units1;
  const int64_t wgs = min(int64_t(gridDim.x), total);
  if (wg >= wgs) return false;
  int64_t item = wg * total / wgs;
  const int64_t end = (wg + 1) * total / wgs;
  int seq = 0;
  int64_t seq_begin = 0;
  for (int base = 0; base < a.kv.seqs; base += 64) {
    Sum mine = mine0, in = in0;
    if (base) {
      mine = share_of(base + lane, length(base + lane));
      in = scan(mine);
    }
    const uint64_t past = __ballot(seq_begin + (int64_t(in) + extra * (lane + 1)) * units1 > item);
    if (past) {
      const int l = __ffsll((unsigned long long)past) - 1;
      seq = base + l;
      seq_begin += (int64_t(readlane(Sum(in - mine), l)) + extra * l) * units1;
      break;
    }
    seq_begin += (int64_t(readlane(in, 63)) + extra * 64) * units1;
  }
  *out = {item, end, total, wgs, seq_begin, seq, extra, len0};
  return true;
}

// Joins the partial results of units (of ROWS rows) that were cut: o = sum o_i 2^(m_i - M),
// the same for l.  Grid (shares of SHARE workgroups of the list, row shares), each
// workgroup the units that those of its share have begun, if any, and one of their rows, so
// that the chains of dependent reads are short: its launch and their latency bound it.
// D / 4 threads hold a column quad each, the rest of the 256 share the parts.
template <class T, int D, int E, bool FEW, int ROWS, int SHARE>
__global__ void __launch_bounds__(256) decode_join_kernel(AttnArgs a, Work work, int wgs) {
  constexpr int kQuads = D / 4, kSplits = 256 / kQuads;
  __shared__ at_f32x4 lds_o[kSplits][kQuads];
  __shared__ float lds_m[kSplits], lds_l[kSplits];
  const int lane = threadIdx.x & 63;
  uint64_t left = SHARE == 1 ? 1 : __ballot(lane < SHARE && blockIdx.x * SHARE + lane < wgs &&
                                            work.cuts[blockIdx.x * SHARE + lane].count > 1);
  for (; left; left &= left - 1) {
    const int wg = SHARE == 1 ? blockIdx.x
                              : blockIdx.x * SHARE + __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)left) - 1);
    const Cut cut = work.cuts[wg];
    if (SHARE == 1 && cut.count <= 1) return;
    const Queries qs = queries_of<FEW>(work, cut.seq);
    const SeqSpan sp = seq_span(a, a.kv.lens[cut.seq], qs.count);
    const int blocks_per_head = (qs.count * a.group + ROWS - 1) / ROWS;
    const int head = cut.unit / blocks_per_head, unit_row = (cut.unit % blocks_per_head) * ROWS;
    const int rows = min(qs.count * a.group - unit_row, ROWS);
    const int quad = threadIdx.x % kQuads, split = threadIdx.x / kQuads;
    for (int r = blockIdx.y; r < rows; r += gridDim.y) {
      float M = kNegInf, L = 0.0f;
      at_f32x4 O = {0, 0, 0, 0};
#pragma unroll 4
      for (int i = split; i < cut.count; i += kSplits) {
        const Partial p = partial_at(work, D, wg + i, i == 0);
        const float m = p.m[r], l = p.l[r];
        const at_f32x4 o = *reinterpret_cast<const at_f32x4*>(p.o + r * D + 4 * quad);
        const float mn = fmaxf(M, m), f = rebase_joined(M, mn), h = rebase_joined(m, mn);
        L = L * f + l * h;
        O = O * f + o * h;
        M = mn;
      }
      __syncthreads();              // the row before has been read
      lds_o[split][quad] = O;
      if (quad == 0) {
        lds_m[split] = M;
        lds_l[split] = L;
      }
      __syncthreads();
      if (split) continue;
      M = lds_m[0];
      for (int i = 1; i < kSplits; ++i) M = fmaxf(M, lds_m[i]);
      L = 0.0f;
      O = (at_f32x4){0, 0, 0, 0};
      for (int i = 0; i < kSplits; ++i) {
        const float f = rebase_joined(lds_m[i], M);
        L += f * lds_l[i];
        O += lds_o[i][quad] * f;
      }
      finish<T, D, E, FEW>(a, work, head, qs, sp, unit_row + r, 4 * quad, M, L, O);
    }
  }
}

// `units`: at most so many.  Where they are few, most workgroups of the list have begun
// none, and 16 at a time are looked at: microseconds of this kernel with 1 / 16, 12 units of
// 7 rows in 768 workgroups 7.2 / 5.4, 24 of 32 rows in 512 7.1 / 5.2; where a workgroup
// in three has begun one the call takes 43.0 / 46.7, in a ragged batch 52.2 / 53.6.
template <class T, int D, int E, bool FEW, int ROWS = kRows>
hipError_t launch_join(const AttnArgs& a, const Work& w, unsigned wgs, int64_t units, hipStream_t stream) {
  constexpr int kShare = 16;
  if (int64_t(wgs) >= 8 * units)
    decode_join_kernel<T, D, E, FEW, ROWS, kShare><<<dim3((wgs + kShare - 1) / kShare, unsigned(w.rows)), 256, 0, stream>>>(
        a, w, int(wgs));
  else
    decode_join_kernel<T, D, E, FEW, ROWS, 1><<<dim3(wgs, unsigned(w.rows)), 256, 0, stream>>>(a, w, int(wgs));
  return hipGetLastError();
}

size_t workspace_bytes(int rows, int D, int wgs) {
  return size_t(wgs) * (2 * size_t(partial_floats(rows, D)) * 4 + sizeof(Cut));
}

// [parts] [cuts]
Work work_at(void* workspace, int rows, int D, int wgs) {
  Work w;
  w.rows = rows;
  w.parts = static_cast<float*>(workspace);
  w.cuts = reinterpret_cast<Cut*>(w.parts + size_t(wgs) * 2 * partial_floats(rows, D));
  w.cu = nullptr;
  w.tokens = 0;
  w.group = fast_div(1);
  return w;
}

}  // namespace
}  // namespace w4a4
