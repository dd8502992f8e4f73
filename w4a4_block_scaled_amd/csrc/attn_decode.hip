// Attention of one new token per sequence, or a few, over the paged cache.
//
// Each kv head of each sequence is a unit with the group's heads as query rows,
// in blocks of 16 (FEW: the heads of its few tokens), and reads its visible keys
// and values once: 4 to 16 fp operations per byte, so HBM bandwidth bounds it.
// The units' visible tokens, in tiles of 128, form one list over all sequences,
// of which every workgroup takes an equal contiguous piece, whatever the lengths
// are, so that the last ones to end end together.  A
// workgroup that holds a unit whole writes its output; a unit cut by the
// pieces' ends leaves partial results (unnormalised sum, reference, sum of
// weights) that a second kernel joins.
//
// Inside a tile each of the 4 waves takes 32 tokens.  Scores come from the
// transposed product S^T = K Q^T (16 x 16 x 32 MFMA, keys as the first operand,
// loaded from the cache straight in operand order), so that a lane holds
// scores of one query row and the 8 tokens 8 g .. 8 g + 7 of its quarter wave
// g; the same registers are the second operand of O^T = V^T P^T.  V's operand
// needs 8 tokens of one d per lane: a lane loads the same d's of 8 tokens and
// transposes them in registers.  No value passes through LDS until the waves
// of a workgroup are merged.  The weights enter the product as two 16-bit parts
// (high and rest, about 16 bits together): the matrix cores idle here, so the
// second product is free and only the output is rounded to 16 bits.
//
// Measured (a plain read of as many bytes runs at 5.4 to 5.7 TB/s here): a
// ragged batch of bf16, 810 MB, 158 us, 5.1 TB/s; three sequences of 90 to 131
// thousand tokens in E4M3, 340 MB, 76 us (69 and 7 of the join); a window of
// 1024 with sinks over 128 fp16 sequences, D = 64, 514 MB, 108 us, 4.8 TB/s; one
// sequence of 2.1 MB 12.4 to 13.6 us: two launches of 7.4 and 2.7 us, and the calls.
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

// ---------------------------------------------------------------- operands --

// Raw keys and values of 32 tokens of one head, in a wave's registers.  E:
// element bytes.
template <class T, int D, int E>
struct Tile {
  static constexpr int kSteps = D / 32;                 // MFMAs of one 16-token score block
  static constexpr int kRun = D >= 128 ? 8 : D / 16;    // consecutive d's per lane of a value row
  static constexpr int kRuns = D / 16 / kRun;
  static constexpr int kVWords = kRun * E / 4;          // dwords per token and run

  at_u32x4 k[2][kSteps * E / 2];
  uint32_t v[8][kRuns][kVWords];

  // First d of the 8 that quarter g holds of step j.  E4M3: one 16-byte load
  // serves the steps 2 c and 2 c + 1.
  static __device__ __forceinline__ int key_dim(int j, int g) {
    return E == 2 ? 32 * j + 8 * g : 64 * (j >> 1) + 16 * g + 8 * (j & 1);
  }
  __device__ __forceinline__ void load_k(int b, const uint8_t* row, int g) {
#pragma unroll
    for (int c = 0; c < kSteps * E / 2; ++c)
      k[b][c] = *reinterpret_cast<const at_u32x4*>(row + 64 * c + 16 * g);
  }
  __device__ __forceinline__ void load_v(int i, const uint8_t* row, int c) {
#pragma unroll
    for (int r = 0; r < kRuns; ++r) {
      const uint8_t* p = row + (r * 128 + c * kRun) * E;
      if constexpr (kVWords == 4) {
        const at_u32x4 x = *reinterpret_cast<const at_u32x4*>(p);
#pragma unroll
        for (int w = 0; w < 4; ++w) v[i][r][w] = x[w];
      } else if constexpr (kVWords == 2) {
        const at_u32x2 x = *reinterpret_cast<const at_u32x2*>(p);
#pragma unroll
        for (int w = 0; w < 2; ++w) v[i][r][w] = x[w];
      } else {
        v[i][r][0] = *reinterpret_cast<const uint32_t*>(p);
      }
    }
  }
  __device__ __forceinline__ void clear_v(int i) {
#pragma unroll
    for (int r = 0; r < kRuns; ++r)
#pragma unroll
      for (int w = 0; w < kVWords; ++w) v[i][r][w] = 0;
  }

  // Key operand of block b, step j.
  __device__ __forceinline__ at_u32x4 key(int b, int j) const {
    if constexpr (E == 2) {
      return k[b][j];
    } else {
      const uint32_t x = k[b][j >> 1][2 * (j & 1)], y = k[b][j >> 1][2 * (j & 1) + 1];
      return (at_u32x4){e4m3_pair<T, false>(x), e4m3_pair<T, true>(x), e4m3_pair<T, false>(y), e4m3_pair<T, true>(y)};
    }
  }
  // Value operands of the elements j and j + 1 (j even) of run r: 8 tokens each.
  __device__ __forceinline__ void values(int r, int j, at_u32x4* lo, at_u32x4* hi) const {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if constexpr (E == 2) {
        const uint32_t x = v[2 * t][r][j / 2], y = v[2 * t + 1][r][j / 2];
        (*lo)[t] = __builtin_amdgcn_perm(y, x, 0x05040100);
        (*hi)[t] = __builtin_amdgcn_perm(y, x, 0x07060302);
      } else {
        const uint32_t x = v[2 * t][r][j / 4], y = v[2 * t + 1][r][j / 4];
        const uint32_t z = __builtin_amdgcn_perm(y, x, j % 4 ? 0x07030602 : 0x05010400);      // codes x_j y_j x_j+1 y_j+1
        (*lo)[t] = e4m3_pair<T, false>(z);
        (*hi)[t] = e4m3_pair<T, true>(z);
      }
    }
  }
};

// Table entries and page rows of the tokens that a lane reads of a tile.
template <bool OCT>
struct Rows {
  int page[OCT ? 2 : 10], slot[OCT ? 2 : 10];      // of the keys, then of the values
};

// ------------------------------------------------------------------ kernel --

// Whether a wave holds two tiles in registers or one, and the workgroups that
// then share a CU.  One tile is enough to keep the memory busy where its bytes
// are few or the rows' addresses take the registers; two gain where a tile is
// large.  Microseconds on 4 to 6 thousand cached tokens each of 32 sequences,
// one tile / two: bf16, D=128 (the ragged batch) 162.3 / 158.2; E4M3, D=128
// 65.5 / 65.0, D=64 85.3 / 90.6, D=256 115.9 / 120.6; token by token (!OCT),
// bf16, D=128 90.7 / 175.3, D=64 108.6 / 124.0 (two tiles spill).  Workgroups,
// for one tile: E4M3, D=64 4 / 3: 79.5 / 85.3, D=256 2 / 1: 94.8 / 115.9,
// D=128 3 / 2 (the long cache): 87.3 / 76.8.
constexpr bool two_tiles(int D, int E, bool oct) { return oct && E == 2 && D < 256; }
constexpr int wgs_per_cu(int D, int E, bool oct) {
  if (D == 256) return oct && E == 1 ? 2 : 1;
  return oct && D == 64 ? (E == 1 ? 4 : 3) : 2;
}

// Tiles that beginning a unit counts as, where a workgroup has 8 tiles or more:
// with 0 the pieces of short sequences, of many units each, end last.  0 / 1 / 2
// on 32 sequences of 100 to 6000 tokens: E4M3, D=128 66.5 / 53.1 / 53.4 us,
// bf16, D=256 157.9 / 147.2 / 148.7; on equal lengths of 3050, 53.6 / 54.8 for
// 0 / 2; the ragged batch 158.9 / 157.5 / 160.1.
constexpr int kStart = 1;
constexpr int kMaxPerCu = 4;     // the workspaces' size

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

// Adds the Inf and NaN of a value operand to the sums of the rows that see them
// (`see`: 1.0 or 0 per token and row), and returns it with zeros in their place.
template <class T>
__device__ __forceinline__ at_u32x4 add_odd(at_u32x4 v, at_u32x4 see, at_f32x4* o) {
  at_u32x4 plus, minus;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t p, n;
    v[k] = T::split_odd(v[k], &p, &n);
    plus[k] = p;
    minus[k] = n;
  }
  const at_f32x4 zero = {0, 0, 0, 0}, up = T::mfma16(plus, see, zero), down = T::mfma16(minus, see, zero);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (up[i] > 0.0f) (*o)[i] -= kNegInf;
    if (down[i] > 0.0f) (*o)[i] += kNegInf;
  }
  return v;
}

// OCT: the page size is a multiple of 8, so 8 tokens from a multiple of 8 lie
// on one page and one lookup serves them; otherwise every row is looked up.
// (32 sequences of 100 to 6000 tokens, 400 MB of bf16, D=128: page 16 87.7 us,
// page 11 92.4.)
// FEW: the sequences have any number of queries (a few, if it is to be fast).
template <class T, int D, int E, bool OCT, bool FEW>
__global__ void __launch_bounds__(256, wgs_per_cu(D, E, OCT)) decode_kernel(AttnArgs a, Work work) {
  typedef Tile<T, D, E> TileT;
  constexpr bool TWO = two_tiles(D, E, OCT);
  static_assert(wgs_per_cu(D, E, OCT) <= kMaxPerCu);
  constexpr int kSteps = TileT::kSteps, kRun = TileT::kRun, kRuns = TileT::kRuns;
  constexpr int kBlocks = D / 16;                        // MFMAs of the value product
  typedef std::conditional_t<FEW, int64_t, int> Sum;     // of tiles (FEW: times units) of 64 sequences
  __shared__ float lds_o[4][kRows][D + 4];
  __shared__ float lds_m[4][kRows], lds_l[4][kRows];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, c = lane & 15;
  const int64_t wg = blockIdx.x;
  if (threadIdx.x == 0) work.cuts[wg].count = 0;

  // This workgroup's piece [item, end) of the list of (sequence, unit, tile),
  // and the sequence that `item` falls in, with the place where that begins.
  // Lane l looks after the sequences l, l + 64, ...; up to 64 sequences take one
  // load of the lengths.
  auto units_of = [&](int count) { return a.kv.heads * ((count * a.group + kRows - 1) / kRows); };
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
  if (wg >= wgs) return;
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

  while (item < end && seq < a.kv.seqs) {
    const Queries qs = queries_of<FEW>(work, seq);
    const SeqSpan sp = seq_span(a, seq < 64 ? __builtin_amdgcn_readlane(len0, seq) : a.kv.lens[seq], qs.count);
    const int units = units_of(qs.count);
    const int64_t in_seq = item - seq_begin;
    const int places = sp.tiles + extra;
    if (in_seq >= int64_t(places) * units) {
      seq_begin += int64_t(places) * units;
      ++seq;
      continue;
    }
    const int unit = int(in_seq / places);
    const int64_t unit_begin = seq_begin + int64_t(unit) * places + extra;    // of its tiles
    const int t0 = int(max(item - unit_begin, int64_t(0)));
    const int t1 = int(min(int64_t(sp.tiles), end - unit_begin));
    item = unit_begin + t1;
    if (t1 <= t0) continue;

    const int blocks_per_head = units / a.kv.heads;
    const int head = unit / blocks_per_head;
    const int unit_row = (unit % blocks_per_head) * kRows;
    const int rows = min(qs.count * a.group - unit_row, kRows);
    // this lane's row: its token and head of the group, and its position
    const int row = unit_row + min(c, rows - 1);
    const int tok = FEW ? work.group.div(row) : 0;
    const int in_group = row - tok * a.group;
    const int past = sp.len - qs.count;
    const int pos = past + tok;
    // positions of the unit's first and last row
    const int pos_min = past + (FEW ? work.group.div(unit_row) : 0);
    const int pos_max = past + (FEW ? work.group.div(unit_row + rows - 1) : 0);
    const float cs = a.scale_log2 * (E == 1 && a.kv.k_scale ? a.kv.k_scale[head] : 1.0f);
    const int32_t* table = a.kv.tables + seq * a.kv.table_stride;
    const uint8_t* kbase = static_cast<const uint8_t*>(a.kv.k) + head * a.kv.head_stride * E;
    const uint8_t* vbase = static_cast<const uint8_t*>(a.kv.v) + head * a.kv.head_stride * E;
    const int64_t step = a.kv.token_stride * E;

    // query operand: row c, zero past the unit's rows
    at_u32x4 q[kSteps];
    {
      const int at = FEW ? min(max(qs.first + tok, 0), work.tokens - 1) : seq;
      const uint16_t* qp = static_cast<const uint16_t*>(a.q) + at * a.q_row + (int64_t(head) * a.group + in_group) * a.q_head;
#pragma unroll
      for (int j = 0; j < kSteps; ++j) {
        q[j] = *reinterpret_cast<const at_u32x4*>(qp + TileT::key_dim(j, g));
        if (c >= rows) q[j] = (at_u32x4){0, 0, 0, 0};
      }
    }

    at_f32x4 o[kBlocks];
    float m, l;
    bool bad = sp.over, odd = false;      // odd: the second time, for Inf and NaN among the values

    // first token of this wave's part of tile t, and the end of its range
    auto tile_at = [&](int t, int* stop) {
      const bool sink = t < sp.sink_tiles;
      *stop = sink ? sp.sink_end : sp.len;
      return (sink ? t * kTile : sp.start + (t - sp.sink_tiles) * kTile) + wave * 32;
    };
    // whether any row of the sequence sees token t, and whether this lane's does
    auto seen = [&](int t, int stop) { return t < stop && (t >= sp.low || t < a.sinks); };
    auto sees = [&](int t, int stop) {
      if (!FEW) return seen(t, stop);
      return t < stop && t <= pos && (!a.window || t > pos - a.window || t < a.sinks);
    };
    // Tokens past the end of the range take the place of its last one (last 8
    // tokens).  Only reads the table: what it gave is looked at in load(), an
    // iteration later.
    auto find = [&](Rows<OCT>& r, int t) {
      int stop;
      const int base = tile_at(t, &stop);
      auto place = [&](int i, int u) {
        const int j = a.kv.page.div(max(u, 0));
        r.slot[i] = max(u, 0) - j * int(a.kv.page.d);
        r.page[i] = table[j];
      };
      if constexpr (OCT) {
        const int last = (stop - 1) & ~7;
        place(0, min(base + 8 * (c >> 2), last));
        place(1, min(base + 8 * g, last));
      } else {
#pragma unroll
        for (int b = 0; b < 2; ++b) place(b, min(base + 8 * (c >> 2) + 4 * b + (c & 3), stop - 1));
#pragma unroll
        for (int i = 0; i < 8; ++i) place(2 + i, min(base + 8 * g + i, stop - 1));
      }
    };
    // An entry outside the cache is read as page 0, and spoils the result if a
    // query sees a token there (the keys' entries are the values').
    auto row_at = [&](const Rows<OCT>& r, int i) -> int64_t {
      const int p = uint32_t(r.page[i]) < uint32_t(a.kv.pages) ? r.page[i] : 0;
      return (int64_t(p) * a.kv.page_stride + int64_t(r.slot[i]) * a.kv.token_stride) * E;
    };
    auto load_keys = [&](TileT& x, const Rows<OCT>& r, int t) {
      int stop;
      const int base = tile_at(t, &stop);
      if constexpr (OCT) {
        const int kt = base + 8 * (c >> 2);
        bad |= uint32_t(r.page[0]) >= uint32_t(a.kv.pages) && kt < stop &&
               (min(kt + 7, stop - 1) >= sp.low || kt < a.sinks);
      } else {
#pragma unroll
        for (int b = 0; b < 2; ++b)
          bad |= uint32_t(r.page[b]) >= uint32_t(a.kv.pages) && seen(base + 8 * (c >> 2) + 4 * b + (c & 3), stop);
      }
      const int64_t k0 = row_at(r, 0);
#pragma unroll
      for (int b = 0; b < 2; ++b) x.load_k(b, kbase + (OCT ? k0 + (4 * b + (c & 3)) * step : b ? row_at(r, 1) : k0), g);
    };
    auto load_values = [&](TileT& x, const Rows<OCT>& r) {
      const int64_t v0 = row_at(r, OCT ? 1 : 2);
#pragma unroll
      for (int i = 0; i < 8; ++i) x.load_v(i, vbase + (OCT ? v0 + i * step : i ? row_at(r, OCT ? 1 : 2 + i) : v0), c);
    };
    auto load = [&](TileT& x, const Rows<OCT>& r, int t) {
      load_keys(x, r, t);
      load_values(x, r);
    };
    // `keys_done` and `values_done` run where the tile's keys and values are no
    // longer needed.
    auto compute = [&](TileT& x, int t, auto keys_done, auto values_done) {
      int stop;
      const int base = tile_at(t, &stop);
      if (base >= stop) {
        keys_done();
        values_done();
        return;
      }
      at_f32x4 s[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
      for (int j = 0; j < kSteps; ++j)
#pragma unroll
        for (int b = 0; b < 2; ++b) s[b] = T::mfma16(x.key(b, j), q[j], s[b]);
      keys_done();
      float p[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = s[i >> 2][i & 3] * cs;
      const bool whole = FEW ? base + 32 <= min(stop, pos_min + 1) &&
                                   (!a.window || base > pos_max - a.window || base + 32 <= a.sinks)
                             : base + 32 <= stop && (base >= sp.low || base + 32 <= a.sinks);
      if (!whole) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (!sees(base + 8 * g + i, stop)) p[i] = kNegInf;
          if (!seen(base + 8 * g + i, stop)) x.clear_v(i);      // 0 x Inf and 0 x NaN would reach the sum
        }
      }
      float mx = p[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) mx = fmaxf(mx, p[i]);
      mx = max_xor32(max_xor16(mx));
      if (__any(mx > m + (kGrowth + T::kRaise))) {
        const float mn = fmaxf(m, mx - T::kRaise), f = fmaxf(rebase(m, mn), odd ? kLeast : 0.0f);
#pragma unroll
        for (int j = 0; j < kBlocks; ++j) o[j] *= f;
        l *= f;
        m = mn;
      }
      const float mm = m == kNegInf ? 0.0f : m;
      at_u32x4 hi, lo;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        p[i] = exp2_fast(p[i] - mm);
        l += p[i];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        hi[i] = T::pack(p[2 * i], p[2 * i + 1]);
        lo[i] = T::pack(p[2 * i] - T::low(hi[i]), p[2 * i + 1] - T::high(hi[i]));
      }
#pragma unroll
      for (int r = 0; r < kRuns; ++r)
#pragma unroll
        for (int j = 0; j < kRun; j += 2) {
          at_u32x4 v0, v1;
          x.values(r, j, &v0, &v1);
          if (odd) {
            at_u32x4 see;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              see[i] = (sees(base + 8 * g + 2 * i, stop) ? T::kOne : 0) | (sees(base + 8 * g + 2 * i + 1, stop) ? T::kOne << 16 : 0);
            v0 = add_odd<T>(v0, see, &o[r * kRun + j]);
            v1 = add_odd<T>(v1, see, &o[r * kRun + j + 1]);
          }
          o[r * kRun + j] = T::mfma16(v0, hi, o[r * kRun + j]);
          o[r * kRun + j + 1] = T::mfma16(v1, hi, o[r * kRun + j + 1]);
          o[r * kRun + j] = T::mfma16(v0, lo, o[r * kRun + j]);
          o[r * kRun + j + 1] = T::mfma16(v1, lo, o[r * kRun + j + 1]);
        }
      values_done();
    };
    auto nothing = [] {};

    // Two tiles in registers: one is computed while the next one's loads (and
    // the table lookups of the one after it) are in flight.  A sum that is not
    // finite is taken again: Inf and NaN among the values then do not enter the
    // products (a weight's second part may be 0 or negative, and a row that does
    // not see the token has the weight 0: times Inf that is NaN), but are added to
    // the rows that see them.
    for (;;) {
#pragma unroll
      for (int j = 0; j < kBlocks; ++j) o[j] = (at_f32x4){0, 0, 0, 0};
      m = kNegInf;
      l = 0.0f;
      // No load depends on a condition inside the loop, and a tile's table
      // entries are read before the loads of the tile ahead of it: loads come
      // back in order, and waiting for either leaves the later ones in flight.
      if constexpr (TWO) {
        TileT x, y;
        Rows<OCT> r, n;
        auto at = [&](int t) { return min(t, t1 - 1); };
        find(r, t0);
        find(n, at(t0 + 1));
        load(x, r, t0);
        int t = t0;
        for (; t + 2 < t1; t += 2) {
          find(r, t + 2);
          load(y, n, t + 1);
          __builtin_amdgcn_sched_barrier(0);
          compute(x, t, nothing, nothing);
          __builtin_amdgcn_sched_barrier(0);
          find(n, at(t + 3));
          load(x, r, t + 2);
          __builtin_amdgcn_sched_barrier(0);
          compute(y, t + 1, nothing, nothing);
          __builtin_amdgcn_sched_barrier(0);
        }
        if (t + 1 < t1) {
          load(y, n, t + 1);
          compute(x, t, nothing, nothing);
          compute(y, t + 1, nothing, nothing);
        } else {
          compute(x, t, nothing, nothing);
        }
      } else {
        // one tile: its keys make way for the next one's after the scores, its
        // values after the sums
        TileT x;
        Rows<OCT> r;
        find(r, t0);
        load(x, r, t0);
        for (int t = t0; t + 1 < t1; ++t) {
          find(r, t + 1);
          __builtin_amdgcn_sched_barrier(0);
          compute(x, t, [&] { load_keys(x, r, t + 1); }, [&] { load_values(x, r); });
          __builtin_amdgcn_sched_barrier(0);
        }
        compute(x, t1 - 1, nothing, nothing);
      }
      if (odd) break;
#pragma unroll
      for (int j = 0; j < kBlocks; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) odd |= !(fabsf(o[j][i]) < -kNegInf);
      odd = __any(odd);
      if (!odd) break;
    }

    // merge the waves
    l = sum_xor32(sum_xor16(l));
    if (__any(bad)) l = __builtin_nanf("");
    if (c < rows) {
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          lds_o[wave][c][(b / kRun) * 128 + (4 * g + i) * kRun + b % kRun] = o[b][i];
      if (g == 0) {
        lds_m[wave][c] = m;
        lds_l[wave][c] = l;
      }
    }
    __syncthreads();
    const bool whole = t0 == 0 && t1 == sp.tiles;
    if (t0 == 0 && !whole && threadIdx.x == 0) {
      const int64_t last = unit_begin + sp.tiles - 1;      // the unit's last item is in workgroup ...
      work.cuts[wg] = {seq, unit, int32_t(((last + 1) * wgs - 1) / total - wg + 1), 0};
    }
    const Partial part = partial_at(work, D, wg, t0 == 0);
    for (int e = threadIdx.x; e < rows * (D / 4); e += 256) {
      const int r = e / (D / 4), d = 4 * (e - r * (D / 4));
      float M = kNegInf;
#pragma unroll
      for (int w = 0; w < 4; ++w) M = fmaxf(M, lds_m[w][r]);
      float L = 0.0f;
      at_f32x4 O = {0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float f = rebase_joined(lds_m[w][r], M);
        L += f * lds_l[w][r];
        O += *reinterpret_cast<const at_f32x4*>(&lds_o[w][r][d]) * f;
      }
      if (whole) {
        finish<T, D, E, FEW>(a, work, head, qs, sp, unit_row + r, d, M, L, O);
      } else {
        *reinterpret_cast<at_f32x4*>(part.o + r * D + d) = O;
        if (d == 0) {
          part.m[r] = M;
          part.l[r] = L;
        }
      }
    }
    __syncthreads();
  }
}

// Joins the partial results of units that were cut: o = sum o_i 2^(m_i - M),
// the same for l.  Grid (workgroups, row shares), each workgroup the unit that
// the one of its number has begun, if any, and one of its rows, so that the
// chains of dependent reads are short: its launch and their latency bound it.
// D / 4 threads hold a column quad each, the rest of the 256 share the parts.
// 2.8 us for 8 units of one sequence, 4 to 5 for a batch, 7 where a unit has up
// to 43 parts.
template <class T, int D, int E, bool FEW>
__global__ void __launch_bounds__(256) decode_join_kernel(AttnArgs a, Work work) {
  constexpr int kQuads = D / 4, kSplits = 256 / kQuads;
  __shared__ at_f32x4 lds_o[kSplits][kQuads];
  __shared__ float lds_m[kSplits], lds_l[kSplits];
  const Cut cut = work.cuts[blockIdx.x];
  if (cut.count <= 1) return;
  const Queries qs = queries_of<FEW>(work, cut.seq);
  const SeqSpan sp = seq_span(a, a.kv.lens[cut.seq], qs.count);
  const int blocks_per_head = (qs.count * a.group + kRows - 1) / kRows;
  const int head = cut.unit / blocks_per_head, unit_row = (cut.unit % blocks_per_head) * kRows;
  const int rows = min(qs.count * a.group - unit_row, kRows);
  const int quad = threadIdx.x % kQuads, split = threadIdx.x / kQuads;
  for (int r = blockIdx.y; r < rows; r += gridDim.y) {
    float M = kNegInf, L = 0.0f;
    at_f32x4 O = {0, 0, 0, 0};
#pragma unroll 4
    for (int i = split; i < cut.count; i += kSplits) {
      const Partial p = partial_at(work, D, blockIdx.x + i, i == 0);
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

// Workgroups of a full card.
int full_card(int D, int E, bool oct) { return 256 * wgs_per_cu(D, E, oct); }
constexpr int kMaxWgs = 256 * kMaxPerCu;

int64_t all_units(int64_t seqs, int q_heads, int heads) {
  return seqs * heads * ((q_heads / heads + kRows - 1) / kRows);
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

template <class T, int D, int E, bool OCT, bool FEW>
hipError_t launch_kernels(const AttnArgs& a, const Work& w, unsigned grid, hipStream_t stream) {
  decode_kernel<T, D, E, OCT, FEW><<<grid, 256, 0, stream>>>(a, w);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  decode_join_kernel<T, D, E, FEW><<<dim3(grid, unsigned(w.rows)), 256, 0, stream>>>(a, w);
  return hipGetLastError();
}

template <class T, int D, int E>
hipError_t launch(const AttnArgs& a, const int32_t* cu, int64_t tokens, void* workspace, hipStream_t stream) {
  const bool oct = a.kv.page.d % 8 == 0;
  const int wgs = full_card(D, E, oct);
  Work w = work_at(workspace, cu ? kRows : std::min(a.group, kRows), D, wgs);
  w.cu = cu;
  w.tokens = int(tokens);
  w.group = fast_div(uint32_t(a.group));
  // no more workgroups than tiles that the tables can hold
  const int64_t units = cu ? a.kv.heads * (tokens * a.group / kRows + a.kv.seqs) : all_units(a.kv.seqs, a.q_heads, a.kv.heads);
  const int64_t tiles = (int64_t(a.kv.max_pages) * a.kv.page.d + kTile - 1) / kTile + 2;
  const unsigned grid = unsigned(std::min<int64_t>(wgs, units * tiles));
  if (cu) return launch_kernels<T, D, E, true, true>(a, w, grid, stream);
  return oct ? launch_kernels<T, D, E, true, false>(a, w, grid, stream)
             : launch_kernels<T, D, E, false, false>(a, w, grid, stream);
}

template <class T, int E>
hipError_t launch_dim(const AttnArgs& a, const int32_t* cu, int64_t tokens, int D, void* workspace, hipStream_t stream) {
  if (D == 64) return launch<T, 64, E>(a, cu, tokens, workspace, stream);
  if (D == 128) return launch<T, 128, E>(a, cu, tokens, workspace, stream);
  return launch<T, 256, E>(a, cu, tokens, workspace, stream);
}

hipError_t launch_any(const AttnArgs& a, const int32_t* cu, int64_t tokens, int cache_dtype, int dtype, int D,
                      void* workspace, hipStream_t stream) {
  const bool e4m3 = cache_dtype == W4A4_E4M3;
  if (dtype == W4A4_BF16)
    return e4m3 ? launch_dim<Bf16, 1>(a, cu, tokens, D, workspace, stream)
                : launch_dim<Bf16, 2>(a, cu, tokens, D, workspace, stream);
  return e4m3 ? launch_dim<F16, 1>(a, cu, tokens, D, workspace, stream)
              : launch_dim<F16, 2>(a, cu, tokens, D, workspace, stream);
}

}  // namespace

size_t attn_decode_workspace(int q_heads, int heads, int head_dim) {
  return workspace_bytes(std::min(q_heads / heads, kRows), head_dim, kMaxWgs);
}

hipError_t launch_attn_decode(const AttnArgs& a, int cache_dtype, int dtype, int head_dim, void* workspace,
                              hipStream_t stream) {
  return launch_any(a, nullptr, a.kv.seqs, cache_dtype, dtype, head_dim, workspace, stream);
}

// Up to 16 rows of a kv head per sequence, on average: one unit, as in decoding.
// More rows would read the keys once per 16; the row tiles of attn_prefill read
// them once.  Here / there, 8 sequences of 8000 tokens, 8 kv heads of 4, D = 128:
// 2 tokens each, bf16 64.2 / 81.2 us, E4M3 43.6 / 65.3; 4 tokens (16 rows) 69.7 /
// 80.6 and 48.2 / 66.5.  With two blocks of 16 rows for 8 tokens it gained
// nothing over attn_prefill's 79.6 and 69.5.  The average hides one long chunk among
// sequences without new tokens, which either way serves alike where they are many:
// 256 tokens on 8000 beside 63 of 1000, bf16, 169 / 172 us (alone, as row tiles with
// the keys split, 74).
bool attn_few_serves(int64_t seqs, int64_t tokens, int group, int page_size) {
  return page_size % 8 == 0 && tokens * group <= seqs * kRows;
}

size_t attn_few_workspace(int head_dim) { return workspace_bytes(kRows, head_dim, kMaxWgs); }

hipError_t launch_attn_few(const AttnArgs& a, const int32_t* cu, int64_t tokens, int cache_dtype, int dtype,
                           int head_dim, void* workspace, hipStream_t stream) {
  return launch_any(a, cu, tokens, cache_dtype, dtype, head_dim, workspace, stream);
}

}  // namespace w4a4
