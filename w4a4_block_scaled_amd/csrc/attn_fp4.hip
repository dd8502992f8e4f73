// Attention of one new token per sequence, or a few, over a paged cache held in
// 4 bits (E2M1 codes with a scale byte for every 32 values).
//
// The work is cut as in attn_decode.hip.  A tile of 128 tokens is 4 waves x 32; the
// bytes are a quarter of 16 bits', so what would wait there for memory has to be
// cheap here:
//
// Scores S^T = K Q^T come from the scaled 16 x 16 x 128 MFMA, which takes the codes and
// the scale bytes as they are in the cache.  Its other operand has to be small too: a
// query's blocks of 32 are split into four parts in FP6 (E2M3), each with a scale of
// its own (attn_fp4.h).  (Products of 2 and 4 significant bits add up in fp32; measured
// against 64 bits 2^-23 of the sum of their sizes where a block's values are of one size,
// 2^-16 where they span 2^16.)  D = 64 fills the instruction's 128 products with two parts.
//
// O^T = V^T P^T as in attn_decode.hip: V's operand is 8 tokens of one d per lane, so the
// codes are widened to BF16 (one instruction per pair, which takes the scale) and pairs
// of tokens interleaved.  Weights and values are BF16 whatever the queries' type is,
// the weights in two parts (16 bits together): the widened values are exact, and of the
// range that the cache's scales have.
//
// Measured, D = 128, whole calls in a loop, and (in a trace, which is slower) kernel + join: 48
// sequences of 37 to 8191 tokens, 8 kv heads of 4, 216 MB 52 to 53 us (47.5 + 4.9; the kernel's
// loads without its arithmetic 43: values come 4 bytes per lane; the vector unit is busy
// 46%, the matrix cores 16% of the time); 3 of 90001 to 131071, 4 heads of 7, 180 MB 45 to 46 us
// (40.6 + 5.6; loads 36); 5 and 9 tokens on 30000 and 33333, 8 heads of 4, 69 MB 39 to 40 us (38.1
// + 5.3: the chain of scores, softmax and sums with two waves per SIMD).  A plain read takes
// 36, 30 and 12 us.  A second tile in registers does not pay where it fits either (4 tokens
// on 33000 25.5 us, 28.1 with it).
#include <algorithm>

#include "attn_fp4.h"
#include "attn_list.h"

namespace w4a4 {
namespace {

constexpr int kParts = 4;                                // of a query's block
constexpr uint32_t kPastRange = 253;     // scale bytes from here on: 4 * 2^126 is past BF16's range, 255 NaN

// Keys in the codes k with the scale byte ks, times part `PART`'s operand; its scale is
// byte BYTE of qs.
template <int BYTE>
__device__ __forceinline__ at_f32x4 mfma_scores(at_u32x4 k, uint32_t ks, at_u32x6 q, uint32_t qs, at_f32x4 c) {
  const at_i32x8 a = {int(k.x), int(k.y), int(k.z), int(k.w), 0, 0, 0, 0};
  const at_i32x8 b = {int(q[0]), int(q[1]), int(q[2]), int(q[3]), int(q[4]), int(q[5]), 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, 2, 0, int(ks), BYTE, int(qs));
}

// Raw keys and values of 32 tokens of one head in a wave's registers: of the keys a
// lane has one block of the tokens 8 (c / 4) + c % 4 and 4 more (D = 256: two blocks;
// D = 64: the upper quarters again those of the lower), of the values the bytes of
// kRun consecutive d's of the tokens 8 g .. 8 g + 7.
template <int D, bool OCT>
struct Fp4Tile {
  static constexpr int kSteps = D == 256 ? 2 : 1;              // of 128 d's
  static constexpr int kRun = D >= 128 ? 8 : 4;
  static constexpr int kRuns = D / 16 / kRun;
  at_u32x4 k[2][kSteps];
  uint32_t ks[2][kSteps];
  uint32_t v[8][kRuns];
  uint32_t vs[kRuns][OCT ? 2 : 8];      // scale bytes of 4 tokens each, or of one
};

// Byte i of the 4 in x where a scale is wanted: bits 23 .. 30 are looked at alone.
__device__ __forceinline__ float scale_of(uint32_t x, int i) {
  return __builtin_bit_cast(float, i == 0 ? x << 23 : i == 1 ? x << 15 : i == 2 ? x << 7 : x >> 1);
}

template <int B>
__device__ __forceinline__ uint32_t widen(uint32_t u, float s) { return fp4_pair<Bf16, B>(u, s); }
__device__ __forceinline__ uint32_t widen_byte(uint32_t u, float s, int b) {
  return b == 0 ? widen<0>(u, s) : b == 1 ? widen<1>(u, s) : b == 2 ? widen<2>(u, s) : widen<3>(u, s);
}

constexpr int kAheadOct = 16, kAheadAny = 2;             // tiles that one load of the table serves
// Workgroups that share a CU: as many as the registers leave without spilling (but for three
// blocks at D = 128, where 10 go to scratch; these have not been timed with one workgroup).
// Microseconds with 4 / 3 / 2 / 1: D = 64 (32 sequences of 100 to 6000 tokens) 37.7 / 40.5 /
// 53.0 / 83.4; D = 128, the ragged batch 62.5 (spills) / 52.3 / 56.0 / 75.3, pages of 11
// 152 / 70 (spills) / 39.2 / 54.4, 2 tokens of each of 8 sequences on 8000 37.6 / 25.5 / 23.5
// / 23.6; D = 256 (32 sequences of 100 to 6000) - / 55.5 (spills) / 40.8 / 40.2, 64 of 128 to 1025
// 16.8 / 18.9 with two and one (the LDS has room for two).
constexpr int wgs_per_cu(int D, bool oct, bool few, int nb) {
  if (D == 256 || nb > 1 || !oct) return 2;
  return D == 64 ? 4 : few ? 2 : 3;
}
constexpr int kMaxPerCu = 4;

// NB: a unit's blocks of 16 rows.  OCT: the page size is a multiple of 8, so 8 tokens
// from a multiple of 8 lie on one page.  FEW: the sequences have any number of queries.
// whole_units: a workgroup has the unit of its number, and nothing is left to join.
template <class T, int D, bool OCT, bool FEW, int NB>
__global__ void __launch_bounds__(256, wgs_per_cu(D, OCT, FEW, NB)) fp4_kernel(AttnArgs a, Work work, bool whole_units) {
  typedef Fp4Tile<D, OCT> TileT;
  constexpr int kSteps = TileT::kSteps, kRun = TileT::kRun, kRuns = TileT::kRuns;
  constexpr int kUnit = kRows * NB, kBlocks = D / 16, kRow = D / 2;
  constexpr int kOps = D == 64 ? 2 : kParts * kSteps;          // score MFMAs per block of rows and 16 tokens
  // the query operands: in registers, or where they are too many in LDS
  constexpr bool kLdsQ = NB > 1 || kOps > 4;
  constexpr int kQ = kLdsQ ? NB * kOps : 1;
  __shared__ at_u32x4 lds_q4[kQ][64];
  __shared__ at_u32x2 lds_q2[kQ][64];
  __shared__ uint32_t lds_qs[kLdsQ ? NB * kSteps : 1][64];
  __shared__ float lds_o[4][kRows][D + 4];
  __shared__ float lds_m[4][kRows], lds_l[4][kRows];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, c = lane & 15;
  const int64_t wg = blockIdx.x;
  const bool whole = !FEW && whole_units;
  if (!whole && threadIdx.x == 0) work.cuts[wg].count = 0;
  Piece pc;
  if (whole) {
    const int units = a.kv.heads * ((a.group + kUnit - 1) / kUnit), s = int(wg) / units;
    const int64_t tiles = seq_span(a, a.kv.lens[s], 1).tiles, first = (int(wg) - s * units) * tiles;
    pc = {first, first + tiles, units * tiles, units, 0, s, 0, 0};
  } else if (!find_piece<FEW>(a, work, kUnit, lane, &pc)) {
    return;
  }
  int64_t item = pc.item, seq_begin = pc.seq_begin;
  int seq = pc.seq;
  const uint32_t page_stride = uint32_t(a.kv.page_stride);       // less than 2^31 (a launch's condition)
  const int page_size = int(a.kv.page.d);

  while (item < pc.end && seq < a.kv.seqs) {
    const Queries qs = queries_of<FEW>(work, seq);
    const SeqSpan sp = seq_span(a, !whole && seq < 64 ? __builtin_amdgcn_readlane(pc.len0, seq) : a.kv.lens[seq], qs.count);
    const int blocks_per_head = (qs.count * a.group + kUnit - 1) / kUnit;
    const int units = a.kv.heads * blocks_per_head;
    const int64_t in_seq = item - seq_begin;
    const int places = sp.tiles + pc.extra;
    if (in_seq >= int64_t(places) * units) {
      seq_begin += int64_t(places) * units;
      ++seq;
      continue;
    }
    const int unit = int(in_seq / places);
    const int64_t unit_begin = seq_begin + int64_t(unit) * places + pc.extra;    // of its tiles
    const int t0 = int(max(item - unit_begin, int64_t(0)));
    const int t1 = int(min(int64_t(sp.tiles), pc.end - unit_begin));
    item = unit_begin + t1;
    if (t1 <= t0) continue;

    const int head = unit / blocks_per_head;
    const int unit_row = (unit % blocks_per_head) * kUnit;
    const int rows = min(qs.count * a.group - unit_row, kUnit);
    const int past = sp.len - qs.count;
    // positions of the unit's first and last row
    const int pos_min = past + (FEW ? work.group.div(unit_row) : 0);
    const int pos_max = past + (FEW ? work.group.div(unit_row + rows - 1) : 0);
    const float cs = a.scale_log2;
    const int32_t* table = a.kv.tables + seq * a.kv.table_stride;

    // what a lane reads lies at these, plus its tokens' places in their pages
    const uint8_t* const kcode = static_cast<const uint8_t*>(a.kv.k) + head * a.kv.head_stride +
                                 (OCT ? (c & 3) * kRow : 0) + 16 * (D == 64 ? g & 1 : g);
    const uint8_t* const kscale = static_cast<const uint8_t*>(a.kv.k) + a.kv.scale_at + head * a.kv.scale_head +
                                  (OCT ? c & 3 : 0) + (D == 64 ? g & 1 : g) * page_size;
    const uint8_t* const vcode = static_cast<const uint8_t*>(a.kv.v) + head * a.kv.head_stride + c * (kRun / 2);
    const uint8_t* const vscale = static_cast<const uint8_t*>(a.kv.v) + a.kv.scale_at + head * a.kv.scale_head +
                                  (D == 64 ? c >> 3 : c >> 2) * page_size;

    at_f32x4 o[NB][kBlocks];
    float m[NB], l[NB];
    bool bad = sp.over;
#pragma unroll
    for (int n = 0; n < NB; ++n) {
#pragma unroll
      for (int j = 0; j < kBlocks; ++j) o[n][j] = (at_f32x4){0, 0, 0, 0};
      m[n] = kNegInf;
      l[n] = 0.0f;
    }

    // first token of this wave's part of tile t, and the end of its range
    auto tile_at = [&](int t, int* stop) {
      const bool sink = t < sp.sink_tiles;
      *stop = sink ? sp.sink_end : sp.len;
      return (sink ? t * kTile : sp.start + (t - sp.sink_tiles) * kTile) + wave * 32;
    };
    // whether any row of the sequence sees token t, and whether a row at position p does
    auto seen = [&](int t, int stop) { return t < stop && (t >= sp.low || t < a.sinks); };
    auto sees = [&](int t, int stop, int p) {
      if (!FEW) return seen(t, stop);
      return t < stop && t <= p && (!a.window || t > p - a.window || t < a.sinks);
    };
    // Lane l looks up the page of 8 tokens (OCT: number l % 4 of tile t + l / 4), or of one
    // (l % 32 of tile t + l / 32).  Tokens past the end of the range take the place of its
    // last one; an entry outside the cache is read as page 0, and spoils the result if a
    // query sees a token there (the keys' entries are the values').
    constexpr int kAhead = OCT ? kAheadOct : kAheadAny;
    int look_page = 0, look_slot = 0;
    auto look = [&](int t) {
      int stop;
      const int tl = min(t + (OCT ? lane >> 2 : lane >> 5), t1 - 1);
      const int tk = tile_at(tl, &stop) + (OCT ? 8 * (lane & 3) : lane & 31);
      const int u = max(min(tk, OCT ? (stop - 1) & ~7 : stop - 1), 0), j = a.kv.page.div(u);
      look_slot = u - j * page_size;
      const int p = table[j];
      const bool good = uint32_t(p) < uint32_t(a.kv.pages);
      look_page = good ? p : 0;
      bad |= !good && tk < stop && (min(tk + (OCT ? 7 : 0), stop - 1) >= sp.low || tk < a.sinks);
    };
    struct Place {
      int page, slot;
    };
    auto place = [&](int from) -> Place {
      return {__builtin_amdgcn_ds_bpermute(from << 2, look_page), __builtin_amdgcn_ds_bpermute(from << 2, look_slot)};
    };
    auto code_at = [&](const uint8_t* base, const Place& p) {
      return base + uint64_t(uint32_t(p.page)) * page_stride + uint32_t(p.slot) * uint32_t(kRow);
    };
    auto scale_at = [&](const uint8_t* base, const Place& p) {
      return base + uint64_t(uint32_t(p.page)) * page_stride + uint32_t(p.slot);
    };
    auto load_keys = [&](TileT& x, int n) {
      Place p[2];
      if constexpr (OCT) p[0] = p[1] = place(4 * n + (c >> 2));
      else p[0] = place(32 * n + 8 * (c >> 2) + (c & 3)), p[1] = place(32 * n + 8 * (c >> 2) + 4 + (c & 3));
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const uint8_t* row = code_at(kcode, p[b]) + (OCT ? 4 * b * kRow : 0);
        const uint8_t* scale = scale_at(kscale, p[b]) + (OCT ? 4 * b : 0);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          x.k[b][i] = *reinterpret_cast<const at_u32x4*>(row + 64 * i);
          x.ks[b][i] = scale[4 * i * page_size];
        }
      }
    };
    auto load_values = [&](TileT& x, int n) {
      Place p = place(OCT ? 4 * n + g : 32 * n + 8 * g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (!OCT && i) p = place(32 * n + 8 * g + i);
        const uint8_t* row = code_at(vcode, p) + (OCT ? i * kRow : 0);
#pragma unroll
        for (int r = 0; r < kRuns; ++r) {
          if constexpr (D == 64) x.v[i][r] = *reinterpret_cast<const uint16_t*>(row);
          else x.v[i][r] = *reinterpret_cast<const uint32_t*>(row + 64 * r);
        }
        const uint8_t* scale = scale_at(vscale, p);
#pragma unroll
        for (int r = 0; r < kRuns; ++r) {
          if constexpr (!OCT) {
            x.vs[r][i] = scale[4 * r * page_size];
          } else if (i == 0) {
            const at_u32x2 z = *reinterpret_cast<const at_u32x2*>(scale + 4 * r * page_size);
            x.vs[r][0] = z.x;
            x.vs[r][1] = z.y;
          }
        }
      }
    };

    // this lane's rows, one of each block: positions and query operands (a row past the
    // unit's last one is that one again, and is not written)
    int pos[NB];
    at_u32x6 q[kLdsQ ? 1 : kOps];
    uint32_t qscale[kLdsQ ? 1 : kSteps];
    auto split_queries = [&] {
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        const int row = unit_row + min(kRows * n + c, rows - 1);
        const int tok = FEW ? work.group.div(row) : 0;
        pos[n] = past + tok;
        const int at = FEW ? min(max(qs.first + tok, 0), work.tokens - 1) : seq;
        const uint16_t* qp = static_cast<const uint16_t*>(a.q) + at * a.q_row +
                             (int64_t(head) * a.group + row - tok * a.group) * a.q_head;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          if (kLdsQ && (n * kSteps + i) % 4 != wave) continue;       // the waves share them
          at_u32x6 part[kParts];
          uint32_t bytes = split_query<T, kParts>(qp + (D == 64 ? 32 * (g & 1) : 128 * i + 32 * g), part);
          if constexpr (D == 64) {        // quarters 0, 1: parts 0 and 2; quarters 2, 3: parts 1 and 3
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int w = 0; w < 6; ++w) part[k][w] = g < 2 ? part[2 * k][w] : part[2 * k + 1][w];
            bytes = g < 2 ? bytes : bytes >> 8;       // bytes 0 and 2
          }
          constexpr int kOf = kOps / kSteps;
#pragma unroll
          for (int p = 0; p < kOf; ++p) {
            if constexpr (kLdsQ) {
              const int k = n * kOps + i * kOf + p;
              lds_q4[k][lane] = (at_u32x4){part[p][0], part[p][1], part[p][2], part[p][3]};
              lds_q2[k][lane] = (at_u32x2){part[p][4], part[p][5]};
            } else {
              q[i * kOf + p] = part[p];
            }
          }
          if constexpr (kLdsQ) lds_qs[n * kSteps + i][lane] = bytes;
          else qscale[i] = bytes;
        }
      }
      if constexpr (kLdsQ) __syncthreads();
    };
    auto operand = [&](int n, int k) {
      if constexpr (!kLdsQ) return q[k];
      const at_u32x4 u = lds_q4[n * kOps + k][lane];
      const at_u32x2 v = lds_q2[n * kOps + k][lane];
      return (at_u32x6){u.x, u.y, u.z, u.w, v.x, v.y};
    };
    auto operand_scale = [&](int n, int i) { return kLdsQ ? lds_qs[n * kSteps + i][lane] : qscale[kLdsQ ? 0 : i]; };

    // One tile in registers: its keys make way for the next one's after the scores, its
    // values after the sums.  D = 256, where registers are short: the queries are split behind
    // the first loads, so that what that needs is not held beside the places (microseconds
    // before / behind, 32 sequences of 100 to 6000 tokens 45.4 / 40.9; D = 128, the ragged batch
    // 52.0 / 52.8, 4 tokens on 33000 25.6 / 26.6).
    constexpr bool kLoadsFirst = D == 256;
    if constexpr (!kLoadsFirst) split_queries();
    TileT x;
    look(t0);
    load_keys(x, 0);
    load_values(x, 0);
    if constexpr (kLoadsFirst) split_queries();

    // `keys_done` and `values_done` run where the tile's keys and values are no longer needed.
    auto compute = [&](TileT& x, int t, auto keys_done, auto values_done) {
      int stop;
      const int base = tile_at(t, &stop);
      if (base >= stop) {
        keys_done();
        values_done();
        return;
      }
      at_f32x4 s[NB][2];
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int b = 0; b < 2; ++b) s[n][b] = (at_f32x4){0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          // the smallest parts first; the two blocks of tokens in turn
          const uint32_t qsc = operand_scale(n, i);
          auto part = [&](auto which) {
            constexpr int P = decltype(which)::value;
            const at_u32x6 z = operand(n, D == 64 ? P / 2 : kParts * i + P);
#pragma unroll
            for (int b = 0; b < 2; ++b) s[n][b] = mfma_scores<P>(x.k[b][i], x.ks[b][i], z, qsc, s[n][b]);
          };
          if constexpr (D != 64) part(std::integral_constant<int, 3>());
          part(std::integral_constant<int, 2>());
          if constexpr (D != 64) part(std::integral_constant<int, 1>());
          part(std::integral_constant<int, 0>());
        }
      keys_done();
      const bool whole = FEW ? base + 32 <= min(stop, pos_min + 1) &&
                                   (!a.window || base > pos_max - a.window || base + 32 <= a.sinks)
                             : base + 32 <= stop && (base >= sp.low || base + 32 <= a.sinks);
      if (!whole) {
        bool odd = false;
        auto past_range = [&](uint32_t y, int i) { return (OCT ? y >> (8 * (i & 3)) & 0xffu : y) >= kPastRange; };
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const bool any = seen(base + 8 * g + i, stop);
#pragma unroll
          for (int n = 0; n < NB; ++n)
            if (!sees(base + 8 * g + i, stop, pos[n])) s[n][i >> 2][i & 3] = kNegInf;
#pragma unroll
          for (int r = 0; r < kRuns; ++r) {      // 0 x NaN and 0 x Inf would reach the sum
            uint32_t& y = x.vs[r][OCT ? i >> 2 : i];
            if (!any) y &= ~(0xffu << (OCT ? 8 * (i & 3) : 0));
            odd |= past_range(y, i);
          }
        }
        if constexpr (FEW) {
          // Blocks of NaN, or with scales that may make Inf, that some row sees and another one may
          // not: the sums of the rows that see them become NaN, then the blocks are cleared.
          if (__any(odd)) {
#pragma unroll
            for (int r = 0; r < kRuns; ++r) {
              at_u32x4 is;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                uint32_t two = 0;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const int i = 2 * k + h;
                  uint32_t& y = x.vs[r][OCT ? i >> 2 : i];
                  if (past_range(y, i)) {
                    two |= Bf16::kOne << (16 * h);
                    y &= ~(0xffu << (OCT ? 8 * (i & 3) : 0));
                  }
                }
                is[k] = two;
              }
#pragma unroll
              for (int n = 0; n < NB; ++n) {
                at_u32x4 see;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  see[k] = (sees(base + 8 * g + 2 * k, stop, pos[n]) ? Bf16::kOne : 0) |
                           (sees(base + 8 * g + 2 * k + 1, stop, pos[n]) ? Bf16::kOne << 16 : 0);
                const at_f32x4 hit = Bf16::mfma16(is, see, (at_f32x4){0, 0, 0, 0});
#pragma unroll
                for (int j = 0; j < kRun; ++j)
#pragma unroll
                  for (int i = 0; i < 4; ++i)
                    if (hit[i] > 0.0f) o[n][r * kRun + j][i] = __builtin_nanf("");
              }
            }
          }
        }
      }
      at_u32x4 hi[NB], lo[NB];
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        float mx = s[n][0][0];
#pragma unroll
        for (int i = 1; i < 8; ++i) mx = fmaxf(mx, s[n][i >> 2][i & 3]);
        mx = max_xor32(max_xor16(mx)) * cs;
        if (__any(mx > m[n] + kGrowth)) {
          const float mn = fmaxf(m[n], mx), f = rebase(m[n], mn);
#pragma unroll
          for (int j = 0; j < kBlocks; ++j) o[n][j] *= f;
          l[n] *= f;
          m[n] = mn;
        }
        const float mm = m[n] == kNegInf ? 0.0f : m[n];
        float p[8], rest[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          p[i] = exp2_fast(__builtin_fmaf(s[n][i >> 2][i & 3], cs, -mm));
          l[n] += p[i];
          // the first part is the upper half of the bits, the second one the rest, rounded
          rest[i] = p[i] - __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, p[i]) & 0xffff0000u);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          hi[n][i] = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, p[2 * i + 1]), __builtin_bit_cast(uint32_t, p[2 * i]),
                                           0x07060302);
          lo[n][i] = Bf16::pack(rest[2 * i], rest[2 * i + 1]);
        }
      }
#pragma unroll
      for (int r = 0; r < kRuns; ++r) {
        float vs[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) vs[i] = OCT ? scale_of(x.vs[r][i >> 2], i & 3) : scale_of(x.vs[r][i], 0);
#pragma unroll
        for (int j = 0; j < kRun; j += 2) {
          at_u32x4 v0, v1;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t y = widen_byte(x.v[2 * k][r], vs[2 * k], j / 2), z = widen_byte(x.v[2 * k + 1][r], vs[2 * k + 1], j / 2);
            v0[k] = __builtin_amdgcn_perm(z, y, 0x05040100);
            v1[k] = __builtin_amdgcn_perm(z, y, 0x07060302);
          }
#pragma unroll
          for (int n = 0; n < NB; ++n) {
            at_f32x4 &o0 = o[n][r * kRun + j], &o1 = o[n][r * kRun + j + 1];
            o0 = Bf16::mfma16(v0, hi[n], o0);
            o1 = Bf16::mfma16(v1, hi[n], o1);
            o0 = Bf16::mfma16(v0, lo[n], o0);
            o1 = Bf16::mfma16(v1, lo[n], o1);
          }
        }
      }
      values_done();
    };
    auto nothing = [] {};

    for (int t = t0; t + 1 < t1; ++t) {
      const int n = (t + 1 - t0) % kAhead;
      if (n == 0) look(t + 1);
      compute(x, t, [&] { load_keys(x, n); }, [&] { load_values(x, n); });
    }
    compute(x, t1 - 1, nothing, nothing);

    // merge the waves, a block of rows at a time
    const bool unit_whole = t0 == 0 && t1 == sp.tiles;
    if (t0 == 0 && !unit_whole && threadIdx.x == 0) {
      const int64_t last = unit_begin + sp.tiles - 1;      // the unit's last item is in workgroup ...
      work.cuts[wg] = {seq, unit, int32_t(((last + 1) * pc.wgs - 1) / pc.total - wg + 1), 0};
    }
    const Partial part = partial_at(work, D, wg, t0 == 0);
    bad = __any(bad);
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      const int here = min(rows - kRows * n, kRows);
      if (here <= 0) break;
      const float sum = bad ? __builtin_nanf("") : sum_xor32(sum_xor16(l[n]));
      if (c < here) {
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            lds_o[wave][c][(b / kRun) * 128 + (4 * g + i) * kRun + b % kRun] = o[n][b][i];
        if (g == 0) {
          lds_m[wave][c] = m[n];
          lds_l[wave][c] = sum;
        }
      }
      __syncthreads();
      for (int e = threadIdx.x; e < here * (D / 4); e += 256) {
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
        if (unit_whole) {
          finish<T, D, 0, FEW>(a, work, head, qs, sp, unit_row + kRows * n + r, d, M, L, O);
        } else {
          *reinterpret_cast<at_f32x4*>(part.o + (kRows * n + r) * D + d) = O;
          if (d == 0) {
            part.m[kRows * n + r] = M;
            part.l[kRows * n + r] = L;
          }
        }
      }
      __syncthreads();
    }
  }
}

// Units are not cut where the tables hold this many tokens at most, since the search in the
// list, the second launch and the partial results cost what some tiles do.  Microseconds per
// call, cut / not cut, D = 128 with 8 kv heads: one sequence of 513 tokens 13.0 / 10.1, of
// 1025 13.0 / 11.1, of 1537 13.0 / 13.9; 64 of 64 to 513 19.8 / 10.7, of 256 to 2049
// 29.7 / 22.9; 128 of 512 to 4097 77.7 / 80.1.  D = 256 with 4 heads: one of 1025
// 13.6 / 16.0, 64 of 128 to 1025 23.8 / 16.8.
int64_t whole_tokens(int D, int64_t units) {
  if (units >= 1 << 24) return 0;                        // more workgroups than a launch takes
  return units >= 256 ? 2048 : D == 256 ? 640 : 1024;
}

constexpr int kMaxWgs = 256 * kMaxPerCu;

template <class T, int D, bool OCT, bool FEW, int NB>
hipError_t launch_kernels(const AttnArgs& a, const int32_t* cu, int64_t tokens, void* workspace, hipStream_t stream) {
  const int wgs = 256 * wgs_per_cu(D, OCT, FEW, NB);
  Work w = work_at(workspace, FEW ? kRows * NB : std::min(a.group, kRows), D, wgs);
  w.cu = cu;
  w.tokens = int(tokens);
  w.group = fast_div(uint32_t(a.group));
  // no more workgroups than tiles that the tables can hold
  const int64_t units = FEW ? a.kv.heads * (tokens * a.group / (kRows * NB) + a.kv.seqs)
                            : a.kv.seqs * a.kv.heads * ((a.group + kRows - 1) / kRows);
  const int64_t tiles = (int64_t(a.kv.max_pages) * a.kv.page.d + kTile - 1) / kTile + 2;
  const unsigned grid = unsigned(std::min<int64_t>(wgs, units * tiles));
  if (!FEW && int64_t(a.kv.max_pages) * a.kv.page.d <= whole_tokens(D, units)) {
    fp4_kernel<T, D, OCT, FEW, NB><<<unsigned(units), 256, 0, stream>>>(a, w, true);
    return hipGetLastError();
  }
  fp4_kernel<T, D, OCT, FEW, NB><<<grid, 256, 0, stream>>>(a, w, false);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return launch_join<T, D, 0, FEW, kRows * NB>(a, w, grid, units, stream);
}

template <class T, int D>
hipError_t launch_dim(const AttnArgs& a, const int32_t* cu, int64_t tokens, void* workspace, hipStream_t stream) {
  if (!cu)
    return a.kv.page.d % 8 == 0 ? launch_kernels<T, D, true, false, 1>(a, cu, tokens, workspace, stream)
                                : launch_kernels<T, D, false, false, 1>(a, cu, tokens, workspace, stream);
  const int blocks = attn_fp4_blocks(a.kv.seqs, tokens, a.group, D);
  if constexpr (D < 256) {
    if (blocks == 3) return launch_kernels<T, D, true, true, 3>(a, cu, tokens, workspace, stream);
    if (blocks == 2) return launch_kernels<T, D, true, true, 2>(a, cu, tokens, workspace, stream);
  }
  return launch_kernels<T, D, true, true, 1>(a, cu, tokens, workspace, stream);
}

template <class T>
hipError_t launch(const AttnArgs& a, const int32_t* cu, int64_t tokens, int D, void* workspace, hipStream_t stream) {
  if (D == 64) return launch_dim<T, 64>(a, cu, tokens, workspace, stream);
  if (D == 128) return launch_dim<T, 128>(a, cu, tokens, workspace, stream);
  return launch_dim<T, 256>(a, cu, tokens, workspace, stream);
}

}  // namespace

int attn_fp4_blocks(int64_t seqs, int64_t tokens, int group, int head_dim) {
  const int64_t blocks = std::max<int64_t>((tokens * group + seqs * kRows - 1) / (seqs * kRows), 1);
  return blocks <= (head_dim == 256 ? 1 : 3) ? int(blocks) : 0;
}

size_t attn_fp4_workspace(int rows, int head_dim) { return workspace_bytes(rows, head_dim, kMaxWgs); }

hipError_t launch_attn_fp4(const AttnArgs& a, const int32_t* cu, int64_t tokens, int dtype, int head_dim,
                           void* workspace, hipStream_t stream) {
  return dtype == W4A4_BF16 ? launch<Bf16>(a, cu, tokens, head_dim, workspace, stream)
                            : launch<F16>(a, cu, tokens, head_dim, workspace, stream);
}

}  // namespace w4a4
