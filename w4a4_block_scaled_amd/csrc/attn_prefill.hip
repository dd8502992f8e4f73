// Attention of chunks of new tokens over the paged cache, causal, with an
// optional window and sinks.
//
// The rows of a kv head are its (token, head of the group) pairs, token by
// token, in tiles of 128: the heads of a group share every key and value that
// a workgroup stages, and a tile spans few positions, so few of its products
// fall on masked pairs.  Per workgroup 4 waves of 32 rows; keys and values in
// tiles of 64 tokens, double buffered in LDS.
//
// S^T = K Q^T with 32 x 32 x 16 MFMAs (keys from LDS as the first operand, the
// queries stay in registers), so that a lane holds 32 scores of one row: the
// row's maximum and sum need one exchange with the lane 32 further.  The same
// registers, rounded to 16 bits, are the second operand of O^T = V^T P^T; V's
// operand comes from the row-major tile by transposing LDS reads, in the token
// order that the scores' registers have.
//
// The matrix cores bound it: 4 D operations per visible pair.  Beside them the
// vector unit has some 5 instructions per 32 x 32 x 16 product to place: a step
// computes the scores of the next tile and the weighted sum of this one, and
// between any two MFMAs stands a slice of the softmax, of the masks or of the
// next copies, held there by scheduling barriers (the two in turn, as written
// without them: 577 us on the ragged chunks; interleaved 507).  Sums are
// rebased only where a maximum has grown by more than 2^8, so they are rarely touched.
// Copies go straight to LDS: by buffer loads, which LDS reads do not wait for.
//
// The weights are rounded to 16 bits (bf16: the relative error is 1.9e-3 against
// 64 bits, of which the output's own rounding is 1.6e-3; fp16: 2.7e-4, of which
// 2.0e-4; a second part would double the second product).  Where the keys are split
// the matrix cores are idle, and two parts are taken, as in decoding.
//
// FP4 (4-bit caches): keys lie in LDS as the cache has them, codes and scale bytes, and the
// scores come from the scaled 32 x 32 x 64 MFMA, the queries in four FP6 parts (attn_fp4.h);
// values are widened on their way to LDS, as from E4M3, to the queries' type: to BF16 exactly, to
// FP16 below 2^-13 in its steps of 2^-24 (half of one is what the output's own rounding is off by
// there) and past its range to Inf, for products at the 16-bit rate without a second type.
// (Ragged chunks over 28 / 4 heads 506 us, 560 with the keys widened to 16 bits too; three
// parts of the queries, right to 2^-14 of a block's largest value, miss the bound on lse.)
// The parts do not all fit: at D = 128 19 registers go to scratch (where rows are looked up one
// by one 29 with BF16 queries, 35 with FP16), at D = 256 4 and 13, with the keys split 73 and 75.
//
// Measured, 32 / 8 heads, D = 128, causal 8192 bf16: 512 to 528 us, 1.05 PFLOP/s (a
// library product of 8192^3 reaches 1.44 here; the MFMAs are busy 55% of the
// time on the ragged chunks, at 1.65 GHz), E4M3 537 to 557 us, D = 64 320 to 337;
// 4096 at D = 256 332 to 346 us.  Ragged chunks over 28 / 4 heads, 526 GFLOP:
// 491 to 514 us.  82 tokens: 10.5 us, 8.7 of them the kernel's.  FP4: causal 8192 514 us, D = 64
// 320, 4096 at D = 256 176 over 16 / 4 heads; ragged chunks 506 to 528; keys split, 100 and 60
// tokens on 30000 and 20000, 32 / 8 heads 174 us (bf16 163), 16 / 4 of D = 256 385 (bf16 667).
#include <algorithm>
#include <type_traits>
#include <utility>

#include "attn_fp4.h"

namespace w4a4 {
namespace {

#define LDS_AS __attribute__((address_space(3)))

constexpr int kBM = 128;      // rows per workgroup
constexpr int kBN = 64;       // tokens per step
constexpr int kMaxSplits = 64;  // of the keys of a row tile: two per lane of the join

struct PrefillWork {
  const int32_t* cu;
  float* parts;               // [row tiles x heads x splits] of kBM x (D + 2), or unused
  int32_t* used;              // [row tiles x heads]: splits that hold results
  int32_t tokens, row_tiles, splits;
  FastDiv group;
};

// The sequence and tile of the sequence that row tile `ti` is; false past the end.
// Tiles of a sequence are handed out from its end, where rows see most keys, and
// up to 64 sequences by length, the longest first: the last workgroups to start
// are short ones.
struct RowTile {
  int seq, tile, first_token, count, len;
  bool over;
};
__device__ __forceinline__ bool find_tile(const AttnArgs& a, const PrefillWork& w, int ti, RowTile* out) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int base = 0; base < a.kv.seqs; base += 64) {
    int s = base + lane, n = 0;
    if (s < a.kv.seqs) n = min(max(w.cu[s + 1] - w.cu[s], 0), w.tokens);
    if (a.kv.seqs <= 64 && a.kv.seqs > 1) {
      const int len = s < a.kv.seqs ? a.kv.lens[s] : INT32_MIN;
      int rank = 0;
      for (int i = 0; i < a.kv.seqs; ++i) {
        const int other = __builtin_amdgcn_readlane(len, i);
        rank += other > len || (other == len && i < lane);
      }
      if (s >= a.kv.seqs) rank = lane;               // behind all sequences, each at its own place
      s = __builtin_amdgcn_ds_permute(rank << 2, s);
      n = __builtin_amdgcn_ds_permute(rank << 2, n);
    }
    const int t = int((int64_t(n) * a.group + kBM - 1) / kBM);
    int in = t;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int y = __shfl_up(in, d);
      if (lane >= d) in += y;
    }
    const uint64_t past = __ballot(before + in > ti);
    if (past) {
      const int l = __ffsll((unsigned long long)past) - 1;
      out->seq = __builtin_amdgcn_readlane(s, l);
      out->count = __builtin_amdgcn_readlane(n, l);
      out->tile = before + __builtin_amdgcn_readlane(in, l) - 1 - ti;
      out->first_token = w.cu[out->seq];
      const int cap = int(min(int64_t(a.kv.max_pages) * a.kv.page.d, int64_t(1) << 30));
      const int len = a.kv.lens[out->seq];
      out->over = len > cap;
      out->len = max(min(len, cap), 0);      // so that len - count does not wrap
      return true;
    }
    before += __builtin_amdgcn_readlane(in, 63);
  }
  return false;
}

// 16-byte chunk swizzles of the LDS tiles (row r, chunk c at slot c ^ swz(r)).
// Keys: 16 consecutive rows of one chunk fall on 16 different 16-byte bank
// groups; values: so do 4 consecutive rows of four chunks (32 lanes' pieces).
template <int D>
__device__ __forceinline__ int key_swz(int r) { return D == 64 ? (r >> 1) & 7 : r & 15; }
template <int D>
__device__ __forceinline__ int value_swz(int r) { return D == 64 ? (r & 2) << 1 : (r & 3) << 2; }

typedef LDS_AS uint16_t Lds16;

// s_waitcnt vmcnt(n) alone: vmcnt in bits 3:0 and 15:14, expcnt 6:4 and lgkmcnt
// 11:8 at their maxima.
constexpr int wait_vmcnt(int n) { return (n & 15) | (n >> 4) << 14 | 0x0f70; }

// 16 bytes per lane from `src` to LDS, lane l writing `dst` + 16 l (dst is
// wave-uniform).
__device__ __forceinline__ void copy_to_lds(const uint8_t* src, Lds16* dst) {
  __builtin_amdgcn_global_load_lds(src, (LDS_AS void*)dst, 16, 0, 0);
}
// The same from `base` (uniform) + `off`.  A buffer load: the compiler counts a
// global load to LDS as an access of both kinds that may come back in any order,
// and then waits for every LDS read before the first one's use.
__device__ __forceinline__ void copy_to_lds(const uint8_t* base, uint32_t off, Lds16* dst) {
  const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, -1, 0x00020000);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (LDS_AS void*)dst, 16, int(off), 0, 0, 0);
}
__device__ __forceinline__ at_u32x4 read16(const Lds16* p) { return *reinterpret_cast<const LDS_AS at_u32x4*>(p); }
// Two dwords (4 elements) of column l % 16 of 4 rows x 16 columns, from the
// 8 bytes that each of 16 lanes points at.
__device__ __forceinline__ at_u32x2 transpose_from_lds(const Lds16* src) {
  typedef short s4 __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(at_u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS s4*)src));
}

// f(0) .. f(N - 1), the numbers as types.
template <int N, class F, int... I>
__device__ __forceinline__ void unroll(F f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>()), ...);
}
template <int N, class F>
__device__ __forceinline__ void unroll(F f) {
  unroll<N>(f, std::make_integer_sequence<int, N>());
}

// ONE: the page size is a multiple of 16, so that 16 tokens from a multiple of
// 16 lie on one page, and one lookup serves the wave that stages them (causal
// 8192: 512 us; row by row, page 11, 566).
// SPLIT: the keys are split over workgroups.  The matrix cores then have time to
// spare, and the weights enter as two 16-bit parts, as in decoding (0 x Inf has
// to be kept out of every tile, since the second part may be 0).
template <class T, int D, int E, bool ONE, bool SPLIT>
__global__ void __launch_bounds__(256, D == 256 ? 1 : 2) prefill_kernel(AttnArgs a, PrefillWork w) {
  constexpr bool FP4 = E == 0;
  constexpr int kUnit = FP4 ? 1 : E;              // bytes that the cache's strides count
  constexpr int kChunks = D / 8;                  // 16-byte chunks of a row of 16-bit elements
  constexpr int kPiece = FP4 && D == 64 ? 8 : 16; // bytes of a load
  constexpr int kRowLoads = FP4 ? D / 2 / kPiece : D * E / 16;       // of a cache row
  constexpr int kLoads = kBN * kRowLoads / 256;   // per thread and tensor
  // Score MFMAs per 32 tokens: of 16 d's; FP4: of 64 d's and a part of the queries each (as
  // long together as 16-bit ones, without widening the keys: ragged chunks over 28 / 4 heads
  // 528 -> 506 us.  Three parts, 477 us, would leave 2^-13 of a block's unit, which a query
  // with an outlier feels).
  constexpr int kParts = FP4 ? 4 : 1;
  constexpr int kSteps = FP4 ? D / 64 * kParts : D / 16;
  constexpr int kKeyOps = FP4 ? D / 64 : D / 16;  // key operands of 32 tokens
  constexpr int kKeyLoads = FP4 ? (D == 256 ? 2 : 1) : 1;       // FP4: 16-byte copies of a tile's keys per thread
  constexpr int kBlocks = D / 32;                 // value blocks
  // Two tiles of keys, two of values, and three words.  One object: with several,
  // the compiler no longer sees that copies into one tile leave the others alone,
  // and waits for them before every read.
  // (FP4: keys as they are in the cache, and their scale bytes.)
  __shared__ __align__(16) uint16_t smem[4 * kBN * D + 8];
  volatile LDS_AS int* const flags = (volatile LDS_AS int*)((Lds16*)smem + 4 * kBN * D);
  constexpr int kBad = 2;                         // [0], [1]: the tile with Inf or NaN among its values

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = lane >> 5, col = lane & 31;
  // kv heads vary fastest: with 8 of them each XCD serves one head, whose keys
  // and values its L2 then holds for all row tiles
  const int head = blockIdx.x % a.kv.heads;
  const int ti = (blockIdx.x / a.kv.heads) % w.row_tiles, split = blockIdx.x / a.kv.heads / w.row_tiles;
  RowTile rt;
  if (!find_tile(a, w, ti, &rt)) return;
  if (threadIdx.x == 0) {
    flags[kBad] = rt.over;
    flags[0] = flags[1] = -1;
  }

  // this lane's row
  const int all_rows = rt.count * a.group;        // at most tokens * q_heads < 2^31
  const int row = rt.tile * kBM + wave * 32 + col;
  const int rc = min(row, all_rows - 1);
  const int tok = w.group.div(rc), in_group = rc - tok * a.group;
  const int qi = rt.first_token + tok;
  const bool valid = row < all_rows && qi >= 0 && qi < w.tokens;
  const int past = rt.len - rt.count;             // may be negative: rows before position 0 see nothing
  const int pos = past + tok;
  const int pos_min = past + w.group.div(rt.tile * kBM);
  const int pos_max = past + w.group.div(min(rt.tile * kBM + kBM, all_rows) - 1);

  // visible tokens of the whole tile: [0, sink_end) and [start, hi)
  const int hi = max(pos_max + 1, 0);
  const int low = a.window ? max(pos_min - a.window + 1, 0) : 0;
  const int start = min(low, hi) & ~15;
  const int sink_end = min(a.sinks, start);
  const int sink_tiles = (sink_end + kBN - 1) / kBN;
  const int tiles = sink_tiles + (hi - start + kBN - 1) / kBN;
  const int used = SPLIT ? min(w.splits, max(tiles / 4, 1)) : 1;      // a split has at least 4 tiles
  if (split >= used) return;
  if (SPLIT && split == 0 && threadIdx.x == 0) w.used[ti * a.kv.heads + head] = used;
  const int t0 = int(int64_t(tiles) * split / used), t1 = int(int64_t(tiles) * (split + 1) / used);

  const float cs = a.scale_log2 * (E == 1 && a.kv.k_scale ? a.kv.k_scale[head] : 1.0f);
  const int32_t* table = a.kv.tables + rt.seq * a.kv.table_stride;
  const uint8_t* kbase = static_cast<const uint8_t*>(a.kv.k) + head * a.kv.head_stride * kUnit;
  const uint8_t* vbase = static_cast<const uint8_t*>(a.kv.v) + head * a.kv.head_stride * kUnit;

  std::conditional_t<FP4, at_u32x6, at_u32x4> q[kSteps];
  uint32_t q_scale[FP4 ? D / 64 : 1];         // FP4: the parts' scale bytes of 64 d's
  {
    const uint16_t* qp = static_cast<const uint16_t*>(a.q) + int64_t(min(max(qi, 0), w.tokens - 1)) * a.q_row +
                         (int64_t(head) * a.group + in_group) * a.q_head;
    if constexpr (FP4) {
#pragma unroll
      for (int j = 0; j < D / 64; ++j) {
        at_u32x6 part[kParts];
        q_scale[j] = split_query<T, kParts>(qp + 64 * j + 32 * half, part);
#pragma unroll
        for (int p = 0; p < kParts; ++p) q[kParts * j + p] = part[p];
      }
    } else {
#pragma unroll
      for (int j = 0; j < kSteps; ++j) q[j] = *reinterpret_cast<const at_u32x4*>(qp + 8 * half + 16 * j);
    }
  }

  auto tile_at = [&](int t, int* stop) {
    const bool sink = t < sink_tiles;
    *stop = sink ? sink_end : hi;
    return sink ? t * kBN : start + (t - sink_tiles) * kBN;
  };
  // Staging.  A wave takes 16 tokens of a tile: its load j brings 64 pieces of 16
  // bytes, kRowLoads of a cache row.  16-bit caches are copied to LDS directly
  // (lane l of a wave writes 16 bytes at 16 l, so the lane picks the chunk that
  // belongs there), E4M3 goes through registers.
  constexpr int kRows = 64 / kRowLoads;           // rows of one load
  auto load_row = [&](int j) { return j * kRows + lane / kRowLoads; };           // of the wave's 16
  auto chunk = [&](int j, bool v) {
    const int r = 16 * wave + load_row(j), c = lane % kRowLoads;
    return E != 2 ? c : c ^ (v ? value_swz<D>(r) : key_swz<D>(r));
  };
  // Where the rows are.  Lane l looks up one page for the tiles ahead: the wave's
  // 16 tokens of tile t + l if they lie on one page (ONE), or its token l % 16 of
  // tile t + l / 16.  So one load of the table serves 64 or 4 tiles.  Tokens past
  // the end take the last one's place, and an entry outside the cache is read as
  // page 0 and spoils the workgroup's rows if any of them may see a token there.
  constexpr int kAhead = ONE ? 64 : 4;
  bool bad = false;
  int64_t where = 0;          // byte offset of the lane's row
  int64_t where_scale = 0;    // FP4: of its first scale byte
  const int64_t head_scales = FP4 ? a.kv.scale_at + head * a.kv.scale_head : 0;
  auto look_ahead = [&](int t) {
    const int tl = min(t + (ONE ? lane : lane >> 4), t1 - 1);
    int stop;
    const int tk = tile_at(tl, &stop) + 16 * wave + (ONE ? 0 : lane & 15);
    const int u = min(tk, ONE ? (stop - 1) & ~15 : stop - 1), i = a.kv.page.div(u);
    const int slot = u - i * int(a.kv.page.d), p = table[i];
    const bool good = uint32_t(p) < uint32_t(a.kv.pages);
    bad |= !good && tk < stop && (min(tk + (ONE ? 16 : 1), stop) > low || tk < a.sinks);
    where = (int64_t(good ? p : 0) * a.kv.page_stride + int64_t(slot) * a.kv.token_stride) * kUnit;
    if constexpr (FP4) where_scale = int64_t(good ? p : 0) * a.kv.page_stride + head_scales + slot;
  };
  // ONE: what a lane reads is at a fixed offset from the first token's row.
  uint32_t koff[kLoads], voff[kLoads];
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    const uint32_t row = ONE ? uint32_t(load_row(j)) * uint32_t(a.kv.token_stride * kUnit) : 0;
    koff[j] = row + kPiece * chunk(j, false);
    voff[j] = row + kPiece * chunk(j, true);
  }
  // FP4.  Of the values a thread has one piece per load, all of one block, and its scale
  // byte; the keys are copied as they are, kKeyLoads pieces per thread (D = 64: the upper
  // half of a wave again those of the lower, to a place that is not read), and one scale
  // byte per 4 blocks, of the wave's token lane % 16.
  const uint32_t soff = FP4 ? (lane % kRowLoads * kPiece / 16) * a.kv.page.d : 0;
  constexpr int kKeyRow = D / 2;                  // bytes
  auto key_row = [&](int j) { return D == 64 ? (lane & 31) >> 1 : (j * 64 + lane) / (kKeyRow / 16); };       // of the wave's 16
  auto raw_swz = [](int r) { return D == 64 ? (r >> 3) & 1 : D == 128 ? (r >> 2) & 3 : (r >> 1) & 7; };
  auto key_chunk = [&](int j) { return lane % (kKeyRow / 16) ^ raw_swz(key_row(j)); };
  struct Raw {
    at_u32x4 x;
    uint32_t scale;
  };
  Raw raw_k[E != 2 ? kLoads : 1], raw_v[E != 2 ? kLoads : 1];
  struct Place {
    int64_t at[ONE ? 1 : kLoads], scale[ONE ? 1 : kLoads];
    int64_t key[!ONE && FP4 ? kKeyLoads : 1], key_scale;
  };
  auto place_of = [&](int t) {
    const int n = (t - t0) % kAhead;
    if (n == 0) look_ahead(t);
    auto uniform = [&](int64_t x) {
      return int64_t(uint32_t(__builtin_amdgcn_readlane(int(x), n))) | int64_t(__builtin_amdgcn_readlane(int(x >> 32), n)) << 32;
    };
    auto from_row = [&](int64_t x, int row) {
      const int from = 16 * n + row;
      return int64_t(uint32_t(__shfl(int(x), from))) | int64_t(__shfl(int(x >> 32), from)) << 32;
    };
    Place x;
    if constexpr (ONE) {
      x.at[0] = uniform(where);
      if constexpr (FP4) x.scale[0] = uniform(where_scale);
    } else {
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        x.at[j] = from_row(where, load_row(j));
        if constexpr (FP4) x.scale[j] = from_row(where_scale, load_row(j));
      }
      if constexpr (FP4) {
#pragma unroll
        for (int j = 0; j < kKeyLoads; ++j) x.key[j] = from_row(where, key_row(j));
        x.key_scale = from_row(where_scale, lane & 15);
      }
    }
    return x;
  };
  auto load = [&](Lds16* tile, const uint8_t* base, const Place& x, const uint32_t* offset, Raw* raw, auto values) {
    constexpr bool VALUES = decltype(values)::value;
    if constexpr (FP4 && !VALUES) {
      const uint8_t* cache = base - head * a.kv.head_stride;
#pragma unroll
      for (int j = 0; j < kKeyLoads; ++j) {
        Lds16* const to = tile + (wave * kKeyLoads + j) * 64 * 8;
        const uint32_t off = (ONE ? key_row(j) * kKeyRow : 0) + 16 * key_chunk(j);
        if constexpr (ONE) copy_to_lds(base + x.at[0], off, to);
        else copy_to_lds(base + x.key[j] + off, to);
        raw[j].scale = (cache + (ONE ? x.scale[0] + (lane & 15) : x.key_scale))[uint32_t(min((lane >> 4) + 4 * j, D / 32 - 1)) * a.kv.page.d];
      }
      return;
    }
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const uint8_t* p = base + x.at[ONE ? 0 : j];
      Lds16* const to = tile + (wave * kLoads + j) * 64 * 8;
      if constexpr (FP4) {
        if constexpr (kPiece == 8) {
          const at_u32x2 y = *reinterpret_cast<const at_u32x2*>(p + offset[j]);
          raw[j].x.x = y.x;
          raw[j].x.y = y.y;
        } else {
          raw[j].x = *reinterpret_cast<const at_u32x4*>(p + offset[j]);
        }
        const uint8_t* scales = base - head * a.kv.head_stride + x.scale[ONE ? 0 : j] + (ONE ? load_row(j) : 0);
        raw[j].scale = scales[soff];
      } else if constexpr (E == 1) raw[j].x = *reinterpret_cast<const at_u32x4*>(p + offset[j]);
      else if constexpr (ONE) copy_to_lds(p, offset[j], to);
      else copy_to_lds(p + offset[j], to);
    }
  };
  // The scale bytes of a tile's keys: [64 tokens][D / 32, padded to 4] behind the keys.
  constexpr int kScaleAt = 4 * kKeyLoads * 64 * 16, kScaleRow = D == 256 ? 8 : 4;
  // 8 and 4 bits: the pieces that have come go to LDS as 16-bit elements.
  auto put = [&](Lds16* tile, const Raw* raw, bool v) {
    if (FP4 && !v) {
      LDS_AS uint8_t* const to = (LDS_AS uint8_t*)tile + kScaleAt + (16 * wave + (lane & 15)) * kScaleRow + (lane >> 4);
#pragma unroll
      for (int j = 0; j < kKeyLoads; ++j) to[4 * j] = uint8_t(raw[j].scale);
    } else if constexpr (FP4) {
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const int r = 16 * wave + load_row(j), c = lane % kRowLoads, z = v ? value_swz<D>(r) : key_swz<D>(r);
        const float f = fp4_scale(raw[j].scale);
#pragma unroll
        for (int s = 0; s < kPiece / 4; ++s) {
          const uint32_t x = raw[j].x[s];
          *reinterpret_cast<LDS_AS at_u32x4*>(tile + r * D + 8 * ((kPiece / 4 * c + s) ^ z)) =
              (at_u32x4){fp4_pair<T, 0>(x, f), fp4_pair<T, 1>(x, f), fp4_pair<T, 2>(x, f), fp4_pair<T, 3>(x, f)};
        }
      }
    } else if constexpr (E == 1) {
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const int r = 16 * wave + load_row(j), c = chunk(j, v), z = v ? value_swz<D>(r) : key_swz<D>(r);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const uint32_t x = raw[j].x[2 * s], y = raw[j].x[2 * s + 1];
          *reinterpret_cast<LDS_AS at_u32x4*>(tile + r * D + 8 * ((2 * c + s) ^ z)) =
              (at_u32x4){e4m3_pair<T, false>(x), e4m3_pair<T, true>(x), e4m3_pair<T, false>(y), e4m3_pair<T, true>(y)};
        }
      }
    }
  };
  // Tiles that every row sees whole need no masks: full sink tiles, and those
  // from where the last row's window begins to the first row's position.
  const int whole_sinks = sink_end / kBN;
  const int whole_from = sink_tiles + (a.window ? (max(pos_max - a.window + 1 - start, 0) + kBN - 1) / kBN : 0);
  const int whole_to = sink_tiles + max(min(pos_min + 1, hi) - start, 0) / kBN;
  auto whole = [&](int t) { return t < whole_sinks || (t >= whole_from && t < whole_to); };
  // Looks over the values of a tile that has come.  In one that some row does not
  // see whole, the wave that staged them clears those past the end (whatever the
  // page holds there) and looks for Inf and NaN among the others.
  auto look_over = [&](Lds16* vt, int buf, int t) {
    if (SPLIT || !whole(t)) {
      bool odd = false;
#pragma unroll
      for (int j = 0; j < kChunks / 4; ++j) {
        const int i = (wave * (kChunks / 4) + j) * 64 + lane;        // 16-byte piece of the tile
        int stop;
        if (tile_at(t, &stop) + i / kChunks < stop) {
          const at_u32x4 x = read16(vt + 8 * i);
#pragma unroll
          for (int k = 0; k < 4; ++k) odd |= T::not_finite(x[k]);
        } else {
          *reinterpret_cast<LDS_AS at_u32x4*>(vt + 8 * i) = (at_u32x4){0, 0, 0, 0};
        }
      }
      if (odd) flags[buf] = t;
    }
  };
  auto arrived = [] {
    if constexpr (E != 1) __builtin_amdgcn_s_waitcnt(wait_vmcnt(0));
  };

  at_f32x16 o[kBlocks];
#pragma unroll
  for (int n = 0; n < kBlocks; ++n)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[n][e] = 0.0f;
  float m = kNegInf, l = 0.0f;
  float least = 0.0f;         // of the factors that the sums are rebased by: kLeast from the first Inf or NaN on

  auto sees = [&](int t, int stop) {
    return t < stop && t <= pos && (!a.window || t > pos - a.window || t < a.sinks);
  };
  // Operands.  A lane's element offsets in a tile, apart from constants: of the key
  // operand of step j (32 tokens: row lane % 32, chunk 2 j + lane / 32), and of the
  // value operand of block n (32 d's, by two transposing reads of 4 tokens x 16
  // d's per 16 lanes; a multiple of 8 tokens does not change the swizzle).
  // (FP4: of step j the block 2 j + lane / 32 of 32 d's.  A wave's 16 tokens have kKeyLoads
  // KiB of their own; 32 tokens further the swizzle is the same.)
  int k_at[kKeyOps], v_at[kBlocks];
#pragma unroll
  for (int j = 0; j < kKeyOps; ++j)
    k_at[j] = FP4 ? (col >> 4) * kKeyLoads * 512 + (col & 15) * (kKeyRow / 2) + 8 * ((2 * j + half) ^ raw_swz(col & 15))
                  : col * D + 8 * ((2 * j + half) ^ key_swz<D>(col));
#pragma unroll
  for (int n = 0; n < kBlocks; ++n) {
    const int i = lane & 15, d = 32 * n + 16 * ((lane >> 4) & 1) + 4 * (i & 3), r = 4 * half + (i >> 2);
    v_at[n] = r * D + 8 * ((d >> 3) ^ value_swz<D>(r)) + (d & 4);
  }
  // Key operand of MFMA i of a tile's scores (block i % 2 of 32 tokens, step i / 2).
  // Register e of the block's scores is the token 8 (e / 4) + 4 half + e % 4.
  auto key = [&](const Lds16* kt, int i) {
    return read16(kt + k_at[i >> 1] + (FP4 ? kKeyLoads * 1024 : 32 * D) * (i & 1));
  };
  // FP4: the scale bytes of a tile's keys: of block b of 32 tokens, byte 2 (j % 2) of word j / 2
  // is that of step j and this half.
  struct KeyScales {
    uint32_t w[2][D == 256 ? 2 : 1];
  };
  auto key_scales = [&](const Lds16* kt) {
    KeyScales x = {};
    if constexpr (FP4) {
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int k = 0; k < (D == 256 ? 2 : 1); ++k)
          x.w[b][k] = *reinterpret_cast<const LDS_AS uint32_t*>((const LDS_AS uint8_t*)kt + kScaleAt + (32 * b + col) * kScaleRow + 4 * k) >> (8 * half);
    }
    return x;
  };
  // Score MFMA m of 2 kSteps: by steps, in a step by parts (the smallest first), the two
  // blocks of tokens in turn.  Its key operand, and whether that is done with.
  constexpr auto key_of = [](int m) { return FP4 ? m / (2 * kParts) * 2 + (m & 1) : m; };
  constexpr auto key_done = [](int m) { return !FP4 || m % (2 * kParts) >= 2 * kParts - 2; };
  auto score = [&](auto which, at_u32x4 k, const KeyScales& ks, at_f32x16 c) {
    constexpr int M = decltype(which)::value;
    if constexpr (FP4) {
      constexpr int J = M / (2 * kParts), P = kParts - 1 - M % (2 * kParts) / 2;
      const at_u32x6 z = q[kParts * J + P];
      const at_i32x8 x = {int(k.x), int(k.y), int(k.z), int(k.w), 0, 0, 0, 0};
      const at_i32x8 y = {int(z[0]), int(z[1]), int(z[2]), int(z[3]), int(z[4]), int(z[5]), 0, 0};
      return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, c, 4, 2, 2 * (J % 2), int(ks.w[M & 1][J / 2]), P, int(q_scale[J]));
    } else {
      return T::mfma32(k, q[M >> 1], c);
    }
  };
  // Value operand of block n, 16 tokens from tb.
  auto value = [&](const Lds16* vt, int n, int tb) {
    const at_u32x2 x = transpose_from_lds(vt + v_at[n] + tb * D), y = transpose_from_lds(vt + v_at[n] + (tb + 8) * D);
    return (at_u32x4){x.x, x.y, y.x, y.y};
  };
  // Masks the scores of tile t.
  auto mask = [&](int t, at_f32x16 (&s)[2]) {
    // A bit for each of the 64 tokens, counted from this half's first one: from <=
    // token < to, or a sink.
    int stop;
    const int base = tile_at(t, &stop) + 4 * half;
    const int to = min(stop, pos + 1) - base, sinks = min(a.sinks - base, to);
    const int from = a.window ? pos - a.window + 1 - base : 0;
    auto below = [](int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1; };
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const uint32_t seen = (below(to - 32 * b) & ~below(from - 32 * b)) | below(sinks - 32 * b);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const uint32_t keep = uint32_t(int32_t(seen << (31 - (8 * (e >> 2) + (e & 3)))) >> 31);
        const float x = s[b][e];
        s[b][e] = __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, x) & keep) | (0xff800000u & ~keep));
      }
    }
  };
  // Takes a tile's largest score into the reference of the weights.
  auto rebase_sums = [&](float mx) {
    mx = max_xor32(mx) * cs;
    if (__any(mx > m + (kGrowth + T::kRaise))) {
      const float mn = fmaxf(m, mx - T::kRaise), f = fmaxf(rebase(m, mn), least);
#pragma unroll
      for (int n = 0; n < kBlocks; ++n) o[n] *= f;
      l *= f;
      m = mn;
    }
  };
  // Inf or NaN in a tile that some row does not see whole: 0 x Inf would reach
  // the row's sum.  The rows that see such a value get it added, then it is
  // cleared in the tile.  (All waves get here together: the flag is the tile's.)
  auto settle_odd = [&](Lds16* vt, int t) {
    if (SPLIT) least = kLeast;
    int stop;
    const int base = tile_at(t, &stop);
#pragma unroll 1
    for (int r = 0; r < kBN; ++r) {
      const bool see = sees(base + r, stop);
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const at_u32x2 x = *reinterpret_cast<const LDS_AS at_u32x2*>(vt + r * D + 8 * (c ^ value_swz<D>(r)) + 4 * half);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float v = k & 1 ? T::high(x[k >> 1]) : T::low(x[k >> 1]);
          if (see && !(fabsf(v) < -kNegInf)) o[c >> 2][4 * (c & 3) + k] += v;
        }
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kBN * D / 2; i += 256) {
      LDS_AS uint32_t* u = reinterpret_cast<LDS_AS uint32_t*>(vt) + i;
      if (T::not_finite(*u)) *u = T::finite(*u);
    }
    __syncthreads();
  };
  // The scores are a tile ahead: the matrix cores take those of tile t + 1 (NEXT),
  // then the values of tile t.  A wave's instructions issue in order, so MFMAs in
  // a row would leave the vector units idle, and the other way round: behind every
  // MFMA comes a share of the vector work.  That is the weights of t, the first
  // kFirst of 16 pairs behind the scores of t + 1, the others behind the values of
  // the first 32 tokens, and behind those of the last 32 the maximum of t + 1.
  // Operands are read kDepth MFMAs ahead.
  auto compute = [&](const Lds16* k_next, const Lds16* v_cur, int t, const at_f32x16 (&s)[2], at_f32x16 (&ahead)[2], auto next) {
    constexpr bool NEXT = decltype(next)::value;
    constexpr int kScores = 2 * kSteps, kKeys = 2 * kKeyOps, kValues = 4 * kBlocks, kDepth = D == 256 ? 2 : 4;
    constexpr int kFirst = 16 * kScores / (kScores + kValues) + 2;      // 10 where both are as many
    const float mm = m == kNegInf ? 0.0f : m;
    at_u32x4 p[4], rest[SPLIT ? 4 : 1];      // weights of 16 tokens as operands (SPLIT: in two parts)
    auto pair = [&](int u) {
      const int i = u >> 2, k = u & 3, e = 8 * (i & 1) + 2 * k;
      const float x = exp2_fast(__builtin_fmaf(s[i >> 1][e], cs, -mm)), y = exp2_fast(__builtin_fmaf(s[i >> 1][e + 1], cs, -mm));
      l += x;
      l += y;
      uint32_t z = T::pack(x, y);
      asm volatile("" : "+v"(z), "+v"(l));      // here, and not where they are used
      p[i][k] = z;
      if constexpr (SPLIT) rest[i][k] = T::pack(x - T::low(z), y - T::high(z));
    };
    auto v_operand = [&](int v) { return value(v_cur, v % kBlocks, 16 * (v / kBlocks)); };
    at_u32x4 f[kDepth];
    if constexpr (NEXT) {
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int e = 0; e < 16; ++e) ahead[b][e] = 0.0f;
      const KeyScales ks = key_scales(k_next);
      auto operand = [&](int i) { return i < kKeys ? key(k_next, i) : v_operand(i - kKeys); };
#pragma unroll
      for (int i = 0; i < kDepth; ++i) f[i] = operand(i);
      unroll<kScores>([&](auto which) {
        constexpr int i = decltype(which)::value, k = key_of(i);
        ahead[i & 1] = score(which, f[k % kDepth], ks, ahead[i & 1]);
        if constexpr (key_done(i)) f[k % kDepth] = operand(k + kDepth);
#pragma unroll
        for (int u = i * kFirst / kScores; u < (i + 1) * kFirst / kScores; ++u) pair(u);
        __builtin_amdgcn_sched_barrier(0);
      });
      if (!whole(t + 1)) mask(t + 1, ahead);
    } else {
#pragma unroll
      for (int i = 0; i < kDepth; ++i) f[(kKeys + i) % kDepth] = v_operand(i);
#pragma unroll
      for (int u = 0; u < kFirst; ++u) pair(u);
    }
    float mx = kNegInf;
#pragma unroll
    for (int v = 0; v < kValues; ++v) {
      const int n = v % kBlocks, i = v / kBlocks;
      at_u32x4& y = f[(kKeys + v) % kDepth];
      o[n] = T::mfma32(y, p[i], o[n]);
      if constexpr (SPLIT) o[n] = T::mfma32(y, rest[i], o[n]);
      if (v + kDepth < kValues) y = v_operand(v + kDepth);
      if (v < kValues / 2) {
#pragma unroll
        for (int u = kFirst + v * (16 - kFirst) / (kValues / 2); u < kFirst + (v + 1) * (16 - kFirst) / (kValues / 2); ++u) pair(u);
      } else if constexpr (NEXT) {
        constexpr int kShare = 64 / kValues;
#pragma unroll
        for (int e = (v - kValues / 2) * kShare; e < (v - kValues / 2 + 1) * kShare; ++e) mx = fmaxf(mx, ahead[e >> 4][e & 15]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (NEXT) {
      rebase_sums(mx);
    }
  };
  // The scores of a tile by themselves, masked and taken into the maximum.
  auto scores = [&](const Lds16* kt, int t, at_f32x16 (&s)[2]) {
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int e = 0; e < 16; ++e) s[b][e] = 0.0f;
    const KeyScales ks = key_scales(kt);
    unroll<2 * kSteps>([&](auto which) {
      constexpr int i = decltype(which)::value;
      s[i & 1] = score(which, key(kt, key_of(i)), ks, s[i & 1]);
    });
    if (!whole(t)) mask(t, s);
    float mx = kNegInf;
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int e = 0; e < 16; ++e) mx = fmaxf(mx, s[b][e]);
    rebase_sums(mx);
  };
  // SPLIT: a wave whose rows are all past the sequence's end only stages.
  const bool busy = rt.tile * kBM + wave * 32 < all_rows;
  // One step: copies start of the keys of t + 2 into the buffer that t's were in,
  // and of the values of t + 1.  That the four tiles are different memory is what
  // lets the reads go on meanwhile.
  Place here;                   // of tile t + 1
  auto settle = [&](Lds16* v_cur, int t, int buf) {
    if ((SPLIT || !whole(t)) && flags[buf] == t) settle_odd(v_cur, t);
  };
  auto tile_step = [&](Lds16* __restrict__ k_in, Lds16* __restrict__ k_next, Lds16* __restrict__ v_cur,
                       Lds16* __restrict__ v_in, int t, int buf, const at_f32x16 (&s)[2], at_f32x16 (&ahead)[2]) {
    load(v_in, vbase, here, voff, raw_v, std::true_type());
    if (t + 2 < t1) {
      here = place_of(t + 2);
      load(k_in, kbase, here, koff, raw_k, std::false_type());
    }
    settle(v_cur, t, buf);
    compute(k_next, v_cur, t, s, ahead, std::true_type());
    arrived();
    put(v_in, raw_v, true);
    if (t + 2 < t1) put(k_in, raw_k, false);
    look_over(v_in, buf ^ 1, t + 1);
    __syncthreads();
  };

  Lds16* const lk = (Lds16*)smem;
  Lds16* const lv = lk + 2 * kBN * D;
  if constexpr (SPLIT) {
    // A share of the keys: what counts is how soon they come, so a tile's copies
    // start a whole step ahead, keys and values, and the step is plain.
    auto split_step = [&](Lds16* __restrict__ k_cur, Lds16* __restrict__ v_cur, Lds16* __restrict__ k_in,
                          Lds16* __restrict__ v_in, int t, int buf) {
      const bool more = t + 1 < t1;
      if (more) {
        here = place_of(t + 1);
        load(k_in, kbase, here, koff, raw_k, std::false_type());
        load(v_in, vbase, here, voff, raw_v, std::true_type());
      }
      at_f32x16 s[2], none[2];
      // Inf is settled after the rebase by this tile's maximum (the first one's is by
      // 0); E4M3 has NaN only, and holds fewer registers this way round.
      if (E != 2) settle(v_cur, t, buf);
      if (busy) scores(k_cur, t, s);
      if (E == 2) settle(v_cur, t, buf);
      if (busy) compute(k_cur, v_cur, t, s, none, std::false_type());
      if (more) {
        arrived();
        put(k_in, raw_k, false);
        put(v_in, raw_v, true);
        look_over(v_in, buf ^ 1, t + 1);
      }
      __syncthreads();
    };
    if (t0 < t1) {
      here = place_of(t0);
      load(lk, kbase, here, koff, raw_k, std::false_type());
      load(lv, vbase, here, voff, raw_v, std::true_type());
      __syncthreads();          // the flags are set before a wave marks its tile in them
      arrived();
      put(lk, raw_k, false);
      put(lv, raw_v, true);
      look_over(lv, 0, t0);
      __syncthreads();
    }
    for (int t = t0; t < t1; ++t) {
      const int buf = (t - t0) & 1, cur = buf * kBN * D, nxt = kBN * D - cur;
      split_step(lk + cur, lv + cur, lk + nxt, lv + nxt, t, buf);
    }
  } else if (t0 < t1) {
    // the keys of t0, its values, and the keys of t0 + 1; the scores of t0 wait
    // for the first only
    here = place_of(t0);
    load(lk, kbase, here, koff, raw_k, std::false_type());
    put(lk, raw_k, false);
    load(lv, vbase, here, voff, raw_v, std::true_type());
    put(lv, raw_v, true);
    if (t0 + 1 < t1) {
      here = place_of(t0 + 1);
      load(lk + kBN * D, kbase, here, koff, raw_k, std::false_type());
      put(lk + kBN * D, raw_k, false);
      if constexpr (E == 2) __builtin_amdgcn_s_waitcnt(wait_vmcnt(2 * kLoads));
    } else if constexpr (E == 2) {
      __builtin_amdgcn_s_waitcnt(wait_vmcnt(kLoads));
    }
    if constexpr (FP4) arrived();
    __syncthreads();
    at_f32x16 s[2], s2[2];
    scores(lk, t0, s);
    arrived();
    look_over(lv, 0, t0);
    __syncthreads();            // also: the keys of t0 have been read by all, theirs is the buffer of t0 + 2
    Lds16 *const k0 = lk, *const k1 = lk + kBN * D, *const v0 = lv, *const v1 = lv + kBN * D;
    int t = t0;
    if constexpr (D == 256) {           // two steps' code would not fit the registers
      for (; t + 1 < t1; ++t) {
        const int cur = ((t - t0) & 1) * kBN * D, nxt = kBN * D - cur;
        tile_step(lk + cur, lk + nxt, lv + cur, lv + nxt, t, (t - t0) & 1, s, s2);
        s[0] = s2[0];
        s[1] = s2[1];
      }
    } else {
      for (; t + 2 < t1; t += 2) {
        tile_step(k0, k1, v0, v1, t, 0, s, s2);
        tile_step(k1, k0, v1, v0, t + 1, 1, s2, s);
      }
      if (t + 1 < t1) {
        tile_step(k0, k1, v0, v1, t, 0, s, s2);
        s[0] = s2[0];
        s[1] = s2[1];
        ++t;
      }
    }
    Lds16* const last = (t - t0) & 1 ? v1 : v0;
    settle(last, t, (t - t0) & 1);
    compute(lk, last, t, s, s2, std::false_type());
  }
  if (bad) flags[kBad] = 1;
  __syncthreads();
  l = sum_xor32(l);
  if (flags[kBad]) l = __builtin_nanf("");

  if (SPLIT && used > 1) {
    float* part = w.parts + (int64_t(ti * a.kv.heads + head) * w.splits + split) * kBM * (D + 2);
    const int r = wave * 32 + col;
#pragma unroll
    for (int n = 0; n < kBlocks; ++n)
#pragma unroll
      for (int f = 0; f < 4; ++f)
        *reinterpret_cast<at_f32x4*>(part + r * D + 32 * n + 8 * f + 4 * half) =
            (at_f32x4){o[n][4 * f], o[n][4 * f + 1], o[n][4 * f + 2], o[n][4 * f + 3]};
    if (half == 0) {
      part[kBM * D + r] = m;
      part[kBM * (D + 1) + r] = l;
    }
    return;
  }
  // A whole tile's Inf goes through the product, where a weight that rounds to 0
  // makes it NaN, and so does a rebase of its sum by 0.  So a sum that is not finite
  // is made again from the Inf and NaN that its row sees: finite values do not matter
  // beside them, and the largest one stands for a sum that has no other cause than
  // its size.  (The wave's lanes look over 64 tokens at a time.)
  if constexpr (!SPLIT && E == 2) {
    constexpr float kLargest = 0x1.fffffep127f;
    float zero[8];              // NaN if any sum is not finite
#pragma unroll
    for (int e = 0; e < 8; ++e) zero[e] = 0.0f;
#pragma unroll
    for (int n = 0; n < kBlocks; ++n)
#pragma unroll
      for (int e = 0; e < 16; ++e) zero[e & 7] = __builtin_fmaf(o[n][e], 0.0f, zero[e & 7]);
#pragma unroll
    for (int e = 4; e; e >>= 1)
#pragma unroll
      for (int k = 0; k < e; ++k) zero[k] += zero[k + e];
    if (__any(zero[0] != 0.0f)) {
#pragma unroll
      for (int n = 0; n < kBlocks; ++n)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (!(fabsf(o[n][e]) < -kNegInf)) o[n][e] = copysignf(kLargest, o[n][e]);
#pragma unroll 1
      for (int base = 0; base < hi; base += 64) {
        const int t = base + lane;
        const uint8_t* row = vbase;
        bool met = false;
        if (t < hi && (t >= low || t < a.sinks)) {
          const int i = a.kv.page.div(t), p = table[i];
          if (uint32_t(p) < uint32_t(a.kv.pages)) {
            row += (int64_t(p) * a.kv.page_stride + int64_t(t - i * int(a.kv.page.d)) * a.kv.token_stride) * E;
#pragma unroll 1
            for (int c = 0; c < kChunks; ++c) {
              const at_u32x4 x = *reinterpret_cast<const at_u32x4*>(row + 16 * c);
              met |= T::not_finite(x[0]) || T::not_finite(x[1]) || T::not_finite(x[2]) || T::not_finite(x[3]);
            }
          }
        }
#pragma unroll 1
        for (uint64_t todo = __ballot(met); todo; todo &= todo - 1) {
          const int from = __ffsll((unsigned long long)todo) - 1;
          const uint8_t* v = reinterpret_cast<const uint8_t*>(__shfl(reinterpret_cast<uintptr_t>(row), from));
          const bool see = sees(base + from, hi);
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            const at_u32x2 x = *reinterpret_cast<const at_u32x2*>(v + 16 * c + 8 * half);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float y = k & 1 ? T::high(x[k >> 1]) : T::low(x[k >> 1]);
              if (see && !(fabsf(y) < -kNegInf)) o[c >> 2][4 * (c & 3) + k] += y;
            }
          }
        }
      }
#pragma unroll
      for (int n = 0; n < kBlocks; ++n)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (fabsf(o[n][e]) == kLargest) o[n][e] = copysignf(-kNegInf, o[n][e]);
    }
  }
  if (!valid) return;
  const int h = head * a.group + in_group;
  const bool none = pos < 0 && !rt.over;
  const float inv = (E == 1 && a.kv.v_scale ? a.kv.v_scale[head] : 1.0f) / l;
  uint16_t* out = static_cast<uint16_t*>(a.out) + qi * a.o_row + h * a.o_head + 4 * half;
#pragma unroll
  for (int n = 0; n < kBlocks; ++n)
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      at_u32x2 y = {T::pack(o[n][4 * f] * inv, o[n][4 * f + 1] * inv), T::pack(o[n][4 * f + 2] * inv, o[n][4 * f + 3] * inv)};
      if (none) y = (at_u32x2){0, 0};
      *reinterpret_cast<at_u32x2*>(out + 32 * n + 8 * f) = y;
    }
  if (a.lse && half == 0) a.lse[int64_t(qi) * a.q_heads + h] = none ? kNegInf : (m + __log2f(l)) * 0.693147180559945f;
}

// Joins the splits of a row tile, as decoding joins its pieces: grid (row tiles
// x heads, kBM / 8); a workgroup joins 8 rows, 32 threads each, so that the
// parts' reads are in flight together.  Their latency bounds it: 8 us for 32
// units of 28 rows.
template <class T, int D, int E>
__global__ void __launch_bounds__(256) prefill_join_kernel(AttnArgs a, PrefillWork w) {
  const int head = blockIdx.x % a.kv.heads, ti = blockIdx.x / a.kv.heads;
  RowTile rt;
  if (!find_tile(a, w, ti, &rt)) return;
  const int used = w.used[blockIdx.x];
  if (used <= 1) return;
  const int r = blockIdx.y * 8 + threadIdx.x / 32, lane = threadIdx.x & 31;
  const int row = rt.tile * kBM + r;
  if (row >= rt.count * a.group) return;
  const int tok = w.group.div(row), qi = rt.first_token + tok;
  if (qi < 0 || qi >= w.tokens) return;
  const float* base = w.parts + int64_t(blockIdx.x) * w.splits * kBM * (D + 2);
  // lane i looks after the splits i, i + 32: their references and sums of weights
  float f0 = kNegInf, f1 = kNegInf, L = 0.0f;
  const int64_t part = int64_t(kBM) * (D + 2);
  if (lane < used) f0 = base[lane * part + kBM * D + r];
  if (lane + 32 < used) f1 = base[(lane + 32) * part + kBM * D + r];
  float M = fmaxf(f0, f1);
#pragma unroll
  for (int d = 16; d; d >>= 1) M = fmaxf(M, __shfl_xor(M, d));
  f0 = rebase_joined(f0, M);
  f1 = rebase_joined(f1, M);
  if (lane < used) L = f0 * base[lane * part + kBM * (D + 1) + r];
  if (lane + 32 < used) L += f1 * base[(lane + 32) * part + kBM * (D + 1) + r];
#pragma unroll
  for (int d = 16; d; d >>= 1) L += __shfl_xor(L, d);
  float O[D / 32];
#pragma unroll
  for (int j = 0; j < D / 32; ++j) O[j] = 0.0f;
  for (int i0 = 0; i0 < used; i0 += 8) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {                     // 8 splits' loads in flight
      const int i = min(i0 + k, used - 1);
      const float f = __shfl(i < 32 ? f0 : f1, (threadIdx.x & 32) + (i & 31));
#pragma unroll
      for (int j = 0; j < D / 64; ++j) {
        const at_f32x2 x = *reinterpret_cast<const at_f32x2*>(base + i * part + r * D + 64 * j + 2 * lane);
        O[2 * j] += i0 + k < used ? f * x.x : 0.0f;
        O[2 * j + 1] += i0 + k < used ? f * x.y : 0.0f;
      }
    }
  }
  const int h = head * a.group + (row - tok * a.group);
  const bool none = rt.len - rt.count + tok < 0 && !rt.over;
  const float inv = (E == 1 && a.kv.v_scale ? a.kv.v_scale[head] : 1.0f) / L;
  uint16_t* out = static_cast<uint16_t*>(a.out) + qi * a.o_row + h * a.o_head + 2 * lane;
#pragma unroll
  for (int j = 0; j < D / 64; ++j)
    *reinterpret_cast<uint32_t*>(out + 64 * j) = none ? 0 : T::pack(O[2 * j] * inv, O[2 * j + 1] * inv);
  if (a.lse && lane == 0) a.lse[int64_t(qi) * a.q_heads + h] = none ? kNegInf : (M + __log2f(L)) * 0.693147180559945f;
}

int64_t row_tiles(int64_t seqs, int64_t tokens, int group) { return tokens * group / kBM + seqs; }

// Splits of the keys: as many as it takes for two workgroups per CU, where the
// row tiles alone leave CUs without work (5 to 9 rows x 4 heads on 33000 E4M3
// tokens, not split / split: 611.8 / 74.2 us; 16 tokens of each of 8 sequences
// on 8000 bf16 tokens 151.7 / 92.4).  Workspace is given for this many; tables that
// hold kNoSplit tokens at most are not split, since the second launch and the
// partial results cost what 15 steps of 64 tokens do: split / not split, a
// prompt of 82 tokens 13.8 / 10.7 us, of 800 33.7 / 21.3, 16 tokens after 700
// 19.5 / 18.8, after 1000 19.3 / 21.8.  Not split, the weights enter as one part.
// (The host knows the tables' width, not the lengths: a short prompt in wide tables
// is split, and where sequences without new tokens bring row tiles enough nothing is:
// 64 tokens on 8000 beside 63 such sequences 166 us, alone 40.)
constexpr int kNoSplit = 1000;
int key_splits(int64_t tiles, int heads) {
  const int64_t wgs = tiles * heads;
  return wgs >= 256 ? 1 : int(std::min<int64_t>((512 + wgs - 1) / wgs, kMaxSplits));
}

template <class T, int D, int E, bool SPLIT>
hipError_t launch_split(const AttnArgs& a, const PrefillWork& w, hipStream_t stream) {
  const unsigned tiles = unsigned(w.row_tiles * a.kv.heads);
  // (a lane's offset from the first of 16 tokens is kept in 32 bits)
  if (a.kv.page.d % 16 == 0 && a.kv.token_stride < (1 << 26))
    prefill_kernel<T, D, E, true, SPLIT><<<tiles * unsigned(w.splits), 256, 0, stream>>>(a, w);
  else
    prefill_kernel<T, D, E, false, SPLIT><<<tiles * unsigned(w.splits), 256, 0, stream>>>(a, w);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !SPLIT) return e;
  prefill_join_kernel<T, D, E><<<dim3(tiles, kBM / 8), 256, 0, stream>>>(a, w);
  return hipGetLastError();
}

template <class T, int D, int E>
hipError_t launch(const AttnArgs& a, const PrefillWork& w, hipStream_t stream) {
  return w.splits > 1 ? launch_split<T, D, E, true>(a, w, stream) : launch_split<T, D, E, false>(a, w, stream);
}

template <class T, int E>
hipError_t launch_dim(const AttnArgs& a, const PrefillWork& w, int D, hipStream_t stream) {
  if (D == 64) return launch<T, 64, E>(a, w, stream);
  if (D == 128) return launch<T, 128, E>(a, w, stream);
  return launch<T, 256, E>(a, w, stream);
}

}  // namespace

// [parts] [used]
size_t attn_prefill_workspace(int64_t seqs, int64_t tokens, int q_heads, int heads, int head_dim, int page_size,
                              int cache_dtype) {
  if (attn_few_serves(seqs, tokens, q_heads / heads, page_size, cache_dtype, head_dim))
    return attn_few_workspace(seqs, tokens, q_heads / heads, cache_dtype, head_dim);
  const int64_t tiles = row_tiles(seqs, tokens, q_heads / heads);
  const int splits = key_splits(tiles, heads);
  if (splits == 1) return 0;
  return size_t(tiles * heads) * (size_t(splits) * kBM * (head_dim + 2) * 4 + 4);
}

// Of the row tiles' launch (few rows have no more than fill the card: 0).
int64_t attn_prefill_workgroups(int64_t seqs, int64_t tokens, int q_heads, int heads, int head_dim, int page_size,
                                int cache_dtype) {
  if (attn_few_serves(seqs, tokens, q_heads / heads, page_size, cache_dtype, head_dim)) return 0;
  const int64_t tiles = row_tiles(seqs, tokens, q_heads / heads);
  return tiles * heads * key_splits(tiles, heads);
}

hipError_t launch_attn_prefill(const AttnArgs& a, const int32_t* cu, int64_t tokens, int cache_dtype, int dtype,
                               int head_dim, void* workspace, hipStream_t stream) {
  if (attn_few_serves(a.kv.seqs, tokens, a.group, int(a.kv.page.d), cache_dtype, head_dim))
    return launch_attn_few(a, cu, tokens, cache_dtype, dtype, head_dim, workspace, stream);
  PrefillWork w;
  w.cu = cu;
  w.tokens = int32_t(tokens);
  w.row_tiles = int32_t(row_tiles(a.kv.seqs, tokens, a.group));
  w.splits = int64_t(a.kv.max_pages) * a.kv.page.d <= kNoSplit ? 1 : key_splits(w.row_tiles, a.kv.heads);
  w.group = fast_div(uint32_t(a.group));
  w.parts = static_cast<float*>(workspace);
  w.used = reinterpret_cast<int32_t*>(w.parts + size_t(w.row_tiles) * a.kv.heads * w.splits * kBM * (head_dim + 2));
  if (cache_dtype == W4A4_E2M1)
    return dtype == W4A4_BF16 ? launch_dim<Bf16, 0>(a, w, head_dim, stream) : launch_dim<F16, 0>(a, w, head_dim, stream);
  const bool e4m3 = cache_dtype == W4A4_E4M3;
  if (dtype == W4A4_BF16)
    return e4m3 ? launch_dim<Bf16, 1>(a, w, head_dim, stream) : launch_dim<Bf16, 2>(a, w, head_dim, stream);
  return e4m3 ? launch_dim<F16, 1>(a, w, head_dim, stream) : launch_dim<F16, 2>(a, w, head_dim, stream);
}

}  // namespace w4a4
