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
// The matrix cores bound it: 4 D operations per visible pair.
#include <algorithm>

#include "attn_common.h"

namespace w4a4 {
namespace {

#define LDS_AS __attribute__((address_space(3)))

constexpr int kBM = 128;      // rows per workgroup
constexpr int kBN = 64;       // tokens per step

struct PrefillWork {
  const int32_t* cu;
  float* parts;               // [row tiles x heads x splits] of kBM x (D + 2), or unused
  int32_t* used;              // [row tiles x heads]: splits that hold results
  int32_t tokens, row_tiles, splits;
  FastDiv group;
};

// The sequence and tile of the sequence that row tile `ti` is; false past the end.
// Tiles of a sequence are handed out from its end, where rows see most keys.
struct RowTile {
  int seq, tile, first_token, count, len;
  bool over;
};
__device__ __forceinline__ bool find_tile(const AttnArgs& a, const PrefillWork& w, int ti, RowTile* out) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int base = 0; base < a.kv.seqs; base += 64) {
    const int s = base + lane;
    int n = 0;
    if (s < a.kv.seqs) n = min(max(w.cu[s + 1] - w.cu[s], 0), w.tokens);
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
      out->seq = base + l;
      out->count = __builtin_amdgcn_readlane(n, l);
      out->tile = before + __builtin_amdgcn_readlane(in, l) - 1 - ti;
      out->first_token = w.cu[base + l];
      const int cap = int(min(int64_t(a.kv.max_pages) * a.kv.page.d, int64_t(1) << 30));
      const int len = a.kv.lens[base + l];
      out->over = len > cap;
      out->len = min(len, cap);
      return true;
    }
    before += __builtin_amdgcn_readlane(in, 63);
  }
  return false;
}

// 16-byte chunk swizzles of the LDS tiles (row r, chunk c at slot c ^ swz(r)).
// Keys: 16 consecutive rows of one chunk fall on 16 different 16-byte bank
// groups; values: so do 4 consecutive rows of two chunks.
template <int D>
__device__ __forceinline__ int key_swz(int r) { return D == 64 ? (r >> 1) & 7 : r & 15; }
template <int D>
__device__ __forceinline__ int value_swz(int r) { return D == 64 ? ((r >> 1) & 3) << 1 : (r & 7) << 1; }

typedef LDS_AS uint16_t Lds16;

// 16 bytes per lane from `src` to LDS, lane l writing `dst` + 16 l (dst is
// wave-uniform).
__device__ __forceinline__ void copy_to_lds(const uint8_t* src, Lds16* dst) {
  __builtin_amdgcn_global_load_lds(src, (LDS_AS void*)dst, 16, 0, 0);
}
__device__ __forceinline__ at_u32x4 read16(const Lds16* p) { return *reinterpret_cast<const LDS_AS at_u32x4*>(p); }
// Two dwords (4 elements) of column l % 16 of 4 rows x 16 columns, from the
// 8 bytes that each of 16 lanes points at.
__device__ __forceinline__ at_u32x2 transpose_from_lds(const Lds16* src) {
  typedef short s4 __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(at_u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS s4*)src));
}

// ONE: the page size is a multiple of 16, so that 16 tokens from a multiple of
// 16 lie on one page, and one lookup serves the wave that stages them.
template <class T, int D, int E, bool ONE>
__global__ void __launch_bounds__(256, D == 256 ? 1 : 2) prefill_kernel(AttnArgs a, PrefillWork w) {
  constexpr int kChunks = D / 8;                  // 16-byte chunks of a row of 16-bit elements
  constexpr int kLoads = kChunks * E / 8;         // 16-byte loads per thread and tensor: 64 rows x D x E bytes
  constexpr int kSteps = D / 16;                  // score MFMAs per 32 tokens
  constexpr int kBlocks = D / 32;                 // value blocks
  // Two tiles of keys, two of values, and three words.  One object: with several,
  // the compiler no longer sees that copies into one tile leave the others alone,
  // and waits for them before every read.
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
  const int used = min(w.splits, max(tiles / 4, 1));      // a split has at least 4 tiles
  if (split >= used) return;
  if (w.splits > 1 && split == 0 && threadIdx.x == 0) w.used[ti * a.kv.heads + head] = used;
  const int t0 = int(int64_t(tiles) * split / used), t1 = int(int64_t(tiles) * (split + 1) / used);

  const float cs = a.scale_log2 * (E == 1 && a.kv.k_scale ? a.kv.k_scale[head] : 1.0f);
  const int32_t* table = a.kv.tables + rt.seq * a.kv.table_stride;
  const uint8_t* kbase = static_cast<const uint8_t*>(a.kv.k) + head * a.kv.head_stride * E;
  const uint8_t* vbase = static_cast<const uint8_t*>(a.kv.v) + head * a.kv.head_stride * E;

  at_u32x4 q[kSteps];
  {
    const uint16_t* qp = static_cast<const uint16_t*>(a.q) + int64_t(min(max(qi, 0), w.tokens - 1)) * a.q_row +
                         (int64_t(head) * a.group + in_group) * a.q_head + 8 * half;
#pragma unroll
    for (int j = 0; j < kSteps; ++j) q[j] = *reinterpret_cast<const at_u32x4*>(qp + 16 * j);
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
  constexpr int kRowLoads = D * E / 16, kRows = 64 / kRowLoads;      // rows of one load
  auto load_row = [&](int j) { return j * kRows + lane / kRowLoads; };           // of the wave's 16
  auto chunk = [&](int j, bool v) {
    const int r = 16 * wave + load_row(j), c = lane % kRowLoads;
    return E == 1 ? c : c ^ (v ? value_swz<D>(r) : key_swz<D>(r));
  };
  // Where the rows are.  Lane l looks up one page for the tiles ahead: the wave's
  // 16 tokens of tile t + l if they lie on one page (ONE), or its token l % 16 of
  // tile t + l / 16.  So one load of the table serves 64 or 4 tiles.  Tokens past
  // the end take the last one's place, and an entry outside the cache is read as
  // page 0 and spoils the workgroup's rows if any of them may see a token there.
  constexpr int kAhead = ONE ? 64 : 4;
  bool bad = false;
  int64_t where = 0;          // byte offset of the lane's row
  auto look_ahead = [&](int t) {
    const int tl = min(t + (ONE ? lane : lane >> 4), t1 - 1);
    int stop;
    const int tk = tile_at(tl, &stop) + 16 * wave + (ONE ? 0 : lane & 15);
    const int u = min(tk, ONE ? (stop - 1) & ~15 : stop - 1), i = a.kv.page.div(u);
    const int slot = u - i * int(a.kv.page.d), p = table[i];
    const bool good = uint32_t(p) < uint32_t(a.kv.pages);
    bad |= !good && tk < stop && (min(tk + (ONE ? 16 : 1), stop) > low || tk < a.sinks);
    where = (int64_t(good ? p : 0) * a.kv.page_stride + int64_t(slot) * a.kv.token_stride) * E;
  };
  // ONE: what a lane reads is at a fixed offset from the first token's row.
  uint32_t koff[kLoads], voff[kLoads];
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    const uint32_t row = ONE ? uint32_t(load_row(j)) * uint32_t(a.kv.token_stride * E) : 0;
    koff[j] = row + 16 * chunk(j, false);
    voff[j] = row + 16 * chunk(j, true);
  }
  at_u32x4 raw_k[E == 1 ? kLoads : 1], raw_v[E == 1 ? kLoads : 1];
  auto load = [&](Lds16* kt, Lds16* vt, int t) {
    const int n = (t - t0) % kAhead;
    if (n == 0) look_ahead(t);
    const int lo = int(where), hi32 = int(where >> 32);
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      int64_t at;
      if constexpr (ONE) {
        at = int64_t(uint32_t(__builtin_amdgcn_readlane(lo, n))) | int64_t(__builtin_amdgcn_readlane(hi32, n)) << 32;
      } else {
        const int from = 16 * n + load_row(j);
        at = int64_t(uint32_t(__shfl(lo, from))) | int64_t(__shfl(hi32, from)) << 32;
      }
      const uint8_t* k = kbase + at + koff[j];
      const uint8_t* v = vbase + at + voff[j];
      if constexpr (E == 2) {
        copy_to_lds(k, kt + (wave * kLoads + j) * 64 * 8);
        copy_to_lds(v, vt + (wave * kLoads + j) * 64 * 8);
      } else {
        raw_k[j] = *reinterpret_cast<const at_u32x4*>(k);
        raw_v[j] = *reinterpret_cast<const at_u32x4*>(v);
      }
    }
  };
  // A tile that every row sees whole needs no masks.
  auto whole = [&](int t) {
    int stop;
    const int base = tile_at(t, &stop);
    return base + kBN <= stop && base + kBN - 1 <= pos_min &&
           (!a.window || base > pos_max - a.window || base + kBN <= a.sinks);
  };
  // Completes a tile.  In one that some row does not see whole, the wave that
  // staged the values clears those past the end (whatever the page holds there)
  // and looks for Inf and NaN among the others.
  auto arrive = [&](Lds16* kt, Lds16* vt, int buf, int t) {
    if constexpr (E == 2) {
      __builtin_amdgcn_s_waitcnt(0x0f70);      // vmcnt(0)
    } else {
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const int r = 16 * wave + load_row(j), c = chunk(j, false);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const uint32_t k0 = raw_k[j][2 * s], k1 = raw_k[j][2 * s + 1], v0 = raw_v[j][2 * s], v1 = raw_v[j][2 * s + 1];
          *reinterpret_cast<LDS_AS at_u32x4*>(kt + r * D + 8 * ((2 * c + s) ^ key_swz<D>(r))) =
              (at_u32x4){e4m3_pair<T, false>(k0), e4m3_pair<T, true>(k0), e4m3_pair<T, false>(k1), e4m3_pair<T, true>(k1)};
          *reinterpret_cast<LDS_AS at_u32x4*>(vt + r * D + 8 * ((2 * c + s) ^ value_swz<D>(r))) =
              (at_u32x4){e4m3_pair<T, false>(v0), e4m3_pair<T, true>(v0), e4m3_pair<T, false>(v1), e4m3_pair<T, true>(v1)};
        }
      }
    }
    if (!whole(t)) {
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
    __syncthreads();
  };

  at_f32x16 o[kBlocks];
#pragma unroll
  for (int n = 0; n < kBlocks; ++n)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[n][e] = 0.0f;
  float m = kNegInf, l = 0.0f;

  auto sees = [&](int t, int stop) {
    return t < stop && t <= pos && (!a.window || t > pos - a.window || t < a.sinks);
  };
  // value operand: block n (32 d's), 16 tokens from tb: two transposing reads of
  // 4 tokens x 16 d's per 16 lanes
  auto value = [&](const Lds16* vt, int n, int tb) {
    const int i = lane & 15, d = 32 * n + 16 * ((lane >> 4) & 1) + 4 * (i & 3);
    at_u32x4 x;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int r = tb + 8 * s + 4 * half + (i >> 2);
      const at_u32x2 y = transpose_from_lds(vt + r * D + 8 * ((d >> 3) ^ value_swz<D>(r)) + (d & 4));
      x[2 * s] = y.x;
      x[2 * s + 1] = y.y;
    }
    return x;
  };
  // Scores of tile t: register e of block b is the token 32 b + 8 (e / 4) + 4
  // half + e % 4 of the tile.
  auto scores = [&](const Lds16* kt, int t, at_f32x16 (&s)[2]) {
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int e = 0; e < 16; ++e) s[b][e] = 0.0f;
#pragma unroll
    for (int j = 0; j < kSteps; ++j)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int r = 32 * b + col;
        s[b] = T::mfma32(read16(kt + r * D + 8 * ((2 * j + half) ^ key_swz<D>(r))), q[j], s[b]);
      }
    if (!whole(t)) {
      // A bit for each of the 64 tokens, counted from this half's first one: from
      // <= token < to, or a sink.
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
    }
  };
  // Scores to weights, with the running maximum and sum.
  auto weights = [&](at_f32x16 (&s)[2]) {
    float mx = s[0][0];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int e = 0; e < 16; ++e) mx = fmaxf(mx, s[b][e]);
    mx = max_xor32(mx) * cs;
    // The sums are rebased only where a maximum has grown by more than 2^8: until
    // then weights go up to 2^8, which costs neither type any accuracy.
    if (__any(mx > m + 8.0f)) {
      const float mn = fmaxf(m, mx), f = rebase(m, mn);
#pragma unroll
      for (int n = 0; n < kBlocks; ++n) o[n] *= f;
      l *= f;
      m = mn;
    }
    const float mm = m == kNegInf ? 0.0f : m;
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        s[b][e] = exp2_fast(__builtin_fmaf(s[b][e], cs, -mm));
        l += s[b][e];
      }
  };
  // Inf or NaN in a tile that some row does not see whole: 0 x Inf would reach
  // the row's sum.  The rows that see such a value get it added, then it is
  // cleared in the tile.  (All waves get here together: the flag is the tile's.)
  auto settle_odd = [&](Lds16* vt, int t) {
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
  auto values = [&](const Lds16* vt, const at_f32x16 (&s)[2]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      at_u32x4 p;        // weights of the tokens 16 i .. 16 i + 15
#pragma unroll
      for (int k = 0; k < 4; ++k) p[k] = T::pack(s[i >> 1][8 * (i & 1) + 2 * k], s[i >> 1][8 * (i & 1) + 2 * k + 1]);
#pragma unroll
      for (int n = 0; n < kBlocks; ++n) o[n] = T::mfma32(value(vt, n, 16 * i), p, o[n]);
    }
  };

  // One step: start the copies of tile t + 1 into `nk`, `nv`, and take tile t from
  // `ck`, `cv`.  That they are different memory is what lets the reads go on while
  // the copies are in flight.
  auto tile_step = [&](Lds16* __restrict__ ck, Lds16* __restrict__ cv, Lds16* __restrict__ nk, Lds16* __restrict__ nv,
                       int t, int buf) {
    if (t + 1 < t1) load(nk, nv, t + 1);
    at_f32x16 s[2];
    scores(ck, t, s);
    weights(s);
    if (flags[buf] == t) settle_odd(cv, t);
    values(cv, s);
  };

  Lds16* const lk = (Lds16*)smem;
  Lds16* const lv = lk + 2 * kBN * D;
  if (t0 < t1) {
    load(lk, lv, t0);
    arrive(lk, lv, 0, t0);
    for (int t = t0; t < t1; ++t) {
      const int buf = (t - t0) & 1, cur = buf * kBN * D, nxt = kBN * D - cur;
      tile_step(lk + cur, lv + cur, lk + nxt, lv + nxt, t, buf);
      if (t + 1 < t1) arrive(lk + nxt, lv + nxt, buf ^ 1, t + 1);
    }
  }
  if (bad) flags[kBad] = 1;
  __syncthreads();
  l = sum_xor32(l);
  if (flags[kBad]) l = __builtin_nanf("");

  if (w.splits > 1 && used > 1) {
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

// Joins the splits of a row tile: grid (row tiles x heads, kBM / 8); a
// workgroup joins 8 rows, 32 threads each.
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
  float M = kNegInf;
  for (int i = 0; i < used; ++i) M = fmaxf(M, base[int64_t(i) * kBM * (D + 2) + kBM * D + r]);
  float L = 0.0f, O[D / 32];
#pragma unroll
  for (int j = 0; j < D / 32; ++j) O[j] = 0.0f;
#pragma unroll 4
  for (int i = 0; i < used; ++i) {
    const float* p = base + int64_t(i) * kBM * (D + 2);
    const float f = rebase(p[kBM * D + r], M);
    L += f * p[kBM * (D + 1) + r];
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
      const at_f32x2 x = *reinterpret_cast<const at_f32x2*>(p + r * D + 64 * j + 2 * lane);
      O[2 * j] += f * x.x;
      O[2 * j + 1] += f * x.y;
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
// row tiles alone leave CUs without work.
int key_splits(int64_t tiles, int heads) {
  const int64_t wgs = tiles * heads;
  return wgs >= 256 ? 1 : int(std::min<int64_t>((512 + wgs - 1) / wgs, 64));
}

template <class T, int D, int E>
hipError_t launch(const AttnArgs& a, const PrefillWork& w, hipStream_t stream) {
  const unsigned tiles = unsigned(w.row_tiles * a.kv.heads);
  // (a lane's offset from the first of 16 tokens is kept in 32 bits)
  if (a.kv.page.d % 16 == 0 && a.kv.token_stride < (1 << 26))
    prefill_kernel<T, D, E, true><<<tiles * unsigned(w.splits), 256, 0, stream>>>(a, w);
  else
    prefill_kernel<T, D, E, false><<<tiles * unsigned(w.splits), 256, 0, stream>>>(a, w);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || w.splits == 1) return e;
  prefill_join_kernel<T, D, E><<<dim3(tiles, kBM / 8), 256, 0, stream>>>(a, w);
  return hipGetLastError();
}

template <class T, int E>
hipError_t launch_dim(const AttnArgs& a, const PrefillWork& w, int D, hipStream_t stream) {
  if (D == 64) return launch<T, 64, E>(a, w, stream);
  if (D == 128) return launch<T, 128, E>(a, w, stream);
  return launch<T, 256, E>(a, w, stream);
}

}  // namespace

// [parts] [used]
size_t attn_prefill_workspace(int64_t seqs, int64_t tokens, int q_heads, int heads, int head_dim) {
  const int64_t tiles = row_tiles(seqs, tokens, q_heads / heads);
  const int splits = key_splits(tiles, heads);
  if (splits == 1) return 0;
  return size_t(tiles * heads) * (size_t(splits) * kBM * (head_dim + 2) * 4 + 4);
}

hipError_t launch_attn_prefill(const AttnArgs& a, const int32_t* cu, int64_t tokens, int cache_dtype, int dtype,
                               int head_dim, void* workspace, hipStream_t stream) {
  PrefillWork w;
  w.cu = cu;
  w.tokens = int32_t(tokens);
  w.row_tiles = int32_t(row_tiles(a.kv.seqs, tokens, a.group));
  w.splits = key_splits(w.row_tiles, a.kv.heads);
  w.group = fast_div(uint32_t(a.group));
  w.parts = static_cast<float*>(workspace);
  w.used = reinterpret_cast<int32_t*>(w.parts + size_t(w.row_tiles) * a.kv.heads * w.splits * kBM * (head_dim + 2));
  const bool e4m3 = cache_dtype == W4A4_E4M3;
  if (dtype == W4A4_BF16)
    return e4m3 ? launch_dim<Bf16, 1>(a, w, head_dim, stream) : launch_dim<Bf16, 2>(a, w, head_dim, stream);
  return e4m3 ? launch_dim<F16, 1>(a, w, head_dim, stream) : launch_dim<F16, 2>(a, w, head_dim, stream);
}

}  // namespace w4a4
