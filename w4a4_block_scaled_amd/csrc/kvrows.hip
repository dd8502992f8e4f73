// Rows of queries, keys and values on their way between a projection and the
// paged cache: the rotation by their positions, alone or with the storing into
// a cache of 16, 8 or 4 bits, and rows read out of a cache.
//
// All of it moves bytes.  Measured: queries of 8191 tokens, 134 MB, 22.2 us (they fit the
// last cache in part); keys, values and queries of 14449 tokens into 4 bits, 245 MB, 51 us, 4.8
// TB/s (a copy of the queries alone by torch 36, by this kernel 34); out of 4 bits 162 MB in
// 28 us.  Small calls are their launch and the chain of lookups behind it: 3.2 us for 16
// tokens, 4.2 with a cache.  In between the vector unit counts, some 350 instructions per
// row of keys and wave: 1795 tokens of 16 / 16 heads of 64 into E4M3, 18 MB, 11.7 us
// (by random scales; see rows_in_kernel for those that are powers of two).
#include <algorithm>
#include <type_traits>

#include "attn_common.h"
#include "mx_quant.h"

namespace w4a4 {
namespace {

// The angle position * freq as a quarter turn's number (mod 4) and the rest x in radians,
// |x| <= pi / 4, in 64 bits: the product of a 31-bit and a 24-bit number is off by 2^-53 of
// itself at most, 1 / (2 pi) is taken in two parts, so the angle of position 2^31 - 1 is
// right to 1e-6 of a turn and that of position 131071 to 2^-48.
struct Angle {
  double x;
  int quarter;
};
__device__ __forceinline__ Angle angle_of(int pos, float freq) {
  constexpr double kInv = 0x1.45f306dc9c883p-3, kInvRest = -0x1.6b01ec5417056p-57;      // 1 / (2 pi)
  const double a = double(pos) * double(freq);
  const double t = a * kInv, rest = __builtin_fma(a, kInv, -t) + a * kInvRest;
  const double u = 4.0 * ((t - __builtin_rint(t)) + rest), k = __builtin_rint(u);
  return {(u - k) * 0x1.921fb54442d18p+0, int(k) & 3};
}
// cos and sin by the Taylor series around the quarter turn, in fp64 right to 2^-50, in fp32
// to 1.3 * 2^-24 and to 2.2 * 2^-24 of themselves; times factor, to 2^-24 of the product.
static __device__ const double kSeries[14] = {
    -1.0 / 1307674368000.0, 1.0 / 6227020800.0, -1.0 / 39916800.0, 1.0 / 362880.0, -1.0 / 5040.0, 1.0 / 120.0,
    -1.0 / 6.0, -1.0 / 87178291200.0, 1.0 / 479001600.0, -1.0 / 3628800.0, 1.0 / 40320.0, -1.0 / 720.0, 1.0 / 24.0,
    -0.5};
template <typename R>
struct Turn {
  R cos, sin;
};
template <typename R>
__device__ __forceinline__ Turn<R> turn_of(int pos, float freq, float factor, bool inverse) {
  const Angle a = angle_of(pos, freq);
  const R x = R(a.x), z = x * x;
  R s, c;
  if constexpr (sizeof(R) == 8) {
    // from memory, read here: as literals they would be kept in registers all along
    const double* k = kSeries;
    asm volatile("" : "+s"(k));
    s = k[0];
    c = k[7];
#pragma unroll
    for (int i = 1; i < 7; ++i) s = __builtin_fma(s, z, k[i]);
#pragma unroll
    for (int i = 8; i < 14; ++i) c = __builtin_fma(c, z, k[i]);
    s = __builtin_fma(s * z, x, x);
    c = __builtin_fma(c, z, R(1.0));
  } else {
    s = R(1.0 / 362880.0);            // x^11 / 11! <= 2^-28.8
    c = R(-1.0 / 3628800.0);          // x^12 / 12! <= 2^-33
    c = __builtin_fmaf(c, z, R(1.0 / 40320.0));
    s = __builtin_fmaf(s, z, R(-1.0 / 5040.0));
    c = __builtin_fmaf(c, z, R(-1.0 / 720.0));
    s = __builtin_fmaf(s, z, R(1.0 / 120.0));
    c = __builtin_fmaf(c, z, R(1.0 / 24.0));
    s = __builtin_fmaf(s, z, R(-1.0 / 6.0));
    c = __builtin_fmaf(c, z, R(-0.5));
    s = __builtin_fmaf(s * z, x, x);
    c = __builtin_fmaf(c, z, R(1.0));
  }
  R cq = a.quarter & 1 ? s : c, sq = a.quarter & 1 ? c : s;
  if (a.quarter == 1 || a.quarter == 2) cq = -cq;
  if (a.quarter >= 2) sq = -sq;
  if (inverse) sq = -sq;
  return {cq * factor, sq * factor};
}

// fp64 -> fp32, inexact results to the neighbour with an odd last bit: a later
// rounding to fewer bits is then that of the fp64 value.
__device__ __forceinline__ float to_odd(double d) {
  const float f = float(d);
  uint32_t b = __float_as_uint(f);
  if (double(f) != d && !(b & 1)) b += __builtin_fabs(d) > double(__builtin_fabsf(f)) ? 1 : -1;
  return __uint_as_float(b);
}

// Where a token of a call is: its place in its sequence, and its page.
struct Place {
  int in;             // it belongs to a sequence
  int pos, page, slot;       // page -1: none
};

// The place of row i (lane l's own; every lane of the wave calls it, active: those with
// one, of consecutive rows).  Up to 63 sequences take one load of cu and lens: the
// sequence of a row is the last one that begins at or before it.
__device__ __forceinline__ Place place_of(const KvView& kv, const int32_t* cu, int i, bool active) {
  const int lane = threadIdx.x & 63;
  Place x = {active && i < kv.seqs, 0, -1, 0};
  int s = i, back = 1, len = 0;      // back: rows from this one to the sequence's last, inclusive
  if (cu && kv.seqs < 64) {
    const int begin = cu[min(lane, kv.seqs)], length = kv.lens[min(lane, kv.seqs - 1)];
    s = -1;
    for (uint64_t todo = __ballot(active); todo; todo &= todo - 1) {
      const int l = __ffsll((unsigned long long)todo) - 1;
      const int row = __builtin_amdgcn_readlane(i, l);
      const int at = __popcll(__ballot(lane < kv.seqs && begin <= row)) - 1;
      if (lane == l) s = at;
    }
    back = __shfl(begin, s + 1) - i;
    len = __shfl(length, max(s, 0));
    x.in = active && s >= 0 && back > 0;
  } else if (active) {
    if (cu) {
      s = find_seq(cu, kv.seqs, i);
      back = cu[s + 1] - i;
      x.in = back > 0 && cu[s] <= i;
    }
    if (x.in) len = kv.lens[s];
  }
  if (!x.in) return x;
  const int64_t pos = int64_t(len) - back;
  x.pos = int(max(pos, int64_t(INT32_MIN)));
  if (pos >= 0) x.page = kv_page(kv, kv.tables + s * kv.table_stride, int(pos), &x.slot);
  return x;
}
__device__ __forceinline__ Place shuffled(const Place& x, int from) {
  return {__shfl(x.in, from), __shfl(x.pos, from), __shfl(x.page, from), __shfl(x.slot, from)};
}

// y / s, from inv = 1 / s, as an E4M3 conversion takes it: fp32 with the last bit odd where
// it is not exact (a quotient of few bits comes out as it, and none becomes one), saturated
// at +-448, NaN kept.
__device__ __forceinline__ float e4m3_quotient(double y, double s, double inv) {
  const double q0 = y * inv, q = __builtin_fma(__builtin_fma(-q0, s, y), inv, q0);
  const float f = float(q0), z = q != q ? f : to_odd(q);        // Inf leaves a NaN behind
  return z != z ? z : fminf(fmaxf(z, -448.0f), 448.0f);
}

constexpr int kAlone = -1;        // CACHE: none
constexpr int kKeys = 1, kValues = 2, kQueries = 4;      // what a workgroup takes
constexpr int kNone = 0, kHalf = 1, kPairs = 2, kHalfAny = 3;      // how the pairs lie
constexpr int kTable = 1024;      // angles of a workgroup's tokens
constexpr int kFlight = 4;        // vectors (one head of one token) in flight per thread

// How 8 consecutive elements of a row, from d, turn: y = x * c + w * s, w the element's
// partner in its pair, s with the sign that this side has; bit e of `turned` for element e.
template <int STYLE>
struct Turn8 {
  static constexpr int kOwn = STYLE == kPairs ? 4 : 8;       // pairs that the elements lie in
  float c[kOwn], s[kOwn];
  uint32_t turned;
};
// Where the angle of pair p lies in LDS: the pairs of one thread a row apart, so that the
// threads of a vector read side by side.
template <int STYLE>
__device__ __forceinline__ int slot_of(int p, int pairs) {
  if (STYLE == kPairs) return (p & 3) * ((pairs + 3) >> 2) + (p >> 2);
  if (STYLE == kHalf) return (p & 7) * (pairs >> 3) + (p >> 3);
  return p;
}
template <int STYLE>
__device__ __forceinline__ int slots_of(int pairs) { return STYLE == kPairs ? (pairs + 3) & ~3 : pairs; }

template <int STYLE>
__device__ __forceinline__ Turn8<STYLE> turns_at(const float2* tab, int d, int pairs) {
  Turn8<STYLE> t;
  t.turned = 0;
  if constexpr (STYLE == kPairs) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int p = (d >> 1) + k;
      const float2 x = tab[slot_of<STYLE>(min(p, pairs - 1), pairs)];
      t.c[k] = x.x;
      t.s[k] = x.y;
      if (p < pairs) t.turned |= 3u << (2 * k);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = d + e, p = i < pairs ? i : min(i - pairs, pairs - 1);
      const float2 x = tab[slot_of<STYLE>(p, pairs)];
      t.c[e] = x.x;
      t.s[e] = i < pairs ? -x.y : x.y;
      if (i < 2 * pairs) t.turned |= 1u << e;
    }
  }
  return t;
}
template <class T, typename R>
__device__ __forceinline__ void widen8(at_u32x4 own, R (&y)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = e & 1 ? T::high(own[e >> 1]) : T::low(own[e >> 1]);
}
// The elements own, with their partners' elements other (kHalf) or their row (kHalfAny), in
// fp32.  y is right to 4 * 2^-24 (|x| + |w|) factor: of |w| factor the error of s, and 2^-24 |s|
// each for the factor, the product and the sum, 3.6 * 2^-24 at most together; of |x| less.
// It is also right to 5.5 * 2^-24 (|x c| + |w s|): 2.2 of s itself and those three.
// SIZES: size becomes |x| |c| + |w| |s|, 0 for an element that stays as it is.
template <class T, int STYLE, bool SIZES = false>
__device__ __forceinline__ void turn8(at_u32x4 own, at_u32x4 other, const uint16_t* row, int d, int pairs,
                                      const Turn8<STYLE>& t, float (&y)[8], float* size = nullptr) {
  widen8<T>(own, y);
  if constexpr (SIZES) {
#pragma unroll
    for (int e = 0; e < 8; ++e) size[e] = 0.0f;
  }
  if (!t.turned) return;
  float w[8], z[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if (STYLE == kPairs) w[e] = y[e ^ 1];
    else if (STYLE == kHalf) w[e] = e & 1 ? T::high(other[e >> 1]) : T::low(other[e >> 1]);
    else w[e] = t.turned >> e & 1 ? T::low(row[d + e < pairs ? d + e + pairs : d + e - pairs]) : 0.0f;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float c = t.c[STYLE == kPairs ? e >> 1 : e], s = t.s[STYLE == kPairs ? e >> 1 : e];
    z[e] = __builtin_fmaf(y[e], c, w[e] * (STYLE == kPairs && !(e & 1) ? -s : s));
    if (SIZES && (STYLE == kHalf || t.turned >> e & 1))
      size[e] = __builtin_fmaf(__builtin_fabsf(y[e]), __builtin_fabsf(c), __builtin_fabsf(w[e] * s));
  }
  if (STYLE == kHalf || t.turned == 0xff) {
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = z[e];
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = t.turned >> e & 1 ? z[e] : y[e];
  }
}
// Largest magnitude of 8 elements, as their type's bits (Inf and NaN above all others).
__device__ __forceinline__ uint32_t top_bits(at_u32x4 u) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  u16x2 m = {0, 0};
#pragma unroll
  for (int k = 0; k < 4; ++k) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, u[k] & 0x7fff7fffu));
  return max(uint32_t(m.x), uint32_t(m.y));
}

__device__ __forceinline__ uint32_t e4m3_codes(const float (&z)[4]) {
  const int p = __builtin_amdgcn_cvt_pk_fp8_f32(z[0], z[1], 0, false);
  return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(z[2], z[3], p, true));
}

// quant8_mx's codes and scale byte of 8 values of a 32-block that are known to within `off`
// (of this lane's); false where that leaves more than one answer, or values are not ordinary ones.
template <int E_MAX>
__device__ __forceinline__ bool quant8_sure(const float (&y)[8], float off, uint32_t& codes, uint32_t& scale) {
  float top = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = fmaxf(top, __builtin_fabsf(y[e]));
  top = fmaxf(top, quad_xor1(top));
  top = fmaxf(top, quad_xor2(top));
  off = fmaxf(off, quad_xor1(off));
  off = fmaxf(off, quad_xor2(off));
  const int field = int(__float_as_uint(top) >> 23);
  const int e = min(field - 129, E_MAX);
  scale = uint32_t(e + 127);
  const float unit = __uint_as_float(uint32_t(127 - e) << 23), room = off * unit;
  float lo[8], hi[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo[i] = __builtin_fmaf(y[i], unit, -room);
    hi[i] = __builtin_fmaf(y[i], unit, room);
  }
  uint32_t above = 0;
  codes = 0;
  codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, lo[0], lo[1], 1.0f, 0);
  codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, lo[2], lo[3], 1.0f, 1);
  codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, lo[4], lo[5], 1.0f, 2);
  codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, lo[6], lo[7], 1.0f, 3);
  above = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(above, hi[0], hi[1], 1.0f, 0);
  above = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(above, hi[2], hi[3], 1.0f, 1);
  above = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(above, hi[4], hi[5], 1.0f, 2);
  above = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(above, hi[6], hi[7], 1.0f, 3);
  return codes == above && field > 30 && field < 240 && off < 0x1p100f &&
         __float_as_uint(top - off) >> 23 == __float_as_uint(top + off) >> 23;
}

template <class T>
__device__ __forceinline__ at_u32x4 pack8(const float (&y)[8]) {
  return (at_u32x4){T::pack(y[0], y[1]), T::pack(y[2], y[3]), T::pack(y[4], y[5]), T::pack(y[6], y[7])};
}

// The workgroups of a launch, in up to three parts by what they take: from where on, and
// of each part the tokens of a workgroup and the workgroups that share those.
struct Parts {
  int count, kinds[3], begin[3], tok_bits[3], splits[3];
};

// A workgroup takes queries, keys and values, or one kind of them, of per_wg tokens, a
// power of two, so that every thread has one token and one chunk of 8 elements, and
// walks over its share of the heads.  The first rows'
// loads start first; meanwhile the tokens are looked up, and
// the cos and sin of all their pairs computed once and handed out through LDS: a thread
// keeps those of its elements for all its vectors.
//
// What is kept in 16 bits is rotated in fp32.  Keys on their way to 8 or 4 bits, and
// quotients by E4M3's scales, are rounded from the values themselves, not from an fp32
// rounding of them: in fp32 they are known to within a bound; where both ends of that
// give the same codes these are the right ones, else the wave takes its 512 values again in
// fp64.  Of random ones by a scale that is no power of two that is one wave in 50 (turned
// keys into 8 bits), 100 (into 4 bits) or 200 (values into 8 bits).  In doubt are also
//  - ties, which quotients by a power of two often are: a value in 16 (BF16) or 128 (FP16),
//    that is nearly every wave of values and of keys that turn in part, also without scales
//    (1795 tokens of 16 / 16 heads of 64 into E4M3: a quarter of the head turned 18.3 us, 11.5
//    to 12.6 by other scales; all of it 14.1 and 12.4 to 12.9; by graph replay)
//  - zeros, for their sign: of E4M3's negative ones, and of turned pairs or blocks into 4
//    bits (14449 tokens, 28 / 4 heads of 128: none 61 us, half of the rows 77, all 95; one
//    value in a hundred 62).
// FLIGHT: vectors in flight per thread, 1 where none has more than one of a kind: the code
// that the unrolled steps would skip has to be read too (1795 tokens of 16 / 16 heads of 64
// into E4M3 11.8 us, 12.7 with 4; into FP16 8.1 and 9.4).
template <class T, int CACHE, int STYLE, int FLIGHT>
__global__ void __launch_bounds__(256) rows_in_kernel(RowsIn a, Parts parts, int lane_bits, FastDiv by_pairs) {
  constexpr bool SMALL = CACHE == W4A4_E4M3 || CACHE == W4A4_E2M1;
  __shared__ float2 tab[STYLE ? kTable : 1];
  const int block = blockIdx.x;
  int part = 0;
  if (CACHE != kAlone && parts.count > 1)
    part = block < parts.begin[1] ? 0 : parts.count == 2 || block < parts.begin[2] ? 1 : 2;
  const int kinds = CACHE == kAlone ? kQueries : parts.kinds[part];
  const int tok_bits = parts.tok_bits[part], splits = parts.splits[part];
  const int at_block = block - parts.begin[part], bx = at_block / splits, by = at_block - bx * splits;
  const int lanes = 1 << lane_bits, group = threadIdx.x >> lane_bits;
  const int d = 8 * (threadIdx.x & (lanes - 1));
  const int per_wg = 1 << tok_bits, tok = group & (per_wg - 1);
  const int phases = (256 >> lane_bits >> tok_bits) * splits;
  const int first = by * (256 >> lane_bits >> tok_bits) + (group >> tok_bits);
  const int64_t row0 = int64_t(bx) << tok_bits, i = row0 + tok;
  const int pairs = a.rot >> 1;
  const bool here = i < a.tokens && d < a.dim;

  // Rows on their way: the heads h, h + phases, ... from `p` on.
  struct Rows {
    const uint16_t* p;
    int64_t step;
    int h, heads;
    at_u32x4 own[FLIGHT], other[FLIGHT];
  };
  const int partner = d < pairs ? d + pairs : d - pairs;
  auto rows_of = [&](const void* base, int64_t row, int64_t head, int h, int heads) {
    Rows r;
    r.p = static_cast<const uint16_t*>(base) + i * row + h * head;
    r.step = phases * head;
    r.h = h;
    r.heads = heads;
    return r;
  };
  auto load = [&](Rows& r, bool turns) {
#pragma unroll
    for (int j = 0; j < FLIGHT; ++j)
      if (here && r.h + j * phases < r.heads) {
        const uint16_t* p = r.p + j * r.step;
        r.own[j] = *reinterpret_cast<const at_u32x4*>(p + d);
        if (STYLE == kHalf && turns && d < a.rot) r.other[j] = *reinterpret_cast<const at_u32x4*>(p + partner);
      }
  };
  auto advance = [&](Rows& r) {
    r.p += FLIGHT * r.step;
    r.h += FLIGHT * phases;
  };
  Rows rows = kinds & kQueries ? rows_of(a.q, a.q_row, a.q_head, first, a.q_heads)
              : kinds & kKeys  ? rows_of(a.k, a.k_row, a.k_head, first, a.kv.heads)
                               : rows_of(a.v, a.v_row, a.v_head, first, a.kv.heads);
  load(rows, kinds != kValues);

  // every wave looks up all tokens of the workgroup, lane l token l
  const int lane = threadIdx.x & 63;
  const bool active = lane < per_wg && row0 + lane < a.tokens;
  Place mine = {active, 0, -1, 0};
  int turn = 0;
  float freq0 = 0.0f;         // of the thread's first angle
  if (STYLE != kNone && int(threadIdx.x) < pairs << tok_bits)
    freq0 = a.freqs[int(threadIdx.x) - by_pairs.div(threadIdx.x) * pairs];
  if (a.positions && active) turn = a.positions[row0 + lane];
  if constexpr (CACHE != kAlone) {
    mine = place_of(a.kv, a.cu, int(row0) + lane, active);
    if (!a.positions) turn = mine.pos;
  }
  Turn8<STYLE> turns;
  if (STYLE != kNone && kinds != kValues) {
    const int angles = pairs << tok_bits;
    for (int e0 = 0; e0 < angles; e0 += 256) {
      const int e = e0 + threadIdx.x, t = by_pairs.div(e), p = e - t * pairs;
      const int pos = __shfl(turn, t & 63);
      if (e < angles) {
        const Turn<float> x = turn_of<float>(pos, e0 ? a.freqs[p] : freq0, a.factor, a.inverse);
        tab[t * slots_of<STYLE>(pairs) + slot_of<STYLE>(p, pairs)] = {x.cos, x.sin};
      }
    }
    __syncthreads();
    turns = turns_at<STYLE>(tab + tok * slots_of<STYLE>(pairs), d, pairs);
  }
  const Place at = shuffled(mine, tok);
  const int my_turn = __shfl(turn, tok);
  if (!here || !at.in) return;

  if (kinds & kQueries) {
    uint16_t* out = static_cast<uint16_t*>(a.out) + i * a.o_row + first * a.o_head + d;
    const int64_t out_step = phases * a.o_head;
    while (rows.h < rows.heads) {
#pragma unroll
      for (int j = 0; j < FLIGHT; ++j)
        if (rows.h + j * phases < rows.heads) {
          float y[8];
          if constexpr (STYLE != kNone)
            turn8<T, STYLE>(rows.own[j], rows.other[j], rows.p + j * rows.step, d, pairs, turns, y);
          // out may be q itself: every lane of the row has read its partners
          if (STYLE == kHalfAny) __builtin_amdgcn_wave_barrier();
          *reinterpret_cast<at_u32x4*>(out + j * out_step) = pack8<T>(y);
        }
      out += FLIGHT * out_step;
      advance(rows);
      if (rows.h < rows.heads) load(rows, true);
    }
  }
  if (CACHE == kAlone || kinds == kQueries || at.page < 0) return;

  // where the row's element d of head `first` goes
  const int64_t page = at.page * a.kv.page_stride;
  const int64_t to = page + at.slot * a.kv.token_stride;
  const int64_t scale_to = page + a.kv.scale_at + (d >> 5) * int64_t(a.kv.page.d) + at.slot;
  auto store_all = [&](Rows& r, void* cache, const float* scales, auto which) {
    constexpr bool KEY = decltype(which)::value && STYLE != kNone;      // turned
    uint8_t* const base = static_cast<uint8_t*>(cache);
    // Stores a row of 16 bits, or its codes; whether (in any lane) these are in doubt.
    auto take = [&](int head, const at_u32x4& own, const at_u32x4& other, const uint16_t* row) {
      const int64_t there = to + head * a.kv.head_stride;
      float y[8];
      if constexpr (!SMALL) {
        at_u32x4 z = own;
        if constexpr (KEY) {
          turn8<T, STYLE>(own, other, row, d, pairs, turns, y);
          z = pack8<T>(y);
        }
        *reinterpret_cast<at_u32x4*>(base + (there + d) * 2) = z;
        return false;
      }
      if constexpr (CACHE == W4A4_E4M3) {
        float size[8];
        if constexpr (KEY) turn8<T, STYLE, true>(own, other, row, d, pairs, turns, y, size);
        else widen8<T>(own, y);
        const float f = scales ? scales[head] : 1.0f, inv = 1.0f / f;
        at_u32x2 codes, above;
        float top = 0.0f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float lo[4], hi[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            // y is off by 5.5 * 2^-24 of its size, the quotient by 2 * 2^-24 of itself, and the bounds'
            // ends are rounded by 2^-24 of it: 2^-21 of both
            const float q = y[4 * k + e] * inv;
            const float room = KEY ? __builtin_fmaf(size[4 * k + e], inv, __builtin_fabsf(q)) * 0x1p-21f : q * 0x1p-21f;
            lo[e] = __builtin_amdgcn_fmed3f(q - room, -448.0f, 448.0f);
            hi[e] = __builtin_amdgcn_fmed3f(q + room, -448.0f, 448.0f);
            if (KEY) top = __builtin_fmaf(size[4 * k + e], 0.0f, top);      // NaN from NaN and Inf
          }
          codes[k] = e4m3_codes(lo);
          above[k] = e4m3_codes(hi);
        }
        *reinterpret_cast<at_u32x2*>(base + there + d) = codes;
        // (the clamp drops NaN; Inf is as good)
        const bool odd = top_bits(own) >= T::kExp || top != 0.0f || !(inv < 0x1p100f && inv > 0x1p-100f);
        return bool(__any(codes[0] != above[0] || codes[1] != above[1] || odd));
      } else {
        uint32_t codes = 0, scale = 0;
        bool sure = true;
        if constexpr (KEY) {
          // what the values are off by: 4 * 2^-24 of both values of a pair, at most 8 * 2^-24 of
          // the largest one here; the bounds' ends round by 2 * 2^-24 of it
          turn8<T, STYLE>(own, other, row, d, pairs, turns, y);
          uint32_t top = top_bits(own);
          if (STYLE == kHalf && turns.turned) top = max(top, top_bits(other));
          if constexpr (STYLE == kHalfAny) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (turns.turned >> e & 1)
                top = max(top, uint32_t(row[d + e < pairs ? d + e + pairs : d + e - pairs] & 0x7fff));
          }
          float off = T::low(top) * a.factor * 0x1p-20f;
          if (!turns.turned) off = 0.0f;
          if (top >= T::kExp) off = -kNegInf;        // NaN too
          sure = quant8_sure<T::kFp4Exp>(y, off, codes, scale);
        } else {
          widen8<T>(own, y);
          quant8_mx<MXFP4, T::kFp4Exp>(y, codes, scale);
        }
        *reinterpret_cast<uint32_t*>(base + there + d / 2) = codes;
        if (!(d & 24)) base[scale_to + head * a.kv.scale_head] = uint8_t(scale);
        return bool(__any(!sure));
      }
    };
    // The codes in doubt again, from the exact values (E4M3: quotients), two at a time in a loop
    // that is not unrolled: where nothing else is in registers.
    auto again = [&](int head, const uint16_t* row) {
      at_u32x4 u = *reinterpret_cast<const at_u32x4*>(row + d);
      const float f = CACHE == W4A4_E4M3 && scales ? scales[head] : 1.0f;
      const double inv = 1.0 / double(f);
      float y[8];
#pragma unroll 1
      for (int n = d; n < d + 8; n += 2) {
        double x[2] = {T::low(u[0]), T::high(u[0])};
        if constexpr (KEY) {
          const double before[2] = {x[0], x[1]};
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (n + e >= a.rot) continue;
            const bool front = STYLE == kPairs ? e == 0 : n + e < pairs;
            const int q = STYLE == kPairs ? n >> 1 : front ? n + e : n + e - pairs;
            const Turn<double> t = turn_of<double>(my_turn, a.freqs[q], a.factor, a.inverse);
            const double w = STYLE == kPairs ? before[e ^ 1] : double(T::low(row[front ? q + pairs : q]));
            x[e] = front ? x[e] * t.cos - w * t.sin : x[e] * t.cos + w * t.sin;
          }
        }
#pragma unroll
        for (int k = 0; k < 3; ++k) u[k] = u[k + 1];
#pragma unroll
        for (int k = 0; k < 6; ++k) y[k] = y[k + 2];
#pragma unroll
        for (int e = 0; e < 2; ++e) y[6 + e] = CACHE == W4A4_E4M3 ? e4m3_quotient(x[e], f, inv) : to_odd(x[e]);
      }
      const int64_t there = to + head * a.kv.head_stride;
      if constexpr (CACHE == W4A4_E4M3) {
        const float one[4] = {y[0], y[1], y[2], y[3]}, two[4] = {y[4], y[5], y[6], y[7]};
        *reinterpret_cast<at_u32x2*>(base + there + d) = (at_u32x2){e4m3_codes(one), e4m3_codes(two)};
      } else {
        uint32_t codes, scale;
        quant8_mx<MXFP4, T::kFp4Exp>(y, codes, scale);
        *reinterpret_cast<uint32_t*>(base + there + d / 2) = codes;
        if (!(d & 24)) base[scale_to + head * a.kv.scale_head] = uint8_t(scale);
      }
    };
    while (r.h < r.heads) {
      uint32_t doubt = 0;
#pragma unroll
      for (int j = 0; j < FLIGHT; ++j)
        if (r.h + j * phases < r.heads && take(r.h + j * phases, r.own[j], r.other[j], r.p + j * r.step))
          doubt |= 1u << j;
      if constexpr (SMALL) {
#pragma unroll 1
        for (int j = 0; j < FLIGHT; ++j)
          if (doubt >> j & 1) again(r.h + j * phases, r.p + j * r.step);
      }
      advance(r);
      if (r.h < r.heads) load(r, decltype(which)::value);
    }
  };
  if (kinds & kKeys) {
    if (kinds & kQueries) {
      rows = rows_of(a.k, a.k_row, a.k_head, first, a.kv.heads);
      load(rows, true);
    }
    store_all(rows, const_cast<void*>(a.kv.k), a.kv.k_scale, std::true_type());
  }
  if (kinds & kValues) {
    if (kinds != kValues) {
      rows = rows_of(a.v, a.v_row, a.v_head, first, a.kv.heads);
      load(rows, false);
    }
    store_all(rows, const_cast<void*>(a.kv.v), a.kv.v_scale, std::false_type());
  }
}

// ---------------------------------------------------------------------- out --

template <class T, int CACHE>
__global__ void __launch_bounds__(256) rows_out_kernel(RowsOut a, int lane_bits, int tok_bits) {
  const int lanes = 1 << lane_bits, group = threadIdx.x >> lane_bits;
  const int d = 8 * (threadIdx.x & (lanes - 1));
  const int per_wg = 1 << tok_bits, tok = group & (per_wg - 1);
  const int phases = (256 >> lane_bits >> tok_bits) * gridDim.y;
  const int first = blockIdx.y * (256 >> lane_bits >> tok_bits) + (group >> tok_bits);
  const int64_t i = (int64_t(blockIdx.x) << tok_bits) + tok;
  const int vectors = 2 * a.kv.heads;
  const int lane = threadIdx.x & 63;
  const int64_t row0 = int64_t(blockIdx.x) << tok_bits;
  const Place at = shuffled(place_of(a.kv, a.cu, int(row0) + lane, lane < per_wg && row0 + lane < a.tokens), tok);
  if (i >= a.tokens || !at.in) return;
  const int64_t page = int64_t(max(at.page, 0)) * a.kv.page_stride;
  const int64_t from = page + at.slot * a.kv.token_stride;
  for (int v0 = first; v0 < vectors; v0 += kFlight * phases) {
    at_u32x4 raw[kFlight];
    uint32_t scale[kFlight];
    float head_scale[kFlight];
#pragma unroll
    for (int j = 0; j < kFlight; ++j) {
      const int v = v0 + j * phases;
      if (v >= vectors) break;
      const bool key = v < a.kv.heads;
      const int head = key ? v : v - a.kv.heads;
      const uint8_t* cache = static_cast<const uint8_t*>(key ? a.kv.k : a.kv.v);
      const int64_t p = from + head * a.kv.head_stride;
      if constexpr (CACHE == W4A4_E2M1) {
        raw[j].x = *reinterpret_cast<const uint32_t*>(cache + p + d / 2);
        scale[j] = cache[page + a.kv.scale_at + head * a.kv.scale_head + (d >> 5) * int64_t(a.kv.page.d) + at.slot];
      } else if constexpr (CACHE == W4A4_E4M3) {
        const at_u32x2 x = *reinterpret_cast<const at_u32x2*>(cache + p + d);
        raw[j].x = x.x;
        raw[j].y = x.y;
        const float* scales = key ? a.kv.k_scale : a.kv.v_scale;
        head_scale[j] = scales ? scales[head] : 1.0f;
      } else {
        raw[j] = *reinterpret_cast<const at_u32x4*>(cache + (p + d) * 2);
      }
    }
#pragma unroll
    for (int j = 0; j < kFlight; ++j) {
      const int v = v0 + j * phases;
      if (v >= vectors) break;
      const bool key = v < a.kv.heads;
      const int head = key ? v : v - a.kv.heads;
      at_u32x4 y = raw[j];
      if constexpr (CACHE == W4A4_E2M1) {
        const float s = fp4_scale(scale[j]);
        y = (at_u32x4){fp4_pair<T, 0>(raw[j].x, s), fp4_pair<T, 1>(raw[j].x, s), fp4_pair<T, 2>(raw[j].x, s),
                       fp4_pair<T, 3>(raw[j].x, s)};
      } else if constexpr (CACHE == W4A4_E4M3) {
        const float s = head_scale[j];
        const uint32_t x[2] = {raw[j].x, raw[j].y};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t z = k & 1 ? e4m3_pair<Bf16, true>(x[k >> 1]) : e4m3_pair<Bf16, false>(x[k >> 1]);     // exact
          y[k] = T::pack(Bf16::low(z) * s, Bf16::high(z) * s);
        }
      }
      if (at.page < 0) y = (at_u32x4){T::kNanPair, T::kNanPair, T::kNanPair, T::kNanPair};
      uint16_t* to = key ? static_cast<uint16_t*>(a.k) + i * a.k_row + head * a.k_head
                         : static_cast<uint16_t*>(a.v) + i * a.v_row + head * a.v_head;
      *reinterpret_cast<at_u32x4*>(to + d) = y;
    }
  }
}

// Lanes of a vector (one head of one token), tokens of a workgroup, workgroups that share
// them.  No more vectors of a token at a time than there are, and many tokens only where that
// leaves workgroups enough: 8191 tokens of 32 heads 22.2 us with 8 tokens each, 27 with 16.
struct Shape {
  int lane_bits, tok_bits;
  int64_t x, y;
  dim3 grid() const { return dim3(unsigned(x), unsigned(y)); }
};
Shape shape_of(int64_t tokens, int64_t vectors, int dim) {
  Shape s = {3, 0, 1, 1};
  while (8 << s.lane_bits < dim) ++s.lane_bits;
  const int groups = 256 >> s.lane_bits;
  while (1 << s.tok_bits < groups &&
         (groups >> s.tok_bits > vectors || (tokens >> s.tok_bits) > 2048))
    ++s.tok_bits;
  s.x = (tokens + (int64_t(1) << s.tok_bits) - 1) >> s.tok_bits;
  const int phases = groups >> s.tok_bits;
  while (s.x * s.y < 512 && s.y * phases < vectors) s.y *= 2;
  return s;
}
// One part where its workgroups are enough for the card (each looks up its tokens and
// computes their angles once for all kinds: 14449 tokens, 28 / 4 heads of 128 into 4 bits,
// 51 us in one part, 63 in three; 1795 of 16 / 16 of 64 into FP16 9.4 and 11.4), else a part
// for each kind, so that the kinds' chains of loads run side by side (one token each of 48
// sequences 4.4 us, 5.5 in one part).
constexpr int kOnePart = 512;
// *most: vectors of a kind that a thread has at most.
Parts parts_of(int64_t tokens, int64_t q_heads, int64_t kv_heads, int dim, int64_t* grid, int* lane_bits,
               int64_t* most) {
  Parts p = {};
  *grid = 0;
  *most = 1;
  auto add = [&](int kinds, int64_t heads) {
    const Shape s = shape_of(tokens, heads, dim);
    const int64_t phases = (256 >> s.lane_bits >> s.tok_bits) * s.y;
    const int64_t rows = std::max(kinds & kQueries ? q_heads : 0, kinds == kQueries ? 0 : kv_heads);
    *most = std::max(*most, (rows + phases - 1) / phases);
    p.kinds[p.count] = kinds;
    p.begin[p.count] = int(*grid);
    p.tok_bits[p.count] = s.tok_bits;
    p.splits[p.count] = int(s.y);
    ++p.count;
    *grid += s.x * s.y;
    *lane_bits = s.lane_bits;
  };
  if (kv_heads == 0) {
    add(kQueries, q_heads);
  } else if (shape_of(tokens, q_heads ? std::min(q_heads, kv_heads) : kv_heads, dim).x >= kOnePart) {
    add((q_heads ? kQueries : 0) | kKeys | kValues, q_heads ? std::min(q_heads, kv_heads) : kv_heads);
  } else {
    add(kKeys, kv_heads);
    add(kValues, kv_heads);
    if (q_heads) add(kQueries, q_heads);
  }
  return p;
}

template <class T, int CACHE>
hipError_t launch_in(const RowsIn& a, hipStream_t stream) {
  int64_t grid, most;
  int lane_bits;
  const Parts parts = parts_of(a.tokens, a.q_heads, a.kv.heads, a.dim, &grid, &lane_bits, &most);
  const FastDiv by_pairs = fast_div(uint32_t(std::max(a.rot / 2, 1)));
  auto go = [&](auto style) {
    constexpr int S = decltype(style)::value;
    const auto kernel = most == 1 ? rows_in_kernel<T, CACHE, S, 1> : rows_in_kernel<T, CACHE, S, kFlight>;
    kernel<<<unsigned(grid), 256, 0, stream>>>(a, parts, lane_bits, by_pairs);
    return hipGetLastError();
  };
  if constexpr (CACHE == W4A4_E2M1)
    if (a.rot == 0) return go(std::integral_constant<int, kNone>());
  if (a.interleaved) return go(std::integral_constant<int, kPairs>());
  return a.rot % 16 == 0 ? go(std::integral_constant<int, kHalf>()) : go(std::integral_constant<int, kHalfAny>());
}

}  // namespace

int64_t rows_workgroups(int64_t tokens, int64_t q_heads, int64_t kv_heads, int dim) {
  int64_t grid, most;
  int lane_bits;
  parts_of(tokens, q_heads, kv_heads, dim, &grid, &lane_bits, &most);
  return grid;
}

hipError_t launch_rows_in(const RowsIn& a, int cache_dtype, int dtype, hipStream_t stream) {
  const bool bf16 = dtype == W4A4_BF16;
  if (a.kv.heads == 0) return bf16 ? launch_in<Bf16, kAlone>(a, stream) : launch_in<F16, kAlone>(a, stream);
  if (cache_dtype == W4A4_E4M3) return bf16 ? launch_in<Bf16, W4A4_E4M3>(a, stream) : launch_in<F16, W4A4_E4M3>(a, stream);
  if (cache_dtype == W4A4_E2M1) return bf16 ? launch_in<Bf16, W4A4_E2M1>(a, stream) : launch_in<F16, W4A4_E2M1>(a, stream);
  return bf16 ? launch_in<Bf16, W4A4_BF16>(a, stream) : launch_in<F16, W4A4_BF16>(a, stream);
}

hipError_t launch_rows_out(const RowsOut& a, int cache_dtype, int dtype, hipStream_t stream) {
  const Shape s = shape_of(a.tokens, 2 * a.kv.heads, a.dim);
  const bool bf16 = dtype == W4A4_BF16;
  auto go = [&](auto kernel) {
    kernel<<<s.grid(), 256, 0, stream>>>(a, s.lane_bits, s.tok_bits);
    return hipGetLastError();
  };
  if (cache_dtype == W4A4_E2M1)
    return bf16 ? go(rows_out_kernel<Bf16, W4A4_E2M1>) : go(rows_out_kernel<F16, W4A4_E2M1>);
  if (cache_dtype == W4A4_E4M3)
    return bf16 ? go(rows_out_kernel<Bf16, W4A4_E4M3>) : go(rows_out_kernel<F16, W4A4_E4M3>);
  return bf16 ? go(rows_out_kernel<Bf16, W4A4_BF16>) : go(rows_out_kernel<F16, W4A4_BF16>);
}

}  // namespace w4a4
