// Rows of queries, keys and values on their way between a projection and the
// paged cache: the rotation by their positions, alone or with the storing into
// a cache of 16, 8 or 4 bits, and rows read out of a cache.
//
// All of it moves bytes; HBM bandwidth bounds it, for small calls the launch and
// the chain of lookups behind it.
#include <algorithm>

#include "attn_common.h"
#include "mx_quant.h"

namespace w4a4 {
namespace {

// cos and sin of position * freq, times factor.  The angle in turns, in 64 bits:
// the product of a 31-bit and a 24-bit number is off by 2^-53 of itself at most,
// 1 / (2 pi) is taken in two parts, so the angle of position 2^31 - 1 is right to
// 1e-6 of a turn and that of position 131071 to 2^-48.  Then the nearest quarter
// turn is taken off and the Taylor series of the rest, |x| <= pi / 4, is off by less
// than 2^-50.
struct Turn {
  double cos, sin;
};
__device__ __forceinline__ Turn turn_of(int pos, float freq, float factor, bool inverse) {
  constexpr double kInv = 0x1.45f306dc9c883p-3, kInvRest = -0x1.6b01ec5417056p-57;      // 1 / (2 pi)
  const double a = double(pos) * double(freq);
  const double t = a * kInv, rest = __builtin_fma(a, kInv, -t) + a * kInvRest;
  const double u = 4.0 * ((t - __builtin_rint(t)) + rest), k = __builtin_rint(u);
  const double x = (u - k) * 0x1.921fb54442d18p+0, z = x * x;
  double s = -1.0 / 1307674368000.0, c = -1.0 / 87178291200.0;
  s = __builtin_fma(s, z, 1.0 / 6227020800.0);
  s = __builtin_fma(s, z, -1.0 / 39916800.0);
  s = __builtin_fma(s, z, 1.0 / 362880.0);
  s = __builtin_fma(s, z, -1.0 / 5040.0);
  s = __builtin_fma(s, z, 1.0 / 120.0);
  s = __builtin_fma(s, z, -1.0 / 6.0);
  s = __builtin_fma(s * z, x, x);
  c = __builtin_fma(c, z, 1.0 / 479001600.0);
  c = __builtin_fma(c, z, -1.0 / 3628800.0);
  c = __builtin_fma(c, z, 1.0 / 40320.0);
  c = __builtin_fma(c, z, -1.0 / 720.0);
  c = __builtin_fma(c, z, 1.0 / 24.0);
  c = __builtin_fma(c, z, -0.5);
  c = __builtin_fma(c, z, 1.0);
  const int q = int(k) & 3;
  double cq = q & 1 ? s : c, sq = q & 1 ? c : s;
  if (q == 1 || q == 2) cq = -cq;
  if (q >= 2) sq = -sq;
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

// Where token i of a call is: the sequence's place of it, and its page.
struct Place {
  bool in;            // it belongs to a sequence
  int pos, page, slot;       // page -1: none
};
__device__ __forceinline__ Place place_of(const KvView& kv, const int32_t* cu, int i) {
  Place x = {i < kv.seqs, 0, -1, 0};
  int s = i, back = 1;      // back: tokens from this one to the sequence's last, inclusive
  if (cu) {
    s = find_seq(cu, kv.seqs, i);
    back = cu[s + 1] - i;
    x.in = back > 0 && cu[s] <= i;
  }
  if (!x.in) return x;
  const int64_t pos = int64_t(kv.lens[s]) - back;
  x.pos = int(max(pos, int64_t(INT32_MIN)));
  if (pos >= 0) x.page = kv_page(kv, kv.tables + s * kv.table_stride, int(pos), &x.slot);
  return x;
}

constexpr int kAlone = -1;        // CACHE: none
constexpr int kNone = 0, kHalf = 1, kPairs = 2, kHalfAny = 3;      // how the pairs lie
constexpr int kMaxToks = 32;      // tokens of a workgroup
constexpr int kTable = 1024;      // angles of a workgroup's tokens
constexpr int kFlight = 4;        // vectors (one head of one token) in flight per thread

// Elements of 8 at d: of cos and sin `tab`, of the row x and, for halves, of the
// partners y (kHalfAny: read one by one).
template <class T, int STYLE, typename R, typename CS>
__device__ __forceinline__ void turn8(at_u32x4 own, at_u32x4 other, const uint16_t* row, int d, int pairs, const CS* tab,
                                      R (&y)[8]) {
  float x[8], z[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    x[e] = e & 1 ? T::high(own[e >> 1]) : T::low(own[e >> 1]);
    z[e] = e & 1 ? T::high(other[e >> 1]) : T::low(other[e >> 1]);
  }
  if constexpr (STYLE == kPairs) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const int p = (d + e) >> 1;
      if (p < pairs) {
        const CS t = tab[p];
        y[e] = R(x[e]) * t.x - R(x[e + 1]) * t.y;
        y[e + 1] = R(x[e]) * t.y + R(x[e + 1]) * t.x;
      } else {
        y[e] = x[e];
        y[e + 1] = x[e + 1];
      }
    }
  } else if constexpr (STYLE == kHalf) {
    const bool back = d >= pairs;
    const CS* at = tab + (back ? d - pairs : d);
    if (d < 2 * pairs) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const CS t = at[e];
        const R s = back ? t.y : -t.y;
        y[e] = R(x[e]) * t.x + R(z[e]) * s;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = x[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      y[e] = x[e];
      if (STYLE == kHalfAny && d + e < 2 * pairs) {
        const bool back = d + e >= pairs;
        const int p = back ? d + e - pairs : d + e;
        const CS t = tab[p];
        const float w = T::low(row[back ? p : p + pairs]);
        y[e] = R(x[e]) * t.x + R(w) * (back ? t.y : -t.y);
      }
    }
  }
}

template <class T>
__device__ __forceinline__ at_u32x4 pack8(const float (&y)[8]) {
  return (at_u32x4){T::pack(y[0], y[1]), T::pack(y[2], y[3]), T::pack(y[4], y[5]), T::pack(y[6], y[7])};
}

// A workgroup takes per_wg tokens (a power of two, so that every thread has one
// token and one chunk of 8 elements, and walks over heads) and a share of the
// vectors.  The rows' loads start first; meanwhile the tokens are looked up, and the
// cos and sin of all their pairs computed once and left in LDS.
// What is kept in 16 bits is rotated in 32.  Keys on their way to 8 or 4 bits are
// rotated in 64, so that the codes are those of the rotated values and not of a
// rounding of them.
template <class T, int CACHE, int STYLE>
__global__ void __launch_bounds__(256) rows_in_kernel(RowsIn a, int lane_bits, int tok_bits) {
  constexpr bool SMALL = CACHE == W4A4_E4M3 || CACHE == W4A4_E2M1;
  __shared__ float2 tab[STYLE ? kTable : 1];
  __shared__ double2 tab64[SMALL && STYLE ? kTable : 1];
  __shared__ Place places[kMaxToks];
  const int lanes = 1 << lane_bits, group = threadIdx.x >> lane_bits;
  const int d = 8 * (threadIdx.x & (lanes - 1));
  const int per_wg = 1 << tok_bits, tok = group & (per_wg - 1);
  const int phases = (256 >> lane_bits >> tok_bits) * gridDim.y;
  const int first = blockIdx.y * (256 >> lane_bits >> tok_bits) + (group >> tok_bits);
  const int64_t i = (int64_t(blockIdx.x) << tok_bits) + tok;
  const int kv_heads = a.kv.heads, vectors = a.q_heads + 2 * kv_heads;
  const int pairs = a.rot >> 1;
  const bool here = i < a.tokens && d < a.dim;

  auto row_of = [&](int v) {
    const uint16_t* p = static_cast<const uint16_t*>(a.q) + i * a.q_row + v * a.q_head;
    if (v >= a.q_heads) {
      const int h = v - a.q_heads;
      p = h < kv_heads ? static_cast<const uint16_t*>(a.k) + i * a.k_row + h * a.k_head
                       : static_cast<const uint16_t*>(a.v) + i * a.v_row + (h - kv_heads) * a.v_head;
    }
    return p;
  };
  at_u32x4 own[kFlight], other[kFlight];
  auto load = [&](int v0) {
#pragma unroll
    for (int j = 0; j < kFlight; ++j) {
      const int v = v0 + j * phases;
      if (here && v < vectors) {
        const uint16_t* p = row_of(v);
        own[j] = *reinterpret_cast<const at_u32x4*>(p + d);
        if (STYLE == kHalf && v < a.q_heads + kv_heads && d < a.rot)
          other[j] = *reinterpret_cast<const at_u32x4*>(p + (d < pairs ? d + pairs : d - pairs));
      }
    }
  };
  load(first);

  if (int(threadIdx.x) < per_wg) {
    const int64_t t = (int64_t(blockIdx.x) << tok_bits) + threadIdx.x;
    Place x = {t < a.tokens, 0, -1, 0};
    if (CACHE != kAlone && x.in) x = place_of(a.kv, a.cu, int(t));
    if (x.in && a.positions) x.pos = a.positions[t];
    places[threadIdx.x] = x;
  }
  __syncthreads();
  if constexpr (STYLE != kNone) {
    for (int e = threadIdx.x; e < pairs << tok_bits; e += 256) {
      const int t = e / pairs, p = e - t * pairs;
      const Turn x = turn_of(places[t].pos, a.freqs[p], a.factor, a.inverse);
      tab[e] = {float(x.cos), float(x.sin)};
      if constexpr (SMALL) tab64[e] = {x.cos, x.sin};
    }
    __syncthreads();
  }
  const Place at = places[tok];
  if (!here || !at.in) return;

  const float2* turns = tab + tok * pairs;
  const double2* turns64 = tab64 + (SMALL ? tok * pairs : 0);
  for (int v0 = first; v0 < vectors; v0 += kFlight * phases) {
    if (v0 != first) load(v0);
#pragma unroll
    for (int j = 0; j < kFlight; ++j) {
      const int v = v0 + j * phases;
      if (v >= vectors) break;
      const uint16_t* row = row_of(v);
      if (v < a.q_heads) {
        float y[8];
        turn8<T, STYLE>(own[j], other[j], row, d, pairs, turns, y);
        // out may be q itself: every lane of the row has read its partners
        if (STYLE == kHalfAny) __builtin_amdgcn_wave_barrier();
        *reinterpret_cast<at_u32x4*>(static_cast<uint16_t*>(a.out) + i * a.o_row + v * a.o_head + d) = pack8<T>(y);
        continue;
      }
      if constexpr (CACHE != kAlone) {
        if (at.page < 0) continue;
        const int h = v - a.q_heads;
        const bool key = h < kv_heads;
        const int head = key ? h : h - kv_heads;
        uint8_t* page = const_cast<uint8_t*>(static_cast<const uint8_t*>(key ? a.kv.k : a.kv.v));
        const int64_t to = at.page * a.kv.page_stride + at.slot * a.kv.token_stride + head * a.kv.head_stride;
        if constexpr (!SMALL) {
          at_u32x4 z = own[j];
          if (STYLE != kNone && key) {
            float y[8];
            turn8<T, STYLE>(own[j], other[j], row, d, pairs, turns, y);
            z = pack8<T>(y);
          }
          *reinterpret_cast<at_u32x4*>(page + (to + d) * 2) = z;
        } else {
          double y[8];
          if (STYLE != kNone && key) turn8<T, STYLE>(own[j], other[j], row, d, pairs, turns64, y);
          else turn8<T, kNone>(own[j], own[j], row, d, 0, turns64, y);
          float x[8];
          if constexpr (CACHE == W4A4_E4M3) {
            const float* scales = key ? a.kv.k_scale : a.kv.v_scale;
            const double s = scales ? scales[head] : 1.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const double z = y[e] / s;
              x[e] = z != z ? float(z) : to_odd(fmin(fmax(z, -448.0), 448.0));
            }
            at_u32x2 w;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              int p = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * k], x[4 * k + 1], 0, false);
              w[k] = uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(x[4 * k + 2], x[4 * k + 3], p, true));
            }
            *reinterpret_cast<at_u32x2*>(page + to + d) = w;
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = to_odd(y[e]);
            uint32_t codes, scale;
            quant8_mx<MXFP4, T::kFp4Exp>(x, codes, scale);
            *reinterpret_cast<uint32_t*>(page + to + d / 2) = codes;
            if (!(d & 24))
              page[at.page * a.kv.page_stride + a.kv.scale_at + head * a.kv.scale_head + (d >> 5) * int64_t(a.kv.page.d) +
                   at.slot] = uint8_t(scale);
          }
        }
      }
    }
  }
}

// ---------------------------------------------------------------------- out --

template <class T, int CACHE>
__global__ void __launch_bounds__(256) rows_out_kernel(RowsOut a, int lane_bits, int tok_bits) {
  __shared__ Place places[kMaxToks];
  const int lanes = 1 << lane_bits, group = threadIdx.x >> lane_bits;
  const int d = 8 * (threadIdx.x & (lanes - 1));
  const int per_wg = 1 << tok_bits, tok = group & (per_wg - 1);
  const int phases = (256 >> lane_bits >> tok_bits) * gridDim.y;
  const int first = blockIdx.y * (256 >> lane_bits >> tok_bits) + (group >> tok_bits);
  const int64_t i = (int64_t(blockIdx.x) << tok_bits) + tok;
  const int vectors = 2 * a.kv.heads;
  if (int(threadIdx.x) < per_wg) {
    const int64_t t = (int64_t(blockIdx.x) << tok_bits) + threadIdx.x;
    Place x = {false, 0, -1, 0};
    if (t < a.tokens) x = place_of(a.kv, a.cu, int(t));
    places[threadIdx.x] = x;
  }
  __syncthreads();
  const Place at = places[tok];
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

// Lanes of a vector, tokens of a workgroup, workgroups per token group.
struct Shape {
  int lane_bits, tok_bits;
  int64_t x, y;
  dim3 grid() const { return dim3(unsigned(x), unsigned(y)); }
};
Shape shape_of(int64_t tokens, int64_t vectors, int dim) {
  Shape s = {3, 0, 1, 1};
  while (8 << s.lane_bits < dim) ++s.lane_bits;
  const int groups = 256 >> s.lane_bits;
  while (1 << s.tok_bits < groups && (tokens >> s.tok_bits) > 1024) ++s.tok_bits;
  s.x = (tokens + (int64_t(1) << s.tok_bits) - 1) >> s.tok_bits;
  const int phases = groups >> s.tok_bits;
  while (s.x * s.y < 512 && s.y * phases < vectors) s.y *= 2;
  return s;
}

template <class T, int CACHE>
hipError_t launch_in(const RowsIn& a, hipStream_t stream) {
  const Shape s = shape_of(a.tokens, a.q_heads + 2 * a.kv.heads, a.dim);
  const int style = a.rot == 0 ? kNone : a.interleaved ? kPairs : a.rot % 16 == 0 ? kHalf : kHalfAny;
  if constexpr (CACHE == W4A4_E2M1) {
    if (style == kNone) {
      rows_in_kernel<T, CACHE, kNone><<<s.grid(), 256, 0, stream>>>(a, s.lane_bits, s.tok_bits);
      return hipGetLastError();
    }
  }
  if (style == kHalf) rows_in_kernel<T, CACHE, kHalf><<<s.grid(), 256, 0, stream>>>(a, s.lane_bits, s.tok_bits);
  else if (style == kPairs) rows_in_kernel<T, CACHE, kPairs><<<s.grid(), 256, 0, stream>>>(a, s.lane_bits, s.tok_bits);
  else rows_in_kernel<T, CACHE, kHalfAny><<<s.grid(), 256, 0, stream>>>(a, s.lane_bits, s.tok_bits);
  return hipGetLastError();
}

}  // namespace

int64_t rows_workgroups(int64_t tokens, int64_t vectors, int dim) {
  const Shape s = shape_of(tokens, vectors, dim);
  return s.x * s.y;
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
