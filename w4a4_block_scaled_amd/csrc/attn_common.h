// Element types, matrix instructions and small reductions shared by the two
// attention kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kvcache.h"

namespace w4a4 {

typedef uint32_t at_u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t at_u32x4 __attribute__((ext_vector_type(4)));
typedef float at_f32x2 __attribute__((ext_vector_type(2)));
typedef float at_f32x4 __attribute__((ext_vector_type(4)));
typedef float at_f32x16 __attribute__((ext_vector_type(16)));

constexpr float kNegInf = -__builtin_huge_valf();

// Whether either half of u is Inf or NaN (all bits of the exponent EXP set).
template <uint32_t EXP>
__device__ __forceinline__ bool has_odd(uint32_t u) {
  return (u & EXP) == EXP || (u >> 16 & EXP) == EXP;
}
// u with 0 in the place of the halves that are Inf or NaN.
template <uint32_t EXP>
__device__ __forceinline__ uint32_t without_odd(uint32_t u) {
  return ((u & EXP) == EXP ? 0 : u & 0xffffu) | ((u >> 16 & EXP) == EXP ? 0 : u & 0xffff0000u);
}

// u with 0 in the place of the halves that are Inf or NaN; *plus gets ONE for +Inf
// and NaN, *minus for -Inf and NaN, 0 elsewhere.
template <uint32_t EXP, uint32_t ONE>
__device__ __forceinline__ uint32_t split_odd16(uint32_t u, uint32_t* plus, uint32_t* minus) {
  uint32_t keep = 0, p = 0, n = 0;
#pragma unroll
  for (int s = 0; s < 32; s += 16) {
    const uint32_t x = u >> s & 0xffffu;
    const bool odd = (x & EXP) == EXP, nan = odd && (x & 0x7fffu) != EXP;
    keep |= odd ? 0 : x << s;
    p |= odd && (nan || x < 0x8000u) ? ONE << s : 0;
    n |= odd && (nan || x >= 0x8000u) ? ONE << s : 0;
  }
  *plus = p;
  *minus = n;
  return keep;
}

// The reference m of a row's softmax weights 2^(score - m).  It follows the row's
// maximum, kRaise below it, and is moved only where the maximum has grown by more
// than kGrowth since, so that sums are rarely rebased and weights go up to
// 2^(kGrowth + kRaise).  kRaise uses FP16's range: a weight is lost (rounded to a
// step of 2^-24) only at 2^-32 of the largest one, where 131071 tokens together
// weigh 2^-15 of it; without, at 2^-25, half a percent each.  BF16 has fp32's range.
constexpr float kGrowth = 8.0f;

// 16-bit element types.  pack(a, b): two fp32 to two elements, RNE, a in the
// low half.  mfma16: 16 x 16 x 32, mfma32: 32 x 32 x 16; operands 8 elements
// per lane.
struct Bf16 {
  static constexpr uint32_t kExp = 0x7f80u, kOne = 0x3f80u;      // the exponent of Inf and NaN; 1.0
  static constexpr uint32_t kNanPair = 0x7fc07fc0u;
  static constexpr int kFp4Exp = 127;             // largest exponent of a 4-bit block stored from this type
  static constexpr float kRaise = 0.0f;
  static __device__ __forceinline__ bool not_finite(uint32_t u) { return has_odd<kExp>(u); }
  static __device__ __forceinline__ uint32_t finite(uint32_t u) { return without_odd<kExp>(u); }
  static __device__ __forceinline__ uint32_t split_odd(uint32_t u, uint32_t* plus, uint32_t* minus) {
    return split_odd16<kExp, kOne>(u, plus, minus);
  }
  typedef __bf16 x8 __attribute__((ext_vector_type(8)));
  typedef __bf16 x2 __attribute__((ext_vector_type(2)));
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((at_f32x2){a, b}, x2));
  }
  template <bool HI>
  static __device__ __forceinline__ x2 from_e4m3(uint32_t u) {
    return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(u, 1.0f, HI);
  }
  template <int B>
  static __device__ __forceinline__ x2 from_fp4(uint32_t u, float scale) {
    return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(u, scale, B);
  }
  static __device__ __forceinline__ float low(uint32_t u) { return __builtin_bit_cast(float, u << 16); }
  static __device__ __forceinline__ float high(uint32_t u) { return __builtin_bit_cast(float, u & 0xffff0000u); }
  static __device__ __forceinline__ at_f32x4 mfma16(at_u32x4 a, at_u32x4 b, at_f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(x8, a), __builtin_bit_cast(x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ at_f32x16 mfma32(at_u32x4 a, at_u32x4 b, at_f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(x8, a), __builtin_bit_cast(x8, b), c, 0, 0, 0);
  }
};
struct F16 {
  static constexpr uint32_t kExp = 0x7c00u, kOne = 0x3c00u;      // the exponent of Inf and NaN; 1.0
  static constexpr uint32_t kNanPair = 0x7e007e00u;
  static constexpr int kFp4Exp = 13;              // so that 6 * 2^13 stays in range
  static constexpr float kRaise = 7.0f;
  static __device__ __forceinline__ bool not_finite(uint32_t u) { return has_odd<kExp>(u); }
  static __device__ __forceinline__ uint32_t finite(uint32_t u) { return without_odd<kExp>(u); }
  static __device__ __forceinline__ uint32_t split_odd(uint32_t u, uint32_t* plus, uint32_t* minus) {
    return split_odd16<kExp, kOne>(u, plus, minus);
  }
  typedef _Float16 x8 __attribute__((ext_vector_type(8)));
  typedef _Float16 x2 __attribute__((ext_vector_type(2)));
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((at_f32x2){a, b}, x2));
  }
  template <bool HI>
  static __device__ __forceinline__ x2 from_e4m3(uint32_t u) {
    return __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(u, 1.0f, HI);
  }
  template <int B>
  static __device__ __forceinline__ x2 from_fp4(uint32_t u, float scale) {
    return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(u, scale, B);
  }
  static __device__ __forceinline__ float low(uint32_t u) {
    return float(__builtin_bit_cast(x2, u).x);
  }
  static __device__ __forceinline__ float high(uint32_t u) {
    return float(__builtin_bit_cast(x2, u).y);
  }
  static __device__ __forceinline__ at_f32x4 mfma16(at_u32x4 a, at_u32x4 b, at_f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(x8, a), __builtin_bit_cast(x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ at_f32x16 mfma32(at_u32x4 a, at_u32x4 b, at_f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(x8, a), __builtin_bit_cast(x8, b), c, 0, 0, 0);
  }
};

// Two E4M3 codes (the low or the high half of u) as two elements of T, exact.
template <class T, bool HI>
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t u) {
  return __builtin_bit_cast(uint32_t, T::template from_e4m3<HI>(u));
}

// The two E2M1 codes of byte B of u times a block's scale, as two elements of T;
// the scale is 2^(byte - 127), NaN for byte 255.
template <class T, int B>
__device__ __forceinline__ uint32_t fp4_pair(uint32_t u, float scale) {
  return __builtin_bit_cast(uint32_t, T::template from_fp4<B>(u, scale));
}
__device__ __forceinline__ float fp4_scale(uint32_t byte) { return __builtin_bit_cast(float, byte << 23); }

// x of the lanes l and l ^ 32 (l ^ 16), in either order: halves (odd and even
// quarters) of two registers change places.
struct Pair {
  float a, b;
};
__device__ __forceinline__ Pair pair_of(at_u32x2 r) {
  const uint32_t x = r.x, y = r.y;      // a bit cast of r.y itself would read r.x
  return {__builtin_bit_cast(float, x), __builtin_bit_cast(float, y)};
}
__device__ __forceinline__ Pair pair_xor32(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  return pair_of(__builtin_amdgcn_permlane32_swap(u, u, false, false));
}
__device__ __forceinline__ Pair pair_xor16(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  return pair_of(__builtin_amdgcn_permlane16_swap(u, u, false, false));
}
__device__ __forceinline__ float max_xor32(float x) {
  const Pair p = pair_xor32(x);
  return fmaxf(p.a, p.b);
}
__device__ __forceinline__ float sum_xor32(float x) {
  const Pair p = pair_xor32(x);
  return p.a + p.b;
}
__device__ __forceinline__ float max_xor16(float x) {
  const Pair p = pair_xor16(x);
  return fmaxf(p.a, p.b);
}
__device__ __forceinline__ float sum_xor16(float x) {
  const Pair p = pair_xor16(x);
  return p.a + p.b;
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// exp2(x - m) as the weight of a partial result with reference x against m;
// 0 for a partial result without a visible token.
__device__ __forceinline__ float rebase(float x, float m) { return x == kNegInf ? 0.0f : exp2_fast(x - m); }

// The least such factor of a sum that may be Inf, the least positive value: a factor
// that underflows to 0 would make it NaN, and every positive weight makes Inf.  What
// it leaves of a finite sum is far below the rounding of the others.
constexpr float kLeast = 0x1p-149f;
__device__ __forceinline__ float rebase_joined(float x, float m) {
  return x == kNegInf ? 0.0f : fmaxf(exp2_fast(x - m), kLeast);
}

}  // namespace w4a4
