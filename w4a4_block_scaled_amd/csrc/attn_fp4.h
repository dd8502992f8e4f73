// A query's operand of the scaled MFMA, whose other one is a 4-bit cache's keys as they
// are: codes and scale bytes.
#pragma once

#include "attn_common.h"

namespace w4a4 {
namespace {

typedef int at_i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t at_u32x6 __attribute__((ext_vector_type(6)));
typedef float at_f32x32 __attribute__((ext_vector_type(32)));
typedef __bf16 at_bf16x32 __attribute__((ext_vector_type(32)));

__host__ __device__ constexpr int part_shift(int p) { return p == 0 ? 0 : 5 * p - 1; }

// The PARTS (up to 4) FP6 parts of 32 values of a query, and their scale bytes (one each;
// NaN's byte where a value is Inf or NaN).  With the largest value in [2, 4) 2^e, the parts'
// units are 2^e, 2^(e - 4), 2^(e - 9) and 2^(e - 14).  E2M3 has steps of 2^-2 in [2, 4) and of
// 2^-3 below, so the first part is right to 2^-3 of its unit, which is two of the next one's;
// each of those is right to 2^-4 of its own, two again of the next: all four together to
// 2^(e - 18).  Exponents below -108 count as that, where this is 2^-126: what is rounded on
// the way to a part is then never a subnormal that matters.
template <class T, int PARTS>
__device__ __forceinline__ uint32_t split_query(const uint16_t* row, at_u32x6 (&part)[PARTS]) {
  float x[32];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const at_u32x4 u = *reinterpret_cast<const at_u32x4*>(row + 8 * i);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[8 * i + 2 * k] = T::low(u[k]);
      x[8 * i + 2 * k + 1] = T::high(u[k]);
    }
  }
#pragma unroll
  for (int i = 0; i < 32; ++i) top = max(top, __builtin_bit_cast(uint32_t, x[i]) & 0x7fffffffu);
  const bool odd = top >= 0x7f800000u;
  const int e = max(int(top >> 23) - 128, -108);
  uint32_t bytes = 0;
#pragma unroll
  for (int p = 0; p < PARTS; ++p) {
    const uint32_t byte = uint32_t(e - part_shift(p) + 127);
    const float scale = __builtin_bit_cast(float, byte << 23);
    at_bf16x32 b;
#pragma unroll
    for (int i = 0; i < 32; ++i) b[i] = (__bf16)x[i];
    part[p] = __builtin_amdgcn_cvt_scalef32_pk32_fp6_bf16(b, scale);
    if (p + 1 < PARTS) {
      const at_f32x32 y = __builtin_amdgcn_cvt_scalef32_pk32_f32_fp6(part[p], scale);
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] -= y[i];
    }
    bytes |= (odd ? 255u : byte) << (8 * p);
  }
  return bytes;
}

}  // namespace
}  // namespace w4a4
