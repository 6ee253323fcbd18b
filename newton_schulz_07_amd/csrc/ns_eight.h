// ns_eight.h - 8-bit values (e4m3) with a power of two as the scale of a block.
#pragma once

#include "ns_device.h"
#include "ns_lanes.h"

namespace ns {

// The scale of a block, as its E8M0 byte b (2^(b - 127)): the least power of two
// from 2^-126 on with largest <= 448 scale.  448 = 1.75 * 2^8, so it is the
// largest's own power of two less 8, and one more if its mantissa is above 1.75
// (the addition then carries into the exponent).
__device__ __forceinline__ unsigned scale_byte(float largest) {
  const int b = (int)((__float_as_uint(largest) + 0x1fffffu) >> 23) - 8;
  return (unsigned)(b > 1 ? b : 1);
}
__device__ __forceinline__ float inverse_scale(unsigned b) { return __uint_as_float((254u - b) << 23); }  // b: scale_byte's
// |v|, and 0 for what no scale can hold (infinities and NaN: they become NaN)
__device__ __forceinline__ float finite_magnitude(float v) {
  const float a = fabsf(v);
  return a < __builtin_inff() ? a : 0.0f;
}

// 8 values divided by their scale, each rounded to the nearest e4m3 value, ties to even.
__device__ __forceinline__ uint2 to_eight(const float* f, float inverse) {
  int a = 0, b = 0;
  a = __builtin_amdgcn_cvt_pk_fp8_f32(f[0] * inverse, f[1] * inverse, a, false);
  a = __builtin_amdgcn_cvt_pk_fp8_f32(f[2] * inverse, f[3] * inverse, a, true);
  b = __builtin_amdgcn_cvt_pk_fp8_f32(f[4] * inverse, f[5] * inverse, b, false);
  b = __builtin_amdgcn_cvt_pk_fp8_f32(f[6] * inverse, f[7] * inverse, b, true);
  return make_uint2((unsigned)a, (unsigned)b);
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// A scale as the fp32 operand of a conversion, which reads its exponent only (0: 2^-127).
__device__ __forceinline__ float scale_exponent(unsigned b) { return __uint_as_float(b << 23); }

// 4 e4m3 values times 2^(b - 127), exact but where the result is below the type's normal range.
__device__ __forceinline__ uint2 from_eight4(unsigned v, float scale, bf16) {
  const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, scale, false);
  const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, scale, true);
  return make_uint2(__builtin_bit_cast(unsigned, lo), __builtin_bit_cast(unsigned, hi));
}
__device__ __forceinline__ uint4 from_eight4(unsigned v, float scale, float) {
  const f32x2 lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(v, scale, false);
  const f32x2 hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(v, scale, true);
  return make_uint4(__float_as_uint(lo[0]), __float_as_uint(lo[1]), __float_as_uint(hi[0]), __float_as_uint(hi[1]));
}

}  // namespace ns
