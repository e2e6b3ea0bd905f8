// Element-level pieces of MXFP4 (blocks of 32 E2M1 elements with an E8M0 scale) and
// of the kernels that write BF16: shared by the norm, the MXFP4 cast and its product.
//
// E2M1 (OCP Microscaling Formats): 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives,
// code = sign << 3 | index.  Two elements per byte, the even one in the low half.
#pragma once

#include "cast_common.h"

namespace fp8ds {

constexpr int kE2M1 = 2;

// What an element of a NaN block is stored as (the block's scale code 255 makes its
// values NaN; E2M1 has no NaN of its own): eight codes of 6.
constexpr uint32_t kFp4NanBlock = 0x77777777u;

// fp32 -> BF16, round to nearest even; NaN stays NaN.  gfx950 converts in hardware.
__device__ __forceinline__ uint32_t bf16_pair_rne(float a, float b) {
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  const bf16x2_t v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ uint16_t bf16_bits_rne(float a) {
  return __builtin_bit_cast(uint16_t, (__bf16)a);
}
__device__ __forceinline__ float bf16_round(float a) {
  return __uint_as_float((uint32_t)bf16_bits_rne(a) << 16);
}

// E8M0 code of a block whose largest |value| has fp32 bits `a`, for elements whose
// largest exponent is emax (2: E2M1, 8: E4M3, 15: E5M2): floor(log2 a) - emax + 127,
// which is the biased exponent of `a` less emax, 0 where that is negative (zero,
// subnormal and tiny blocks), 255 if the block holds an infinity or NaN.
__device__ __forceinline__ uint32_t mx_code(uint32_t a, uint32_t emax) {
  const uint32_t f = a >> 23;
  return f == 255u ? 255u : f > emax ? f - emax : 0u;
}

// 2^(127 - code) for a code below 255.
__device__ __forceinline__ float mx_multiplier(uint32_t code) {
  return __uint_as_float((254u - code) << 23);
}

// Eight E2M1 codes of v / 2^(code - 127) (code < 255): the multiplication is exact
// wherever the element does not round to zero, gfx950's conversion rounds to nearest
// even and saturates at 6.
__device__ __forceinline__ uint32_t fp4_codes8(const float (&v)[8], uint32_t code) {
  const float m = mx_multiplier(code);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0] * m, v[1] * m, 1.0f, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2] * m, v[3] * m, 1.0f, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4] * m, v[5] * m, 1.0f, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6] * m, v[7] * m, 1.0f, 3);
  return w;
}
__device__ __forceinline__ uint32_t fp4_code1(float v) {
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v, 0.0f, 1.0f, 0) & 15u;
}


// The eight values of a dword of codes with scale code `s`: exact in fp32 (2^-127 is
// subnormal there, and a product of it with an element is too).
__device__ __forceinline__ void fp4_values8(uint32_t c, uint32_t s, float (&v)[8]) {
  const float x = __uint_as_float(s == 255u ? 0x7FC00000u : s == 0u ? 0x00400000u : s << 23);
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0);
  const f32x2_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1);
  const f32x2_t d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2);
  const f32x2_t e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3);
  v[0] = a.x * x; v[1] = a.y * x; v[2] = b.x * x; v[3] = b.y * x;
  v[4] = d.x * x; v[5] = d.y * x; v[6] = e.x * x; v[7] = e.y * x;
}

}  // namespace fp8ds
