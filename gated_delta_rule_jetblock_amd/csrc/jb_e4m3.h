// jb_e4m3.h -- values in 8 bits: e4m3 codes (1 sign, 4 exponent and 3 fraction bits, bias
// 7; largest 448, 0x7f and 0xff NaN, no infinity) times a power-of-two scale that is held as
// its exponent e: 2^(e - 127), 255 NaN.  A code times a scale is a bf16 value, but where it
// is 2^128 or more (scales from 2^120 on), which bf16 and fp32 read as an infinity.
#pragma once

#include <math.h>

#include "jb_device.h"

namespace jb {

typedef unsigned int e4m3_u4_t __attribute__((ext_vector_type(4)));
typedef float e4m3_f2_t __attribute__((ext_vector_type(2)));

// The scale as the conversion to bf16 takes it: it looks at the exponent bits only, and
// reads all zeros as 2^-127 and all ones as NaN (checked for every code and exponent; what
// falls below bf16's smallest number is rounded, what passes its largest is an infinity).
__device__ __forceinline__ float scale_of(uint32_t e) { return __uint_as_float(e << 23); }

// 8 codes, in order, as bf16
__device__ __forceinline__ e4m3_u4_t bf16_of_e4m3(uint32_t lo, uint32_t hi, float scale) {
  return e4m3_u4_t{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true))};
}

// 2^(e - 127) as a number
__device__ __forceinline__ float scale_value(uint32_t e) {
  return e == 255u ? NAN : __uint_as_float(e ? e << 23 : 1u << 22);
}

// 4 codes as floats
__device__ __forceinline__ float4 floats_of_e4m3(uint32_t u, uint32_t e) {
  const e4m3_f2_t a = __builtin_amdgcn_cvt_pk_f32_fp8(u, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(u, true);
  const float s = scale_value(e);
  return make_float4(a[0] * s, a[1] * s, b[0] * s, b[1] * s);
}

}  // namespace jb
