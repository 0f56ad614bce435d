// NVFP4 codes and block scales to bf16, as the weight-only products stage them (gfx950).
#pragma once

#include "common.h"

namespace nvq {

typedef float f32x2c __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2c __attribute__((ext_vector_type(2)));

// Byte B of word (two codes, low nibble first) under block scale value s ->
// packed bf16 pair of e2m1 * s.  The E2M1 decode is the hardware's FP4
// conversion at scale 1 (its scale operand applies only a power of two, so
// the E4M3 scale is multiplied in fp32; the product has at most 6
// significant bits and is exact, as is its bf16 conversion).
template <int B>
__device__ __forceinline__ uint32_t dq_byte(uint32_t word, float s) {
  const f32x2c v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, 1.0f, B);
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2c{v.x * s, v.y * s}, bf16x2c));
}
__device__ __forceinline__ uint32_t dq_byte(uint32_t word, float s, int b) {   // b known after unrolling
  switch (b) {
    case 0: return dq_byte<0>(word, s);
    case 1: return dq_byte<1>(word, s);
    case 2: return dq_byte<2>(word, s);
    default: return dq_byte<3>(word, s);
  }
}

// Signed E4M3 value of byte B of word, NaN for 0x7F and 0xFF (the scale of a
// row that the quantizer rejected): the hardware's FP8 conversion, whose
// OCP format on gfx950 is E4M3FN.
template <int B>
__device__ __forceinline__ float e4m3_byte(uint32_t word) {
  return __builtin_amdgcn_cvt_f32_fp8((int)word, B);
}

}  // namespace nvq
