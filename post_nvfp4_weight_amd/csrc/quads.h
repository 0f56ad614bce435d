// How the few-row kernels deal a product's operands to the lanes (gfx950).
//
// A matrix instruction's operands take row l % 16 in lane l, so that four
// neighbouring lanes read four rows, and a load instruction costs the address
// unit a cycle for each of them where four lanes in one line cost one: 64 cycles
// instead of 16 for 1024 bytes.  Where weights are read once from memory and the
// matrix cores idle, the lanes are dealt otherwise.  Lane l = 16 q + 4 a + b, and
// k in chunks of 16 pieces of 32:
//   A, load i (of four): channel 4 a + i, piece 4 q + b, so that four neighbours
//      read 64 consecutive bytes of 4-bit codes;  row 4 a + b of the product is
//      channel 4 a + i over the pieces b, 4 + b, 8 + b and 12 + b alone;
//   B: column 4 t + b is token t over the same pieces.
// The result at row 4 a + b, column 4 t + b is channel 4 a + i, token t over those
// pieces, and its sum over b is the whole (entries of a row and a column with
// different b mean nothing).  A product thus serves 4 tokens instead of 16.
#pragma once

#include "common.h"

namespace nvq {

__device__ __forceinline__ int quad_piece(int lane) { return 4 * (lane >> 4) + (lane & 3); }
__device__ __forceinline__ int quad_column(int lane) { return (lane >> 2) & 3; }   // a of A, the token of B

// The sums of 16 channels and 4 tokens out of the four loads' products: the lane
// gets channel 4 q + b and its column's token, q = l / 16, b = l % 4.
__device__ __forceinline__ float quad_sum(const f32x4 (&acc)[4], int lane) {
  const int b = lane & 3;
  float r = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // (register b of lane 16 q + 4 t + b: row 4 q + b, column 4 t + b)
    float v = b == 0 ? acc[i][0] : b == 1 ? acc[i][1] : b == 2 ? acc[i][2] : acc[i][3];
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xF, 0xF, false));   // lanes 1, 0, 3, 2
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xF, 0xF, false));   // lanes 2, 3, 0, 1
    r = b == i ? v : r;
  }
  return r;
}

}  // namespace nvq
