// Row tiles of 16-bit elements in LDS and the matrix operands read from them.
#pragma once

#include "gdn_common.h"

namespace gdn {

typedef float f32x16 __attribute__((ext_vector_type(16)));

// Rows of D 16-bit elements in LDS, 16-byte pieces of a row permuted by the row's number
// (xor), for 64 banks of 4 bytes: the 16 rows that a cycle of a row-wise operand read takes,
// one piece each, and the 4 rows x 4 pieces of half a wave's transposing read then all lie in
// different banks (with the rows' numbers as they are, every transposing read took twice as long).
// The permutation has a period of 16 rows, so it is a constant of the lane.
template <int D>
__device__ __forceinline__ int piece_of(int row) {
  if constexpr (D >= 128) return ((row & 3) << 2) | ((row >> 2) & 3);  // 16 pieces to the banks
  else return (((row >> 1) & 1) << 2) | ((row >> 2) & 3);              // 8 pieces, two rows
}
// element offset of column c (a multiple of 4) of a row
template <int D>
__device__ __forceinline__ int at(int row, int c) {
  return row * D + (((c >> 3) ^ piece_of<D>(row)) << 3) + (c & 4);
}

// A value that the compiler must not keep computed things of across the loop:
// the LDS offsets that follow from it by one xor cost a register each otherwise.
__device__ __forceinline__ int fresh(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// A lane's column (lane % 16 of its group's 16) of 8 rows by two transposing reads
// of 4 rows (see lds_tr16), at element offsets a and b.
__device__ __forceinline__ uint4 column8(const uint16_t* tile, int a, int b) {
  const uint2 x = lds_tr16(tile + a), y = lds_tr16(tile + b);
  return make_uint4(x.x, x.y, y.x, y.y);
}

}  // namespace gdn
