// Matrix-core steps on rows held as 16-byte chunks (gfx950, wave64).
//
// Both operands of a step are rows whose elements run along the summed axis.
// Lane l holds a chunk of row (or column) l % 16; its quarter q = l / 16 says
// which of four neighbouring chunks.  Both operands use the same chunk for the
// same quarter, so the order in which the hardware sums a chunk's elements
// does not matter.  The result tile is 16 x 16 float32: lane l holds rows
// 4q .. 4q+3 (of the first operand) of column l % 16 (of the second).
#pragma once

#include "device_common.h"

namespace moe {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// acc += rows(a) . columns(b) over four chunks of the summed axis: one
// 16x16x32 instruction for bfloat16, four 16x16x4 for float32 (element j of
// every lane's chunk in the j-th).
template <int DT>
__device__ __forceinline__ f32x4 mma_chunk(const u32x4 a, const u32x4 b, f32x4 acc) {
  if constexpr (DT == kBF16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                   acc, 0, 0, 0);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[j]), __uint_as_float(b[j]), acc, 0, 0, 0);
    return acc;
  }
}

}  // namespace moe
