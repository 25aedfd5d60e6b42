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

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Two floats as bfloat16, nearest even (one instruction).
__device__ __forceinline__ uint32_t round_bf16x2(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

// Rows in memory as a buffer of `bytes` from p (uniform over the wave): a load
// whose offset is past the end gives zeros and touches no memory, so the ends
// of rows and tiles need no branches.  Offsets are 32 bits; kOutside lies past
// every buffer made here (each below 2 GiB).
constexpr uint32_t kOutside = 0x80000000u;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rows(const void* p, size_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)(uint32_t)bytes, 0x00027000);
}

// The chunk at byte `lane_off` (per lane) + `off` (uniform).  ONCE: read by
// nobody else, so marked non-temporal; that pays only where one instruction
// takes whole 128-byte lines.
template <bool ONCE = false>
__device__ __forceinline__ u32x4 load_rows(__amdgpu_buffer_rsrc_t rows, uint32_t lane_off, uint32_t off) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rows, (int)lane_off, (int)off, ONCE ? 2 : 0));
}

// Keeps loads and products in the order they are written in: left alone, the
// compiler gathers the loads of a software pipeline and waits for all of them.
__device__ __forceinline__ void in_order() { __builtin_amdgcn_sched_barrier(0); }

}  // namespace moe
