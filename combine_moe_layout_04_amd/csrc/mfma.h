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

// Eight floats as operands of three bfloat16 products: their sign and exponent
// with 8 bits of the significand each, cut off, not rounded, so that hi + mid + lo
// is the float itself and a product keeps all of its 24 bits.
//
// Beyond the finite numbers that is not so: an infinity has no remainder, and an
// infinity in the other operand meets parts that are zero.  Either way the sum
// becomes NaN, and never anything else that is wrong, since a float's parts have
// one sign.  So a product is formed with FINITE parts first, and again with the
// others where the result has a NaN: then an infinity is all in hi, and mid and lo
// meet the other operand's finite_part.
template <bool FINITE>
struct Parts {
  u32x4 hi, mid, lo;
  __device__ __forceinline__ explicit Parts(const float (&f)[8]) {
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      float v[2], r[2], l[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        v[i] = f[2 * d + i];
        r[i] = v[i] - high_half(v[i]);
        if (!FINITE && r[i] != r[i]) r[i] = 0.f;
        l[i] = r[i] - high_half(r[i]);
      }
      hi[d] = high_halves(v[0], v[1]);
      mid[d] = high_halves(r[0], r[1]);
      lo[d] = high_halves(l[0], l[1]);
    }
  }

 private:
  static __device__ __forceinline__ float high_half(float v) { return __uint_as_float(__float_as_uint(v) & 0xFFFF0000u); }
  static __device__ __forceinline__ uint32_t high_halves(float a, float b) {
    return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
  }
};

// A chunk of bfloat16 with zeros for infinities and NaN.
__device__ __forceinline__ u32x4 finite_part(u32x4 c) {
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    if ((c[d] & 0x00007F80u) == 0x00007F80u) c[d] &= 0xFFFF0000u;
    if ((c[d] & 0x7F800000u) == 0x7F800000u) c[d] &= 0x0000FFFFu;
  }
  return c;
}

// acc += bfloat16 rows . eight floats a lane
template <bool FINITE>
__device__ __forceinline__ f32x4 mma_parts(const u32x4 row, const Parts<FINITE>& p, f32x4 acc) {
  const u32x4 rest = FINITE ? row : finite_part(row);
  acc = mma_chunk<kBF16>(row, p.hi, acc);
  acc = mma_chunk<kBF16>(rest, p.mid, acc);
  return mma_chunk<kBF16>(rest, p.lo, acc);
}

// Whether any lane of the wave has a NaN in these results.
template <int N>
__device__ __forceinline__ bool any_nan(const f32x4 (&v)[N]) {
  bool nan = false;
#pragma unroll
  for (int i = 0; i < N; ++i) nan |= __builtin_isunordered(v[i][0], v[i][1]) | __builtin_isunordered(v[i][2], v[i][3]);
  return __ballot(nan) != 0;
}

// Rows in memory as a buffer of `bytes` from p (uniform over the wave): a load
// whose offset is past the end gives zeros and touches no memory, so the ends
// of rows and tiles need no branches.  Offsets are 32 bits; kOutside lies past
// every buffer made here (each below 2 GiB).
constexpr uint32_t kOutside = 0x80000000u;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rows(const void* p, size_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)(uint32_t)bytes, 0x00027000);
}

// The chunk at byte `lane_off` (per lane) + `off` (uniform, inside the buffer:
// it is the lane's part that is held against the end).  ONCE: read by
// nobody else, so marked non-temporal; that pays only where one instruction
// takes whole 128-byte lines.
template <bool ONCE = false>
__device__ __forceinline__ u32x4 load_rows(__amdgpu_buffer_rsrc_t rows, uint32_t lane_off, uint32_t off) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rows, (int)lane_off, (int)off, ONCE ? 2 : 0));
}

// Tiles of 4 rows by 256 bytes of each, one load instruction in which every
// quad of lanes takes 64 contiguous bytes.  That order is what the address unit
// wants: 1 KiB loads from L2 run at 25.6 TB/s so, and at 9.2 TB/s where each
// lane of a quad is on another row (MI355X), as the operand layout above would
// have it.  As an operand the tile's 16 rows are the 4 rows with 4 chunks each
// (every fourth lane quarter's); the other operand's 16 columns are 4 rows
// likewise.  The result's elements that meet in the same chunk are one of the
// four in each lane; a quad of lanes holds the four parts of one sum.  Three
// quarters of the products are not used: where memory is the limit the matrix
// cores have far more to spare.
struct Lane {
  int row, chunk;  // of the 4 rows, of the 16 chunks of its 256 bytes
  __device__ __forceinline__ Lane() : row((lane_id() >> 2) & 3), chunk((lane_id() >> 4) * 4 + (lane_id() & 3)) {}
  // the joined result in this lane: first operand's row, second operand's row
  __device__ __forceinline__ int first() const { return lane_id() >> 4; }
  __device__ __forceinline__ int second() const { return row; }
};

template <int CTRL>
__device__ __forceinline__ float quad_move(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}

// The sum of the parts, in every lane of the quad.
__device__ __forceinline__ float join_parts(f32x4 acc) {
  const int k = lane_id() & 3;
  float v = k == 0 ? acc[0] : k == 1 ? acc[1] : k == 2 ? acc[2] : acc[3];
  v += quad_move<0xB1>(v);  // lanes 1 0 3 2
  v += quad_move<0x4E>(v);  // lanes 2 3 0 1
  return v;
}

// Keeps loads and products in the order they are written in: left alone, the
// compiler gathers the loads of a software pipeline and waits for all of them.
__device__ __forceinline__ void in_order() { __builtin_amdgcn_sched_barrier(0); }

}  // namespace moe
