// Device-side helpers shared by the layout and row kernels (gfx950, wave64).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

constexpr int kWave = 64;

// One 16-byte chunk of a row: 4 fp32 or 8 bf16 elements.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

enum : int { kF32 = 0, kBF16 = 1 };

template <int DT>
struct Elems {
  static constexpr int kPerChunk = DT == kF32 ? 4 : 8;  // elements per 16-byte chunk
};

// bfloat16 -> float32 is exact: bf16 is the upper half of a binary32.
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// float32 -> bfloat16 bits, round to nearest, ties to even.  Adds 0x7FFF plus
// the lowest kept bit, then drops the low half; NaNs are made quiet and keep
// their sign and top payload bits.
__device__ __forceinline__ uint32_t f32_to_bf16(float f) {
  uint32_t b = __float_as_uint(f);
  if ((b & 0x7FFFFFFFu) > 0x7F800000u) return (b >> 16) | 0x40u;
  return (b + 0x7FFFu + ((b >> 16) & 1u)) >> 16;
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  return f32_to_bf16(lo) | (f32_to_bf16(hi) << 16);
}

// Unpack a chunk into its float32 elements (in memory order).
template <int DT>
__device__ __forceinline__ void unpack(const u32x4 c, float* f) {
  if constexpr (DT == kF32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(c[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16_lo(c[i]);
      f[2 * i + 1] = bf16_hi(c[i]);
    }
  }
}

// Pack float32 elements into a chunk, rounding to the row type.
template <int DT>
__device__ __forceinline__ u32x4 pack(const float* f) {
  u32x4 c;
  if constexpr (DT == kF32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = __float_as_uint(f[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
  }
  return c;
}

template <bool NT>
__device__ __forceinline__ void store_chunk(u32x4* p, const u32x4 v) {
  if constexpr (NT) {
    __builtin_nontemporal_store(v, p);
  } else {
    *p = v;
  }
}

__device__ __forceinline__ int lane_id() { return __lane_id(); }

__device__ __forceinline__ uint64_t lanes_below(int lane) {
  return (lane == 0) ? 0ull : (~0ull >> (64 - lane));
}

__device__ __forceinline__ int read_lane_i(int v, int lane) {
  return __builtin_amdgcn_readlane(v, lane);
}

__device__ __forceinline__ float read_lane_f(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

// Data-parallel move of a lane's value (DPP control CTRL, rows of 16 lanes in
// the mask ROWS); lanes without a source get 0.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp0(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}

// Inclusive sum over the lanes up to this one.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
  v += dpp0<0x111, 0xF>(v);  // row_shr 1, 2, 4, 8: rows of 16 lanes
  v += dpp0<0x112, 0xF>(v);
  v += dpp0<0x114, 0xF>(v);
  v += dpp0<0x118, 0xF>(v);
  v += dpp0<0x142, 0xA>(v);  // last lane of a row to the next row
  v += dpp0<0x143, 0xC>(v);  // lane 31 to the upper half
  return v;
}

// Largest value and sum over the wave, in every lane (the total arrives in lane 63).
// All overloads stand here: one in an unnamed namespace would hide these there.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max(v, dpp0<0x111, 0xF>(v));  // row_shr 1, 2, 4, 8: rows of 16 lanes
  v = max(v, dpp0<0x112, 0xF>(v));
  v = max(v, dpp0<0x114, 0xF>(v));
  v = max(v, dpp0<0x118, 0xF>(v));
  v = max(v, dpp0<0x142, 0xA>(v));  // last lane of a row to the next row
  v = max(v, dpp0<0x143, 0xC>(v));  // lane 31 to the upper half
  return (uint32_t)read_lane_i((int)v, 63);
}

__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
  const uint32_t hi = wave_max((uint32_t)(v >> 32));
  const uint32_t lo = wave_max((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
  return ((uint64_t)hi << 32) | lo;
}

__device__ __forceinline__ uint32_t wave_min(uint32_t v) { return ~wave_max(~v); }

template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_float(float v) {
  return __uint_as_float(dpp0<CTRL, ROWS>(__float_as_uint(v)));
}

__device__ __forceinline__ float wave_sum(float v) {
  v += dpp_float<0x111, 0xF>(v);
  v += dpp_float<0x112, 0xF>(v);
  v += dpp_float<0x114, 0xF>(v);
  v += dpp_float<0x118, 0xF>(v);
  v += dpp_float<0x142, 0xA>(v);
  v += dpp_float<0x143, 0xC>(v);
  return read_lane_f(v, 63);
}

// As dpp_float, but lanes without a source keep their own value.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_or_own(float v) {
  const int b = __float_as_int(v);
  return __int_as_float(__builtin_amdgcn_update_dpp(b, b, CTRL, ROWS, 0xF, false));
}

// The largest of the numbers (NaN only where there is nothing else).
__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, dpp_or_own<0x111, 0xF>(v));
  v = fmaxf(v, dpp_or_own<0x112, 0xF>(v));
  v = fmaxf(v, dpp_or_own<0x114, 0xF>(v));
  v = fmaxf(v, dpp_or_own<0x118, 0xF>(v));
  v = fmaxf(v, dpp_or_own<0x142, 0xA>(v));
  v = fmaxf(v, dpp_or_own<0x143, 0xC>(v));
  return read_lane_f(v, 63);
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int s = 32; s >= 1; s >>= 1) v += __shfl_xor(v, s, kWave);
  return v;
}

// Fold the 64 lane partials: for s = 32, 16, ..., 1 every lane adds the
// partial of lane (l xor s).  float32 addition is commutative, so every lane
// ends with the same value, the one partial 0 holds.
__device__ __forceinline__ float fold64(float v) {
#pragma unroll
  for (int s = 32; s >= 1; s >>= 1) {
    float o = __shfl_xor(v, s, kWave);
    v = __fadd_rn(v, o);
  }
  return v;
}

// exp(x) = 2^t (1 + rest) for |x| <= 200: t is the product with log2(e) rounded, and what that
// leaves of it is small.
__device__ __forceinline__ float exp_parts(float x, float& t) {
  t = x * 1.44269502f;  // log2(e) = 1.44269502 + 1.92596303e-8
  return __builtin_fmaf(x, 1.92596303e-8f, __builtin_fmaf(x, 1.44269502f, -t)) * 0.693147182f;
}

}  // namespace moe
