// Rounding to 8-bit integers with a scale for each row.
//
//   s = amax / 127 in float32, at least 2^-126;  q = the integer nearest to x / s,
//   ties to even.
// The quotient is not formed: x times the rounded 1 / s is within one step of it, and
// the remainder x - q s is exact in float32 (it is a multiple of the smaller operand's
// last place and not larger than s), so comparing it with s / 2 settles the rounding.
// That makes the result a function of the numbers alone, the same in every kernel.
#pragma once

#include "device_common.h"

namespace moe {

// bits of the largest |x| (as unsigned integers they are ordered like the values, NaN above all)
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

__device__ __forceinline__ float quant_scale(uint32_t amax_bits) {
  const float s = __uint_as_float(amax_bits) / 127.f;
  return s < 0x1p-126f ? 0x1p-126f : s;  // a NaN stays
}

// A row with an infinity or NaN has that as its scale, and zeros: what is made of it is NaN.
__device__ __forceinline__ int quant_one(float x, float s, float inv) {
  if (!(s < INFINITY)) return 0;
  float q = rintf(x * inv);
  const float r = __builtin_fmaf(-q, s, x), h = 0.5f * s;
  const bool odd = (static_cast<int>(q) & 1) != 0;
  if (r > h || (r == h && odd)) q += 1.f;
  else if (-r > h || (-r == h && odd)) q -= 1.f;
  return static_cast<int>(fminf(fmaxf(q, -127.f), 127.f));
}

// Values of one 16-byte chunk of a row (4 float32, 8 bfloat16) as its 4 or 8 bytes.
template <int V>
__device__ __forceinline__ void store_quant(int8_t* row, int chunk, const float* f, float s, float inv) {
  uint32_t w[V / 4];
#pragma unroll
  for (int d = 0; d < V / 4; ++d) {
    w[d] = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[d] |= ((uint32_t)quant_one(f[4 * d + i], s, inv) & 0xFFu) << (8 * i);
  }
  uint32_t* p = reinterpret_cast<uint32_t*>(row) + (size_t)chunk * (V / 4);
  if constexpr (V == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  else *p = w[0];
}

}  // namespace moe
