// Rounding to 8-bit integers with a scale for each row.
//
//   s = amax / 127 in float32, at least 2^-126;  q = the integer nearest to x / s,
//   ties to even.
// The quotient is not formed: x times about 1 / s is within one step of it, and
// the remainder x - q s is exact in float32 (it is a multiple of the smaller operand's
// last place and not larger than s), so comparing it with s / 2 settles the rounding.
// That makes the result a function of the numbers alone, the same in every kernel.
#pragma once

#include "device_common.h"

namespace moe {

// bits of the largest |x| (as unsigned integers they are ordered like the values, NaN above all)
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// amax / 127, rounded as a division is: the product with the rounded 1 / 127 is within one
// place of it, its remainder is exact, and one step from there rounds right (on the CPU
// equal to the division for every amax of the exponents tried, the ends among them).
__device__ __forceinline__ float quant_scale(uint32_t amax_bits) {
  const float m = __uint_as_float(amax_bits), q = m * (1.f / 127.f);
  const float s = __builtin_fmaf(__builtin_fmaf(-127.f, q, m), 1.f / 127.f, q);
  if (!(m < INFINITY)) return m;  // infinite or NaN, as it is
  return s < 0x1p-126f ? 0x1p-126f : s;
}

// About 1 / scale: what is made with it is corrected where that matters.
__device__ __forceinline__ float quant_inverse(float s) { return __builtin_amdgcn_rcpf(s); }

// The integer (as a float) nearest to x / s: exact, for a finite row.
__device__ __forceinline__ float quant_exact(float x, float s, float inv) {
  float q = rintf(x * inv);
  const float r = __builtin_fmaf(-q, s, x), h = 0.5f * s;
  const bool odd = (static_cast<int>(q) & 1) != 0;
  if (r > h || (r == h && odd)) q += 1.f;
  else if (-r > h || (-r == h && odd)) q -= 1.f;
  return q;
}

// Values of one 16-byte chunk of a row (4 float32, 8 bfloat16) as its 4 or 8 bytes.
// |x / s| is at most 127 (1 + 2^-23) and inv off by 2^-23 of itself, so x * inv is within
// 2^-15 of it: only where that lies nearer than 2^-14 to a half can its rounding be another
// than the quotient's.  A row with an infinity or NaN has that as its scale, and zeros:
// what is made of it is NaN.
template <int V>
__device__ __forceinline__ void store_quant(int8_t* row, int chunk, const float* f, float s, float inv) {
  float q[V], far = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float t = f[i] * inv;
    q[i] = rintf(t);
    far = fmaxf(far, fabsf(t - q[i]));
  }
  if (far > 0.5f - 0x1p-14f)
#pragma unroll
    for (int i = 0; i < V; ++i) q[i] = quant_exact(f[i], s, inv);
  const uint32_t keep = s < INFINITY ? 0xFFFFFFFFu : 0u;
  uint32_t w[V / 4];
#pragma unroll
  for (int d = 0; d < V / 4; ++d) {
    const uint32_t lo = __builtin_amdgcn_perm((uint32_t)(int)q[4 * d + 1], (uint32_t)(int)q[4 * d], 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm((uint32_t)(int)q[4 * d + 3], (uint32_t)(int)q[4 * d + 2], 0x04000C0Cu);
    w[d] = (lo | hi) & keep;
  }
  uint32_t* p = reinterpret_cast<uint32_t*>(row) + (size_t)chunk * (V / 4);
  if constexpr (V == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  else *p = w[0];
}

}  // namespace moe
