// A whole mixture-of-experts layer for a few tokens, in two kernels.
//
//   act[p]  = f(Wg_e x_t) * (Wu_e x_t)          pair p = (t, k), e = topk_idx[t, k]
//   out[t]  = sum_k w[t, k] * W2_e act[t, k]
//
// A decode batch reads far more weight bytes than it computes on: the chosen
// experts' weights, 3 H I elements each, are the floor, and each is read once
// per call.  The matrix cores take 16 weight rows against up to 16 of the
// expert's tokens a tile; one step of 1 KiB of weights costs 16 cycles of
// matrix core for bfloat16, about a twenty-fifth of what the bytes cost.
//
// No layout runs before: a call has at most 512 pairs, every wave holds their
// ids in registers, and ballots give an expert's pairs.  A workgroup of the
// first kernel owns (expert, 16 columns of act); its four waves split the sum
// over H.  A workgroup of the second owns 16 columns of out for all pairs: its
// waves share out the experts, leave each pair's 16 values in LDS, and the
// top-k sum is formed there in k order, so that no second pass over pairs, no
// atomics and no order left to chance remain.  An id outside [0, E) belongs to
// no expert here and adds nothing.
#include "device_common.h"
#include "internal.h"
#include "mfma.h"
#include "../../include/moe_layout.h"

namespace moe {
namespace {

// The ids of all pairs, pair 64 r + lane in register r; -1 where there is no
// pair or no expert.
template <int NR>
__device__ __forceinline__ void load_ids(const FewArgs& a, int (&id)[NR]) {
  const int lane = lane_id();
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const int p = r * kWave + lane;
    id[r] = -1;
    if (p < a.pairs) {
      const int64_t e = a.itype == MOE_I32 ? (int64_t)static_cast<const int*>(a.idx)[p]
                                           : static_cast<const int64_t*>(a.idx)[p];
      if (e >= 0 && e < a.E) id[r] = (int)e;
    }
  }
}

// Group g of the call: with fewer pairs than experts the expert of pair g,
// unless an earlier pair has the same one (-1 then); else expert g.
template <int NR>
__device__ __forceinline__ int group_expert(const FewArgs& a, const int (&id)[NR], int g) {
  if (a.pairs > a.E) return g;
  int e = -1;
#pragma unroll
  for (int r = 0; r < NR; ++r)
    if (g / kWave == r) e = read_lane_i(id[r], g % kWave);
  if (e < 0) return -1;
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const uint64_t same = __ballot(id[r] == e);
    if (same) return r * kWave + __builtin_ctzll(same) == g ? e : -1;
  }
  return -1;
}

// The pairs of expert e in ascending order, written to `list`; their number.
template <int NR>
__device__ __forceinline__ int list_pairs(const int (&id)[NR], int e, uint16_t* list) {
  const int lane = lane_id();
  int n = 0;
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const uint64_t mine = __ballot(id[r] == e);
    if (id[r] == e) list[n + __popcll(mine & lanes_below(lane))] = (uint16_t)(r * kWave + lane);
    n += __popcll(mine);
  }
  return n;
}

__device__ __forceinline__ float gated(float g, float u, int act) {
  if (act == MOE_ACT_SILU) return g / (1.f + expf(-g)) * u;
  const float y = 0.7978845608028654f * (g + 0.044715f * g * g * g);  // sqrt(2/pi)
  return 0.5f * g * (1.f + tanhf(y)) * u;
}

// One 64-byte step of 16 rows: this lane's chunk, zero past the row's end.
__device__ __forceinline__ u32x4 row_chunk(const u32x4* row, int j, int n) {
  u32x4 v = {0u, 0u, 0u, 0u};
  if (j < n) v = row[j];
  return v;
}

constexpr int kUpWaves = 4;

// act for 16 columns of one expert.  Steps go to the waves in pairs (128
// bytes of a row), so that a wave reads whole cache lines.
template <int DT, int NR, int NT>
__global__ __launch_bounds__(kUpWaves* kWave) void few_up_kernel(FewArgs a) {
  constexpr int kUnits = NT == 1 ? 4 : 2;  // pairs of steps in flight
  __shared__ uint16_t list[kFewMaxPairs];
  __shared__ f32x4 part[kUpWaves][NT][2][kWave];
  const int lane = lane_id(), wave = (int)(threadIdx.x / kWave);
  const int col = lane & 15, q = lane >> 4;

  int id[NR];
  load_ids(a, id);
  const int e = group_expert(a, id, blockIdx.y);
  if (e < 0) return;  // the whole workgroup: every wave holds the same ids
  int n = 0;
  if (wave == 0) {
    n = list_pairs(id, e, list);
  } else {
#pragma unroll
    for (int r = 0; r < NR; ++r) n += __popcll(__ballot(id[r] == e));
  }
  if (n == 0) return;
  __syncthreads();

  const int nch = a.hch;  // chunks of an x or w13 row
  const int i0 = blockIdx.x * 16;
  const int i = min(i0 + col, a.I - 1);  // rows past the end repeat the last one and are not stored
  const u32x4* w13 = static_cast<const u32x4*>(a.w13) + (size_t)e * 2 * a.I * nch;
  const u32x4* wg = w13 + (size_t)i * nch;
  const u32x4* wu = w13 + (size_t)(a.I + i) * nch;
  const u32x4* x = static_cast<const u32x4*>(a.x);

  for (int first = 0; first < n; first += 16 * NT) {
    const u32x4* xr[NT];
#pragma unroll
    for (int c = 0; c < NT; ++c) {  // columns past the last pair repeat it and are not stored
      const int p = list[min(first + c * 16 + col, n - 1)];
      xr[c] = x + (size_t)(p / a.K) * nch;
    }
    f32x4 g[NT], u[NT];
#pragma unroll
    for (int c = 0; c < NT; ++c) g[c] = u[c] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int j0 = wave * 8 + q; j0 - q < nch; j0 += kUpWaves * 8 * kUnits) {
      u32x4 ag[2 * kUnits], au[2 * kUnits], b[2 * kUnits][NT];
#pragma unroll
      for (int s = 0; s < 2 * kUnits; ++s) {
        const int j = j0 + (s / 2) * kUpWaves * 8 + (s & 1) * 4;
        ag[s] = row_chunk(wg, j, nch);
        au[s] = row_chunk(wu, j, nch);
#pragma unroll
        for (int c = 0; c < NT; ++c) b[s][c] = row_chunk(xr[c], j, nch);
      }
#pragma unroll
      for (int s = 0; s < 2 * kUnits; ++s)
#pragma unroll
        for (int c = 0; c < NT; ++c) {
          g[c] = mma_chunk<DT>(ag[s], b[s][c], g[c]);
          u[c] = mma_chunk<DT>(au[s], b[s][c], u[c]);
        }
    }
#pragma unroll
    for (int c = 0; c < NT; ++c) {
      part[wave][c][0][lane] = g[c];
      part[wave][c][1][lane] = u[c];
    }
    __syncthreads();
    for (int c = wave; c < NT; c += kUpWaves) {
      f32x4 sg = part[0][c][0][lane], su = part[0][c][1][lane];
#pragma unroll
      for (int v = 1; v < kUpWaves; ++v) {
        sg += part[v][c][0][lane];
        su += part[v][c][1][lane];
      }
      const int at = first + c * 16 + col;
      if (at < n) {
        const size_t row = (size_t)list[at] * a.I;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int ii = i0 + q * 4 + r;
          if (ii < a.I) {
            const float v = gated(sg[r], su[r], a.act);
            // act is rounded to the element type: the second product's
            // operand, as between two separate products
            if constexpr (DT == kF32) static_cast<float*>(a.mid)[row + ii] = v;
            else static_cast<uint16_t*>(a.mid)[row + ii] = (uint16_t)f32_to_bf16(v);
          }
        }
      }
    }
    __syncthreads();
  }
}

// 16 columns of out, for every pair.  Wave items are (group, part of the sum
// over I); each leaves its pairs' 16 values in y[part][pair].
template <int DT, int NR, int W>
__global__ __launch_bounds__(W* kWave) void few_down_kernel(FewArgs a) {
  constexpr int kSteps = 8;
  extern __shared__ f32x4 lds[];
  f32x4* y = lds;  // [split][pairs][4]: 16 columns as four quads
  uint16_t* lists = reinterpret_cast<uint16_t*>(lds + (size_t)a.split * a.pairs * 4);  // [W][pairs]
  const int lane = lane_id(), wave = (int)(threadIdx.x / kWave);
  const int col = lane & 15, q = lane >> 4;
  uint16_t* list = lists + (size_t)wave * a.pairs;

  int id[NR];
  load_ids(a, id);
  const int nch = a.ich;  // chunks of an act or w2 row
  const int h0 = blockIdx.x * 16;
  const int h = min(h0 + col, a.H - 1);
  const u32x4* mid = static_cast<const u32x4*>(a.mid);
  const int items = a.groups * a.split;
  for (int it = wave; it < items; it += W) {
    const int grp = it / a.split, part = it - grp * a.split;
    const int e = group_expert(a, id, grp);
    if (e < 0) continue;
    const int n = list_pairs(id, e, list);
    const u32x4* w2 = static_cast<const u32x4*>(a.w2) + ((size_t)e * a.H + h) * nch;
    const int lo = part * a.part_ch, hi = min(lo + a.part_ch, nch);
    for (int first = 0; first < n; first += 16) {
      const int p = list[min(first + col, n - 1)];
      const u32x4* row = mid + (size_t)p * nch;
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
      for (int j0 = lo + q; j0 - q < hi; j0 += 4 * kSteps) {
        u32x4 w[kSteps], b[kSteps];
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          w[s] = row_chunk(w2, j0 + 4 * s, hi);
          b[s] = row_chunk(row, j0 + 4 * s, hi);
        }
#pragma unroll
        for (int s = 0; s < kSteps; ++s) acc = mma_chunk<DT>(w[s], b[s], acc);
      }
      if (first + col < n) y[((size_t)part * a.pairs + p) * 4 + q] = acc;
    }
  }
  __syncthreads();

  const float* yf = reinterpret_cast<const float*>(y);
  for (int o = threadIdx.x; o < a.T * 16; o += W * kWave) {
    const int t = o >> 4, c = o & 15;
    if (h0 + c >= a.H) continue;
    float sum = 0.f;
    for (int k = 0; k < a.K; ++k) {
      const int p = t * a.K + k;
      const int64_t e = a.itype == MOE_I32 ? (int64_t)static_cast<const int*>(a.idx)[p]
                                           : static_cast<const int64_t*>(a.idx)[p];
      if (e < 0 || e >= a.E) continue;
      float v = yf[(size_t)p * 16 + c];
      for (int s = 1; s < a.split; ++s) v += yf[((size_t)s * a.pairs + p) * 16 + c];
      sum = __fadd_rn(sum, a.w ? __fmul_rn(a.w[p], v) : v);
    }
    const size_t at = (size_t)t * a.H + h0 + c;
    if constexpr (DT == kF32) static_cast<float*>(a.out)[at] = sum;
    else static_cast<uint16_t*>(a.out)[at] = (uint16_t)f32_to_bf16(sum);
  }
}

template <int DT, int NR>
hipError_t launch_few_typed(const FewArgs& a, hipStream_t s) {
  const dim3 up((a.I + 15) / 16, a.groups);
  if (a.pairs <= 8 * a.E)
    hipLaunchKernelGGL((few_up_kernel<DT, NR, 1>), up, dim3(kUpWaves * kWave), 0, s, a);
  else
    hipLaunchKernelGGL((few_up_kernel<DT, NR, 4>), up, dim3(kUpWaves * kWave), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  constexpr int W = 8;
  const size_t lds = (size_t)a.split * a.pairs * 64 + (size_t)W * a.pairs * 2;
  hipLaunchKernelGGL((few_down_kernel<DT, NR, W>), dim3((a.H + 15) / 16), dim3(W * kWave), lds, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_few(const FewArgs& args, hipStream_t s) {
  FewArgs a = args;
  a.groups = a.pairs > a.E ? a.E : a.pairs;
  a.split = 1;
  while (a.groups * a.split < 8 && 2 * a.split * a.pairs <= kFewMaxPairs) a.split *= 2;
  a.part_ch = ((a.ich + a.split - 1) / a.split + 7) / 8 * 8;  // whole cache lines
  if (a.pairs <= kWave)
    return a.dtype == MOE_F32 ? launch_few_typed<kF32, 1>(a, s) : launch_few_typed<kBF16, 1>(a, s);
  return a.dtype == MOE_F32 ? launch_few_typed<kF32, 8>(a, s) : launch_few_typed<kBF16, 8>(a, s);
}

}  // namespace moe
