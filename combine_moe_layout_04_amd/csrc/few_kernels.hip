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
// over H.  A workgroup of the second owns 8 columns of out for all pairs: its
// waves share out the experts, leave each pair's 8 values in LDS, and the
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

constexpr int kUpWaves = 4;
constexpr int kUpDepth = 4;  // units of two steps in flight

// act for 16 columns of one expert.  A unit is 128 bytes of each row (two
// steps), so that a wave reads whole cache lines; units go to the waves in
// turn, and each wave keeps kUpDepth of them in flight.
template <int DT, int NR, int NT>
__global__ __launch_bounds__(kUpWaves* kWave) void few_up_kernel(FewArgs a) {
  constexpr int kDepth = NT == 1 ? kUpDepth : 2;
  __shared__ uint16_t list[kFewMaxPairs];
  __shared__ f32x4 part[kUpWaves][NT][2][kWave];
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave));
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
  const uint32_t row_bytes = (uint32_t)nch * 16;
  const int i0 = blockIdx.x * 16;
  const char* w13 = static_cast<const char*>(a.w13) + ((size_t)e * 2 * a.I + i0) * row_bytes;
  // rows past the last one are outside the buffer and read as zeros
  const size_t tile_bytes = (size_t)min(16, a.I - i0) * row_bytes;
  const auto gate = make_rows(w13, tile_bytes);
  const auto up = make_rows(w13 + (size_t)a.I * row_bytes, tile_bytes);
  const auto xs = make_rows(a.x, (size_t)a.T * row_bytes);
  const uint32_t w_off = (uint32_t)col * row_bytes + q * 16;
  const int units = (nch + 7) / 8;

  for (int first = 0; first < n; first += 16 * NT) {
    uint32_t x_off[NT];
#pragma unroll
    for (int c = 0; c < NT; ++c) {  // columns past the last pair repeat it and are not stored
      const int p = list[min(first + c * 16 + col, n - 1)];
      x_off[c] = (uint32_t)(p / a.K) * row_bytes + q * 16;
    }
    f32x4 g[NT], u[NT];
#pragma unroll
    for (int c = 0; c < NT; ++c) g[c] = u[c] = f32x4{0.f, 0.f, 0.f, 0.f};
    u32x4 wg[kDepth][2], wu[kDepth][2], b[kDepth][2][NT];
    auto fetch = [&](int d, int unit) {
      const int ch = unit * 8;
      const bool in0 = ch + q < nch, in1 = ch + 4 + q < nch;
      const uint32_t off = (uint32_t)ch * 16;
      wg[d][0] = load_rows(gate, in0 ? w_off : kOutside, off);
      wg[d][1] = load_rows(gate, in1 ? w_off + 64 : kOutside, off);
      wu[d][0] = load_rows(up, in0 ? w_off : kOutside, off);
      wu[d][1] = load_rows(up, in1 ? w_off + 64 : kOutside, off);
#pragma unroll
      for (int c = 0; c < NT; ++c) {
        b[d][0][c] = load_rows(xs, in0 ? x_off[c] : kOutside, off);
        b[d][1][c] = load_rows(xs, in1 ? x_off[c] + 64 : kOutside, off);
      }
    };
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      fetch(d, wave + d * kUpWaves);
      in_order();
    }
    for (int unit = wave; unit < units; unit += kDepth * kUpWaves) {
#pragma unroll
      for (int d = 0; d < kDepth; ++d) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int c = 0; c < NT; ++c) {
            g[c] = mma_chunk<DT>(wg[d][s], b[d][s][c], g[c]);
            u[c] = mma_chunk<DT>(wu[d][s], b[d][s][c], u[c]);
          }
        in_order();
        fetch(d, unit + (d + kDepth) * kUpWaves);  // past the end: zeros
        in_order();
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

// 8 columns of out, for every pair.  A wave's item is (group, part of the sum
// over I).  The 16 rows of a matrix-core tile are 8 rows of W2 twice, once for
// each half of the item's part, its 16 columns 8 pairs twice likewise; the two
// diagonal quarters of the result are the halves' sums, the others are not
// used.  So a workgroup needs 8 columns of out only, and there are enough
// workgroups for the chip at the usual widths.  Each item leaves its pairs' 8
// values in y[part][pair].
constexpr int kDownWaves = 16;

template <int DT, int NR>
__global__ __launch_bounds__(kDownWaves* kWave) void few_down_kernel(FewArgs a) {
  constexpr int kDepth = 6;  // steps in flight
  extern __shared__ f32x4 lds[];
  f32x4* y = lds;  // [split][pairs][2]: 8 columns as two quads
  uint16_t* lists = reinterpret_cast<uint16_t*>(lds + (size_t)a.split * a.pairs * 2);  // [kDownWaves][pairs]
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave));
  const int col = lane & 7, half = (lane >> 3) & 1, q = lane >> 4;
  uint16_t* list = lists + (size_t)wave * a.pairs;

  int id[NR];
  load_ids(a, id);
  const int nch = a.ich;  // chunks of an act or w2 row
  const uint32_t row_bytes = (uint32_t)nch * 16;
  const int h0 = blockIdx.x * 8;
  const size_t tile_bytes = (size_t)min(8, a.H - h0) * row_bytes;
  const auto mid = make_rows(a.mid, (size_t)a.pairs * row_bytes);
  const int items = a.groups * a.split;
  for (int it = wave; it < items; it += kDownWaves) {
    const int grp = it / a.split, part = it - grp * a.split;
    const int e = group_expert(a, id, grp);
    if (e < 0) continue;
    const int n = list_pairs(id, e, list);
    const auto w2 = make_rows(static_cast<const char*>(a.w2) + ((size_t)e * a.H + h0) * row_bytes, tile_bytes);
    // chunks [lo, hi) of this half of the part
    const int lo = part * a.part_ch + half * (a.part_ch / 2);
    const int hi = min(lo + a.part_ch / 2, nch);
    const int steps = a.part_ch / 8;
    const uint32_t w_off = (uint32_t)col * row_bytes + (lo + q) * 16;
    for (int first = 0; first < n; first += 8) {
      const int p = list[min(first + col, n - 1)];
      const uint32_t m_off = (uint32_t)p * row_bytes + (lo + q) * 16;
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
      u32x4 w[kDepth], b[kDepth];
      auto fetch = [&](int d, int step) {
        const bool in = lo + step * 4 + q < hi;
        w[d] = load_rows(w2, in ? w_off : kOutside, (uint32_t)step * 64);
        b[d] = load_rows(mid, in ? m_off : kOutside, (uint32_t)step * 64);
      };
#pragma unroll
      for (int d = 0; d < kDepth; ++d) {
        fetch(d, d);
        in_order();
      }
      for (int step = 0; step < steps; step += kDepth) {
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
          acc = mma_chunk<DT>(w[d], b[d], acc);
          in_order();
          fetch(d, step + kDepth + d);  // past the end: zeros
          in_order();
        }
      }
      // result rows 4q..4q+3 of column lane % 16: the second half's diagonal
      // quarter (q >= 2, columns 8..15) joins the first's
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] += __shfl(acc[i], lane + 40, kWave);
      if (q < 2 && half == 0 && first + col < n) y[((size_t)part * a.pairs + p) * 2 + q] = acc;
    }
  }
  __syncthreads();

  const float* yf = reinterpret_cast<const float*>(y);
  for (int o = threadIdx.x; o < a.T * 8; o += kDownWaves * kWave) {
    const int t = o >> 3, c = o & 7;
    if (h0 + c >= a.H) continue;
    float sum = 0.f;
    for (int k = 0; k < a.K; ++k) {
      const int p = t * a.K + k;
      const int64_t e = a.itype == MOE_I32 ? (int64_t)static_cast<const int*>(a.idx)[p]
                                           : static_cast<const int64_t*>(a.idx)[p];
      if (e < 0 || e >= a.E) continue;
      float v = yf[(size_t)p * 8 + c];
      for (int s = 1; s < a.split; ++s) v += yf[((size_t)s * a.pairs + p) * 8 + c];
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
  const size_t lds = (size_t)a.split * a.pairs * 32 + (size_t)kDownWaves * a.pairs * 2;
  hipLaunchKernelGGL((few_down_kernel<DT, NR>), dim3((a.H + 7) / 8), dim3(kDownWaves * kWave), lds, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_few(const FewArgs& args, hipStream_t s) {
  FewArgs a = args;
  a.groups = a.pairs > a.E ? a.E : a.pairs;
  a.split = 1;
  while (a.groups * a.split < kDownWaves && 2 * a.split * a.pairs <= kFewMaxPairs) a.split *= 2;
  a.part_ch = ((a.ich + a.split - 1) / a.split + 15) / 16 * 16;  // two halves of whole cache lines
  if (a.pairs <= kWave)
    return a.dtype == MOE_F32 ? launch_few_typed<kF32, 1>(a, s) : launch_few_typed<kBF16, 1>(a, s);
  return a.dtype == MOE_F32 ? launch_few_typed<kF32, 8>(a, s) : launch_few_typed<kBF16, 8>(a, s);
}

}  // namespace moe
