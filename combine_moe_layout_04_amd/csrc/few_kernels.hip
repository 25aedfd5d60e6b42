// A whole mixture-of-experts layer for a few tokens, in two kernels.
//
//   act[p]  = f(Wg_e x_t) * (Wu_e x_t)          pair p = (t, k), e = topk_idx[t, k]
//   out[t]  = sum_k w[t, k] * W2_e act[t, k]
//
// A decode batch reads far more weight bytes than it computes on: the chosen
// experts' weights, 3 H I elements each, are the floor, and each is read once
// per call.  The matrix cores take 8 weight rows against up to 8 of the
// expert's tokens a tile; 1 KiB of weights costs 16 cycles of one matrix core
// for bfloat16, about a twenty-fifth of what the bytes cost.
//
// No layout runs before: a call has at most 512 pairs, every wave holds their
// ids in registers, and ballots give an expert's pairs.  A workgroup of the
// first kernel owns (expert, columns of act); its four waves split the sum over H.
//  A workgroup of the second owns 8 columns of out for all pairs: its
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

// A weight tile is 8 rows by one 128-byte line of each, one load instruction
// of whole lines.  As an operand its 16 rows are the 8 rows twice, with the
// first and the second half of the line; the 16 columns of the other operand
// are 8 tokens twice likewise.  Two diagonal quarters of the result are the
// halves' sums over the line, the other two are not used: the matrix cores
// have far more to spare than the memory has.  (Streaming 0.8 GB of rows of 4
// KiB on MI355X: 16 rows by 64 bytes an instruction 6.2 TB/s, whole lines
// non-temporal 6.9 TB/s.)
struct Lane {
  int row, half, q;  // row (or token) of the tile, half of its line, chunk of the half
  __device__ __forceinline__ Lane() : row(lane_id() & 7), half((lane_id() >> 3) & 1), q(lane_id() >> 4) {}
  __device__ __forceinline__ int chunk() const { return half * 4 + q; }
};

// Rows 4q..4q+3 (q < 2) of column `row` in the lanes of the first half: the
// second half's quarter (rows 8.., columns 8..) joins the first's.
__device__ __forceinline__ f32x4 join_halves(f32x4 acc) {
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] += __shfl(acc[i], lane_id() + 40, kWave);
  return acc;
}

constexpr int kUpWaves = 4;

// act for 8 RT columns of one expert, NT tiles of 8 of its pairs at a time.
// The lines of a row go to the waves in turn; a wave keeps `kDepth` lines of
// every row of its tiles in flight.
template <int DT, int NR, int RT, int NT>
__global__ __launch_bounds__(kUpWaves* kWave) void few_up_kernel(FewArgs a) {
  constexpr int kDepth = NT == 1 ? 4 : 2;
  __shared__ uint16_t list[kFewMaxPairs];
  __shared__ f32x4 part[kUpWaves][NT][RT][2][kWave / 4];
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave));
  const Lane at;

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
  const int i0 = blockIdx.x * 8 * RT;
  const char* w13 = static_cast<const char*>(a.w13) + ((size_t)e * 2 * a.I + i0) * row_bytes;
  // rows past the last one are outside the buffer and read as zeros
  const size_t tile_bytes = (size_t)min(8 * RT, a.I - i0) * row_bytes;
  const auto gate = make_rows(w13, tile_bytes);
  const auto up = make_rows(w13 + (size_t)a.I * row_bytes, tile_bytes);
  const auto xs = make_rows(a.x, (size_t)a.T * row_bytes);
  const uint32_t w_off = (uint32_t)at.row * row_bytes + at.chunk() * 16;
  const int lines = (nch + 7) / 8;

  for (int first = 0; first < n; first += 8 * NT) {
    uint32_t x_off[NT];
#pragma unroll
    for (int c = 0; c < NT; ++c) {  // columns past the last pair repeat it and are not stored
      const int p = list[min(first + c * 8 + at.row, n - 1)];
      x_off[c] = (uint32_t)(p / a.K) * row_bytes + at.chunk() * 16;
    }
    f32x4 g[NT][RT], u[NT][RT];
#pragma unroll
    for (int c = 0; c < NT; ++c)
#pragma unroll
      for (int r = 0; r < RT; ++r) g[c][r] = u[c][r] = f32x4{0.f, 0.f, 0.f, 0.f};
    u32x4 wg[kDepth][RT], wu[kDepth][RT], b[kDepth][NT];
    auto fetch = [&](int d, int line) {
      const bool in = line * 8 + at.chunk() < nch;
      const uint32_t off = (uint32_t)line * 128;
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        wg[d][r] = load_rows<true>(gate, in ? w_off + r * 8 * row_bytes : kOutside, off);
        wu[d][r] = load_rows<true>(up, in ? w_off + r * 8 * row_bytes : kOutside, off);
      }
#pragma unroll
      for (int c = 0; c < NT; ++c) b[d][c] = load_rows(xs, in ? x_off[c] : kOutside, off);
    };
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      fetch(d, wave + d * kUpWaves);
      in_order();
    }
    for (int line = wave; line < lines; line += kDepth * kUpWaves) {
#pragma unroll
      for (int d = 0; d < kDepth; ++d) {
#pragma unroll
        for (int c = 0; c < NT; ++c)
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            g[c][r] = mma_chunk<DT>(wg[d][r], b[d][c], g[c][r]);
            u[c][r] = mma_chunk<DT>(wu[d][r], b[d][c], u[c][r]);
          }
        in_order();
        fetch(d, line + (d + kDepth) * kUpWaves);  // past the end: zeros
        in_order();
      }
    }
#pragma unroll
    for (int c = 0; c < NT; ++c)
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const f32x4 sg = join_halves(g[c][r]), su = join_halves(u[c][r]);
        if (at.half == 0 && at.q < 2) {
          part[wave][c][r][0][at.q * 8 + at.row] = sg;
          part[wave][c][r][1][at.q * 8 + at.row] = su;
        }
      }
    __syncthreads();
    // 16 lanes per tile: quad and pair
    for (int i = threadIdx.x; i < NT * RT * 16; i += kUpWaves * kWave) {
      const int slot = i & 15, r = (i >> 4) % RT, c = (i >> 4) / RT;
      f32x4 sg = part[0][c][r][0][slot], su = part[0][c][r][1][slot];
#pragma unroll
      for (int v = 1; v < kUpWaves; ++v) {
        sg += part[v][c][r][0][slot];
        su += part[v][c][r][1][slot];
      }
      const int pos = first + c * 8 + (slot & 7);
      if (pos < n) {
        const size_t row = (size_t)list[pos] * a.I;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int ii = i0 + r * 8 + (slot >> 3) * 4 + k;
          if (ii < a.I) {
            const float v = gated(sg[k], su[k], a.act);
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
// over I); it leaves its pairs' 8 values in y[part][pair].
constexpr int kDownWaves = 16;

template <int DT, int NR>
__global__ __launch_bounds__(kDownWaves* kWave) void few_down_kernel(FewArgs a) {
  constexpr int kDepth = 6;  // lines in flight
  extern __shared__ f32x4 lds[];
  f32x4* y = lds;  // [split][pairs][2]: 8 columns as two quads
  uint16_t* lists = reinterpret_cast<uint16_t*>(lds + (size_t)a.split * a.pairs * 2);  // [kDownWaves][pairs]
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave));
  const Lane at;
  uint16_t* list = lists + (size_t)wave * a.pairs;

  int id[NR];
  load_ids(a, id);
  const int nch = a.ich;  // chunks of an act or w2 row
  const uint32_t row_bytes = (uint32_t)nch * 16;
  const int h0 = blockIdx.x * 8;
  const size_t tile_bytes = (size_t)min(8, a.H - h0) * row_bytes;
  const auto mid = make_rows(a.mid, (size_t)a.pairs * row_bytes);
  const uint32_t w_off = (uint32_t)at.row * row_bytes + at.chunk() * 16;
  const int lines = (nch + 7) / 8;
  const int items = a.groups * a.split;
  for (int it = wave; it < items; it += kDownWaves) {
    const int grp = it / a.split, part = it - grp * a.split;
    const int e = group_expert(a, id, grp);
    if (e < 0) continue;
    const int n = list_pairs(id, e, list);
    const auto w2 = make_rows(static_cast<const char*>(a.w2) + ((size_t)e * a.H + h0) * row_bytes, tile_bytes);
    const int lo = part * a.part_lines, hi = min(lo + a.part_lines, lines);
    for (int first = 0; first < n; first += 8) {
      const int p = list[min(first + at.row, n - 1)];
      const uint32_t m_off = (uint32_t)p * row_bytes + at.chunk() * 16;
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
      u32x4 w[kDepth], b[kDepth];
      auto fetch = [&](int d, int line) {
        const bool in = line < hi && line * 8 + at.chunk() < nch;
        w[d] = load_rows<true>(w2, in ? w_off : kOutside, (uint32_t)line * 128);
        b[d] = load_rows(mid, in ? m_off : kOutside, (uint32_t)line * 128);
      };
#pragma unroll
      for (int d = 0; d < kDepth; ++d) {
        fetch(d, lo + d);
        in_order();
      }
      for (int line = lo; line < hi; line += kDepth) {
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
          acc = mma_chunk<DT>(w[d], b[d], acc);
          in_order();
          fetch(d, line + kDepth + d);  // past the end: zeros
          in_order();
        }
      }
      acc = join_halves(acc);
      if (at.half == 0 && at.q < 2 && first + at.row < n) y[((size_t)part * a.pairs + p) * 2 + at.q] = acc;
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
    const size_t pos = (size_t)t * a.H + h0 + c;
    if constexpr (DT == kF32) static_cast<float*>(a.out)[pos] = sum;
    else static_cast<uint16_t*>(a.out)[pos] = (uint16_t)f32_to_bf16(sum);
  }
}

template <int DT, int NR>
hipError_t launch_few_typed(const FewArgs& a, hipStream_t s) {
  constexpr int RT = 2;
  const dim3 up((a.I + 8 * RT - 1) / (8 * RT), a.groups);
  if (a.pairs <= 8 * a.E)
    hipLaunchKernelGGL((few_up_kernel<DT, NR, RT, 1>), up, dim3(kUpWaves * kWave), 0, s, a);
  else
    hipLaunchKernelGGL((few_up_kernel<DT, NR, RT, 4>), up, dim3(kUpWaves * kWave), 0, s, a);
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
  a.part_lines = ((a.ich + 7) / 8 + a.split - 1) / a.split;
  if (a.pairs <= kWave)
    return a.dtype == MOE_F32 ? launch_few_typed<kF32, 1>(a, s) : launch_few_typed<kBF16, 1>(a, s);
  return a.dtype == MOE_F32 ? launch_few_typed<kF32, 8>(a, s) : launch_few_typed<kBF16, 8>(a, s);
}

}  // namespace moe
