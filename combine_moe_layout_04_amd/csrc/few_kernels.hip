// A whole mixture-of-experts layer for a few tokens, in two kernels.
//
//   act[p]  = f(Wg_e x_t) * (Wu_e x_t)          pair p = (t, k), e = topk_idx[t, k]
//   out[t]  = sum_k w[t, k] * W2_e act[t, k]
//
// A decode batch reads far more weight bytes than it computes on: the chosen
// experts' weights, 3 H I elements each, are the floor, and each is read once
// per call.  The matrix cores take 4 weight rows against 4 of the expert's
// tokens a tile; 1 KiB of weights costs 16 cycles of one matrix core for
// bfloat16, three times that in the second product, about a twenty-fifth and an
// eighth of what the bytes cost.
//
// No layout runs before: a call has at most 512 pairs, and every workgroup
// groups them by expert in its LDS as it starts.  A workgroup of the first
// kernel takes (expert, 8 columns of act) after another; its waves split the
// sum over H.  A workgroup of the second owns 4 or 8 columns of out for all pairs:
// its waves share out the experts, leave each pair's values in LDS, and the
// top-k sum is formed there in k order, so that no second pass over pairs and
// no order left to chance remain.  An id outside [0, E) belongs to no expert
// here and adds nothing.
//
// act goes from one kernel to the other as float32; for bfloat16's matrix
// instructions the second kernel cuts it into three parts (Parts in mfma.h), which
// lose nothing.  Rounded to one bfloat16 it would make the result half as wrong
// again (against the formula in 64 bits 2.4e-3 instead of 1.7e-3, the result's own
// rounding); in two rounded parts it lost the last 8 bits, and cost, with two and
// three parts, 193 and 198 us at 64 tokens of 128 experts, 19.6 and 19.8 at one
// token, 106 and 113 at 16 pairs for each of 32 experts.
#include <algorithm>

#include "device_common.h"
#include "internal.h"
#include "mfma.h"
#include "../../include/moe_layout.h"

namespace moe {
namespace {

__device__ __forceinline__ int pair_expert(const FewArgs& a, int p) {  // -1: none of this call's experts
  const int64_t e = a.itype == MOE_I32 ? (int64_t)static_cast<const int*>(a.idx)[p]
                                       : static_cast<const int64_t*>(a.idx)[p];
  return e >= 0 && e < a.E ? (int)e : -1;
}

// Chunks of act for one of w2: act is float32, and stands in the workspace so
// that the loads of both go alike.  For bfloat16 a pair's row is the first four
// of every eight columns, then the last four.
template <int DT>
constexpr int kActChunks = DT == kBF16 ? 2 : 1;

// The pairs of a call grouped by expert, in a workgroup's LDS.
struct Groups {
  int count[MOE_MAX_E];
  uint32_t used[kFewMaxPairs];   // experts with pairs, ascending: expert << 20 | first place << 10 | pairs
  uint16_t pairs[kFewMaxPairs];  // grouped by expert
};

// Fills g for the whole workgroup (at least kFewMaxPairs / PER threads, each
// with PER pairs); the number of experts with pairs.  The order of an
// expert's pairs is left to the LDS atomics: it only says which column of a
// tile a pair takes, and a column's value does not depend on its place.
template <int PER>
__device__ __forceinline__ int group_pairs(const FewArgs& a, Groups& g) {
  int e[PER], place[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int p = threadIdx.x + i * blockDim.x;
    e[i] = p < a.pairs ? pair_expert(a, p) : -1;
  }
  for (int i = threadIdx.x; i < a.E; i += blockDim.x) g.count[i] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < PER; ++i) place[i] = e[i] >= 0 ? atomicAdd(&g.count[e[i]], 1) : 0;
  __syncthreads();
  // every wave counts the experts, the first one notes them and turns the
  // counts into first places
  const int lane = lane_id();
  int n = 0;
  uint32_t first = 0;
  for (int i = 0; i < a.E; i += kWave) {
    const uint32_t c = i + lane < a.E ? (uint32_t)g.count[i + lane] : 0u;
    const uint64_t mask = __ballot(c != 0);
    if (threadIdx.x < kWave) {
      const uint32_t end = wave_scan(c);
      if (c) g.used[n + __popcll(mask & lanes_below(lane))] = (uint32_t)(i + lane) << 20 | (first + end - c) << 10 | c;
      first += (uint32_t)read_lane_i((int)end, 63);
    }
    n += __popcll(mask);
  }
  __syncthreads();
  if (threadIdx.x < kWave) {
    for (int j = lane; j < n; j += kWave) g.count[g.used[j] >> 20] = (int)(g.used[j] >> 10 & 1023);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (e[i] >= 0) g.pairs[g.count[e[i]] + place[i]] = (uint16_t)(threadIdx.x + i * blockDim.x);
  __syncthreads();
  return n;
}

__device__ __forceinline__ float gated(float g, float u, int act) {
  if (act == MOE_ACT_SILU) return g / (1.f + expf(-g)) * u;
  const float y = 0.7978845608028654f * (g + 0.044715f * g * g * g);  // sqrt(2/pi)
  return 0.5f * g * (1.f + tanhf(y)) * u;
}

// Whether one tile of 4 pairs does: the host goes by all pairs of a call, of which
// many may belong to other ranks' experts (13 tokens, top 8 of 256, 32 of them here,
// 7168 x 2048, bfloat16: the second kernel 67 us with the two tiles that the pairs
// call for, 59 with one; float32 gains nothing, and the choice costs it 3%).  The
// border, 9/4 pairs for an expert that has any, is the host's 2 for each there is:
// chosen at random, 2 for each leave one in seven without.  A call with one tile
// and with the host's, us, 2048 x 768: 64 experts of 256, 2.1 pairs 88 and 96; of 128,
// 2.2 92 and 94, 3.2 112 and 109, 4.1 133 and 111; 2048 x 1024, 32 of 128, 2.3 64 and
// 73, 3.1 76 and 84, 3.9 90 and 86.
__device__ __forceinline__ bool one_tile(const Groups& g, int experts) {
  if (experts == 0) return true;
  const uint32_t last = (uint32_t)__builtin_amdgcn_readfirstlane((int)g.used[experts - 1]);
  return 4 * (int)((last >> 10 & 1023) + (last & 1023)) <= 9 * experts;
}

// Workgroups go to the 8 XCDs in turn: of every 64, 8 neighbouring places go to
// one, whose L2 joins what they write to the same lines.
__device__ __forceinline__ int place_of_block() {
  const int b = blockIdx.x;
  return b < (int)(gridDim.x & ~63u) ? (b & ~63) + (b & 7) * 8 + (b >> 3 & 7) : b;
}

// act, in items of (expert, 8 columns).  A workgroup's waves take the 256-byte
// lines of the item's rows in turn and meet in LDS; they work in rounds of
// kDepth lines each and ask for the next round's while they multiply this
// one's, from item to item too.  NT tiles of 4 of the expert's pairs at a time.
//
// What decides how near to the memory's rate this comes (64 tokens, 126 experts
// of 768 columns and rows of 4 KiB, 0.79 GB):
//   - the order of lanes in a load (mfma.h): 134 -> 125 us;
//   - neighbouring places to one XCD: 132 -> 120 us, the last of the four (act's
//     lines, written in pieces from 8 L2s, had cost 6 us by then), 6.6 TB/s;
//   - workgroup b takes items b, b + grid, ..., so that all of them together
//     move through a narrow window of the weights: 164 us with even runs of
//     neighbouring items, 140 us in steps;
//   - each workgroup starts at another line of its rows (and goes round): rows
//     4 KiB apart read at the same place at the same time meet in a few memory
//     channels.  140 -> 134 us.  The order of the sum depends on the workgroup
//     alone, so it is the same in every run.
constexpr int kUpWaves = 8;
constexpr int kUpGroups = 512;  // workgroups at most: two a CU

template <int DT, int NT>
__device__ __forceinline__ void few_up(const FewArgs& a, const Groups& groups, int items, float* parts) {
  constexpr int kDepth = 1;  // the other waves' lines are in flight meanwhile
  // wave, tile of pairs, tile of rows, gate or up, row * 4 + pair
  auto& part = *reinterpret_cast<float(*)[kUpWaves][NT][2][2][16]>(parts);
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave));
  const Lane at;

  const int slabs = (a.I + 7) / 8;
  int item = place_of_block();

  const int nch = a.hch;  // chunks of an x or w13 row
  const uint32_t row_bytes = (uint32_t)nch * 16;
  const uint32_t w_off = (uint32_t)at.row * row_bytes + at.chunk * 16;
  const int lines = (nch + 15) / 16;
  const int rounds = (lines + kUpWaves * kDepth - 1) / (kUpWaves * kDepth);
  const int start = item * 2 % lines;
  const auto xs = make_rows(a.x, (size_t)a.T * row_bytes);

  u32x4 wg[kDepth][2], wu[kDepth][2], b[kDepth][NT];
  uint32_t x_off[NT];
  auto gate = make_rows(a.w13, 0), up = gate;
  int slab = 0, n = 0;  // of the item being fetched
  const uint16_t* list = groups.pairs;
  auto fetch_item = [&]() {
    slab = item % slabs;
    const uint32_t group = (uint32_t)__builtin_amdgcn_readfirstlane((int)groups.used[item / slabs]);
    const int e = (int)(group >> 20);
    list = groups.pairs + (group >> 10 & 1023);
    n = (int)(group & 1023);
    // rows past the last one are outside the buffer and read as zeros
    const size_t first = (size_t)e * 2 * a.I + slab * 8;
    const size_t bytes = (size_t)min(8, a.I - slab * 8) * row_bytes;
    gate = make_rows(static_cast<const char*>(a.w13) + first * row_bytes, bytes);
    up = make_rows(static_cast<const char*>(a.w13) + (first + a.I) * row_bytes, bytes);
  };
  auto tokens = [&](int first) {  // columns past the last pair are zeros and not stored
#pragma unroll
    for (int c = 0; c < NT; ++c) {
      const int pos = first + c * 4 + at.row;
      const uint32_t off = (uint32_t)(list[min(pos, n - 1)] / a.K) * row_bytes + at.chunk * 16;
      x_off[c] = pos < n ? off : kOutside;
    }
  };
  auto fetch = [&](int d, int i) {  // the i-th line after `start`; past the last: zeros
    const int line = i >= lines ? 0 : i + start < lines ? i + start : i + start - lines;
    const bool in = i < lines && line * 16 + at.chunk < nch;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const uint32_t off = in ? w_off + r * 4 * row_bytes : kOutside;
      wg[d][r] = load_rows<true>(gate, off, (uint32_t)line * 256);
      wu[d][r] = load_rows<true>(up, off, (uint32_t)line * 256);
    }
#pragma unroll
    for (int c = 0; c < NT; ++c) b[d][c] = load_rows(xs, in ? x_off[c] : kOutside, (uint32_t)line * 256);
  };

  fetch_item();
  tokens(0);
#pragma unroll
  for (int d = 0; d < kDepth; ++d) {
    fetch(d, wave + d * kUpWaves);
    in_order();
  }
  f32x4 g[NT][2], u[NT][2];
#pragma unroll
  for (int c = 0; c < NT; ++c)
#pragma unroll
    for (int r = 0; r < 2; ++r) g[c][r] = u[c][r] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int first = 0, round = 0; item < items;) {
    const int this_i = slab * 8, this_n = n, this_first = first;
    const uint16_t* this_list = list;
    int next = wave + (round + 1) * kDepth * kUpWaves;
    if (++round == rounds) {
      round = 0;
      next = wave;
      first += 4 * NT;
      if (first >= n) {
        first = 0;
        item += gridDim.x;
        if (item < items) fetch_item();
        else next = lines;  // nothing more to fetch
      }
      tokens(first);
    }
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
#pragma unroll
      for (int c = 0; c < NT; ++c)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          g[c][r] = mma_chunk<DT>(wg[d][r], b[d][c], g[c][r]);
          u[c][r] = mma_chunk<DT>(wu[d][r], b[d][c], u[c][r]);
        }
      in_order();
      fetch(d, next + d * kUpWaves);
      in_order();
    }
    if (round == 0) {
      __syncthreads();  // the last results have been read
#pragma unroll
      for (int c = 0; c < NT; ++c)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float sg = join_parts(g[c][r]), su = join_parts(u[c][r]);
          g[c][r] = u[c][r] = f32x4{0.f, 0.f, 0.f, 0.f};
          if ((lane_id() & 3) == 0) {
            part[wave][c][r][0][at.first() * 4 + at.second()] = sg;
            part[wave][c][r][1][at.first() * 4 + at.second()] = su;
          }
        }
      __syncthreads();
      for (int i = threadIdx.x; i < NT * 32; i += kUpWaves * kWave) {
        // neighbouring threads: neighbouring columns of one pair
        const int column = i & 7, t = (i >> 3) & 3, c = i >> 5;
        const int slot = (column & 3) * 4 + t;
        float sg = part[0][c][column >> 2][0][slot], su = part[0][c][column >> 2][1][slot];
#pragma unroll
        for (int v = 1; v < kUpWaves; ++v) {
          sg += part[v][c][column >> 2][0][slot];
          su += part[v][c][column >> 2][1][slot];
        }
        const int pos = this_first + c * 4 + t;
        if (pos < this_n && this_i + column < a.I) {
          const float v = gated(sg, su, a.act);
          // (bfloat16: I is a multiple of 8)
          const int place = DT == kF32 ? this_i + column : (column >> 2) * (a.I / 2) + this_i / 2 + (column & 3);
          a.mid[(size_t)this_list[pos] * a.I + place] = v;
        }
      }
    }
  }
}

template <int DT, int NT>
__global__ __launch_bounds__(kUpWaves* kWave) void few_up_kernel(FewArgs a) {
  __shared__ Groups groups;
  __shared__ float parts[kUpWaves * NT * 64];
  const int experts = group_pairs<kFewMaxPairs / (kUpWaves * kWave)>(a, groups);
  const int items = experts * ((a.I + 7) / 8);
  if (place_of_block() >= items) return;  // the whole workgroup
  if (DT == kBF16 && NT > 1 && one_tile(groups, experts)) few_up<DT, 1>(a, groups, items, parts);
  else few_up<DT, NT>(a, groups, items, parts);
}

// 4 NR columns of out, for every pair.  A wave's item is (expert, part of the sum
// over I); it leaves its pairs' values in y[part][pair].  The waves stream
// their items' weights in rounds of kDepth lines, the next round's (of the same
// item or the next) under way during this one.  (64 tokens, 126 experts of 768
// columns, rows of 1.5 KiB, 0.4 GB: 82 us, 4.9 TB/s; 66 us with act rounded to one
// part.)
constexpr int kDownWaves = 16;

// FINITE: see Parts.  Returns whether this wave's values hold a NaN.
template <int DT, int NT, int NR, bool FINITE>
__device__ __forceinline__ bool few_down(const FewArgs& a, const Groups& groups, int experts, float* y) {
  // 13 tokens, 32 experts of 4096 x 2048: 274, 271, 279 us a call with 1, 2, 3; the
  // most tiles have no registers for two
  constexpr int kDepth = NT * NR < 8 ? 2 : 1;
  constexpr int kCols = 4 * NR, kChunks = kActChunks<DT>;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave));
  const Lane at;

  const int items = experts * a.split;
  // the split divides the number of waves: a wave has one part of all its experts
  const int part = wave % a.split;

  const int nch = a.ich;  // chunks of an act or w2 row
  const uint32_t row_bytes = (uint32_t)nch * 16;
  const int h0 = place_of_block() * kCols;
  const size_t tile_bytes = (size_t)min(kCols, a.H - h0) * row_bytes;
  const auto mid = make_rows(a.mid, (size_t)a.pairs * kChunks * row_bytes);
  const uint32_t w_off = (uint32_t)at.row * row_bytes + at.chunk * 16;
  const int lo = part * a.part_lines, hi = min(lo + a.part_lines, (nch + 15) / 16);
  const int rounds = (a.part_lines + kDepth - 1) / kDepth;

  u32x4 w[kDepth][NR], b[kDepth][NT][kChunks];
  auto w2 = make_rows(a.w2, 0);
  uint32_t m_off[NT];
  int n = 0;  // pairs of the fetched item
  const uint16_t* list = groups.pairs;
  auto item = [&](int j) {
    const uint32_t group = (uint32_t)__builtin_amdgcn_readfirstlane((int)groups.used[j / a.split]);
    list = groups.pairs + (group >> 10 & 1023);
    n = (int)(group & 1023);
    w2 = make_rows(static_cast<const char*>(a.w2) + ((size_t)(group >> 20) * a.H + h0) * row_bytes, tile_bytes);
  };
  auto pairs_of = [&](int first) {  // columns past the last pair are zeros and not stored
#pragma unroll
    for (int c = 0; c < NT; ++c) {
      const int pos = first + c * 4 + at.row;
      const uint32_t off = (uint32_t)list[min(pos, n - 1)] * kChunks * row_bytes + at.chunk * 16;
      m_off[c] = pos < n ? off : kOutside;
    }
  };
  auto fetch = [&](int d, int next) {  // past the part's last line: zeros
    const int line = min(next, hi - 1);
    const bool in = next < hi && line * 16 + at.chunk < nch;
#pragma unroll
    for (int r = 0; r < NR; ++r)
      w[d][r] = load_rows<true>(w2, in ? w_off + r * 4 * row_bytes : kOutside, (uint32_t)line * 256);
#pragma unroll
    for (int c = 0; c < NT; ++c)
#pragma unroll
      for (int i = 0; i < kChunks; ++i)
        b[d][c][i] = load_rows(mid, in ? m_off[c] : kOutside, (uint32_t)line * 256 + i * row_bytes);
  };
  if (wave < items) {
    item(wave);
    pairs_of(0);
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      fetch(d, lo + d);
      in_order();
    }
  }
  f32x4 acc[NT][NR];
#pragma unroll
  for (int c = 0; c < NT; ++c)
#pragma unroll
    for (int r = 0; r < NR; ++r) acc[c][r] = f32x4{0.f, 0.f, 0.f, 0.f};
  bool nan = false;
  for (int j = wave, first = 0, round = 0; j < items;) {
    const uint16_t* this_list = list;
    const int this_n = n;
    int next_j = j, next_first = first, next_round = round + 1;
    if (next_round == rounds) {
      next_round = 0;
      next_first += 4 * NT;
      if (next_first >= n) {
        next_first = 0;
        next_j += kDownWaves;
        if (next_j < items) item(next_j);
      }
      if (next_j < items) pairs_of(next_first);
    }
    const int next_line = next_j < items ? lo + next_round * kDepth : hi;
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
#pragma unroll
      for (int c = 0; c < NT; ++c) {
        if constexpr (DT == kF32) {
#pragma unroll
          for (int r = 0; r < NR; ++r) acc[c][r] = mma_chunk<DT>(w[d][r], b[d][c][0], acc[c][r]);
        } else {
          float f[8];
          unpack<kF32>(b[d][c][0], *reinterpret_cast<float(*)[4]>(f));
          unpack<kF32>(b[d][c][1], *reinterpret_cast<float(*)[4]>(f + 4));
          const Parts<FINITE> act(f);
#pragma unroll
          for (int r = 0; r < NR; ++r) acc[c][r] = mma_parts(w[d][r], act, acc[c][r]);
        }
      }
      in_order();
      fetch(d, next_line + d);  // past the end: zeros
      in_order();
    }
    if (next_round == 0) {
#pragma unroll
      for (int c = 0; c < NT; ++c) {
        const int pos = first + c * 4 + at.second();
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const float v = join_parts(acc[c][r]);
          acc[c][r] = f32x4{0.f, 0.f, 0.f, 0.f};
          if ((lane_id() & 3) == 0 && pos < this_n) {
            y[((size_t)part * a.pairs + this_list[pos]) * kCols + r * 4 + at.first()] = v;
            nan |= v != v;
          }
        }
      }
    }
    j = next_j;
    first = next_first;
    round = next_round;
  }
  return __ballot(nan) != 0;
}

template <int DT, int NT, int NR>
__device__ __forceinline__ void down(const FewArgs& a, const Groups& groups, int experts, float* y) {
  const bool nan = few_down<DT, NT, NR, true>(a, groups, experts, y);
  if (DT == kBF16 && nan) few_down<DT, NT, NR, false>(a, groups, experts, y);  // a wave writes what it wrote before
}

template <int DT, int NT, int NR>
__global__ __launch_bounds__(kDownWaves* kWave) void few_down_kernel(FewArgs a) {
  constexpr int kCols = 4 * NR;
  __shared__ Groups groups;
  __shared__ float weight[kFewMaxPairs];
  __shared__ uint8_t here[kFewMaxPairs];
  extern __shared__ float y[];  // [split][pairs][kCols]
  if (threadIdx.x < a.pairs) {
    weight[threadIdx.x] = a.w ? a.w[threadIdx.x] : 1.f;
    here[threadIdx.x] = pair_expert(a, threadIdx.x) >= 0;
  }
  const int experts = group_pairs<1>(a, groups);
  if (DT == kBF16 && NT > 1 && one_tile(groups, experts)) down<DT, 1, NR>(a, groups, experts, y);
  else down<DT, NT, NR>(a, groups, experts, y);
  const int h0 = place_of_block() * kCols;
  __syncthreads();

  for (int o = threadIdx.x; o < a.T * kCols; o += kDownWaves * kWave) {
    const int t = o / kCols, c = o % kCols;
    if (h0 + c >= a.H) continue;
    float sum = 0.f;
    for (int k = 0; k < a.K; ++k) {
      const int p = t * a.K + k;
      if (!here[p]) continue;
      float v = y[(size_t)p * kCols + c];
      for (int i = 1; i < a.split; ++i) v += y[((size_t)i * a.pairs + p) * kCols + c];
      sum = __fadd_rn(sum, __fmul_rn(weight[p], v));
    }
    const size_t pos = (size_t)t * a.H + h0 + c;
    if constexpr (DT == kF32) static_cast<float*>(a.out)[pos] = sum;
    else static_cast<uint16_t*>(a.out)[pos] = (uint16_t)f32_to_bf16(sum);
  }
}

template <int DT, int NT>
hipError_t launch_few_typed(const FewArgs& a, hipStream_t s) {
  const int up = (int)std::min<int64_t>(kUpGroups, (int64_t)a.groups * ((a.I + 7) / 8));
  hipLaunchKernelGGL((few_up_kernel<DT, NT>), dim3(up), dim3(kUpWaves * kWave), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 block(kDownWaves * kWave);
  const size_t column = (size_t)a.split * a.pairs * sizeof(float);
  // 4 columns of out a workgroup where 8 would leave CUs without one (the kernel with
  // 8 and 4, us: 57 tokens, top 6 of 60, 288 x 140 float32 24.0 and 15.4; 30, top 8 of
  // 40, 1024 x 400 bfloat16 23.4 and 19.3; 1, top 4 of 64, 512 x 256 5.8 and 5.3)
  if (a.H < 8 * 256)
    hipLaunchKernelGGL((few_down_kernel<DT, NT, 1>), dim3((a.H + 3) / 4), block, column * 4, s, a);
  else
    hipLaunchKernelGGL((few_down_kernel<DT, NT, 2>), dim3((a.H + 7) / 8), block, column * 8, s, a);
  return hipGetLastError();
}

template <int DT>
hipError_t launch_few_tiles(const FewArgs& a, hipStream_t s) {
  // By the pairs an expert of the call has on average.  More tiles read fewer
  // weights twice and multiply more zeros, which float32's matrix rate feels
  // first (2048 x 768, 32 experts of all that are chosen from; us with 1, 2, 3, 4
  // tiles.  bfloat16, 1 pair: 24 26 28 31, 4: 70 57 60 66, 8: 113 81 69 73, 16: 197
  // 134 113 109; float32, 1: 42 41 52 64, 4: 127 109 137 168, 8: 221 154 151 175, 16:
  // 400 270 264 281).  Each a kernel of its own: the registers of the most tiles
  // would cost the others their second workgroup on a CU (32 tokens, top 2 of 16,
  // 512 x 256, bfloat16: 12.2 us so, 14.0 with all in one).
  if (a.pairs <= 2 * a.E) return launch_few_typed<DT, 1>(a, s);
  if (a.pairs <= (DT == kF32 ? 8 : 4) * a.E) return launch_few_typed<DT, 2>(a, s);
  if constexpr (DT == kBF16) {
    if (a.pairs > 8 * a.E) return launch_few_typed<DT, 4>(a, s);
  }
  return launch_few_typed<DT, 3>(a, s);
}

}  // namespace

hipError_t launch_few(const FewArgs& args, hipStream_t s) {
  FewArgs a = args;
  a.groups = std::min(a.pairs, a.E);
  a.split = 1;  // parts for every wave of a workgroup of the second product, when experts are few
  while (a.groups * a.split < kDownWaves && 2 * a.split * a.pairs <= kFewMaxPairs) a.split *= 2;
  a.part_lines = ((a.ich + 15) / 16 + a.split - 1) / a.split;
  return a.dtype == MOE_F32 ? launch_few_tiles<kF32>(a, s) : launch_few_tiles<kBF16>(a, s);
}

}  // namespace moe
