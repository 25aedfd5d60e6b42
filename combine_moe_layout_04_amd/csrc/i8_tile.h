// Products of 8-bit rows and 8-bit weights, grouped by expert (moe_matmul_i8).
//
//   acc[p,n] = sum_k q[p,k] w[e,n,k]        exact, in 32-bit integers
//   y[p,n]   = float(acc) * s[p] * sw[e,n]  in float32, rounded once to the output type
//   gated:     f(y[p,i]) * y[p,I+i]         formed before that rounding
//
// A workgroup's tile is BM rows of one expert by BN channels; both operands run
// through LDS in steps of 128 bytes of each row, loaded there directly (no registers
// on the way) into one of three stages: two steps are on their way while the matrix
// cores work on a third, with one barrier a step.  Rows of 128 bytes, whole lines: with
// steps of 64 bytes the address units give half the rate (17 to 22 TB/s from L2, 33 to 35
// with 128).  The stages are separate arrays, so that the compiler sees that reads of one
// need not wait for loads into another.  The weights are the first operand of the matrix
// instruction: a lane then holds four neighbouring channels of one row.  A row's chunks
// are stored permuted (by the row's bits), so that the 16 rows of an operand lie in
// different banks: no bank conflict is counted.
//
// Workgroups stay and take tile after tile, and the stages go on from one to the next:
// during a tile's last two steps the first two of the tile after it are loaded, so that
// they are there when this one is scaled and written (32768 rows, 768 x 2048: 113 us with
// a beginning for every tile, 100 so).  A tile begins as many stages on as it has steps
// modulo 3, which is therefore known when the kernel is compiled.  What is on its way is
// counted, not waited for: every tile issues the same number of loads of scales and of
// stores, what is not there from or to nowhere (a store that may be left out makes the
// compiler wait for all of them; copying registers that are still being loaded as well).
// An expert of n rows has ceil(n / BM) tiles of equal size; a tile leaves out the
// products of 16-row parts that it has no rows for.  The tiles are found from the experts'
// offsets on the device: the host knows only how many there can be.
//
// Rows past an expert's last and chunks past a row's end have an offset outside the
// buffer: the hardware reads nothing and puts zeros into LDS.  A tile starts its sum at a
// step of its own, so that workgroups do not all ask for the same part of their rows at
// the same time.
//
// Measured (MI355X): one projection of 4096 rows, 7168 x 4096, gated: 102 to 113 us, 2.1 to
// 2.3 POP/s, half of what the matrix cores could do (a library's product of two 8192 x 8192
// int8 matrices reaches 2.4); the loads alone take 77 us, the products alone 57.  4096 tokens
// of 8 of 128 experts, 2048 x 1536, gated: 154 to 162 us; loads alone 128 (520 to 570 MB are read,
// 403 of them weights), products alone 70.  64 tokens there: 73 to 76 us, 5.2 to 5.5 TB/s
// of weights; a plain read of as much reaches 6.15.
#pragma once

#include "device_common.h"
#include "internal.h"
#include "mfma.h"
#include "quant.h"
#include "../../include/moe_layout.h"
#include <type_traits>

namespace moe {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// The wait for all but the last n of a wave's memory operations, and all of its LDS ones.
constexpr int wait_for(int n) { return (n & 15) | (7 << 4) | ((n >> 4) << 14); }

constexpr int kMaxExperts = 1024;           // MOE_MAX_E
constexpr uint32_t kNowhere = 0xFFFFFFF0u;  // past every buffer

constexpr int kStep = 8;  // 16-byte chunks of a row in a step

// Steps of a tile: two are asked for ahead.
__host__ __device__ constexpr int steps_of(int kch) { return kch > kStep ? (kch + kStep - 1) / kStep : 2; }

struct Tile {
  int e, row, rows, col;  // expert, first receive row, rows (0: no such tile), channel tile
};

// The tiles of a call, numbered by expert, band of kBand row tiles, channel tile and row
// tile, the last fastest: what an XCD works on at a time is about as high as wide, and
// reads fewer rows and weights into its L2 than a column of tiles would (4096 rows of
// 7168 x 4096: 107 us when this was tried, in columns 110).
constexpr int kBand = 8;

struct Tiles {
  const int* before;  // [E+1] in LDS: row tiles of the experts before each
  const int* first;   // [E+1] in LDS: first receive row of each
  int E, cols;

  __device__ __forceinline__ uint32_t total() const { return (uint32_t)before[E] * cols; }

  __device__ __forceinline__ Tile at(uint32_t id) const {  // the same in every lane
    const int key = (int)(id / cols), block = (E + kWave - 1) / kWave;
    // the expert whose run of row tiles holds number `key`: 64 blocks, then 16 of a block
    int e = __popcll(__ballot(before[min(E, (lane_id() + 1) * block)] <= key)) * block;
    e += __popcll(__ballot(lane_id() < block && before[min(E, e + lane_id() + 1)] <= key));
    e = __builtin_amdgcn_readfirstlane(min(e, E - 1));
    const int b = __builtin_amdgcn_readfirstlane(before[e]), tiles = __builtin_amdgcn_readfirstlane(before[e + 1]) - b;
    const int row = __builtin_amdgcn_readfirstlane(first[e]), n = __builtin_amdgcn_readfirstlane(first[e + 1]) - row;
    const int r = (int)(id - (uint32_t)b * cols);
    const int step = ((n + tiles - 1) / tiles + 15) & ~15;  // rows of a tile
    const int band = r / (kBand * cols), high = min(kBand, tiles - band * kBand), s = r - band * kBand * cols;
    const int m = band * kBand + s % high;
    return {e, row + m * step, min(step, n - m * step), s / high};
  }
};

// f(g) = g sigmoid(x): x = g (silu), or 2 sqrt(2 / pi) (g + 0.044715 g^3), since
// (1 + tanh(x / 2)) / 2 = sigmoid(x).  The exponential is off by 4 u of itself (u = 2^-24),
// the sum by u, the reciprocal by 2 u and the product by u: silu by 8 u of itself down to g =
// -87, below which it is under 2^-118 and may be 0.  (The exponential's first part alone is
// off by (|x| + 2) u.  4096 tokens of 8 of 128 experts, 2048 x 1536: 154 us, with the first
// part alone 152, with expf and a division 168.)
__device__ __forceinline__ float activate(float g, int act) {
  const float x = act == MOE_ACT_SILU ? g : 1.5957691216057308f * (g + 0.044715f * g * g * g);
  float t;
  const float y = __builtin_amdgcn_fmed3f(-x, -200.f, 200.f);  // past it 0 or infinite, as it is
  const float rest = exp_parts(y, t);
  return g * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(t) * (1.f + rest));
}

// Which channel of a tile a row of the B stage holds.  A lane has the four channels
// 4 g .. 4 g + 3 (g = lane / 16) of each 16 x 16 result; the channels are dealt so that
// what a lane stores together is 16 contiguous bytes and what a wave stores of a row 64:
// float32 by itself; bfloat16 takes two results, channels 8 g + 4 j + v of 32.  Gated:
// 16 gate channels (`up` 0) and the up channels (`up` 1) of the same outputs in turn.
template <int DT, bool GATED, int NB>
struct Channels {
  static constexpr bool kPaired = DT == kBF16 && NB % (GATED ? 4 : 2) == 0;
  static __device__ __forceinline__ int of_row(int r, int& up) {
    const int m = r % 16, g = m / 4, v = m % 4;
    int b = r / 16;  // result
    up = 0;
    if (GATED) {
      up = b & 1;
      b >>= 1;
    }
    return kPaired ? b / 2 * 32 + 8 * g + 4 * (b & 1) + v : b * 16 + m;
  }
  // the first of the four channels of result b (of the gate and up results: pair b)
  static __device__ __forceinline__ int of_result(int b, int g) {
    return kPaired ? b / 2 * 32 + 8 * g + 4 * (b & 1) : b * 16 + 4 * g;
  }
};

// MB x NB tiles of 16 x 16 a wave, WM x WN waves.  REST: steps of a tile, modulo 3.
template <int DT, bool GATED, int MB, int NB, int WM, int WN, int REST, int EU>
__global__ __launch_bounds__(WM* WN* kWave, EU) void i8_kernel(I8Args a, int cols) {
  constexpr int BM = 16 * MB * WM, BN = 16 * NB * WN, kWaves = WM * WN;
  constexpr int kRowsPer = kWave / kStep;  // rows of one load instruction
  constexpr int kLoadsA = (BM + kRowsPer * kWaves - 1) / (kRowsPer * kWaves), kLoadsB = BN / kRowsPer / kWaves;
  static_assert(kRowsPer * kWaves % 16 == 0);
  static_assert(kLoadsB >= 1 && BN % (kRowsPer * kWaves) == 0);
  constexpr int kStageA = kLoadsA * kWaves * kWave, kStageB = BN * kStep;
  __shared__ u32x4 a0[kStageA], b0[kStageB], a1[kStageA], b1[kStageB], a2[kStageA], b2[kStageB];
  auto stage_a = [&](auto I) __attribute__((always_inline)) -> u32x4* {
    if constexpr (I == 0) return a0;
    else if constexpr (I == 1) return a1;
    else return a2;
  };
  auto stage_b = [&](auto I) __attribute__((always_inline)) -> u32x4* {
    if constexpr (I == 0) return b0;
    else if constexpr (I == 1) return b1;
    else return b2;
  };
  __shared__ int sums_of_waves[kWaves];
  extern __shared__ int tables[];  // before [E+1], first [E+1]
  int *before = tables, *first = tables + a.E + 1;
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wm = wave % WM, wn = wave / WM;
  // the bits of a row that its chunks are permuted by: 16 rows over all banks
  auto key = [](int row) { return (row >> 1) & 7; };
  const int N = GATED ? a.N / 2 : a.N;  // channels of the output
  const int64_t width = (int64_t)a.kch * 16;

  // the experts' row tiles
  {
    constexpr int kEach = (kMaxExperts + kWaves * kWave - 1) / (kWaves * kWave);  // experts of a thread
    int start[kEach + 1], tiles[kEach], sum = 0;
#pragma unroll
    for (int i = 0; i <= kEach; ++i) {
      const int e = min(kEach * (int)threadIdx.x + i, a.E);
      start[i] = a.offset ? min(max(a.offset[e], 0), a.R) : e ? a.M : 0;
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      tiles[i] = (max(start[i + 1] - start[i], 0) + BM - 1) / BM;
      sum += tiles[i];
    }
    const int upto = (int)wave_scan((uint32_t)sum);
    if (lane == 63) sums_of_waves[wave] = upto;
    __syncthreads();
    int b = upto - sum;
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
      if (w < wave) b += sums_of_waves[w];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int e = kEach * (int)threadIdx.x + i;
      if (e <= a.E) {
        before[e] = b;
        first[e] = start[i];
      }
      b += tiles[i];
    }
    if (threadIdx.x == kWaves * kWave - 1 && kEach * kWaves * kWave <= a.E) {
      before[a.E] = b;
      first[a.E] = start[kEach];
    }
    __syncthreads();
  }
  const Tiles list = {before, first, a.E, cols};
  // XCD x (workgroups x, x + 8, ..) takes the x-th eighth of the tiles, its workgroups in turn
  const uint32_t total = (uint32_t)__builtin_amdgcn_readfirstlane((int)list.total()), per = (total + 7) / 8;
  const uint32_t from = (blockIdx.x & 7) * per, end = min(total, from + per), stride = gridDim.x / 8;
  uint32_t id = from + blockIdx.x / 8;
  auto tile_at = [&](uint32_t i) __attribute__((always_inline)) {
    Tile none = {0, 0, 0, 0};
    return i < end ? list.at(i) : none;
  };

  const int mine = wave * kRowsPer + lane / kStep;  // this lane's row of a wave's first load
  const int chunk = lane % kStep ^ key(mine);       // the same in all of them
  const int full = (a.kch + kStep - 1) / kStep, steps = steps_of(a.kch);  // the second may have one without a load
  Tile t = tile_at(id);
  if (t.rows == 0) return;  // uniform over the workgroup

  // What a tile's rows are made of: rows of q (-1: none) for this lane's loads, and for its
  // results' scales.
  struct Rows {
    int load[kLoadsA], scale[MB];
  };
  auto rows_of = [&](const Tile& x, Rows& to) __attribute__((always_inline)) {
    auto one = [&](int r) __attribute__((always_inline)) {
      if (r >= x.rows) return -1;
      return a.recv_token ? a.recv_token[x.row + r] : x.row + r;
    };
#pragma unroll
    for (int i = 0; i < kLoadsA; ++i) to.load[i] = one(i * kWaves * kRowsPer + mine);
#pragma unroll
    for (int i = 0; i < MB; ++i) to.scale[i] = one((i * WM + wm) * 16 + (lane & 15));
  };
  uint32_t offa[kLoadsA], offb[kLoadsB];
  __amdgpu_buffer_rsrc_t rq, rw;
  int begin = 0;
  auto aim = [&](const Tile& x, const Rows& rows) __attribute__((always_inline)) {
    // rows of q: the tile's own, or any
    const int first_row = a.recv_token ? 0 : x.row;
    const int64_t qrows = a.recv_token ? a.M : x.rows, qbase = first_row * width;
    rq = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(a.q) + qbase, 0, (int)(uint32_t)(qrows * width), 0x00027000);
    const int n0 = x.col * (GATED ? BN / 2 : BN);
    const int64_t wbase = ((int64_t)x.e * a.N + n0) * width;
    rw = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(a.w) + wbase, 0, (int)(uint32_t)((a.N - n0) * width),
                                           0x00027000);
#pragma unroll
    for (int i = 0; i < kLoadsA; ++i) {
      const int row = rows.load[i] - first_row;  // negative: none
      offa[i] = (uint32_t)row < (uint32_t)qrows ? (uint32_t)(row * width) + chunk * 16 : kNowhere;
    }
#pragma unroll
    for (int i = 0; i < kLoadsB; ++i) {
      const int r = i * kWaves * kRowsPer + mine;
      int up;
      const int n = Channels<DT, GATED, NB>::of_row(r, up);
      offb[i] = x.rows != 0 && n0 + n < N ? (uint32_t)((n + (up ? N : 0)) * width) + chunk * 16 : kNowhere;
    }
    begin = (int)((uint32_t)(x.e * cols + x.col) % (uint32_t)full);
  };
  // Load n of a step: those of q first.  Every load of a step is issued, past the rows'
  // end too, so that their number is known.
  auto load = [&](auto STAGE, int s, auto n) __attribute__((always_inline)) {
    int step = s + begin;
    if (step >= full) step -= full;
    const int left = s < full ? a.kch - step * kStep : 0;  // chunks of the row from there on (a select, no branch)
    const bool in = chunk < left;
    const int at = step * kStep * 16;
    if constexpr (n < kLoadsA) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rq, (__attribute__((address_space(3))) void*)(stage_a(STAGE) + (n * kWaves + wave) * kWave), 16,
          (int)(in ? offa[n] : kNowhere), at, 0, 0);
    } else {
      constexpr int m = n - kLoadsA;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rw, (__attribute__((address_space(3))) void*)(stage_b(STAGE) + (m * kWaves + wave) * kWave), 16,
          (int)(in ? offb[m] : kNowhere), at, 0, 0);
    }
  };
  // loads FROM to TO - 1 of a step
  auto loads = [&](auto STAGE, int s, auto FROM, auto TO) __attribute__((always_inline)) {
    auto each = [&](auto self, auto n) __attribute__((always_inline)) {
      if constexpr (n < TO) {
        load(STAGE, s, n);
        self(self, std::integral_constant<int, n + 1>{});
      }
    };
    each(each, FROM);
  };
  constexpr std::integral_constant<int, 0> s0;
  constexpr std::integral_constant<int, 1> s1;
  constexpr std::integral_constant<int, kLoadsA + kLoadsB> every;
  using Ch = Channels<DT, GATED, NB>;
  constexpr int kOuts = GATED ? NB / 2 : NB;  // results of a wave in a row tile
  constexpr int kStores = MB * (Ch::kPaired ? kOuts / 2 : kOuts);  // of a wave, for a whole tile
  i32x4 acc[MB][NB];
  // the sums, of the first B row tiles of each wave, from stage FIRST on; follow(): aims
  // the loads at the tile that follows and asks for the scales of this one
  auto sums = [&](auto B, auto FIRST, auto follow) __attribute__((always_inline)) {
    // step FIRST + AT: wait for its loads, let the stage before it be filled again with step
    // `to`, multiply.  first: one of a tile's first two; last: how many are left, of the last two
    auto work = [&](auto AT, int to, auto first, auto last) __attribute__((always_inline)) {
      constexpr std::integral_constant<int, (FIRST + AT) % 3> I;
      // memory operations complete in their order, and these may still be on their way: the
      // next step's loads, the stores of the tile before (they came after the loads of this
      // one's first two steps), and before the last step the scales
      constexpr int kFlying = kLoadsA + kLoadsB + (first ? kStores : 0) + (last == 1 ? MB + NB : 0);
      __asm__ __volatile__("" ::: "memory");  // the barrier alone does not keep LDS reads on their side of it
      __builtin_amdgcn_s_waitcnt(wait_for(kFlying));
      __builtin_amdgcn_s_barrier();
      __asm__ __volatile__("" ::: "memory");
      if constexpr (last == 2) follow();
      constexpr std::integral_constant<int, (I + 2) % 3> before_it;
      const u32x4 *la = stage_a(I), *lb = stage_b(I);
      const int r = lane & 15, c = lane >> 4;
      constexpr int kParts = kStep / 4;
      i32x4 fa[kParts][B], fb[kParts][NB];
#pragma unroll
      for (int k = 0; k < kParts; ++k) {
        const int slot = (4 * k + c) ^ key(r);  // 16 more rows have the same key
#pragma unroll
        for (int j = 0; j < NB; ++j) fb[k][j] = __builtin_bit_cast(i32x4, lb[((wn * NB + j) * 16 + r) * kStep + slot]);
#pragma unroll
        for (int i = 0; i < B; ++i) fa[k][i] = __builtin_bit_cast(i32x4, la[((i * WM + wm) * 16 + r) * kStep + slot]);
      }
      if constexpr (first) in_order();  // else the compiler waits for more than it has to
      // a load takes the address unit as long as a product the matrix unit: one by one between them
      constexpr int kGroups = kParts * B;
      auto group = [&](auto self, auto g) __attribute__((always_inline)) {
        if constexpr (g < kGroups) {
          constexpr int k = g / B, i = g % B;
          loads(before_it, to, std::integral_constant<int, g * every / kGroups>{},
                std::integral_constant<int, (g + 1) * every / kGroups>{});
#pragma unroll
          for (int j = 0; j < NB; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[k][j], fa[k][i], acc[i][j], 0, 0, 0);
          in_order();
          self(self, std::integral_constant<int, g + 1>{});
        }
      };
      group(group, s0);
    };
    constexpr std::integral_constant<int, 2> s2;
    constexpr std::false_type no;
    constexpr std::true_type yes;
    if constexpr (REST == 2) {
      if (steps == 2) {
        work(s0, 0, yes, s2);
        work(s1, 1, yes, s1);
        return;
      }
    }
    if constexpr (REST == 0) {
      if (steps == 3) {
        work(s0, 2, yes, s0);
        work(s1, 0, yes, s2);
        work(s2, 1, no, s1);
        return;
      }
    }
    work(s0, 2, yes, s0);
    work(s1, 3, yes, s0);
    int to = 4;
    for (; to + 3 <= steps; to += 3) {
      work(s2, to, no, s0);
      work(s0, to + 1, no, s0);
      work(s1, to + 2, no, s0);
    }
    constexpr int kLeft = (REST + 2) % 3;  // (steps - 4) modulo 3
    if constexpr (kLeft >= 1) work(s2, to, no, s0);
    if constexpr (kLeft >= 2) work(s0, to + 1, no, s0);
    work(std::integral_constant<int, 2 + kLeft>{}, 0, no, s2);
    work(std::integral_constant<int, 3 + kLeft>{}, 1, no, s1);
  };

  // lane: row l % 16 of a row tile
  const int g = lane >> 4;
  // A tile's scales, MB + NB loads whatever is there: their number is counted on.
  f32x4 scale_w[NB];
  float scale_q[MB];
  int scale_row[MB];
  const __amdgpu_buffer_rsrc_t rqs =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(a.qs), 0, (int)((uint32_t)a.M * 4), 0x00027000);
  auto scales_of = [&](const Tile& x) __attribute__((always_inline)) {
    const int n0 = x.col * (GATED ? BN / 2 : BN);
    const __amdgpu_buffer_rsrc_t r =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(a.ws) + (int64_t)x.e * a.N, 0, a.N * 4, 0x00027000);
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int n = n0 + Ch::of_result(wn * kOuts + (GATED ? j / 2 : j), g);
      const uint32_t at = n < N ? (uint32_t)(n + (GATED && (j & 1) ? N : 0)) * 4 : kNowhere;
      scale_w[j] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0));
    }
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      const uint32_t at = (uint32_t)scale_row[i] < (uint32_t)a.M ? (uint32_t)scale_row[i] * 4 : kNowhere;
      scale_q[i] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rqs, at, 0, 0));
    }
  };
  Rows rows;
  rows_of(t, rows);
  aim(t, rows);
#pragma unroll
  for (int i = 0; i < MB; ++i) scale_row[i] = rows.scale[i];
  Tile next = tile_at(id += stride);
  rows_of(next, rows);
  loads(s0, 0, s0, every);
  loads(s1, 1, s0, every);
  __builtin_amdgcn_s_waitcnt(wait_for(0));  // from here on the number of what is on its way is known
  // A tile from stage FIRST on; false after the last.
  auto tile = [&](auto FIRST) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    auto follow = [&]() __attribute__((always_inline)) {
      aim(next, rows);
      scales_of(t);
      in_order();
    };
    const int tiles = (t.rows + 16 * WM - 1) / (16 * WM);
    if constexpr (MB == 1) {
      sums(std::integral_constant<int, 1>{}, FIRST, follow);
    } else if constexpr (MB == 2) {
      if (tiles == 1) sums(std::integral_constant<int, 1>{}, FIRST, follow);
      else sums(std::integral_constant<int, 2>{}, FIRST, follow);
    } else {
      static_assert(MB == 4);
      if (tiles == 1) sums(std::integral_constant<int, 1>{}, FIRST, follow);
      else if (tiles == 2) sums(std::integral_constant<int, 2>{}, FIRST, follow);
      else if (tiles == 3) sums(std::integral_constant<int, 3>{}, FIRST, follow);
      else sums(std::integral_constant<int, 4>{}, FIRST, follow);
    }
    __asm__ __volatile__("" ::: "memory");
    bool token[MB];  // a row without one is zero, whatever the channels' scales are
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      token[i] = scale_row[i] >= 0;
      scale_row[i] = rows.scale[i];
    }
    const Tile after = tile_at(id += stride);
    rows_of(after, rows);
    in_order();
    __asm__ __volatile__("" ::: "memory");  // the stores below come after these loads
    in_order();
    // kStores stores, whatever is there: their number is counted on
    const int n0 = t.col * (GATED ? BN / 2 : BN);
    constexpr int kBytes = DT == kF32 ? 4 : 2;
    const __amdgpu_buffer_rsrc_t ro = __builtin_amdgcn_make_buffer_rsrc(
        static_cast<char*>(a.out) + (int64_t)t.row * N * kBytes, 0, (int)((uint32_t)t.rows * N * kBytes), 0x00027000);
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      const int r = (i * WM + wm) * 16 + (lane & 15);
      const bool there = (i * WM + wm) * 16 < t.rows;  // of the 16 rows any
      // an output that is not there: nowhere
      auto at = [&](int j) __attribute__((always_inline)) {
        const int n = n0 + Ch::of_result(wn * kOuts + j, g);
        return r < t.rows && n < N ? ((uint32_t)r * N + n) * kBytes : kNowhere;
      };
      float y[kOuts][4];
#pragma unroll
      for (int j = 0; j < kOuts; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          y[j][v] = 0.f;
          if (!there) continue;
          if constexpr (GATED)
            y[j][v] = activate((float)acc[i][2 * j][v] * scale_q[i] * scale_w[2 * j][v], a.act) *
                      ((float)acc[i][2 * j + 1][v] * scale_q[i] * scale_w[2 * j + 1][v]);
          else
            y[j][v] = (float)acc[i][j][v] * scale_q[i] * scale_w[j][v];
          if (!token[i]) y[j][v] = 0.f;
        }
      if constexpr (DT == kF32) {
#pragma unroll
        for (int j = 0; j < kOuts; ++j)
          __builtin_amdgcn_raw_buffer_store_b128(
              __builtin_bit_cast(u32x4, f32x4{y[j][0], y[j][1], y[j][2], y[j][3]}), ro, at(j), 0, 0);
      } else if constexpr (Ch::kPaired) {
#pragma unroll
        for (int j = 0; j < kOuts; j += 2)  // N is whole 16-byte chunks: all 8 channels there, or none
          __builtin_amdgcn_raw_buffer_store_b128(
              u32x4{round_bf16x2(y[j][0], y[j][1]), round_bf16x2(y[j][2], y[j][3]), round_bf16x2(y[j + 1][0], y[j + 1][1]),
                    round_bf16x2(y[j + 1][2], y[j + 1][3])},
              ro, at(j), 0, 0);
      } else {
#pragma unroll
        for (int j = 0; j < kOuts; ++j)
          __builtin_amdgcn_raw_buffer_store_b64(
              u32x2{round_bf16x2(y[j][0], y[j][1]), round_bf16x2(y[j][2], y[j][3])}, ro, at(j), 0, 0);
      }
    }
    if (next.rows == 0) return false;
    t = next;
    next = after;
    return true;
  };
  // the stages go on from tile to tile: a tile begins REST stages after the one before
  for (;;) {
    if (!tile(s0)) break;
    if constexpr (REST != 0) {
      if (!tile(std::integral_constant<int, REST>{})) break;
      if (!tile(std::integral_constant<int, 3 - REST>{})) break;
    }
  }
  __builtin_amdgcn_s_waitcnt(wait_for(0));  // nothing on its way to LDS that another workgroup may have next
}

// Tiles of rows there can be at most (whole ones, and one of each expert that is not
// whole) times tiles of channels: the host does not know the experts' rows.
int64_t most_tiles(const I8Args& a, int bm, int bn) {
  const int64_t rows = a.offset ? a.R : a.M, partial = a.offset ? (rows < a.E ? rows : a.E) : 1;
  return (rows / bm + partial) * ((a.N + bn - 1) / bn);
}

template <int MB, int NB, int WM, int WN, int REST, int EU>
hipError_t launch_steps(const I8Args& a, hipStream_t s) {
  constexpr int BM = 16 * MB * WM, BN = 16 * NB * WN;
  const bool gated = a.act != MOE_ACT_NONE;
  const int cols = (a.N + BN - 1) / BN;  // gated: BN / 2 of N / 2 outputs each
  const int64_t most = (most_tiles(a, BM, BN) + 7) / 8 * 8, fit = 256 * (4 * EU / (WM * WN));  // what the GPU holds at once
  const unsigned grid = (unsigned)(most < fit ? most : fit);
  const uint32_t lds = 2 * (a.E + 1) * sizeof(int);
  if (a.dtype == kF32) {
    if (gated) i8_kernel<kF32, true, MB, NB, WM, WN, REST, EU><<<grid, WM * WN * kWave, lds, s>>>(a, cols);
    else i8_kernel<kF32, false, MB, NB, WM, WN, REST, EU><<<grid, WM * WN * kWave, lds, s>>>(a, cols);
  } else {
    if (gated) i8_kernel<kBF16, true, MB, NB, WM, WN, REST, EU><<<grid, WM * WN * kWave, lds, s>>>(a, cols);
    else i8_kernel<kBF16, false, MB, NB, WM, WN, REST, EU><<<grid, WM * WN * kWave, lds, s>>>(a, cols);
  }
  return hipGetLastError();
}

template <int MB, int NB, int WM, int WN, int EU>
hipError_t launch_tile(const I8Args& a, hipStream_t s) {
  switch (steps_of(a.kch) % 3) {
    case 0: return launch_steps<MB, NB, WM, WN, 0, EU>(a, s);
    case 1: return launch_steps<MB, NB, WM, WN, 1, EU>(a, s);
    default: return launch_steps<MB, NB, WM, WN, 2, EU>(a, s);
  }
}

}  // namespace

// The three sizes of tiles, each in a source file of its own (they compile side by side).
hipError_t launch_i8_large(const I8Args& a, hipStream_t s);   // 128 x 256
hipError_t launch_i8_middle(const I8Args& a, hipStream_t s);  // 64 x 128
hipError_t launch_i8_small(const I8Args& a, hipStream_t s);   // 64 x 64

}  // namespace moe
