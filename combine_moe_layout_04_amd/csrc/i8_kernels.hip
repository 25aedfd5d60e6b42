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
// Workgroups stay and take tile after tile: a tile's first loads are asked for before the
// tile before it is scaled and written, and its rows' tokens while that one is summed.
// An expert of n rows has ceil(n / BM) tiles of equal size; a tile leaves out the
// products of 16-row parts that it has no rows for.  The tiles are found from the experts'
// offsets on the device: the host knows only how many there can be.
//
// Rows past an expert's last and chunks past a row's end have an offset outside the
// buffer: the hardware reads nothing and puts zeros into LDS.  A tile starts its sum at a
// step of its own, so that workgroups do not all ask for the same part of their rows at
// the same time.
//
// Measured (MI355X): one projection of 4096 rows, 7168 x 4096, gated: 103 to 113 us, 2.1 to
// 2.3 POP/s, half of what the matrix cores could do (a library's product of two 8192 x 8192
// int8 matrices reaches 2.4); the loads alone take 77 us, the products alone 57.  4096 tokens
// of 8 of 128 experts, 2048 x 1536, gated: 156 us; loads alone 128 (520 to 570 MB are read,
// 403 of them weights), products alone 70.  64 tokens there: 73 us, 5.5 TB/s of weights,
// which is what memory gives.
#include "device_common.h"
#include "internal.h"
#include "mfma.h"
#include "quant.h"
#include "../../include/moe_layout.h"
#include <type_traits>

namespace moe {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// The wait for all but the last n of a wave's memory operations, and all of its LDS ones.
constexpr int wait_for(int n) { return (n & 15) | (7 << 4) | ((n >> 4) << 14); }

constexpr int kMaxExperts = 1024;           // MOE_MAX_E
constexpr uint32_t kNowhere = 0xFFFFFFF0u;  // past every buffer

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
// (1 + tanh(x / 2)) / 2 = sigmoid(x).  The fast exponential is off by (|x| + 2) u of
// itself (u = 2^-24) and the reciprocal by 2 u, so f by (0.28 + 5) u |g|: s (1 - s) |x|
// is at most 0.23.
__device__ __forceinline__ float activate(float g, int act) {
  const float x = act == MOE_ACT_SILU ? g : 1.5957691216057308f * (g + 0.044715f * g * g * g);
  return g * __builtin_amdgcn_rcpf(1.f + __expf(-x));
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

// MB x NB tiles of 16 x 16 a wave, WM x WN waves.
template <int DT, bool GATED, int MB, int NB, int WM, int WN, int KC, int STAGES, int EU>
__global__ __launch_bounds__(WM* WN* kWave, EU) void i8_kernel(I8Args a, int cols) {
  constexpr int BM = 16 * MB * WM, BN = 16 * NB * WN, kWaves = WM * WN;
  constexpr int kRowsPer = kWave / KC;  // rows of one load instruction
  constexpr int kLoadsA = (BM + kRowsPer * kWaves - 1) / (kRowsPer * kWaves), kLoadsB = BN / kRowsPer / kWaves;
  static_assert(kRowsPer * kWaves % 16 == 0);
  static_assert(kLoadsB >= 1 && BN % (kRowsPer * kWaves) == 0);
  constexpr int kStageA = kLoadsA * kWaves * kWave, kStageB = BN * KC;
  __shared__ u32x4 a0[kStageA], b0[kStageB], a1[kStageA], b1[kStageB], a2[STAGES > 2 ? kStageA : 1],
      b2[STAGES > 2 ? kStageB : 1], a3[STAGES > 3 ? kStageA : 1], b3[STAGES > 3 ? kStageB : 1];
  auto stage_a = [&](auto I) __attribute__((always_inline)) -> u32x4* {
    if constexpr (I == 0) return a0;
    else if constexpr (I == 1) return a1;
    else if constexpr (I == 2) return a2;
    else return a3;
  };
  auto stage_b = [&](auto I) __attribute__((always_inline)) -> u32x4* {
    if constexpr (I == 0) return b0;
    else if constexpr (I == 1) return b1;
    else if constexpr (I == 2) return b2;
    else return b3;
  };
  __shared__ int sums_of_waves[kWaves];
  extern __shared__ int tables[];  // before [E+1], first [E+1]
  int *before = tables, *first = tables + a.E + 1;
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wm = wave % WM, wn = wave / WM;
  // the bits of a row that its chunks are permuted by: 16 rows over all banks
  auto key = [](int row) { return KC >= 16 ? row & 15 : KC == 8 ? (row >> 1) & 7 : (row >> 2) & 3; };
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

  const int mine = wave * kRowsPer + lane / KC;  // this lane's row of a wave's first load
  const int chunk = lane % KC ^ key(mine);       // the same in all of them
  const int steps = (a.kch + KC - 1) / KC;
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
      offb[i] = n0 + n < N ? (uint32_t)((n + (up ? N : 0)) * width) + chunk * 16 : kNowhere;
    }
    begin = (int)((uint32_t)(x.e * cols + x.col) % (uint32_t)steps);
  };
  // Load n of a step: those of q first.  Every load of a step is issued, past the rows'
  // end too, so that their number is known.
  auto load = [&](auto STAGE, int s, auto n) __attribute__((always_inline)) {
    int step = s + begin;
    if (step >= steps) step -= steps;
    const bool in = s < steps && chunk < a.kch - step * KC;  // a step there is, not past the row's end
    const int at = step * KC * 16;
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
  constexpr std::integral_constant<int, 2> s2;
  constexpr std::integral_constant<int, 3> s3;
  constexpr std::integral_constant<int, kLoadsA + kLoadsB> every;
  auto start = [&]() __attribute__((always_inline)) {  // the steps before the first
    loads(s0, 0, s0, every);
    if constexpr (STAGES > 2) loads(s1, 1, s0, every);
    if constexpr (STAGES > 3) loads(s2, 2, s0, every);
  };
  using Ch = Channels<DT, GATED, NB>;
  constexpr int kOuts = GATED ? NB / 2 : NB;  // results of a wave in a row tile
  constexpr int kStores = MB * (Ch::kPaired ? kOuts / 2 : kOuts);  // of a wave, for a whole tile
  int stored = 0;  // stores that the tile before ended with, at least
  i32x4 acc[MB][NB];
  // the sums, of the first B row tiles of each wave
  auto sums = [&](auto B) __attribute__((always_inline)) {
    // step s in stage I: wait for its loads, let the stage before it be filled again, multiply
    auto work = [&](auto I, int s) __attribute__((always_inline)) {
      constexpr int kFlying = (STAGES - 2) * (kLoadsA + kLoadsB);  // loads that may still be on their way
      __asm__ __volatile__("" ::: "memory");  // the barrier alone does not keep LDS reads on their side of it
      // memory operations complete in their order: the stores of the tile before came after
      // this one's first loads, and need not be waited for with them
      if (s < STAGES - 1 && stored == kStores) __builtin_amdgcn_s_waitcnt(wait_for(kFlying + kStores));
      else if (s < STAGES - 1 && stored >= kStores / 2) __builtin_amdgcn_s_waitcnt(wait_for(kFlying + kStores / 2));
      else __builtin_amdgcn_s_waitcnt(wait_for(kFlying));
      __builtin_amdgcn_s_barrier();
      __asm__ __volatile__("" ::: "memory");
      constexpr std::integral_constant<int, (I + STAGES - 1) % STAGES> before_it;
      const u32x4 *la = stage_a(I), *lb = stage_b(I);
      const int r = lane & 15, c = lane >> 4;
      constexpr int kParts = KC / 4;
      i32x4 fa[kParts][B], fb[kParts][NB];
#pragma unroll
      for (int k = 0; k < kParts; ++k) {
        const int slot = (4 * k + c) ^ key(r);  // 16 more rows have the same key
#pragma unroll
        for (int j = 0; j < NB; ++j) fb[k][j] = __builtin_bit_cast(i32x4, lb[((wn * NB + j) * 16 + r) * KC + slot]);
#pragma unroll
        for (int i = 0; i < B; ++i) fa[k][i] = __builtin_bit_cast(i32x4, la[((i * WM + wm) * 16 + r) * KC + slot]);
      }
      // a load takes the address unit as long as a product the matrix unit: one by one between them
      constexpr int kGroups = kParts * B;
      auto group = [&](auto self, auto g) __attribute__((always_inline)) {
        if constexpr (g < kGroups) {
          constexpr int k = g / B, i = g % B;
          loads(before_it, s + STAGES - 1, std::integral_constant<int, g * every / kGroups>{},
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
    int s = 0;
    for (; s + STAGES <= steps; s += STAGES) {
      work(s0, s);
      work(s1, s + 1);
      if constexpr (STAGES > 2) work(s2, s + 2);
      if constexpr (STAGES > 3) work(s3, s + 3);
    }
    if (s < steps) work(s0, s);
    if constexpr (STAGES > 2)
      if (s + 1 < steps) work(s1, s + 1);
    if constexpr (STAGES > 3)
      if (s + 2 < steps) work(s2, s + 2);
  };

  // lane: row l % 16 of a row tile
  const int g = lane >> 4;
  struct Scales {
    f32x4 w[NB];
    float q[MB];
  };
  typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
  auto scales_of = [&](const Tile& x, const Rows& rows, Scales& to) __attribute__((always_inline)) {
    const int n0 = x.col * (GATED ? BN / 2 : BN);
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int n = n0 + Ch::of_result(wn * kOuts + (GATED ? j / 2 : j), g);
      const float* p = a.ws + (int64_t)x.e * a.N + n + (GATED && (j & 1) ? N : 0);
      to.w[j] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (n < N) to.w[j] = *reinterpret_cast<const f32x4_any*>(p);
    }
#pragma unroll
    for (int i = 0; i < MB; ++i) to.q[i] = (uint32_t)rows.scale[i] < (uint32_t)a.M ? a.qs[rows.scale[i]] : 0.f;
  };
  Rows rows;
  Scales now, then;
  rows_of(t, rows);
  aim(t, rows);
  scales_of(t, rows, now);
  Tile next = tile_at(id += stride);
  rows_of(next, rows);
  start();
  for (;;) {
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    const int tiles = (t.rows + 16 * WM - 1) / (16 * WM);
    if constexpr (MB == 1) {
      sums(std::integral_constant<int, 1>{});
    } else if constexpr (MB == 2) {
      if (tiles == 1) sums(std::integral_constant<int, 1>{});
      else sums(std::integral_constant<int, 2>{});
    } else if constexpr (MB == 4) {
      if (tiles == 1) sums(std::integral_constant<int, 1>{});
      else if (tiles == 2) sums(std::integral_constant<int, 2>{});
      else if (tiles == 3) sums(std::integral_constant<int, 3>{});
      else sums(std::integral_constant<int, 4>{});
    } else {
      if (tiles <= 2) sums(std::integral_constant<int, 2>{});
      else if (tiles <= 4) sums(std::integral_constant<int, 4>{});
      else if (tiles == 5) sums(std::integral_constant<int, 5>{});
      else if (tiles == 6) sums(std::integral_constant<int, 6>{});
      else if (tiles == 7) sums(std::integral_constant<int, 7>{});
      else if (tiles == 8 && MB > 8) sums(std::integral_constant<int, 8>{});
      else sums(std::integral_constant<int, MB>{});
    }
    __asm__ __volatile__("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(wait_for(0));  // nothing on its way to a stage, or from one
    Tile after = {0, 0, 0, 0};
    if (next.rows != 0) {  // its first loads run while this tile is written
      __builtin_amdgcn_s_barrier();
      __asm__ __volatile__("" ::: "memory");
      aim(next, rows);
      scales_of(next, rows, then);
      after = tile_at(id += stride);
      rows_of(after, rows);
      in_order();
      start();
      __asm__ __volatile__("" ::: "memory");  // the stores below come after these loads
      in_order();
    }
    const int n0 = t.col * (GATED ? BN / 2 : BN);
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      const int r = (i * WM + wm) * 16 + (lane & 15);
      if (r >= t.rows) continue;
      const int64_t p = (int64_t)t.row + r;
      float y[kOuts][4];
#pragma unroll
      for (int j = 0; j < kOuts; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          if constexpr (GATED)
            y[j][v] = activate((float)acc[i][2 * j][v] * now.q[i] * now.w[2 * j][v], a.act) *
                      ((float)acc[i][2 * j + 1][v] * now.q[i] * now.w[2 * j + 1][v]);
          else
            y[j][v] = (float)acc[i][j][v] * now.q[i] * now.w[j][v];
        }
      if constexpr (DT == kF32) {
        float* out = static_cast<float*>(a.out) + p * N;
#pragma unroll
        for (int j = 0; j < kOuts; ++j) {
          const int n = n0 + Ch::of_result(wn * kOuts + j, g);
          if (n < N) *reinterpret_cast<float4*>(out + n) = make_float4(y[j][0], y[j][1], y[j][2], y[j][3]);
        }
      } else {
        uint16_t* out = static_cast<uint16_t*>(a.out) + p * N;
        if constexpr (Ch::kPaired) {
#pragma unroll
          for (int j = 0; j < kOuts; j += 2) {  // N is whole 16-byte chunks: all 8 channels there, or none
            const int n = n0 + Ch::of_result(wn * kOuts + j, g);
            if (n < N)
              *reinterpret_cast<u32x4*>(out + n) = u32x4{round_bf16x2(y[j][0], y[j][1]), round_bf16x2(y[j][2], y[j][3]),
                                                         round_bf16x2(y[j + 1][0], y[j + 1][1]),
                                                         round_bf16x2(y[j + 1][2], y[j + 1][3])};
          }
        } else {
#pragma unroll
          for (int j = 0; j < kOuts; ++j) {
            const int n = n0 + Ch::of_result(wn * kOuts + j, g);
            if (n < N)
              *reinterpret_cast<uint2*>(out + n) = make_uint2(round_bf16x2(y[j][0], y[j][1]), round_bf16x2(y[j][2], y[j][3]));
          }
        }
      }
    }
    if (next.rows == 0) return;
    // row tiles of this wave with a row, where every channel is there
    const int with_rows = min(MB, max(0, (t.rows - wm * 16 + 16 * WM - 1) / (16 * WM)));
    stored = n0 + (GATED ? BN / 2 : BN) <= N ? with_rows * (kStores / MB) : 0;
    t = next;
    next = after;
    now = then;
  }
}

// Tiles of rows there can be at most (whole ones, and one of each expert that is not
// whole) times tiles of channels: the host does not know the experts' rows.
int64_t most_tiles(const I8Args& a, int bm, int bn) {
  const int64_t rows = a.offset ? a.R : a.M, partial = a.offset ? (rows < a.E ? rows : a.E) : 1;
  return (rows / bm + partial) * ((a.N + bn - 1) / bn);
}

template <int MB, int NB, int WM, int WN, int KC, int STAGES, int EU>
hipError_t launch_tile(const I8Args& a, hipStream_t s) {
  constexpr int BM = 16 * MB * WM, BN = 16 * NB * WN;
  const bool gated = a.act != MOE_ACT_NONE;
  const int cols = (a.N + BN - 1) / BN;  // gated: BN / 2 of N / 2 outputs each
  const int64_t most = (most_tiles(a, BM, BN) + 7) / 8 * 8, fit = 256 * (4 * EU / (WM * WN));  // what the GPU holds at once
  const unsigned grid = (unsigned)(most < fit ? most : fit);
  const uint32_t lds = 2 * (a.E + 1) * sizeof(int);
  if (a.dtype == kF32) {
    if (gated) i8_kernel<kF32, true, MB, NB, WM, WN, KC, STAGES, EU><<<grid, WM * WN * kWave, lds, s>>>(a, cols);
    else i8_kernel<kF32, false, MB, NB, WM, WN, KC, STAGES, EU><<<grid, WM * WN * kWave, lds, s>>>(a, cols);
  } else {
    if (gated) i8_kernel<kBF16, true, MB, NB, WM, WN, KC, STAGES, EU><<<grid, WM * WN * kWave, lds, s>>>(a, cols);
    else i8_kernel<kBF16, false, MB, NB, WM, WN, KC, STAGES, EU><<<grid, WM * WN * kWave, lds, s>>>(a, cols);
  }
  return hipGetLastError();
}

}  // namespace

// Tiles of 128 x 256, one workgroup a CU, where there are enough of them; else of 64 x
// 128, two workgroups a CU; else of 64 x 64.  Rows of 2 KiB and more hide a tile's
// beginning and end better, so fewer large ones will do.  In us, large / middle / small:
//   64 tokens of 8 of 128 experts, 2048 x 1536 (792 large tiles at most): 73 / 73 / 77
//   1500 rows, 7168 x 4096 (192): 51 / 58 / 81;   1024 rows (128): 48 / 38 / 52
//   2000 tokens of 2 of 8, 1024 x 2048 (312): 27 / 23 / 26
//   4096 rows, 768 x 1024 (128; 512 of the middle size): 12.5 / 10 / 12.4
//   64 tokens of 2 of 8, 4096 x 2048 (72; 160): 21 / 18 / 14;   1 token of 8 of 128: 14 / 12 / 9
hipError_t launch_i8(const I8Args& a, hipStream_t s) {
  if (most_tiles(a, 128, 256) >= (a.kch >= 128 ? 192 : 400)) return launch_tile<4, 4, 2, 4, 8, 3, 2>(a, s);
  if (most_tiles(a, 64, 128) >= 256) return launch_tile<2, 4, 2, 2, 8, 3, 2>(a, s);
  return launch_tile<1, 2, 4, 2, 8, 3, 4>(a, s);
}

}  // namespace moe
