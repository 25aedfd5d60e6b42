// Products of 8-bit rows and 8-bit weights, grouped by expert (moe_matmul_i8).
//
//   acc[p,n] = sum_k q[p,k] w[e,n,k]        exact, in 32-bit integers
//   y[p,n]   = float(acc) * s[p] * sw[e,n]  in float32, rounded once to the output type
//   gated:     f(y[p,i]) * y[p,I+i]         formed before that rounding
//
// A workgroup's tile is BM rows of one expert by BN channels; both operands run
// through LDS in steps of KC 16-byte chunks a row, loaded there directly (no
// registers on the way) while the matrix cores work on the step before: two stages,
// one barrier a step.  The stages are separate arrays, so that the compiler sees
// that a stage's reads need not wait for the other's loads.  The weights are the
// first operand of the matrix instruction: a lane then holds four neighbouring
// channels of one row.  Chunks of a row are stored permuted (by the row's bits), so
// that the 16 rows of an operand lie in different banks.
//
// Rows past an expert's last and chunks past a row's end have an offset outside the
// buffer: the hardware reads nothing and puts zeros into LDS.
//
// Tiles: an expert of n rows has ceil(n / BM), of equal size; the tile of a
// workgroup is found from the experts' offsets on the device (the host knows only
// how many there can be).  Each XCD takes a run of tiles, the rows' tiles of the
// same channels one after the other, so that weights are read from HBM once and
// found in that XCD's L2 by the others.
#include "device_common.h"
#include "internal.h"
#include "mfma.h"
#include "quant.h"
#include "../../include/moe_layout.h"

namespace moe {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr uint32_t kNowhere = 0xFFFFFFF0u;  // past every buffer

struct Tile {
  int e, row, rows, col;  // expert, first receive row, rows, channel tile
};

// Finds tile `id` of a layout; false past the last one.
__device__ __forceinline__ bool find_tile(const I8Args& a, int bm, int cols, int64_t id, int (&shared)[8], Tile& t) {
  if (!a.offset) {
    const int mt = (a.M + bm - 1) / bm;
    const int64_t total = (int64_t)mt * cols, per = (total + 7) / 8;
    const int64_t at = (id & 7) * per + (id >> 3);
    if ((id >> 3) >= per || at >= total) return false;
    const int m = (int)(at % mt);
    const int step = ((a.M + mt - 1) / mt + 15) & ~15;
    t.e = 0;
    t.col = (int)(at / mt);
    t.row = m * step;
    t.rows = min(step, a.M - t.row);
    return true;
  }
  // each thread has four experts
  const int lane = lane_id(), wave = threadIdx.x / kWave;
  const int e0 = 4 * (int)threadIdx.x;
  int start[5], tiles[4], sum = 0;
#pragma unroll
  for (int i = 0; i < 5; ++i) {
    const int v = a.offset[min(e0 + i, a.E)];
    start[i] = min(max(v, 0), a.R);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    tiles[i] = (max(start[i + 1] - start[i], 0) + bm - 1) / bm;
    sum += tiles[i];
  }
  const int upto = (int)wave_scan((uint32_t)sum);
  if (lane == 63) shared[wave] = upto;
  __syncthreads();
  int before = upto - sum, all = 0;
#pragma unroll
  for (int w = 0; w < kThreads / kWave; ++w) {
    if (w < wave) before += shared[w];
    all += shared[w];
  }
  const int64_t total = (int64_t)all * cols, per = (total + 7) / 8;
  const int64_t at = (id & 7) * per + (id >> 3);
  if ((id >> 3) >= per || at >= total) return false;  // uniform
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t first = (int64_t)before * cols;
    if (tiles[i] > 0 && at >= first && at < first + (int64_t)tiles[i] * cols) {
      const int r = (int)(at - first), n = start[i + 1] - start[i];
      const int step = ((n + tiles[i] - 1) / tiles[i] + 15) & ~15;
      const int m = r % tiles[i];
      shared[4] = e0 + i;
      shared[5] = start[i] + m * step;
      shared[6] = min(step, n - m * step);
      shared[7] = r / tiles[i];
    }
    before += tiles[i];
  }
  __syncthreads();
  t.e = shared[4];
  t.row = shared[5];
  t.rows = shared[6];
  t.col = shared[7];
  return true;
}

__device__ __forceinline__ float activate(float g, int act) {
  if (act == MOE_ACT_SILU) return g / (1.f + expf(-g));
  return 0.5f * g * (1.f + tanhf(0.7978845608028654f * (g + 0.044715f * g * g * g)));
}

// MB x NB tiles of 16 x 16 a wave, WM x WN waves.
template <int DT, bool GATED, int MB, int NB, int WM, int WN, int KC>
__global__ __launch_bounds__(kThreads) void i8_kernel(I8Args a, int cols) {
  static_assert(WM * WN * kWave == kThreads);
  constexpr int BM = 16 * MB * WM, BN = 16 * NB * WN, kWaves = WM * WN;
  constexpr int kRowsPer = kWave / KC;                  // rows of one load instruction
  constexpr int kLoadsA = BM / kRowsPer / kWaves, kLoadsB = BN / kRowsPer / kWaves;
  static_assert(kLoadsA >= 1 && kLoadsB >= 1 && BM % (kRowsPer * kWaves) == 0 && BN % (kRowsPer * kWaves) == 0);
  __shared__ u32x4 a0[BM * KC], b0[BN * KC], a1[BM * KC], b1[BN * KC];
  __shared__ int found[8];
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wm = wave % WM, wn = wave / WM;
  // the bits of a row that its chunks are permuted by: 16 rows over all banks
  auto key = [](int row) { return KC >= 16 ? row & 15 : (row >> 1) & 7; };
  const int N = GATED ? a.N / 2 : a.N;  // channels of the output

  for (int64_t id = blockIdx.x;; id += gridDim.x) {  // one tile, unless there are more than the largest grid
    Tile t;
    if (!find_tile(a, BM, cols, id, found, t)) return;
    const int64_t width = (int64_t)a.kch * 16;
    const int n0 = t.col * (GATED ? BN / 2 : BN);
    // rows of q: the tile's own, or any
    const int64_t qbase = a.recv_token ? 0 : (int64_t)t.row * width;
    const int64_t qbytes = min((int64_t)0xFFFFFFE0, (a.recv_token ? (int64_t)a.M : (int64_t)t.rows) * width);
    const auto rq = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(a.q) + qbase, 0, (int)(uint32_t)qbytes, 0x00027000);
    const int64_t wbase = ((int64_t)t.e * a.N + n0) * width;
    const int64_t wbytes = ((int64_t)a.N - n0) * width;  // below 2 GiB
    const auto rw = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(a.w) + wbase, 0, (int)(uint32_t)wbytes, 0x00027000);

    uint32_t offa[kLoadsA], offb[kLoadsB];
    int chunka[kLoadsA], chunkb[kLoadsB];
  #pragma unroll
    for (int i = 0; i < kLoadsA; ++i) {
      const int r = (i * kWaves + wave) * kRowsPer + lane / KC;
      chunka[i] = lane % KC ^ key(r);
      offa[i] = kNowhere;
      if (r < t.rows) {
        int row = r;
        if (a.recv_token) row = a.recv_token[t.row + r];
        if (!a.recv_token || (unsigned)row < (unsigned)a.M) offa[i] = (uint32_t)(row * width) + chunka[i] * 16;
      }
    }
  #pragma unroll
    for (int i = 0; i < kLoadsB; ++i) {
      const int r = (i * kWaves + wave) * kRowsPer + lane / KC;
      chunkb[i] = lane % KC ^ key(r);
      // gated: 16 gate channels, then their 16 up channels
      const int n = GATED ? r / 32 * 16 + r % 16 : r;
      const int row = GATED && (r & 16) ? n + N : n;
      offb[i] = n0 + n < N ? (uint32_t)(row * width) + chunkb[i] * 16 : kNowhere;
    }
    auto load = [&](u32x4* la, u32x4* lb, int step) {
      const int left = a.kch - step * KC;  // chunks from here on
      const int at = step * KC * 16;
  #pragma unroll
      for (int i = 0; i < kLoadsA; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rq, (__attribute__((address_space(3))) void*)(la + (i * kWaves + wave) * kWave), 16,
            (int)(left >= KC || chunka[i] < left ? offa[i] : kNowhere), at, 0, 0);
  #pragma unroll
      for (int i = 0; i < kLoadsB; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rw, (__attribute__((address_space(3))) void*)(lb + (i * kWaves + wave) * kWave), 16,
            (int)(left >= KC || chunkb[i] < left ? offb[i] : kNowhere), at, 0, 0);
    };
    i32x4 acc[MB][NB];
  #pragma unroll
    for (int i = 0; i < MB; ++i)
  #pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    auto multiply = [&](const u32x4* la, const u32x4* lb) {
      const int r = lane & 15, c = lane >> 4;
  #pragma unroll
      for (int k = 0; k < KC / 4; ++k) {
        const int slot = (4 * k + c) ^ key(r);  // 16 more rows have the same key
        i32x4 fa[MB], fb[NB];
  #pragma unroll
        for (int i = 0; i < MB; ++i) fa[i] = __builtin_bit_cast(i32x4, la[((i * WM + wm) * 16 + r) * KC + slot]);
  #pragma unroll
        for (int j = 0; j < NB; ++j) fb[j] = __builtin_bit_cast(i32x4, lb[((wn * NB + j) * 16 + r) * KC + slot]);
  #pragma unroll
        for (int i = 0; i < MB; ++i)
  #pragma unroll
          for (int j = 0; j < NB; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[j], fa[i], acc[i][j], 0, 0, 0);
      }
    };
    const int steps = (a.kch + KC - 1) / KC;
    load(a0, b0, 0);
    for (int s = 0; s < steps; s += 2) {
      __syncthreads();  // stage 0 has landed, stage 1 has been read
      if (s + 1 < steps) load(a1, b1, s + 1);
      multiply(a0, b0);
      __syncthreads();
      if (s + 1 >= steps) break;
      if (s + 2 < steps) load(a0, b0, s + 2);
      multiply(a1, b1);
    }

    // lane: row l % 16 of a row tile, channels 4 (l / 16) + 0..3 of a channel tile
    const int quad = 4 * (lane >> 4);
    float sw[NB][4];
  #pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int b = wn * NB + j;
      const int n = n0 + (GATED ? b / 2 * 16 : b * 16) + quad;
      const float* p = a.ws + (int64_t)t.e * a.N + (GATED && (b & 1) ? N : 0) + n;
  #pragma unroll
      for (int v = 0; v < 4; ++v) sw[j][v] = n < N ? p[v] : 0.f;
    }
  #pragma unroll
    for (int i = 0; i < MB; ++i) {
      const int r = (i * WM + wm) * 16 + (lane & 15);
      if (r >= t.rows) continue;
      const int64_t p = (int64_t)t.row + r;
      int64_t source = p;
      if (a.recv_token) source = a.recv_token[p];
      const float s = source >= 0 && source < a.M ? a.qs[source] : 0.f;
      constexpr int kStep = GATED ? 2 : 1;
  #pragma unroll
      for (int j = 0; j < NB; j += kStep) {
        const int n = n0 + (wn * NB + j) / kStep * 16 + quad;
        float y[4];
  #pragma unroll
        for (int v = 0; v < 4; ++v) {
          y[v] = (float)acc[i][j][v] * s * sw[j][v];
          if constexpr (GATED) y[v] = activate(y[v], a.act) * ((float)acc[i][j + 1][v] * s * sw[j + 1][v]);
        }
        if (n >= N) continue;
        if constexpr (DT == kF32) {
          *reinterpret_cast<float4*>(static_cast<float*>(a.out) + p * N + n) = make_float4(y[0], y[1], y[2], y[3]);
        } else {
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + p * N + n) =
              make_uint2(round_bf16x2(y[0], y[1]), round_bf16x2(y[2], y[3]));
        }
      }
    }
    __syncthreads();  // the stages and `found` are free again
  }
}

template <int MB, int NB, int WM, int WN, int KC>
hipError_t launch_tile(const I8Args& a, hipStream_t s) {
  constexpr int BM = 16 * MB * WM, BN = 16 * NB * WN;
  const bool gated = a.act != MOE_ACT_NONE;
  const int bn = gated ? BN / 2 : BN, N = gated ? a.N / 2 : a.N;
  const int cols = (N + bn - 1) / bn;
  // tiles of rows there can be at most: whole ones, and one of each expert that is not whole
  const int64_t rows = a.offset ? a.R : a.M, partial = a.offset ? (rows < a.E ? rows : a.E) : 1;
  int64_t grid = ((rows / BM + partial) * cols + 7) / 8 * 8;
  if (grid > (1 << 22)) grid = 1 << 22;
  if (a.dtype == kF32) {
    if (gated) i8_kernel<kF32, true, MB, NB, WM, WN, KC><<<(unsigned)grid, kThreads, 0, s>>>(a, cols);
    else i8_kernel<kF32, false, MB, NB, WM, WN, KC><<<(unsigned)grid, kThreads, 0, s>>>(a, cols);
  } else {
    if (gated) i8_kernel<kBF16, true, MB, NB, WM, WN, KC><<<(unsigned)grid, kThreads, 0, s>>>(a, cols);
    else i8_kernel<kBF16, false, MB, NB, WM, WN, KC><<<(unsigned)grid, kThreads, 0, s>>>(a, cols);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_i8(const I8Args& a, hipStream_t s) {
  const int64_t rows = a.offset ? a.R : a.M, per = (rows + a.E - 1) / a.E;  // of an expert, on average
  if (per <= 16) return launch_tile<1, 2, 1, 4, 16>(a, s);
  return launch_tile<4, 4, 2, 2, 8>(a, s);
}

}  // namespace moe
