// Low-rank adapters of many requests beside a shared projection, and their
// gradients, on the rows of a layout with one expert (adapter) per token:
//
//   u[p]    = A_e x_t                      row p of adapter e holds token t
//   out[t]  = base[t] + w_t (u[p] B_e)     A_e [r, H], B_e [r, N]
//   raw[p]  = B_e g_t,  gu[p] = w_t raw[p],  grad_w[t] = <raw[p], u[p]>
//   grad_x[t] = grad_base[t] + gu[p] A_e
//   grad_A_e  = sum_p gu[p]^T x_t,   grad_B_e = sum_p w_t u[p]^T g_t
//
// Three kernels do all of it, because A and B are both held with the rank as
// the row index: `shrink` (to the rank: u, gu), `expand` (back to full width:
// out, grad_x) and `wgrad` (an adapter's sum over its rows).  All are bound by
// the wide rows they read and write; the products are thin (r <= 128).
//
// Rows of an adapter stand together in the layout, so a tile of 16 receive
// rows usually belongs to one adapter and its product is a matrix product.  A
// tile that several adapters share is walked adapter by adapter, the rows of
// the others masked; with few tokens the adapters of a tile go to different
// workgroups (slots).
//
// u and gu stay float32.  Where they are operands of a bfloat16 matrix
// instruction they are split into two bfloat16 parts (their sum is within
// 2^-16 of the value), so that nothing but the result is rounded to bfloat16:
// the second instruction costs nothing beside the memory traffic.
#include "device_common.h"
#include "internal.h"
#include "mfma.h"
#include "../../include/moe_layout.h"

namespace moe {
namespace {

constexpr int kTile = 16;        // receive rows of a tile
constexpr int kMaxOff = 1024 + 1;

template <int DT>
struct Shape {
  static constexpr int V = DT == kBF16 ? 8 : 4;   // elements of a chunk
  static constexpr int JL = V;                    // summed indices a lane holds of a block
  static constexpr int KB = 4 * JL;               // summed indices of a block
  static constexpr int COLS = 16 * V;             // columns of a wave's tile
};

// The tile's adapters: f(e, lo, hi) for each adapter e (or e >= A: rows
// without one) with rows [lo, hi) in the tile, of those that fall to `slot`.
// off: the layout's expert offsets in LDS, E + 1 of them.
template <typename F>
__device__ __forceinline__ void each_adapter(const int* off, int E, int r0, int r1, int slot, int slots, F f) {
  const int lane = lane_id();
  int e = 0;  // the first segment that ends past r0
  for (int i = 0; i < E; i += kWave) e += __popcll(__ballot(i + lane < E && off[i + lane + 1] <= r0));
  int n = 0;
  for (int lo = r0; lo < r1;) {  // wave-uniform: the same values in every lane
    const int hi = e < E ? min(__builtin_amdgcn_readfirstlane(off[e + 1]), r1) : r1;  // behind the last segment: none
    if (hi > lo) {
      if (n % slots == slot) f(e, lo, hi);
      ++n;
      lo = hi;
    }
    ++e;
  }
}

__device__ __forceinline__ void load_offsets(int* off, const LowrankArgs& a) {
  for (int i = threadIdx.x; i <= a.E; i += blockDim.x) off[i] = a.expert_offset[i];
  __syncthreads();
}

// The token of receive row p, -1 for a row without one (padding).
__device__ __forceinline__ int row_token(const LowrankArgs& a, int p) {
  const int t = p < a.R ? a.recv_token[p] : -1;
  return (unsigned)t < (unsigned)a.T ? t : -1;
}

// ---- shrink ---------------------------------------------------------------------
//
// One workgroup per (RT tiles of 16 rows, slot).  Its waves split the sum over
// the row, a 128-byte line of every row each in turn, kDepth lines in flight,
// and meet in LDS; wave rt adds the parts of tile rt and writes its 16 rows of
// r float32.
//
// A wave loads whole lines, eight lanes to a line: the bank is read again for
// every tile, from L2, and L2 gives 25.6 TB/s in that order but 9.2 TB/s in the
// operands' (each lane of a quad on another row).  The lines pass through the
// wave's own piece of LDS, chunks rotated by row so that neither side meets a
// bank twice.  Workgroups start at different lines (and go round): rows a
// power of two apart, read at the same place at once, meet in a few memory
// channels.  FAR: the wide rows reach past what a buffer's 32-bit offsets do (2
// GiB).
template <int JT, int RT>
struct Shrink {
  static constexpr int kMeet = JT * RT <= 4 ? JT : 4 / RT;     // tiles of the rank that meet in LDS together
  static constexpr int kStaged = JT < 4 ? JT : 4;              // tiles of the rank in LDS at a time
  static constexpr int kRows = 16 * (RT + kStaged);            // rows of a stage: the tokens', then the bank's
  static constexpr int kWaves = JT + RT <= 3 ? 8 : 4;
  static constexpr size_t kLds = (size_t)kWaves * kRows * 128;  // at most 48 KiB
};

template <int DT, int JT, int RT, bool FAR>
__global__ __launch_bounds__((Shrink<JT, RT>::kWaves * kWave)) void shrink_kernel(LowrankArgs a) {
  constexpr int kShrinkWaves = Shrink<JT, RT>::kWaves, kMeet = Shrink<JT, RT>::kMeet;
  constexpr int kStaged = Shrink<JT, RT>::kStaged, kRows = Shrink<JT, RT>::kRows;
  constexpr int kDepth = JT + RT <= 2 ? 3 : JT + RT <= 4 ? 2 : 1;
  __shared__ int off[kMaxOff];
  extern __shared__ u32x4 lds[];  // [waves][kRows][8 chunks]; then [waves][RT][kMeet][64] to meet in
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave));
  const int col = lane & 15, q = lane >> 4;  // of an operand
  const int row8 = lane >> 3, chunk = lane & 7;  // of a load: 8 rows by one line
  u32x4* stage = lds + (size_t)wave * kRows * 8;
  f32x4* part = reinterpret_cast<f32x4*>(lds);
  const int nch = a.wch, lines = (nch + 7) / 8;
  const int start = (blockIdx.x + blockIdx.y) * 5 % lines;
  const uint32_t row_bytes = (uint32_t)nch * 16;
  const int r0 = blockIdx.x * kTile * RT, r1 = min(r0 + kTile * RT, a.R);
  int t[RT], load_t[2 * RT];
#pragma unroll
  for (int i = 0; i < 2 * RT; ++i) load_t[i] = max(row_token(a, r0 + i * 8 + row8), 0);
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) t[rt] = row_token(a, r0 + rt * kTile + col);
  load_offsets(off, a);
  each_adapter(off, a.E, r0, r1, blockIdx.y, gridDim.y, [&](int e, int lo, int hi) {
    bool mine[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int p = r0 + rt * kTile + col;
      mine[rt] = p >= lo && p < hi;
    }
    if (e >= a.A) {  // no adapter: u = 0, and no gradient
      for (int i = threadIdx.x; i < (hi - lo) * a.r; i += kShrinkWaves * kWave) a.u[(size_t)lo * a.r + i] = 0.f;
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
        if (a.dot && wave == rt && q == 0 && mine[rt] && t[rt] >= 0) a.dot[t[rt]] = 0.f;
      return;
    }
    // columns of other adapters take their rows (padding the first one); the
    // results are dropped
    const auto wide = make_rows(a.rows, FAR ? 0 : (size_t)a.T * row_bytes);
    const auto bank = make_rows(static_cast<const u32x4*>(a.bank) + (size_t)e * a.r * nch, (size_t)a.r * row_bytes);
    const uint32_t b_off = (uint32_t)row8 * row_bytes + chunk * 16;
    u32x4 in[kDepth][2 * (RT + JT)];
    auto fetch = [&](int d, int i) {  // the i-th line after `start`; past the last: zeros
      const int line = i + start < lines ? i + start : i + start - lines;
      const int c = line * 8 + chunk;
      const bool ok = i < lines && c < nch;
#pragma unroll
      for (int k = 0; k < 2 * RT; ++k) {
        if constexpr (FAR) {
          in[d][k] = static_cast<const u32x4*>(a.rows)[(size_t)load_t[k] * nch + (ok ? c : 0)];
          // the bank's zeros alone would leave NaN where a row holds one
          if (!ok) in[d][k] = u32x4{0u, 0u, 0u, 0u};
        } else {
          in[d][k] = load_rows(wide, ok ? (uint32_t)load_t[k] * row_bytes + chunk * 16 : kOutside, (uint32_t)line * 128);
        }
      }
#pragma unroll
      for (int k = 0; k < 2 * JT; ++k)
        in[d][2 * RT + k] = load_rows(bank, ok ? b_off + (uint32_t)k * 8 * row_bytes : kOutside, (uint32_t)line * 128);
    };
    f32x4 acc[RT][JT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int jt = 0; jt < JT; ++jt) acc[rt][jt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      fetch(d, wave + d * kShrinkWaves);
      in_order();
    }
    for (int i = wave; i < lines; i += kShrinkWaves * kDepth) {
#pragma unroll
      for (int d = 0; d < kDepth; ++d) {
        // row r's chunk c stands at place c ^ (r / 2 % 8)
        auto put = [&](int r, const u32x4 v) { stage[r * 8 + (chunk ^ (r >> 1 & 7))] = v; };
#pragma unroll
        for (int k = 0; k < 2 * RT; ++k) put(k * 8 + row8, in[d][k]);
#pragma unroll
        for (int j0 = 0; j0 < JT; j0 += kStaged) {
#pragma unroll
          for (int k = 0; k < 2 * kStaged; ++k) put((2 * RT + k) * 8 + row8, in[d][2 * RT + 2 * j0 + k]);
          if (j0 + kStaged == JT) {
            in_order();
            fetch(d, i + (d + kDepth) * kShrinkWaves);
            in_order();
          }
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const int place = (s * 4 + q) ^ (col >> 1);
            u32x4 xv[RT];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) xv[rt] = stage[(rt * 16 + col) * 8 + place];
#pragma unroll
            for (int m = 0; m < kStaged; ++m) {
              const u32x4 bv = stage[((RT + m) * 16 + col) * 8 + place];
#pragma unroll
              for (int rt = 0; rt < RT; ++rt) acc[rt][j0 + m] = mma_chunk<DT>(bv, xv[rt], acc[rt][j0 + m]);
            }
          }
        }
        in_order();
      }
    }
    float w = 1.f, dot = 0.f;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
      if (wave == rt && a.w && t[rt] >= 0) w = a.w[t[rt]];
#pragma unroll
    for (int first = 0; first < JT; first += kMeet) {
      __syncthreads();  // every wave is done with its stage, or with the parts before
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int m = 0; m < kMeet; ++m) part[((wave * RT + rt) * kMeet + m) * kWave + lane] = acc[rt][first + m];
      __syncthreads();
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        if (wave != rt) continue;
        const size_t p = r0 + rt * kTile + col;
#pragma unroll
        for (int m = 0; m < kMeet; ++m) {
          f32x4 v = part[(rt * kMeet + m) * kWave + lane];
#pragma unroll
          for (int k = 1; k < kShrinkWaves; ++k) v += part[((k * RT + rt) * kMeet + m) * kWave + lane];
          const int j = (first + m) * 16 + q * 4;
          if (mine[rt] && j < a.r) {
            if (t[rt] < 0) v = f32x4{0.f, 0.f, 0.f, 0.f};  // padding
            if (a.backward) {
              if (a.dot) {
                const f32x4 u = *reinterpret_cast<const f32x4*>(a.saved + p * a.r + j);
#pragma unroll
                for (int i = 0; i < 4; ++i) dot += v[i] * u[i];
              }
              v *= w;
            }
            *reinterpret_cast<f32x4*>(a.u + p * a.r + j) = v;
          }
        }
      }
    }
    if (a.dot) {
      dot += __shfl_xor(dot, 16, kWave);
      dot += __shfl_xor(dot, 32, kWave);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
        if (wave == rt && q == 0 && mine[rt] && t[rt] >= 0) a.dot[t[rt]] = dot;
    }
    __syncthreads();  // the parts have been read
  });
}

// A chunk of V floats rounded to the element type.
template <int DT, int V>
__device__ __forceinline__ u32x4 pack_rows(const float (&f)[V]) {
  u32x4 c;
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = DT == kF32 ? __float_as_uint(f[i]) : round_bf16x2(f[2 * i % V], f[(2 * i + 1) % V]);
  return c;
}

// ---- products over the rank or over rows --------------------------------------------
//
// Here the summed index is the row index of the wide operand (the bank's rows,
// or tokens): a lane loads the same chunk of V neighbouring rows, and element i
// of all of them is its operand for the i-th of V result tiles.  The tile's 16
// columns are then V columns apart, and a lane ends with all V elements of
// chunks 4q .. 4q+3.

// Splits 8 floats into two bfloat16 parts, hi + lo.
__device__ __forceinline__ void split_bf16(const float (&f)[8], u32x4& hi, u32x4& lo) {
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    hi[d] = round_bf16x2(f[2 * d], f[2 * d + 1]);
    const float x = f[2 * d] - bf16_lo(hi[d]), y = f[2 * d + 1] - bf16_hi(hi[d]);
    // beyond the finite numbers the difference is not a number: no second part
    lo[d] = round_bf16x2(x - x == 0.f ? x : 0.f, y - y == 0.f ? y : 0.f);
  }
}

// The operands of V result tiles from the chunks of V rows: for bfloat16
// element i across the rows, for float32 the rows as they are.
template <int DT, int V>
__device__ __forceinline__ void across(const u32x4 (&w)[V], u32x4 (&o)[V]) {
  if constexpr (DT == kBF16) {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int d = 0; d < 4; ++d)
        o[i][d] = __builtin_amdgcn_perm(w[2 * d + 1][i / 2], w[2 * d][i / 2], i & 1 ? 0x07060302u : 0x05040100u);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = w[i];
  }
}

// The other operand: V floats along the summed index.
template <int DT>
struct Factor;
template <>
struct Factor<kBF16> {
  u32x4 hi, lo;
  __device__ __forceinline__ explicit Factor(const float (&f)[8]) { split_bf16(f, hi, lo); }
};
template <>
struct Factor<kF32> {
  float f[4];
  __device__ __forceinline__ explicit Factor(const float (&g)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = g[i];
  }
};

// acc[i] += operand i . factor over a block of the summed index.
template <int DT, int V>
__device__ __forceinline__ void mma_across(const u32x4 (&o)[V], const Factor<DT>& f, f32x4 (&acc)[V]) {
  if constexpr (DT == kBF16) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      acc[i] = mma_chunk<kBF16>(o[i], f.hi, acc[i]);
      acc[i] = mma_chunk<kBF16>(o[i], f.lo, acc[i]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i)
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(o[j][i]), f.f[j], acc[i], 0, 0, 0);
  }
}

// ---- expand ---------------------------------------------------------------------
//
// One wave per (a.tiles tiles of 16 receive rows, COLS columns, slot); it keeps
// its columns of an adapter's bank in registers from tile to tile, and has the
// next tile's rows of base on their way.  BLOCKS blocks of KB ranks.  The
// products pass through LDS, so that base is read and out is written with 16
// lanes to a row.
constexpr int kExpandWaves = 4;

template <int DT, int BLOCKS>
__global__ __launch_bounds__(kExpandWaves* kWave) void expand_lowrank_kernel(LowrankArgs a) {
  using S = Shape<DT>;
  constexpr int V = S::V;
  constexpr int kStride = 16 * V + 4;  // floats of a row in LDS: rows shifted by four banks
  __shared__ int off[kMaxOff];
  __shared__ __align__(16) float products[kExpandWaves][kTile * kStride];
  const int lane = lane_id(), wave = (int)(threadIdx.x / kWave);
  const int col = lane & 15, q = lane >> 4;
  float* prod = products[wave];
  const int nch = a.wch;
  const int c0 = (blockIdx.y * kExpandWaves + wave) * 16;  // first chunk of this wave's columns
  const uint32_t row_bytes = (uint32_t)nch * 16;
  const int my_c = c0 + col;
  const bool in = my_c < nch;
  // ranks and columns past the end are outside the bank and read as zeros
  const uint32_t b_off = in ? (uint32_t)my_c * 16 : kOutside;

  // a tile's rows: the token of row `col`, and base where this lane adds it
  // (rows q, 4 + q, ..., chunk `col`)
  struct Rows {
    int t;
    u32x4 base[4];
  } now, next;
  auto fetch = [&](Rows& r, int t) {
    r.t = t;
    if (a.base) {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int tt = max(__shfl(t, s * 4 + q, kWave), 0);
        r.base[s] = static_cast<const u32x4*>(a.base)[(size_t)tt * nch + min(my_c, nch - 1)];
      }
    }
  };
  int tile = blockIdx.x * a.tiles;
  const int tile_end = min(tile + a.tiles, (a.R + kTile - 1) / kTile);
  int next_t = row_token(a, tile * kTile + col);
  load_offsets(off, a);
  if (c0 >= nch) return;
  fetch(next, next_t);
  next_t = row_token(a, (tile + 1) * kTile + col);

  u32x4 bank[BLOCKS][V];
  int held = -1;  // the adapter whose bank is held
  for (; tile < tile_end; ++tile) {
    now = next;
    const int r0 = tile * kTile, r1 = min(r0 + kTile, a.R);
    const float w = a.w ? a.w[max(now.t, 0)] : 1.f;
    float f[BLOCKS][V];
    const float* u = a.u + (size_t)min(r0 + col, a.R - 1) * a.r;
#pragma unroll
    for (int k = 0; k < BLOCKS; ++k)
#pragma unroll
      for (int j = 0; j < V; j += 4) {
        const int jj = k * S::KB + q * V + j;
        const f32x4 v = *reinterpret_cast<const f32x4*>(u + (jj < a.r ? jj : 0));
#pragma unroll
        for (int i = 0; i < 4; ++i) f[k][j + i] = jj < a.r ? v[i] * w : 0.f;
      }
    if (tile + 1 < tile_end) fetch(next, next_t);
    next_t = row_token(a, (tile + 2) * kTile + col);
    each_adapter(off, a.E, r0, r1, blockIdx.z, gridDim.z, [&](int e, int lo, int hi) {
      if (e < a.A) {
        if (e != held) {
          held = e;
          const auto rows = make_rows(static_cast<const u32x4*>(a.bank) + (size_t)e * a.r * nch, (size_t)a.r * row_bytes);
#pragma unroll
          for (int k = 0; k < BLOCKS; ++k) {
            u32x4 b[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
              const int jj = k * S::KB + q * V + j;
              b[j] = load_rows(rows, jj < a.r ? b_off + (uint32_t)jj * row_bytes : kOutside, 0);
            }
            across<DT, V>(b, bank[k]);
          }
        }
        f32x4 acc[V];
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < BLOCKS; ++k) mma_across<DT, V>(bank[k], Factor<DT>(f[k]), acc);
        // row `col`, chunks 4q .. 4q+3
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int i = 0; i < V; i += 4)
            *reinterpret_cast<f32x4*>(prod + col * kStride + (q * 4 + s) * V + i) =
                f32x4{acc[i][s], acc[i + 1][s], acc[i + 2][s], acc[i + 3][s]};
      }
      // the rows of other adapters are dropped
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int row = s * 4 + q, t = __shfl(now.t, row, kWave);
        float o[V];
        if (a.base) unpack<DT>(now.base[s], o);
        if (e < a.A) {
#pragma unroll
          for (int i = 0; i < V; i += 4) {
            const f32x4 v = *reinterpret_cast<const f32x4*>(prod + row * kStride + col * V + i);
#pragma unroll
            for (int k = 0; k < 4; ++k) o[i + k] = a.base ? o[i + k] + v[k] : v[k];
          }
        } else if (!a.base) {
#pragma unroll
          for (int i = 0; i < V; ++i) o[i] = 0.f;
        }
        if (t >= 0 && r0 + row >= lo && r0 + row < hi && in)
          static_cast<u32x4*>(a.out)[(size_t)t * nch + my_c] = pack_rows<DT>(o);
      }
    });
  }
}

// ---- gradients of the adapters ---------------------------------------------------
//
// grad[e][j][c] = sum over the adapter's rows p of coef[p][j] rows[t_p][c],
// coef = u (times w for grad_B).  One workgroup per (COLS columns, adapter, 16
// JT of the rank): its waves take the adapter's rows in turn, each a block of
// KB rows at a time with the next block's on its way, and meet in LDS.  A
// block's rows of u pass through the wave's own piece of LDS, loaded 16 bytes a
// lane: four bytes a lane, as the operand takes them, cost the address unit
// twice what the wide rows do.  An adapter without rows gets zeros.
constexpr int kWgradWaves = 8;

template <int DT, int JT>
__global__ __launch_bounds__(kWgradWaves* kWave) void wgrad_kernel(LowrankArgs a) {
  using S = Shape<DT>;
  constexpr int V = S::V;
  constexpr int kStride = JT * 16 + 4;                  // floats of a row of u in LDS
  constexpr int kLoads = S::KB * JT * 4 / kWave;        // a block's u, 16 bytes a lane
  __shared__ __align__(16) union {
    float u[kWgradWaves][S::KB * kStride];
    f32x4 part[kWgradWaves][V][kWave];
  } sh;
  auto& part = sh.part;
  const int lane = lane_id(), wave = (int)(threadIdx.x / kWave);
  const int col = lane & 15, q = lane >> 4;
  const int e = blockIdx.y;
  const int nch = a.wch;
  const int parts = (a.r + 16 * JT - 1) / (16 * JT);
  const int c0 = blockIdx.x / parts * 16;
  const int j0 = blockIdx.x % parts * JT * 16;
  const int c = min(c0 + col, nch - 1);  // chunks past the end repeat the last and are not stored
  const int lo = a.expert_offset[e], hi = min(a.expert_offset[e + 1], a.R);
  f32x4 acc[JT][V];
#pragma unroll
  for (int jt = 0; jt < JT; ++jt)
#pragma unroll
    for (int i = 0; i < V; ++i) acc[jt][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  // lane l < KB knows the block's row l: its token, -1 without one
  auto tokens = [&](int p0) {
    const int p = p0 + lane;
    const int v = a.recv_token[min(p, a.R - 1)];
    return lane < S::KB && p < hi && (unsigned)v < (unsigned)a.T ? v : -1;
  };
  u32x4 x[V];
  f32x4 u[kLoads];
  float w = 1.f;
  int t = -1, next_t = -1;
  auto fetch = [&](int p0) {  // the rows whose tokens are in t
#pragma unroll
    for (int k = 0; k < V; ++k)
      x[k] = static_cast<const u32x4*>(a.rows)[(size_t)max(__shfl(t, q * V + k, kWave), 0) * nch + c];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int at = i * kWave + lane, row = at / (JT * 4), j = j0 + at % (JT * 4) * 4;
      u[i] = *reinterpret_cast<const f32x4*>(a.u + (size_t)min(p0 + row, hi - 1) * a.r + min(j, a.r - 4));
    }
    if (a.w) w = a.w[max(t, 0)];
  };
  constexpr int kStep = kWgradWaves * S::KB;
  int p0 = lo + wave * S::KB;
  if (p0 < hi) {
    t = tokens(p0);
    fetch(p0);
    next_t = tokens(p0 + kStep);
  }
  for (; p0 < hi; p0 += kStep) {
    // this block's operands leave their registers, then the next block's rows
    // are asked for
    float* us = sh.u[wave];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int at = i * kWave + lane;
      *reinterpret_cast<f32x4*>(us + at / (JT * 4) * kStride + at % (JT * 4) * 4) = u[i];
    }
    bool there[V];
    float wk[V];
    u32x4 o[V];
    {
      u32x4 z[V];
#pragma unroll
      for (int k = 0; k < V; ++k) {
        there[k] = __shfl(t, q * V + k, kWave) >= 0;
        wk[k] = a.w ? __shfl(w, q * V + k, kWave) : 1.f;
        z[k] = there[k] ? x[k] : u32x4{0u, 0u, 0u, 0u};  // rows without a token
      }
      across<DT, V>(z, o);
    }
    t = next_t;
    fetch(p0 + kStep);
    next_t = tokens(p0 + 2 * kStep);
#pragma unroll
    for (int jt = 0; jt < JT; ++jt) {
      float f[V];
#pragma unroll
      for (int k = 0; k < V; ++k) f[k] = there[k] ? us[(q * V + k) * kStride + jt * 16 + col] * wk[k] : 0.f;
      mma_across<DT, V>(o, Factor<DT>(f), acc[jt]);
    }
  }
#pragma unroll
  for (int jt = 0; jt < JT; ++jt) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < V; ++i) part[wave][i][lane] = acc[jt][i];
    __syncthreads();
    const int j = j0 + jt * 16 + col;
    if (wave < 4) {  // wave s stores the s-th of every lane's four chunks
      float o[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float* f = reinterpret_cast<const float*>(&part[0][i][lane]) + wave;
        o[i] = f[0];
#pragma unroll
        for (int k = 1; k < kWgradWaves; ++k) o[i] += f[(size_t)k * V * kWave * 4];
      }
      const int cc = c0 + q * 4 + wave;
      if (j < a.r && cc < nch) static_cast<u32x4*>(a.out)[((size_t)e * a.r + j) * nch + cc] = pack_rows<DT>(o);
    }
  }
}

template <typename F>
hipError_t launched(F f) {
  f();
  return hipGetLastError();
}

int slots_for(int64_t workgroups, int E) {  // adapters of a tile side by side while workgroups are few
  int s = 1;
  while (s < kTile && s < E && workgroups * s < 512) s *= 2;
  return s;
}

}  // namespace

hipError_t launch_lowrank_shrink(const LowrankArgs& a, hipStream_t s) {
  // two tiles a workgroup, which halves what is read of the banks, when that
  // still leaves a workgroup for every CU
  const bool far = (int64_t)a.T * a.wch * 16 >= (int64_t(1) << 31);
  const int rt = !far && a.r <= 64 && a.R >= 2 * kTile * 256 ? 2 : 1;
  const int tiles = (a.R + kTile * rt - 1) / (kTile * rt);
  const dim3 grid(tiles, slots_for(tiles, a.E));
#define MOE_SHRINK(J, T, F)                                                                             \
  return launched([&] {                                                                                 \
    const dim3 block((Shrink<J, T>::kWaves * kWave));                                                   \
    const size_t lds = (Shrink<J, T>::kLds);                                                            \
    if (a.dtype == MOE_F32) hipLaunchKernelGGL((shrink_kernel<kF32, J, T, F>), grid, block, lds, s, a); \
    else hipLaunchKernelGGL((shrink_kernel<kBF16, J, T, F>), grid, block, lds, s, a);                   \
  })
  if (far) {
    if (a.r <= 32) MOE_SHRINK(2, 1, true);
    MOE_SHRINK(8, 1, true);
  }
  if (rt == 2) {
    if (a.r <= 16) MOE_SHRINK(1, 2, false);
    if (a.r <= 32) MOE_SHRINK(2, 2, false);
    MOE_SHRINK(4, 2, false);
  }
  if (a.r <= 16) MOE_SHRINK(1, 1, false);
  if (a.r <= 32) MOE_SHRINK(2, 1, false);
  if (a.r <= 64) MOE_SHRINK(4, 1, false);
  MOE_SHRINK(8, 1, false);
#undef MOE_SHRINK
}

hipError_t launch_lowrank_expand(const LowrankArgs& args, hipStream_t s) {
  LowrankArgs a = args;
  const int tiles = (a.R + kTile - 1) / kTile;
  const int cols = (a.wch + 16 * kExpandWaves - 1) / (16 * kExpandWaves);
  // as many tiles a wave as leave one generation of workgroups, two a CU (8192
  // rows of 4096 columns in bfloat16, rank 32: 46 us with one tile, 38 with
  // four, 34 with eight)
  a.tiles = 1;
  while (a.tiles < 16 && (int64_t)tiles * cols >= 2 * a.tiles * 512) a.tiles *= 2;
  const int blocks = (tiles + a.tiles - 1) / a.tiles;
  const dim3 grid(blocks, cols, a.tiles > 1 ? 1 : slots_for((int64_t)tiles * cols, a.E)), block(kExpandWaves * kWave);
#define MOE_EXPAND(D, B) \
  return launched([&] { hipLaunchKernelGGL((expand_lowrank_kernel<D, B>), grid, block, 0, s, a); })
  if (a.dtype == MOE_F32) {
    if (a.r <= 16) MOE_EXPAND(kF32, 1);
    if (a.r <= 32) MOE_EXPAND(kF32, 2);
    if (a.r <= 64) MOE_EXPAND(kF32, 4);
    MOE_EXPAND(kF32, 8);
  }
  if (a.r <= 32) MOE_EXPAND(kBF16, 1);
  if (a.r <= 64) MOE_EXPAND(kBF16, 2);
  MOE_EXPAND(kBF16, 4);
#undef MOE_EXPAND
}

hipError_t launch_lowrank_wgrad(const LowrankArgs& a, hipStream_t s) {
  const dim3 block(kWgradWaves * kWave);
  const int cols = (a.wch + 15) / 16;
#define MOE_WGRAD(J)                                                                                   \
  return launched([&] {                                                                                \
    const dim3 grid(cols * ((a.r + 16 * J - 1) / (16 * J)), a.A);                                      \
    if (a.dtype == MOE_F32) hipLaunchKernelGGL((wgrad_kernel<kF32, J>), grid, block, 0, s, a);         \
    else hipLaunchKernelGGL((wgrad_kernel<kBF16, J>), grid, block, 0, s, a);                           \
  })
  if (a.r <= 16) MOE_WGRAD(1);
  MOE_WGRAD(2);
#undef MOE_WGRAD
}

}  // namespace moe
