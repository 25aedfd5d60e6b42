// Low-rank adapters of many requests beside a shared projection, and their
// gradients, on the rows of a layout with one expert (adapter) per token:
//
//   u[p]    = A_e x_t                      row p of adapter e holds token t
//   out[t]  = base[t] + w_t (u[p] B_e)     A_e [r, H], B_e [r, N]
//   raw[p]  = B_e g_t,  gu[p] = w_t raw[p],  grad_w[t] = <raw[p], u[p]>
//   grad_x[t] = grad_base[t] + gu[p] A_e
//   grad_A_e  = sum_p gu[p]^T x_t,   grad_B_e = sum_p w_t u[p]^T g_t
//
// Three steps do all of it, because A and B are both held with the rank as
// the row index: `shrink` (to the rank: u, gu), `expand` (back to full width:
// out, grad_x; small calls take both in one launch) and `wgrad` (an adapter's
// sum over its rows).  All are bound by the wide rows they read and write; the
// products are thin (r <= 128).
//
// Rows of an adapter stand together in the layout, so a tile of 16 receive
// rows usually belongs to one adapter and its product is a matrix product.  A
// tile that several adapters share is walked adapter by adapter, the rows of
// the others masked; with few tokens the adapters of a tile go to different
// workgroups (slots).
//
// u and gu stay float32.  As operands of a bfloat16 matrix instruction they are
// cut into three bfloat16 parts (Parts in mfma.h), which lose nothing: nothing but
// the result is rounded.  (Two rounded parts, 16 bits, save little: a pass of 8192
// rows, rank 32, 4096 columns 66.1 and 66.5 us, forward and backward of 4096 rows,
// rank 64 97 and 101.)
#include <type_traits>

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

// The adapters of rows [r0, r1) (at most 64): f(e, lo, hi) for each adapter e
// (or A <= e < E: rows without one) with rows [lo, hi) of them, of those that fall
// to `slot`.  Rows after the last segment belong to nobody, and what the layout
// holds for them is not defined: they are left out.  off: the layout's expert
// offsets in LDS, E + 1 of them.  Each lane finds its row's adapter by bisection,
// all at once: walking the adapters of a tile one after another cost 0.3 us each.
template <typename F>
__device__ __forceinline__ void each_adapter(const int* off, int E, int r0, int r1, int slot, int slots, F f) {
  const int lane = lane_id(), p = min(r0 + lane, r1 - 1);
  int e = 0;  // the last segment that begins at or before row p: not an empty one
  for (int s = 1 << (31 - __builtin_clz(E)); s > 0; s >>= 1)
    if (e + s <= E && off[e + s] <= p) e += s;
  const int before = __shfl_up(e, 1, kWave);
  uint64_t first = __ballot(r0 + lane < r1 && (lane == 0 || e != before));
  for (int n = 0; first; ++n) {  // wave-uniform
    const int i = __builtin_ctzll(first);
    first &= first - 1;
    if (read_lane_i(e, i) == E) return;
    if (n % slots == slot) f(read_lane_i(e, i), r0 + i, first ? r0 + (int)__builtin_ctzll(first) : r1);
  }
}

__device__ __forceinline__ void load_offsets(int* off, const LowrankArgs& a) {
  for (int i = threadIdx.x; i <= a.E; i += blockDim.x) off[i] = a.expert_offset[i];
  __syncthreads();
}

// Workgroups go to the 8 XCDs in turn.  Of n tiles every XCD takes a run, so that
// its L2 holds the banks of few adapters (4096 rows of 4096 bfloat16, 16 adapters
// of rank 64, to 256 columns: 38 us a pass with tiles in turn, 23 with runs).
__device__ __forceinline__ int xcd_run(int b, int n) {
  const int xcd = b & 7, more = n & 7;
  return xcd * (n >> 3) + min(xcd, more) + (b >> 3);
}

// The token of receive row p, -1 for a row without one (padding).
__device__ __forceinline__ int row_token(const LowrankArgs& a, int p) {
  const int t = p < a.R ? a.recv_token[p] : -1;
  return (unsigned)t < (unsigned)a.T ? t : -1;
}

// ---- shrink ---------------------------------------------------------------------
//
// One workgroup per (RT tiles of 16 rows, slot, 16 JT of the rank).  Its waves split the sum over
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
// GiB).  (8192 rows of 4096 bfloat16, 16 adapters of rank 32: 21 us, 67 MB of rows
// at 3.2 TB/s and as much again of the banks from L2; what is left of the bound is
// the wait for the first lines and for the adapters of a tile.)
template <int JT, int RT>
struct Shrink {
  static constexpr int kMeet = JT * RT <= 4 ? JT : 4 / RT;     // tiles of the rank that meet in LDS together
  static constexpr int kStaged = JT < 4 ? JT : 4;              // tiles of the rank in LDS at a time
  static constexpr int kRows = 16 * (RT + kStaged);            // rows of a stage: the tokens', then the bank's
  static constexpr int kWaves = JT + RT <= 3 ? 8 : 4;
  static constexpr size_t kLds = (size_t)kWaves * kRows * 128;  // at most 48 KiB
  static constexpr int kKeep = JT * 16 + 4;                     // floats of a row of u kept in LDS
};

// Rows [lo, hi) of adapter e, of the RT tiles from r0 on, ranks [j0, j0 + 16 JT);
// the whole workgroup.  keep: where the rows' u go as well, [16][kKeep], or null.  t, load_t: the tokens of this lane's rows as an operand and in a load.
template <int DT, int JT, int RT, bool FAR>
__device__ __forceinline__ void shrink_rows(const LowrankArgs& a, u32x4* lds, int r0, int j0, int e, int lo,
                                            int hi, const int (&t)[RT], const int (&load_t)[2 * RT], float* keep) {
  constexpr int kShrinkWaves = Shrink<JT, RT>::kWaves, kMeet = Shrink<JT, RT>::kMeet;
  constexpr int kStaged = Shrink<JT, RT>::kStaged, kRows = Shrink<JT, RT>::kRows;
  constexpr int kDepth = JT + RT <= 2 ? 3 : JT + RT <= 4 ? 2 : 1;
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave));
  const int col = lane & 15, q = lane >> 4;  // of an operand
  const int row8 = lane >> 3, chunk = lane & 7;  // of a load: 8 rows by one line
  u32x4* stage = lds + (size_t)wave * kRows * 8;      // [kRows][8 chunks], one for each wave
  f32x4* part = reinterpret_cast<f32x4*>(lds);        // then [waves][RT][kMeet][64] to meet in
  const int nch = a.wch, lines = (nch + 7) / 8;
  const int start = (blockIdx.x + blockIdx.y) * 5 % lines;
  const uint32_t row_bytes = (uint32_t)nch * 16;
  bool mine[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int p = r0 + rt * kTile + col;
    mine[rt] = p >= lo && p < hi;
  }
  if (e >= a.A) {  // no adapter: u = 0, and no gradient
    if (j0 > 0) return;
    for (int i = threadIdx.x; i < (hi - lo) * a.r; i += kShrinkWaves * kWave) a.u[(size_t)lo * a.r + i] = 0.f;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
      if (a.dot && wave == rt && q == 0 && mine[rt] && t[rt] >= 0) a.dot[t[rt]] = 0.f;
    return;
  }
  // the columns of other adapters (and padding) are zeros, or with FAR their own
  // rows (padding the first one); the results are dropped either way
  uint32_t x_off[2 * RT];
#pragma unroll
  for (int k = 0; k < 2 * RT; ++k) {
    const int p = r0 + k * 8 + row8;
    x_off[k] = p >= lo && p < hi ? (uint32_t)load_t[k] * row_bytes + chunk * 16 : kOutside;
  }
  const auto wide = make_rows(a.rows, FAR ? 0 : (size_t)a.T * row_bytes);
  const auto bank = make_rows(static_cast<const u32x4*>(a.bank) + ((size_t)e * a.r + j0) * nch, (size_t)(a.r - j0) * row_bytes);
  const uint32_t b_off = (uint32_t)row8 * row_bytes + chunk * 16;
  u32x4 in[kDepth][2 * (RT + JT)];
  auto fetch = [&](int d, int i) {  // the i-th line after `start`; past the last: zeros
    const int line = i >= lines ? 0 : i + start < lines ? i + start : i + start - lines;
    const int c = line * 8 + chunk;
    const bool ok = i < lines && c < nch;
#pragma unroll
    for (int k = 0; k < 2 * RT; ++k) {
      if constexpr (FAR) {
        in[d][k] = static_cast<const u32x4*>(a.rows)[(size_t)load_t[k] * nch + (ok ? c : 0)];
        // the bank's zeros alone would leave NaN where a row holds one
        if (!ok) in[d][k] = u32x4{0u, 0u, 0u, 0u};
      } else {
        in[d][k] = load_rows(wide, ok ? x_off[k] : kOutside, (uint32_t)line * 128);
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
        const int j = j0 + (first + m) * 16 + q * 4;
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
          if (keep) *reinterpret_cast<f32x4*>(keep + col * Shrink<JT, RT>::kKeep + j) = v;
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
}

template <int DT, int JT, int RT, bool FAR>
__global__ __launch_bounds__((Shrink<JT, RT>::kWaves * kWave)) void shrink_kernel(LowrankArgs a) {
  __shared__ int off[kMaxOff];
  extern __shared__ u32x4 lds[];
  const int lane = lane_id();
  const int r0 = xcd_run(blockIdx.x, gridDim.x) * kTile * RT, r1 = min(r0 + kTile * RT, a.R);
  int t[RT], load_t[2 * RT];
#pragma unroll
  for (int i = 0; i < 2 * RT; ++i) load_t[i] = max(row_token(a, r0 + i * 8 + (lane >> 3)), 0);
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) t[rt] = row_token(a, r0 + rt * kTile + (lane & 15));
  load_offsets(off, a);
  each_adapter(off, a.E, r0, r1, blockIdx.y, gridDim.y, [&](int e, int lo, int hi) {
    shrink_rows<DT, JT, RT, FAR>(a, lds, r0, blockIdx.z * JT * 16, e, lo, hi, t, load_t, nullptr);
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

// acc[i] += operand i . the other operand, V floats along a block of the summed
// index.  FINITE: see Parts in mfma.h.
template <int DT, bool FINITE, int V>
__device__ __forceinline__ void mma_across(const u32x4 (&o)[V], const float (&f)[V], f32x4 (&acc)[V]) {
  if constexpr (DT == kBF16) {
    const Parts<FINITE> p(f);
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = mma_parts(o[i], p, acc[i]);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i)
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(o[j][i]), f[j], acc[i], 0, 0, 0);
  }
}

// ---- expand ---------------------------------------------------------------------
//
// The columns of a wave: 16 chunks from c0 on.  A lane reads base and writes
// out at chunk c0 + lane % 16 of rows lane / 16, + 4, + 8, + 12, the products pass
// through LDS, so that 16 lanes share a row's 256 bytes.
template <int DT, int BLOCKS>
struct Expand {
  using S = Shape<DT>;
  static constexpr int V = S::V;
  static constexpr int kStride = 16 * V + 4;          // floats of a row in LDS: rows shifted by four banks
  static constexpr int kProducts = kTile * kStride;   // floats of a wave
  u32x4 bank[BLOCKS][V];                              // its columns of an adapter's bank, as operands

  __device__ __forceinline__ void load_bank(const LowrankArgs& a, int e, int c0) {
    const int col = lane_id() & 15, q = lane_id() >> 4;
    const uint32_t row_bytes = (uint32_t)a.wch * 16;
    const auto rows = make_rows(static_cast<const u32x4*>(a.bank) + (size_t)e * a.r * a.wch, (size_t)a.r * row_bytes);
    // ranks and columns past the end are outside the bank and read as zeros
    const uint32_t off = c0 + col < a.wch ? (uint32_t)(c0 + col) * 16 : kOutside;
#pragma unroll
    for (int k = 0; k < BLOCKS; ++k) {
      u32x4 b[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int jj = k * S::KB + q * V + j;
        b[j] = load_rows(rows, jj < a.r ? off + (uint32_t)jj * row_bytes : kOutside, 0);
      }
      across<DT, V>(b, bank[k]);
    }
  }

  // a row of u, this lane's part of every block (ranks past the last: other ranks')
  static __device__ __forceinline__ void load_u(const LowrankArgs& a, const float* u, f32x4 (&u4)[BLOCKS][V / 4]) {
    const int q = lane_id() >> 4;
#pragma unroll
    for (int k = 0; k < BLOCKS; ++k)
#pragma unroll
      for (int j = 0; j < V; j += 4) {
        const int jj = k * S::KB + q * V + j;
        u4[k][j / 4] = *reinterpret_cast<const f32x4*>(u + (jj < a.r ? jj : 0));
      }
  }

  // w times it; zeros past the last rank, and in a row that is not there
  static __device__ __forceinline__ void weigh(const LowrankArgs& a, const f32x4 (&u4)[BLOCKS][V / 4], float w,
                                               float (&f)[BLOCKS][V], bool there = true) {
    const int q = lane_id() >> 4;
#pragma unroll
    for (int k = 0; k < BLOCKS; ++k)
#pragma unroll
      for (int j = 0; j < V; ++j) f[k][j] = there && k * S::KB + q * V + j < a.r ? u4[k][j / 4][j % 4] * w : 0.f;
  }

  static __device__ __forceinline__ void load_base(const LowrankArgs& a, int t, int c0, u32x4 (&base)[4]) {
    const int col = lane_id() & 15, q = lane_id() >> 4;
    if (!a.base) return;
#pragma unroll
    for (int s = 0; s < 4; ++s)
      base[s] = static_cast<const u32x4*>(a.base)[(size_t)max(__shfl(t, s * 4 + q, kWave), 0) * a.wch + min(c0 + col, a.wch - 1)];
  }

  template <bool FINITE>
  __device__ __forceinline__ void products(const float (&f)[BLOCKS][V], f32x4 (&acc)[V]) const {
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < BLOCKS; ++k) mma_across<DT, FINITE, V>(bank[k], f[k], acc);
  }

  // Rows [lo, hi) of adapter e (e >= A: none) of the tile at r0; t: the token of
  // row lane % 16.  The rows of other adapters are dropped.
  __device__ __forceinline__ void rows(const LowrankArgs& a, float* prod, int r0, int e, int lo, int hi, int t, int c0,
                                       const float (&f)[BLOCKS][V], const u32x4 (&base)[4]) const {
    const int col = lane_id() & 15, q = lane_id() >> 4;
    if (e < a.A) {
      f32x4 acc[V];
      products<true>(f, acc);
      if (DT == kBF16 && any_nan(acc)) products<false>(f, acc);
      // row `col`, chunks 4q .. 4q+3
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int i = 0; i < V; i += 4)
          *reinterpret_cast<f32x4*>(prod + col * kStride + (q * 4 + s) * V + i) =
              f32x4{acc[i][s], acc[i + 1][s], acc[i + 2][s], acc[i + 3][s]};
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int row = s * 4 + q, tt = __shfl(t, row, kWave);
      float o[V];
      if (a.base) unpack<DT>(base[s], o);
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
      if (tt >= 0 && r0 + row >= lo && r0 + row < hi && c0 + col < a.wch)
        static_cast<u32x4*>(a.out)[(size_t)tt * a.wch + c0 + col] = pack_rows<DT>(o);
    }
  }
};

// One wave per (a.tiles tiles of 16 receive rows, 16 chunks of columns, slot);
// it keeps its columns of an adapter's bank in registers from tile to tile, and
// has the next tile's rows of base and u on their way.  BLOCKS blocks of KB ranks.
// (8192 rows of 4096 bfloat16, rank 32: 34 us, 134 MB read and written at 4.0 TB/s;
// 1 us more when u is asked for as it is needed.  What is left is the first tile's
// wait, for tokens, base, offsets and bank one after another, and a mixture of
// reads and writes in pieces of 256 bytes.)
constexpr int kExpandWaves = 4;

template <int DT, int BLOCKS>
__global__ __launch_bounds__(kExpandWaves* kWave, BLOCKS <= 2 ? 2 : 1) void expand_lowrank_kernel(LowrankArgs a) {
  using X = Expand<DT, BLOCKS>;
  __shared__ int off[kMaxOff];
  __shared__ __align__(16) float products[kExpandWaves][X::kProducts];
  const int col = lane_id() & 15, wave = (int)(threadIdx.x / kWave);
  const int c0 = (blockIdx.y * kExpandWaves + wave) * 16;  // first chunk of this wave's columns
  int tile = xcd_run(blockIdx.x, gridDim.x) * a.tiles;
  const int tile_end = min(tile + a.tiles, (a.R + kTile - 1) / kTile);
  int next_t = row_token(a, tile * kTile + col), t = next_t;
  load_offsets(off, a);
  if (c0 >= a.wch) return;
  X x;
  u32x4 base[4], next_base[4];
  f32x4 next_u[BLOCKS][X::V / 4];
  float next_w = 1.f;
  X::load_base(a, next_t, c0, next_base);
  X::load_u(a, a.u + (size_t)min(tile * kTile + col, a.R - 1) * a.r, next_u);
  if (a.w) next_w = a.w[max(next_t, 0)];
  int after_t = row_token(a, (tile + 1) * kTile + col);
  int held = -1;  // the adapter whose bank is held
  for (; tile < tile_end; ++tile) {
    t = next_t;
#pragma unroll
    for (int s = 0; s < 4; ++s) base[s] = next_base[s];
    const int r0 = tile * kTile, r1 = min(r0 + kTile, a.R);
    float f[BLOCKS][X::V];
    X::weigh(a, next_u, next_w, f);
    next_t = after_t;
    if (tile + 1 < tile_end) {
      X::load_base(a, next_t, c0, next_base);
      X::load_u(a, a.u + (size_t)min(r0 + kTile + col, a.R - 1) * a.r, next_u);
      if (a.w) next_w = a.w[max(next_t, 0)];
    }
    after_t = row_token(a, (tile + 2) * kTile + col);
    each_adapter(off, a.E, r0, r1, blockIdx.z, gridDim.z, [&](int e, int lo, int hi) {
      if (e < a.A && e != held) {
        held = e;
        x.load_bank(a, e, c0);
      }
      x.rows(a, products[wave], r0, e, lo, hi, t, c0, f, base);
    });
  }
}

// ---- shrink and expand in one -----------------------------------------------------
//
// For few tokens with small banks: one workgroup per (tile, slot) does both for
// the adapter's rows, where two launches would each pay for starting, reading
// the offsets and the tokens.  It walks the wide columns with its own waves, so
// it is for banks that one CU reads in the time of a launch.  (48 tokens of 2048
// bfloat16, 32 adapters of rank 16: 11.7 us, 0.5 more with u read back from memory; a
// wave issues 1050 instructions in 3 us and waits for loads half of the time.)
template <int DT, int JT>
struct Both {
  static constexpr int kBlocks = DT == kBF16 ? (JT + 1) / 2 : JT;
  using X = Expand<DT, kBlocks>;
  static constexpr int kWaves = Shrink<JT, 1>::kWaves;
  static constexpr size_t kProducts = (size_t)kWaves * X::kProducts * 4;
  static constexpr size_t kStage = Shrink<JT, 1>::kLds > kProducts ? Shrink<JT, 1>::kLds : kProducts;
  static constexpr size_t kLds = kStage + (size_t)kTile * Shrink<JT, 1>::kKeep * 4;
};

template <int DT, int JT>
__global__ __launch_bounds__((Both<DT, JT>::kWaves * kWave)) void lowrank_both_kernel(LowrankArgs s, LowrankArgs a) {
  using X = typename Both<DT, JT>::X;
  constexpr int kWaves = Both<DT, JT>::kWaves;
  __shared__ int off[kMaxOff];
  extern __shared__ u32x4 lds[];
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave));
  const int r0 = blockIdx.x * kTile, r1 = min(r0 + kTile, a.R);
  int t[1], load_t[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) load_t[i] = max(row_token(a, r0 + i * 8 + (lane >> 3)), 0);
  t[0] = row_token(a, r0 + (lane & 15));
  load_offsets(off, a);
  float* prod = reinterpret_cast<float*>(lds) + (size_t)wave * X::kProducts;
  float* keep = reinterpret_cast<float*>(lds) + Both<DT, JT>::kStage / 4;  // u, from one step to the other
  each_adapter(off, a.E, r0, r1, blockIdx.y, gridDim.y, [&](int e, int lo, int hi) {
    // the first columns' bank and base, which do not wait for u, are asked for ahead
    X x;
    u32x4 base[4];
    int c0 = wave * 16;
    if (c0 < a.wch) {
      if (e < a.A) x.load_bank(a, e, c0);
      X::load_base(a, t[0], c0, base);
    }
    shrink_rows<DT, JT, 1, false>(s, lds, r0, 0, e, lo, hi, t, load_t, keep);
    float f[Both<DT, JT>::kBlocks][X::V];
    f32x4 u4[Both<DT, JT>::kBlocks][X::V / 4];
    X::load_u(a, keep + (lane & 15) * Shrink<JT, 1>::kKeep, u4);
    const int p = r0 + (lane & 15);  // only this adapter's rows have been kept
    X::weigh(a, u4, a.w ? a.w[max(t[0], 0)] : 1.f, f, p >= lo && p < hi);
    while (c0 < a.wch) {
      x.rows(a, prod, r0, e, lo, hi, t[0], c0, f, base);
      c0 += kWaves * 16;
      if (c0 < a.wch) {
        if (e < a.A) x.load_bank(a, e, c0);
        X::load_base(a, t[0], c0, base);
      }
    }
    __syncthreads();  // the next adapter's stages take the products' place
  });
}

// ---- gradients of the adapters ---------------------------------------------------
//
// grad[e][j][c] = sum over the adapter's rows p of coef[p][j] rows[t_p][c],
// coef = u (times w for grad_B).  One workgroup per (COLS columns, adapter, 16
// JT of the rank): its waves take the adapter's rows in turn, each a block of
// KB rows at a time with the next block's on its way, and meet in LDS.  A
// block's rows of u pass through the wave's own piece of LDS, loaded 16 bytes a
// lane: four bytes a lane, as the operand takes them, cost the address unit
// twice what the wide rows do.  An adapter without rows gets zeros.  (Both sides
// of 4096 rows of 2048 and 4096 bfloat16, 4 adapters of rank 64: 25 us; every 32
// ranks read the rows again, 100 MB at 4 TB/s.)
//
// With few adapters the rows of one are split over gridDim.z workgroups, whose
// sums wgrad_sum_kernel adds in their order.

// What the gradients of a and of b, in one launch, do not share.
struct WgradSide {
  const void* rows;
  const float* w;
  const float* u;
  void* out;
  int wch;
  float* parts;  // [gridDim.z][A, r, W] with split rows
};

template <int DT, int JT, int W>
__global__ __launch_bounds__((W * kWave)) void wgrad_kernel(LowrankArgs a, WgradSide one, WgradSide two,
                                                                  int one_blocks) {
  using S = Shape<DT>;
  constexpr int V = S::V;
  constexpr int kStride = JT * 16 + 4;                  // floats of a row of u in LDS
  constexpr int kLoads = S::KB * JT * 4 / kWave;        // a block's u, 16 bytes a lane
  __shared__ __align__(16) union {
    float u[W][S::KB * kStride];
    f32x4 part[W][V][kWave];
  } sh;
  auto& part = sh.part;
  const int lane = lane_id(), wave = (int)(threadIdx.x / kWave);
  const int col = lane & 15, q = lane >> 4;
  const int e = blockIdx.y;
  const bool second = (int)blockIdx.x >= one_blocks;
  const int block = second ? blockIdx.x - one_blocks : blockIdx.x;
  const u32x4* rows = static_cast<const u32x4*>(second ? two.rows : one.rows);
  const float* weights = second ? two.w : one.w;
  const float* u_rows = second ? two.u : one.u;
  u32x4* out = static_cast<u32x4*>(second ? two.out : one.out);
  float* parts_out = second ? two.parts : one.parts;
  const int nch = second ? two.wch : one.wch;
  const int parts = (a.r + 16 * JT - 1) / (16 * JT);
  // the parts of the rank that read the same columns 8 workgroups apart: one XCD
  const int whole = (nch + 15) / 16 / 8 * 8 * parts, in = block % (8 * parts);
  const int c0 = (block < whole ? block / (8 * parts) * 8 + in % 8 : block / parts) * 16;
  const int j0 = (block < whole ? in / 8 : block % parts) * JT * 16;
  const int c = min(c0 + col, nch - 1);  // chunks past the end repeat the last and are not stored
  int lo = a.expert_offset[e], hi = min(a.expert_offset[e + 1], a.R);
  const int splits = gridDim.z;
  if (splits > 1) {
    const int share = ((hi - lo + splits - 1) / splits + S::KB - 1) / S::KB * S::KB;
    lo += blockIdx.z * share;
    hi = min(hi, lo + share);
  }
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
      x[k] = rows[(size_t)max(__shfl(t, q * V + k, kWave), 0) * nch + c];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int at = i * kWave + lane, row = at / (JT * 4), j = j0 + at % (JT * 4) * 4;
      u[i] = *reinterpret_cast<const f32x4*>(u_rows + (size_t)min(p0 + row, hi - 1) * a.r + min(j, a.r - 4));
    }
    if (weights) w = weights[max(t, 0)];
  };
  constexpr int kStep = W * S::KB;
  f32x4 acc[JT][V];
  // over this wave's rows; the second time, which is rare, nothing is asked for
  // ahead (the finite parts take the registers)
  auto sums = [&](auto pass) {
    constexpr bool kFinite = decltype(pass)::value;
#pragma unroll
    for (int jt = 0; jt < JT; ++jt)
#pragma unroll
      for (int i = 0; i < V; ++i) acc[jt][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    int p0 = lo + wave * S::KB;
    if (kFinite && p0 < hi) {
      t = tokens(p0);
      fetch(p0);
      next_t = tokens(p0 + kStep);
    }
    for (; p0 < hi; p0 += kStep) {
      if (!kFinite) {
        t = tokens(p0);
        fetch(p0);
      }
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
          wk[k] = weights ? __shfl(w, q * V + k, kWave) : 1.f;
          z[k] = there[k] ? x[k] : u32x4{0u, 0u, 0u, 0u};  // rows without a token
        }
        across<DT, V>(z, o);
      }
      if (kFinite) {
        t = next_t;
        fetch(p0 + kStep);
        next_t = tokens(p0 + 2 * kStep);
      }
#pragma unroll
      for (int jt = 0; jt < JT; ++jt) {
        float f[V];
#pragma unroll
        for (int k = 0; k < V; ++k) f[k] = there[k] ? us[(q * V + k) * kStride + jt * 16 + col] * wk[k] : 0.f;
        mma_across<DT, kFinite, V>(o, f, acc[jt]);
      }
    }
  };
  sums(std::true_type{});
  if constexpr (DT == kBF16) {
    bool nan = false;
#pragma unroll
    for (int jt = 0; jt < JT; ++jt) nan |= any_nan(acc[jt]);
    if (nan) sums(std::false_type{});
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
        for (int k = 1; k < W; ++k) o[i] += f[(size_t)k * V * kWave * 4];
      }
      const int cc = c0 + q * 4 + wave;
      if (j < a.r && cc < nch) {
        const size_t to = ((size_t)e * a.r + j) * nch + cc;
        if (splits == 1) {
          out[to] = pack_rows<DT>(o);
        } else {
          f32x4* f = reinterpret_cast<f32x4*>(parts_out) + ((size_t)blockIdx.z * a.A * a.r * nch + to) * (V / 4);
#pragma unroll
          for (int i = 0; i < V / 4; ++i) f[i] = f32x4{o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]};
        }
      }
    }
  }
}

// The parts' sums, a chunk a thread; first: chunks of the first side.
template <int DT>
__global__ __launch_bounds__(256) void wgrad_sum_kernel(WgradSide one, WgradSide two, int first, int chunks, int splits) {
  constexpr int V = Shape<DT>::V;
  int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= chunks) return;
  const bool second = c >= first;
  const size_t n = second ? chunks - first : first;
  c -= second ? first : 0;
  const f32x4* f = reinterpret_cast<const f32x4*>(second ? two.parts : one.parts) + (size_t)c * (V / 4);
  float o[V];
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    f32x4 v = f[i];
    for (int s = 1; s < splits; ++s) v += f[s * n * (V / 4) + i];
#pragma unroll
    for (int k = 0; k < 4; ++k) o[4 * i + k] = v[k];
  }
  static_cast<u32x4*>(second ? two.out : one.out)[c] = pack_rows<DT>(o);
}

template <typename F>
hipError_t launched(F f) {
  f();
  return hipGetLastError();
}

// lowrank_both_kernel is taken up to so many tiles of rows and bytes of one
// adapter's two banks (us a pass in bfloat16, one launch against two: 256 tokens,
// 512 columns, rank 64, 128 KiB 9.3 against 11.0; 48 tokens, 2048 columns, rank
// 16, 128 KiB 10.9 against 11.5; 48 tokens, 4096 columns, 256 KiB 15.5 against
// 12.4; 1024 tokens, 1024 columns, rank 8, 32 KiB 8.1 against 9.9).
constexpr int kBothTiles = 64;
constexpr int64_t kBothBank = 128 << 10;

// Adapters of a tile side by side while workgroups are few (a forward pass, 4096
// columns, rank 16, one slot against this: 16 tokens of 16 adapters 63 and 12 us,
// 256 of 64 40 and 15, 2048 of 64 26 and 24).
int slots_for(int64_t workgroups, int E) {
  int s = 1;
  while (s < kTile && s < E && workgroups * s < 512) s *= 2;
  return s;
}

}  // namespace

hipError_t launch_lowrank_shrink(const LowrankArgs& a, hipStream_t s) {
  // two tiles a workgroup, which halves what is read of the banks, when that
  // still leaves a workgroup for every CU (a forward pass of 8192 rows, 4096
  // columns, one tile against two: rank 32 66 and 63 us, rank 64 95 and 81)
  const bool far = (int64_t)a.T * a.wch * 16 >= (int64_t(1) << 31);
  const int rt = !far && a.r <= 64 && a.R >= 2 * kTile * 256 ? 2 : 1;
  const int tiles = (a.R + kTile * rt - 1) / (kTile * rt);
  // Few tiles: the rank in parts of 16 or more, since one CU reads a bank slowly
  // (the kernel in one part and in parts, us: 4 float32 rows of 3936, rank 52 26
  // and 10; bfloat16 rows of 4096, rank 64, 8 of them 9.9 and 6.4, 48 11.8 and
  // 6.9; 700 of 2048, rank 32 6.1 and 6.4).  Not with grad_w, a sum over the rank.
  int width = a.r <= 16 ? 1 : a.r <= 32 ? 2 : a.r <= 64 ? 4 : 8;
  auto parts = [&] { return (a.r + 16 * width - 1) / (16 * width); };  // every part has ranks
  if (!far && !a.dot)
    while (width > 1 && tiles * parts() * 2 <= 128) width /= 2;
  const dim3 grid(tiles, slots_for(tiles, a.E), parts());
#define MOE_SHRINK(J, T, F)                                                                             \
  return launched([&] {                                                                                 \
    const dim3 block((Shrink<J, T>::kWaves * kWave));                                                   \
    const size_t lds = (Shrink<J, T>::kLds);                                                            \
    if (a.dtype == MOE_F32) hipLaunchKernelGGL((shrink_kernel<kF32, J, T, F>), grid, block, lds, s, a); \
    else hipLaunchKernelGGL((shrink_kernel<kBF16, J, T, F>), grid, block, lds, s, a);                   \
  })
  if (far) {  // two rank widths: ranks from 33 to 64 multiply as many zeros again
    if (a.r <= 32) MOE_SHRINK(2, 1, true);
    MOE_SHRINK(8, 1, true);
  }
  if (rt == 2) {
    if (a.r <= 16) MOE_SHRINK(1, 2, false);
    if (a.r <= 32) MOE_SHRINK(2, 2, false);
    MOE_SHRINK(4, 2, false);
  }
  if (width == 1) MOE_SHRINK(1, 1, false);
  if (width == 2) MOE_SHRINK(2, 1, false);
  if (width == 4) MOE_SHRINK(4, 1, false);
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

// Both steps of a pass: u = rows -> rank with `s`, then rank -> rows with `a`
// (which reads s.u), in one launch where that is the faster.
hipError_t launch_lowrank_pass(const LowrankArgs& s, const LowrankArgs& a, hipStream_t stream) {
  const int tiles = (s.R + kTile - 1) / kTile;
  const int64_t bank = (int64_t)s.r * ((int64_t)s.wch + a.wch) * 16;
  const bool far = (int64_t)s.T * s.wch * 16 >= (int64_t(1) << 31);
  if (!far && tiles <= kBothTiles && bank <= kBothBank) {
    const dim3 grid(tiles, slots_for(tiles, s.E));
#define MOE_BOTH(J)                                                                                           \
  return launched([&] {                                                                                       \
    const dim3 f32((Both<kF32, J>::kWaves * kWave)), bf16((Both<kBF16, J>::kWaves * kWave));                  \
    if (s.dtype == MOE_F32)                                                                                   \
      hipLaunchKernelGGL((lowrank_both_kernel<kF32, J>), grid, f32, (Both<kF32, J>::kLds), stream, s, a);     \
    else                                                                                                      \
      hipLaunchKernelGGL((lowrank_both_kernel<kBF16, J>), grid, bf16, (Both<kBF16, J>::kLds), stream, s, a);  \
  })
    if (s.r <= 16) MOE_BOTH(1);
    if (s.r <= 32) MOE_BOTH(2);
    if (s.r <= 64) MOE_BOTH(4);
    MOE_BOTH(8);
#undef MOE_BOTH
  }
  const hipError_t e = launch_lowrank_shrink(s, stream);
  return e != hipSuccess ? e : launch_lowrank_expand(a, stream);
}

namespace {

int wgrad_width(int r) {  // ranks of a workgroup
  // a backward pass with 16 against 32: 1024 rows, rank 16 27 and 29 us, 4096
  // rows, rank 64 77 and 69, rank 128 180 and 143
  return r <= 16 ? 16 : 32;
}

int64_t wgrad_blocks(int wch, int r) { return (int64_t)((wch + 15) / 16) * ((r + wgrad_width(r) - 1) / wgrad_width(r)); }

template <int DT, int JT>
hipError_t launch_wgrad(const LowrankArgs& a, const WgradSide& one, const WgradSide& two, int one_blocks, dim3 grid,
                        hipStream_t s) {
  // As many workgroups of 8 waves as the registers let run at once (bfloat16 one
  // a CU, float32 two): more go with 4 waves, all at once again (a backward pass
  // in bfloat16 with 8 and 4 waves: 512 rows of 64 adapters, rank 32, 2048
  // columns 61 and 38 us, 4096 of 16, rank 64, 4096 columns 123 and 99, 4096 of
  // one, 2048 columns 57 and 76).
  const int64_t groups = (int64_t)grid.x * grid.y * grid.z;
  return launched([&] {
    if (groups > (DT == kBF16 ? 256 : 512))
      hipLaunchKernelGGL((wgrad_kernel<DT, JT, 4>), grid, dim3(4 * kWave), 0, s, a, one, two, one_blocks);
    else
      hipLaunchKernelGGL((wgrad_kernel<DT, JT, 8>), grid, dim3(8 * kWave), 0, s, a, one, two, one_blocks);
  });
}

}  // namespace

// Parts that the rows of an adapter are split into: while the workgroups are
// fewer than CUs and every wave keeps two blocks of rows (a backward pass of one
// adapter in bfloat16, whole and split: 4096 rows, rank 64, 2048 columns 57 and 43
// us, 16384 rows, rank 64, 4096 columns 220 and 182; float32, 2048 rows, rank 32,
// 2048 columns 50 and 36).
int lowrank_wgrad_splits(int64_t R, int A, int r, int hch, int nch, int dtype) {
  const int64_t groups = (wgrad_blocks(hch, r) + wgrad_blocks(nch, r)) * A;
  const int64_t rows = 8 * 2 * (dtype == MOE_F32 ? Shape<kF32>::KB : Shape<kBF16>::KB);
  int s = 1;
  while (s < 16 && groups * s * 2 <= 256 && R / A >= rows * s * 2) s *= 2;
  return s;
}

// grad_a from `a` and grad_b from `b`, where their out is not null; parts: room
// for `splits` times both in float32, with splits > 1.
hipError_t launch_lowrank_wgrad(const LowrankArgs& a, const LowrankArgs& b, float* parts, int splits, hipStream_t s) {
  const int64_t one_blocks = a.out ? wgrad_blocks(a.wch, a.r) : 0, two_blocks = b.out ? wgrad_blocks(b.wch, b.r) : 0;
  const int v = a.dtype == MOE_F32 ? 4 : 8;
  const int64_t one_chunks = a.out ? (int64_t)a.A * a.r * a.wch : 0, two_chunks = b.out ? (int64_t)b.A * b.r * b.wch : 0;
  const WgradSide one{a.rows, a.w, a.u, a.out, a.wch, parts};
  const WgradSide two{b.rows, b.w, b.u, b.out, b.wch, splits > 1 ? parts + splits * one_chunks * v : nullptr};
  const dim3 grid(one_blocks + two_blocks, a.A, splits);
  hipError_t e;
  if (a.dtype == MOE_F32)
    e = wgrad_width(a.r) == 16 ? launch_wgrad<kF32, 1>(a, one, two, (int)one_blocks, grid, s)
                               : launch_wgrad<kF32, 2>(a, one, two, (int)one_blocks, grid, s);
  else
    e = wgrad_width(a.r) == 16 ? launch_wgrad<kBF16, 1>(a, one, two, (int)one_blocks, grid, s)
                               : launch_wgrad<kBF16, 2>(a, one, two, (int)one_blocks, grid, s);
  if (e != hipSuccess || splits == 1) return e;
  const int chunks = (int)(one_chunks + two_chunks);
  return launched([&] {
    const dim3 blocks((chunks + 255) / 256);
    if (a.dtype == MOE_F32) hipLaunchKernelGGL(wgrad_sum_kernel<kF32>, blocks, dim3(256), 0, s, one, two, (int)one_chunks, chunks, splits);
    else hipLaunchKernelGGL(wgrad_sum_kernel<kBF16>, blocks, dim3(256), 0, s, one, two, (int)one_chunks, chunks, splits);
  });
}

}  // namespace moe
