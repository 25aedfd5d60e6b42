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

// Chunk of 16 that slot m of an operand takes, chosen so that the four lanes
// of one result column store four neighbouring chunks.
__device__ __forceinline__ int slot_chunk(int m) { return (m & 3) * 4 + (m >> 2); }

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
// One workgroup per (tile, slot).  Its waves split the sum over the row in
// pairs of 64-byte steps and meet in LDS; the first wave adds the parts and
// writes 16 rows of r float32.
constexpr int kShrinkWaves = 8;

template <int DT, int JT>
__global__ __launch_bounds__(kShrinkWaves* kWave) void shrink_kernel(LowrankArgs a) {
  constexpr int kSteps = JT <= 2 ? 4 : 2;  // steps in flight
  __shared__ int off[kMaxOff];
  constexpr int kMeet = JT < 4 ? JT : 4;  // tiles of the rank that meet in LDS together
  __shared__ f32x4 part[kShrinkWaves][kMeet][kWave];
  const int lane = lane_id(), wave = (int)(threadIdx.x / kWave);
  const int col = lane & 15, q = lane >> 4;
  load_offsets(off, a);
  const int r0 = blockIdx.x * kTile, r1 = min(r0 + kTile, a.R);
  each_adapter(off, a.E, r0, r1, blockIdx.y, gridDim.y, [&](int e, int lo, int hi) {
    const int p = r0 + col;
    const bool mine = p >= lo && p < hi;
    const int t = mine ? row_token(a, p) : -1;
    if (e >= a.A) {  // no adapter: u = 0, and no gradient
      if (wave == 0 && mine) {
        for (int j = q * 4; j < a.r; j += 16) *reinterpret_cast<f32x4*>(a.u + (size_t)p * a.r + j) = f32x4{0.f, 0.f, 0.f, 0.f};
        if (a.dot && q == 0 && t >= 0) a.dot[t] = 0.f;
      }
      return;
    }
    // columns of other adapters read a row of this one; their results are dropped
    const int tt = max(row_token(a, mine ? p : lo), 0);
    const int nch = a.wch;
    const u32x4* x = static_cast<const u32x4*>(a.rows) + (size_t)tt * nch;
    const u32x4* bank = static_cast<const u32x4*>(a.bank) + (size_t)e * a.r * nch;
    const u32x4* br[JT];
#pragma unroll
    for (int jt = 0; jt < JT; ++jt) br[jt] = bank + (size_t)min(jt * 16 + col, a.r - 1) * nch;
    f32x4 acc[JT];
#pragma unroll
    for (int jt = 0; jt < JT; ++jt) acc[jt] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int c0 = wave * 4 * kSteps + q; c0 - q < nch; c0 += kShrinkWaves * 4 * kSteps) {
      u32x4 xv[kSteps], bv[kSteps][JT];
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int c = c0 + 4 * s;
        xv[s] = u32x4{0u, 0u, 0u, 0u};
        if (c < nch) xv[s] = x[c];
#pragma unroll
        for (int jt = 0; jt < JT; ++jt) {
          bv[s][jt] = u32x4{0u, 0u, 0u, 0u};
          if (c < nch) bv[s][jt] = br[jt][c];
        }
      }
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int jt = 0; jt < JT; ++jt) acc[jt] = mma_chunk<DT>(bv[s][jt], xv[s], acc[jt]);
    }
    const float w = wave == 0 && a.w && t >= 0 ? a.w[t] : 1.f;
    float dot = 0.f;
#pragma unroll
    for (int first = 0; first < JT; first += kMeet) {
#pragma unroll
      for (int m = 0; m < kMeet; ++m) part[wave][m][lane] = acc[first + m];
      __syncthreads();
      if (wave == 0) {
#pragma unroll
        for (int m = 0; m < kMeet; ++m) {
          f32x4 v = part[0][m][lane];
#pragma unroll
          for (int k = 1; k < kShrinkWaves; ++k) v += part[k][m][lane];
          const int j = (first + m) * 16 + q * 4;
          if (mine && j < a.r) {
            if (t < 0) v = f32x4{0.f, 0.f, 0.f, 0.f};  // padding
            const size_t at = (size_t)p * a.r + j;
            if (a.backward) {
              if (a.dot) {
                const f32x4 u = *reinterpret_cast<const f32x4*>(a.saved + at);
#pragma unroll
                for (int i = 0; i < 4; ++i) dot += v[i] * u[i];
              }
              v *= w;
            }
            *reinterpret_cast<f32x4*>(a.u + at) = v;
          }
        }
      }
      __syncthreads();
    }
    if (wave == 0 && a.dot) {
      dot += __shfl_xor(dot, 16, kWave);
      dot += __shfl_xor(dot, 32, kWave);
      if (q == 0 && t >= 0) a.dot[t] = dot;
    }
  });
}

// ---- expand ---------------------------------------------------------------------

// Splits 8 floats into two bfloat16 parts, hi + lo.
__device__ __forceinline__ void split_bf16(const float (&f)[8], u32x4& hi, u32x4& lo) {
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const uint32_t a = f32_to_bf16(f[2 * d]), b = f32_to_bf16(f[2 * d + 1]);
    hi[d] = a | (b << 16);
    const float x = f[2 * d] - __uint_as_float(a << 16), y = f[2 * d + 1] - __uint_as_float(b << 16);
    // beyond the finite numbers the difference is not a number: no second part
    lo[d] = f32_to_bf16(x - x == 0.f ? x : 0.f) | (f32_to_bf16(y - y == 0.f ? y : 0.f) << 16);
  }
}

// Element i of eight rows' chunks, as one operand chunk along the rows.
__device__ __forceinline__ u32x4 across_rows(const u32x4 (&w)[8], int i) {
  u32x4 o;
#pragma unroll
  for (int d = 0; d < 4; ++d)
    o[d] = __builtin_amdgcn_perm(w[2 * d + 1][i / 2], w[2 * d][i / 2], i & 1 ? 0x07060302u : 0x05040100u);
  return o;
}

// acc[i] += (element i of the rows w) . f over a block of the summed index.
template <int DT, int V>
__device__ __forceinline__ void mma_across(const u32x4 (&w)[V], const float (&f)[V], f32x4 (&acc)[V]) {
  if constexpr (DT == kBF16) {
    u32x4 hi, lo;
    split_bf16(f, hi, lo);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const u32x4 a = across_rows(w, i);
      acc[i] = mma_chunk<kBF16>(a, hi, acc[i]);
      acc[i] = mma_chunk<kBF16>(a, lo, acc[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j)
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(w[j][i]), f[j], acc[i], 0, 0, 0);
  }
}

// One wave per (tile, COLS columns, slot): out of 16 receive rows.
constexpr int kExpandWaves = 4;

template <int DT>
__global__ __launch_bounds__(kExpandWaves* kWave) void expand_lowrank_kernel(LowrankArgs a) {
  using S = Shape<DT>;
  constexpr int V = S::V;
  __shared__ int off[kMaxOff];
  const int lane = lane_id(), wave = (int)(threadIdx.x / kWave);
  const int col = lane & 15, q = lane >> 4;
  load_offsets(off, a);
  const int nch = a.wch;
  const int c0 = (blockIdx.y * kExpandWaves + wave) * 16;  // first chunk of this wave's columns
  if (c0 >= nch) return;
  const int r0 = blockIdx.x * kTile, r1 = min(r0 + kTile, a.R);
  each_adapter(off, a.E, r0, r1, blockIdx.z, gridDim.z, [&](int e, int lo, int hi) {
    const int p = r0 + col;
    const bool mine = p >= lo && p < hi;
    const int t = mine ? row_token(a, p) : -1;
    f32x4 acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (e < a.A) {
      const float w = a.w && t >= 0 ? a.w[t] : 1.f;
      const int c = c0 + slot_chunk(col);
      const u32x4* bank = static_cast<const u32x4*>(a.bank) + (size_t)e * a.r * nch + c;
      const float* u = a.u + (size_t)(mine ? p : lo) * a.r;
      for (int j0 = q * V; j0 - q * V < a.r; j0 += S::KB) {
        u32x4 b[V];
        float f[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
          b[j] = u32x4{0u, 0u, 0u, 0u};
          if (j0 < a.r && c < nch) b[j] = bank[(size_t)(j0 + j) * nch];
        }
#pragma unroll
        for (int j = 0; j < V; j += 4) {
          f32x4 v = {0.f, 0.f, 0.f, 0.f};
          if (j0 < a.r) v = *reinterpret_cast<const f32x4*>(u + j0 + j);
#pragma unroll
          for (int i = 0; i < 4; ++i) f[j + i] = v[i] * w;
        }
        mma_across<DT, V>(b, f, acc);
      }
    }
    if (t < 0) return;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int c = c0 + s * 4 + q;
      if (c < nch) {
        const size_t at = (size_t)t * nch + c;
        float o[V];
        if (a.base) unpack<DT>(static_cast<const u32x4*>(a.base)[at], o);
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = a.base ? o[i] + acc[i][s] : acc[i][s];
        static_cast<u32x4*>(a.out)[at] = pack<DT>(o);
      }
    }
  });
}

// ---- gradients of the adapters ---------------------------------------------------
//
// grad[e][j][c] = sum over the adapter's rows p of coef[p][j] rows[t_p][c],
// coef = u (times w for grad_B).  One workgroup per (COLS columns, adapter, 16
// JT of the rank): its waves take the adapter's rows in turn, each a block of
// KB rows at a time, and meet in LDS.  An adapter without rows gets zeros.
constexpr int kWgradWaves = 4;

template <int DT, int JT>
__global__ __launch_bounds__(kWgradWaves* kWave) void wgrad_kernel(LowrankArgs a) {
  using S = Shape<DT>;
  constexpr int V = S::V;
  __shared__ f32x4 part[kWgradWaves][V][kWave];
  const int lane = lane_id(), wave = (int)(threadIdx.x / kWave);
  const int col = lane & 15, q = lane >> 4;
  const int e = blockIdx.y;
  const int nch = a.wch;
  const int c0 = blockIdx.x * 16;
  const int c = c0 + slot_chunk(col);
  const int j0 = blockIdx.z * JT * 16;
  const int lo = a.expert_offset[e], hi = min(a.expert_offset[e + 1], a.R);
  f32x4 acc[JT][V];
#pragma unroll
  for (int jt = 0; jt < JT; ++jt)
#pragma unroll
    for (int i = 0; i < V; ++i) acc[jt][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int p0 = lo + wave * S::KB; p0 < hi; p0 += kWgradWaves * S::KB) {
    u32x4 x[V];
    float w[V];
    int pp[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int p = p0 + q * V + k;
      const int t = p < hi ? row_token(a, p) : -1;
      pp[k] = t >= 0 ? p : -1;
      x[k] = u32x4{0u, 0u, 0u, 0u};
      if (t >= 0 && c < nch) x[k] = static_cast<const u32x4*>(a.rows)[(size_t)t * nch + c];
      w[k] = a.w && t >= 0 ? a.w[t] : 1.f;
    }
#pragma unroll
    for (int jt = 0; jt < JT; ++jt) {
      const int j = j0 + jt * 16 + col;
      float f[V];
#pragma unroll
      for (int k = 0; k < V; ++k) f[k] = pp[k] >= 0 && j < a.r ? a.u[(size_t)pp[k] * a.r + j] * w[k] : 0.f;
      mma_across<DT, V>(x, f, acc[jt]);
    }
  }
#pragma unroll
  for (int jt = 0; jt < JT; ++jt) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < V; ++i) part[wave][i][lane] = acc[jt][i];
    __syncthreads();
    const int j = j0 + jt * 16 + col;
    // wave s stores the chunks of quad s
    for (int s = wave; s < 4; s += kWgradWaves) {
      float o[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float* f = reinterpret_cast<const float*>(&part[0][i][lane]) + s;
        o[i] = f[0];
#pragma unroll
        for (int k = 1; k < kWgradWaves; ++k) o[i] += f[(size_t)k * V * kWave * 4];
      }
      const int cc = c0 + s * 4 + q;
      if (j < a.r && cc < nch) static_cast<u32x4*>(a.out)[((size_t)e * a.r + j) * nch + cc] = pack<DT>(o);
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
  const int tiles = (a.R + kTile - 1) / kTile;
  const dim3 grid(tiles, slots_for(tiles, a.E)), block(kShrinkWaves * kWave);
#define MOE_SHRINK(J)                                                                                  \
  return launched([&] {                                                                                \
    if (a.dtype == MOE_F32) hipLaunchKernelGGL((shrink_kernel<kF32, J>), grid, block, 0, s, a);        \
    else hipLaunchKernelGGL((shrink_kernel<kBF16, J>), grid, block, 0, s, a);                          \
  })
  if (a.r <= 16) MOE_SHRINK(1);
  if (a.r <= 32) MOE_SHRINK(2);
  if (a.r <= 64) MOE_SHRINK(4);
  MOE_SHRINK(8);
#undef MOE_SHRINK
}

hipError_t launch_lowrank_expand(const LowrankArgs& a, hipStream_t s) {
  const int tiles = (a.R + kTile - 1) / kTile;
  const int cols = (a.wch + 16 * kExpandWaves - 1) / (16 * kExpandWaves);
  const dim3 grid(tiles, cols, slots_for((int64_t)tiles * cols, a.E)), block(kExpandWaves * kWave);
  return launched([&] {
    if (a.dtype == MOE_F32) hipLaunchKernelGGL((expand_lowrank_kernel<kF32>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((expand_lowrank_kernel<kBF16>), grid, block, 0, s, a);
  });
}

hipError_t launch_lowrank_wgrad(const LowrankArgs& a, hipStream_t s) {
  const dim3 block(kWgradWaves * kWave);
  const int cols = (a.wch + 15) / 16;
#define MOE_WGRAD(J)                                                                                   \
  return launched([&] {                                                                                \
    const dim3 grid(cols, a.A, (a.r + 16 * J - 1) / (16 * J));                                         \
    if (a.dtype == MOE_F32) hipLaunchKernelGGL((wgrad_kernel<kF32, J>), grid, block, 0, s, a);         \
    else hipLaunchKernelGGL((wgrad_kernel<kBF16, J>), grid, block, 0, s, a);                           \
  })
  if (a.r <= 16) MOE_WGRAD(1);
  if (a.r <= 32) MOE_WGRAD(2);
  MOE_WGRAD(4);
#undef MOE_WGRAD
}

}  // namespace moe
