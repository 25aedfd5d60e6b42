// The norms before and after a block, with the residual, its scale and the gate,
// and their gradients.
//
//   before:  n = x r w2',   r = 1 / sqrt(mean(x^2) + eps), w' = w + offset
//   after:   out = a x + gate * (y r1 w1')   (without w1: a x + gate * y)
//            n = out r2 w2'                  the next block's norm, from out before its rounding
//   With a layout y is formed on the way: y[t] = sum_k [w[t,k] *] rows[recv_pos[t,k]].
//
// Backward, o^ = out r2 and y^ = y r1:
//   d = grad_out + r2 (w2' gn - o^ mean(w2' gn o^)),   grad_w2 = sum_t gn o^,
//       with out formed again from x and y: from its rounded form grad_w2 had 1.4
//       times the error in bfloat16, and as many rows were read
//   grad_x = a d,  v = gate d,  grad_gate = sum over its tokens of d y^ w1'
//   grad_w1 = sum_t v y^,  grad_y = r1 (w1' v - y^ mean(w1' v y^))
//
// One workgroup per row (forward) or per run of rows (backward), a row's chunks in
// registers from the first read to the last use, so every row is read and written
// once (rows of more than 8192 after a block go backward in two kernels).  Sums over
// a row: each wave's by lane moves, then the waves' in order through LDS.  Sums over
// tokens: a workgroup's run of at most 256 rows in registers, one partial for each run,
// the partials added in the order of the runs and in 64 bits by a second kernel, so that
// results do not depend on timing, nor their errors on the number of tokens.
//
// Bound by HBM.  Measured (MI355X, kernels): 8192 rows of 2816 with their combine of 8
// receive rows: 100 us, 510 MB (a combine alone 70, 415 MB); 4096 x 7168 to 8 bits: 24 us,
// 3.6 TB/s, what the rounding leaves of the bandwidth; 4096 x 2048 after a block: 16.5 us
// forward (67 MB), 29 + 5 backward (101 MB and 13 MB of partials).
#include <algorithm>

#include "device_common.h"
#include "internal.h"
#include "quant.h"
#include "../../include/moe_layout.h"

namespace moe {
namespace {

constexpr int kMaxWaves = 16;

template <int CPL>
struct Block {
  static constexpr int kMax = CPL == 4 ? 1024 : 512;  // threads
};

__device__ __forceinline__ float block_sum(float v, float* red) {
  v = wave_sum(v);
  const int waves = blockDim.x / kWave;
  if (waves == 1) return v;
  if (lane_id() == 0) red[threadIdx.x / kWave] = v;
  __syncthreads();
  v = red[0];
  for (int w = 1; w < waves; ++w) v += red[w];
  return v;
}

__device__ __forceinline__ uint32_t block_max(uint32_t v, float* red) {
  v = wave_max(v);
  const int waves = blockDim.x / kWave;
  if (waves == 1) return v;
  if (lane_id() == 0) red[threadIdx.x / kWave] = __uint_as_float(v);
  __syncthreads();
  v = __float_as_uint(red[0]);
  for (int w = 1; w < waves; ++w) v = max(v, __float_as_uint(red[w]));
  return v;
}

// 1 / sqrt(mean of squares + eps) of the row whose values f are spread over the
// workgroup.  Where the squares leave float32's range (values above 2^64, or below
// 2^-50 beside an eps that small), relative to the largest value.
template <int N>
__device__ float block_rstd(const float (&f)[N], int H, float eps, float* red, float* red2, float* red3) {
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) ss = __builtin_fmaf(f[i], f[i], ss);
  ss = block_sum(ss, red);
  if (ss < 3e38f && (ss > 0x1p-100f || eps > 0x1p-70f)) return 1.f / sqrtf(ss / (float)H + eps);  // uniform
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) top = max(top, abs_bits(f[i]));
  const float m = __uint_as_float(block_max(top, red2));
  if (!(m < INFINITY) || m == 0.f) return 1.f / sqrtf(ss / (float)H + eps);
  float rel = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) rel += (f[i] / m) * (f[i] / m);
  rel = block_sum(rel, red3);
  return (float)(1.0 / sqrt((double)m * m * (rel / (double)H) + eps));
}

// ---- forward ----------------------------------------------------------------------

enum : int { kBefore = 0, kRows = 1, kGather = 2 };  // where y comes from

// A workgroup for each of `rows` rows: a dimension of a grid has fewer than 2^32 threads, so
// from kAcross rows on they go down a second one.
constexpr int kAcross = 1 << 20;
dim3 row_grid(int rows) { return dim3(rows < kAcross ? rows : kAcross, (rows + kAcross - 1) / kAcross); }
__device__ __forceinline__ int row_of_block() { return blockIdx.y * kAcross + blockIdx.x; }

template <int DT, int CPL, int SRC>
__global__ __launch_bounds__(Block<CPL>::kMax) void norm_kernel(NormArgs a) {
  constexpr int V = Elems<DT>::kPerChunk;
  __shared__ float red[7][kMaxWaves];
  const int t = row_of_block(), tid = threadIdx.x, H = a.nch * V;
  if (t >= a.T) return;  // uniform
  const size_t row = (size_t)t * a.nch;
  float f[CPL * V], x[CPL * V];
  u32x4 c[CPL];
  const u32x4 zero = {0, 0, 0, 0};
  auto load = [&](const void* p, size_t at, u32x4(&to)[CPL]) {
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      const int j = tid + i * blockDim.x;
      to[i] = j < a.nch ? static_cast<const u32x4*>(p)[at + j] : zero;
    }
  };
  auto floats = [&](const u32x4(&from)[CPL], float(&to)[CPL * V]) {
#pragma unroll
    for (int i = 0; i < CPL; ++i) unpack<DT>(from[i], to + i * V);
  };
  auto store = [&](void* p, const float(&from)[CPL * V]) {
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      const int j = tid + i * blockDim.x;
      if (j < a.nch) static_cast<u32x4*>(p)[row + j] = pack<DT>(from + i * V);
    }
  };
  // The weights and the gate are asked for with the row, not when its sums are known (4096
  // x 4096 bfloat16: 25.6 us, 28.0 then), except where receive rows need the registers
  // (8192 x 2816: 102 us, 104 with them).
  constexpr bool kEarly = SRC != kGather;
  u32x4 w1[CPL], w2[CPL], gate[CPL], cy[CPL];
  auto weights = [&]() {
    if (SRC != kBefore && a.w1) load(a.w1, 0, w1);
    if (SRC != kBefore && a.gate) load(a.gate, (size_t)(t / a.group) * a.nch, gate);
    if (a.w2) load(a.w2, 0, w2);
  };
  load(a.x, row, c);
  if constexpr (SRC == kRows) load(a.y, row, cy);
  if constexpr (kEarly) weights();
  floats(c, x);
  float r1 = 1.f, r2 = 1.f;
  if constexpr (SRC != kBefore) {
    if constexpr (SRC == kRows) {
      floats(cy, f);
    } else {
#pragma unroll
      for (int i = 0; i < CPL * V; ++i) f[i] = 0.f;
      constexpr int kGatherRows = CPL == 1 ? 8 : 4;  // receive rows in flight
      for (int k0 = 0; k0 < a.K; k0 += kGatherRows) {  // sums in k order from +0
        u32x4 g[kGatherRows][CPL];
        float w[kGatherRows];
        bool good[kGatherRows];  // uniform
#pragma unroll
        for (int k = 0; k < kGatherRows; ++k) {
          const bool there = k0 + k < a.K;
          const int p = there ? a.recv_pos[(size_t)t * a.K + k0 + k] : -1;
          w[k] = there && a.w ? a.w[(size_t)t * a.K + k0 + k] : 1.f;
          good[k] = (unsigned)p < (unsigned)a.R;
          if (there && !good[k] && tid == 0) atomicOr(a.status, MOE_STATUS_BAD_POSITION);
          if (good[k])
#pragma unroll
            for (int i = 0; i < CPL; ++i) {  // read once
              const int j = tid + i * blockDim.x;
              g[k][i] = j < a.nch ? __builtin_nontemporal_load(static_cast<const u32x4*>(a.y) + (size_t)p * a.nch + j) : zero;
            }
        }
#pragma unroll
        for (int k = 0; k < kGatherRows; ++k) {
          if (!good[k]) continue;
          float e[CPL * V];
          floats(g[k], e);
#pragma unroll
          for (int i = 0; i < CPL * V; ++i) f[i] += a.w ? w[k] * e[i] : e[i];
        }
      }
    }
    if (a.w1) {
      r1 = block_rstd(f, H, a.eps, red[0], red[1], red[2]);
      if constexpr (!kEarly) load(a.w1, 0, w1);
      float w[CPL * V];
      floats(w1, w);
#pragma unroll
      for (int i = 0; i < CPL * V; ++i) f[i] = f[i] * r1 * (w[i] + a.offset);
    }
    if (a.gate) {
      if constexpr (!kEarly) load(a.gate, (size_t)(t / a.group) * a.nch, gate);
      float w[CPL * V];
      floats(gate, w);
#pragma unroll
      for (int i = 0; i < CPL * V; ++i) f[i] *= w[i];
    }
#pragma unroll
    for (int i = 0; i < CPL * V; ++i) x[i] = a.residual * x[i] + f[i];
    store(a.out, x);
  }
  if (a.w2) {
    r2 = block_rstd(x, H, a.eps, red[3], red[4], red[5]);
    if constexpr (!kEarly) load(a.w2, 0, w2);
    float w[CPL * V];
    floats(w2, w);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < CPL * V; ++i) {
      x[i] = x[i] * r2 * (w[i] + a.offset);
      top = max(top, abs_bits(x[i]));
    }
    if (a.q) {
      const float s = quant_scale(block_max(top, red[6])), inv = quant_inverse(s);
#pragma unroll
      for (int i = 0; i < CPL; ++i) {
        const int j = tid + i * blockDim.x;
        if (j < a.nch) store_quant<V>(a.q + (size_t)t * H, j, x + i * V, s, inv);
      }
      if (tid == 0) a.scale[t] = s;
    } else {
      store(a.n, x);
    }
  }
  if (tid == 0 && a.rstd) {
    if constexpr (SRC == kBefore) a.rstd[t] = r2;
    else *reinterpret_cast<float2*>(a.rstd + 2 * (size_t)t) = make_float2(r1, r2);
  }
}

// ---- rows to 8 bits -----------------------------------------------------------------

// A wave takes 4 / CPL rows of at most 64 CPL chunks, four chunks a lane in all; wider
// rows a workgroup each.
template <int DT, int CPL>
__global__ __launch_bounds__(256) void quant_wave_kernel(NormArgs a) {
  constexpr int V = Elems<DT>::kPerChunk, kRows = 4 / CPL;
  const int64_t t0 = ((int64_t)blockIdx.x * 4 + threadIdx.x / kWave) * kRows;
  const int lane = lane_id();
  u32x4 c[kRows][CPL];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const u32x4* p = static_cast<const u32x4*>(a.x) + (size_t)(t0 + r) * a.nch;
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      const int j = lane + i * kWave;
      c[r][i] = t0 + r < a.T && j < a.nch ? p[j] : u32x4{0, 0, 0, 0};
    }
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int64_t t = t0 + r;
    if (t >= a.T) return;  // wave-uniform
    float f[CPL * V];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < CPL; ++i) unpack<DT>(c[r][i], f + i * V);
#pragma unroll
    for (int i = 0; i < CPL * V; ++i) top = max(top, abs_bits(f[i]));
    const float s = quant_scale(wave_max(top)), inv = quant_inverse(s);
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      const int j = lane + i * kWave;
      if (j < a.nch) store_quant<V>(a.q + (size_t)t * a.nch * V, j, f + i * V, s, inv);
    }
    if (lane == 0) a.scale[t] = s;
  }
}

template <int DT>
__global__ __launch_bounds__(1024) void quant_block_kernel(NormArgs a) {
  constexpr int V = Elems<DT>::kPerChunk;
  __shared__ float red[kMaxWaves];
  const size_t t = row_of_block();
  if (t >= (size_t)a.T) return;  // uniform
  const u32x4* p = static_cast<const u32x4*>(a.x) + t * a.nch;
  uint32_t top = 0;
  for (int j = threadIdx.x; j < a.nch; j += blockDim.x) {
    float f[V];
    unpack<DT>(p[j], f);
#pragma unroll
    for (int i = 0; i < V; ++i) top = max(top, abs_bits(f[i]));
  }
  const float s = quant_scale(block_max(top, red)), inv = quant_inverse(s);
  for (int j = threadIdx.x; j < a.nch; j += blockDim.x) {  // the row again, from the caches
    float f[V];
    unpack<DT>(p[j], f);
    store_quant<V>(a.q + t * a.nch * V, j, f, s, inv);
  }
  if (threadIdx.x == 0) a.scale[t] = s;
}

// ---- backward ---------------------------------------------------------------------

// The tokens of a run: a part of one gate's tokens, or whole gates.
__device__ __forceinline__ void tokens_of_run(const NormBwdArgs& a, int run, int& t0, int& t1) {
  if (a.parts > 1) {
    const int group = run / a.parts, part = run % a.parts;
    t0 = group * a.group + part * a.rows;
    t1 = min(t0 + a.rows, (group + 1) * a.group);
  } else {
    t0 = (int)min((int64_t)run * a.rows, (int64_t)a.T);
    t1 = (int)min((int64_t)t0 + a.rows, (int64_t)a.T);
  }
}

// A chunk of a row after a block: y^, y^ weight' (y^ without a norm), gate.
template <int DT, int V>
__device__ __forceinline__ void block_chunk(const NormBwdArgs& a, u32x4 yc, u32x4 wc, u32x4 gatec, float r1, float (&y)[V],
                                            float (&yn)[V], float (&gate)[V]) {
  float w[V];
  unpack<DT>(yc, y);
  unpack<DT>(wc, w);
  unpack<DT>(gatec, gate);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    y[v] *= r1;
    yn[v] = a.w1 ? y[v] * (w[v] + a.offset) : y[v];
    if (!a.gate) gate[v] = 1.f;
  }
}

// A chunk of the norm before the next block: z^ (from out as the forward pass had it, or
// x), grad_n, grad_n next'.
template <int DT, bool BLOCK, int V>
__device__ __forceinline__ void next_chunk(const NormBwdArgs& a, u32x4 xc, u32x4 gnc, u32x4 wc, float r2, const float (&yn)[V],
                                           const float (&gate)[V], float (&z)[V], float (&gn)[V], float (&gw)[V]) {
  float w[V];
  unpack<DT>(xc, z);
  unpack<DT>(gnc, gn);
  unpack<DT>(wc, w);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if constexpr (BLOCK) z[v] = a.residual * z[v] + gate[v] * yn[v];
    z[v] *= r2;
    gw[v] = gn[v] * (w[v] + a.offset);
  }
}

// Rows of up to 512 chunks are asked for a row ahead; wider ones have no registers for
// that (7168 bfloat16, 4096 rows: 110 us without, 118 with).  The chunks stay as they were
// read, and each of the three passes over them (the first sum, the second, the end) makes
// its numbers again, a chunk at a time: what lives over a pass is the sums over the run and
// v.
template <int DT, int CPL, bool BLOCK, bool kAhead, int MOST>
__global__ __launch_bounds__(MOST) void norm_bwd_kernel(NormBwdArgs a) {
  constexpr int V = Elems<DT>::kPerChunk, N = CPL * V;
  __shared__ float red[4][kMaxWaves];
  const int tid = threadIdx.x, run = blockIdx.x, H = a.nch * V;
  int t0, t1;
  tokens_of_run(a, run, t0, t1);
  const u32x4 zero = {0, 0, 0, 0};
  auto chunks = [&](const void* p, int row, u32x4(&to)[CPL]) {
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      const int j = tid + i * blockDim.x;
      to[i] = p && j < a.nch ? static_cast<const u32x4*>(p)[(size_t)row * a.nch + j] : zero;
    }
  };
  auto store = [&](void* p, int row, int i, const float* from) {
    const int j = tid + i * blockDim.x;
    if (j < a.nch) static_cast<u32x4*>(p)[(size_t)row * a.nch + j] = pack<DT>(from);
  };
  auto partial = [&](float* p, const float(&from)[N]) {
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      const int j = tid + i * blockDim.x;
      if (j < a.nch)
#pragma unroll
        for (int v = 0; v < V; v += 4)
          *reinterpret_cast<float4*>(p + (size_t)run * H + (size_t)j * V + v) =
              make_float4(from[i * V + v], from[i * V + v + 1], from[i * V + v + 2], from[i * V + v + 3]);
    }
  };
  struct Row {
    u32x4 g[CPL], gn[CPL], x[CPL], y[CPL], gate[CPL];
    float r1, r2;
  };
  auto fetch = [&](int t, Row& r) {
    chunks(a.g, t, r.g);
    chunks(a.gn, t, r.gn);
    chunks(a.gn ? a.x : nullptr, t, r.x);
    r.r1 = 1.f;
    if constexpr (BLOCK) {
      chunks(a.y, t, r.y);
      chunks(a.gate, t / a.group, r.gate);
      r.r1 = a.rstd[2 * (size_t)t];
      r.r2 = a.rstd[2 * (size_t)t + 1];
    } else {
      r.r2 = a.rstd[t];
    }
  };
  float s1[N], s2[N], sg[N];  // sums over the run
#pragma unroll
  for (int i = 0; i < N; ++i) s1[i] = s2[i] = sg[i] = 0.f;
  u32x4 w1[CPL], w2[CPL];
  chunks(BLOCK ? a.w1 : nullptr, 0, w1);
  chunks(a.w2, 0, w2);
  Row row;
  if (t0 < t1) fetch(t0, row);
  for (int t = t0; t < t1; ++t) {
    Row r = row;
    if constexpr (kAhead) {
      if (t + 1 < t1) fetch(t + 1, row);
    }
    const int odd = (t - t0) & 1;  // two rows' sums lie apart: one barrier a sum
    auto block_values = [&](int i, float(&y)[V], float(&yn)[V], float(&gate)[V]) {
      block_chunk<DT>(a, r.y[i], w1[i], r.gate[i], r.r1, y, yn, gate);
    };
    auto next_values = [&](int i, const float(&yn)[V], const float(&gate)[V], float(&z)[V], float(&gn)[V], float(&gw)[V]) {
      next_chunk<DT, BLOCK>(a, r.x[i], r.gn[i], w2[i], r.r2, yn, gate, z, gn, gw);
    };
    float m2 = 0.f;
    if (a.gn) {
#pragma unroll
      for (int i = 0; i < CPL; ++i) {
        float y[V], yn[V], gate[V], z[V], gn[V], gw[V];
        if constexpr (BLOCK) block_values(i, y, yn, gate);
        next_values(i, yn, gate, z, gn, gw);
#pragma unroll
        for (int v = 0; v < V; ++v) m2 = __builtin_fmaf(gw[v], z[v], m2);
      }
      m2 = block_sum(m2, red[odd]) / (float)H;
    }
    float d[N], m1 = 0.f;
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      if constexpr (CPL > 1) __asm__ __volatile__("" ::: "memory");  // a chunk at a time
      float y[V], yn[V], gate[V];
      float* di = d + i * V;
      if constexpr (BLOCK) block_values(i, y, yn, gate);
      unpack<DT>(r.g[i], di);
      if (a.gn) {
        float z[V], gn[V], gw[V];
        next_values(i, yn, gate, z, gn, gw);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          s2[i * V + v] += gn[v] * z[v];
          di[v] += r.r2 * (gw[v] - z[v] * m2);
        }
      }
      if constexpr (!BLOCK) {
        if (a.gx) store(a.gx, t, i, di);
      } else {
        if (a.gx) {
          float gx[V];
#pragma unroll
          for (int v = 0; v < V; ++v) gx[v] = a.residual * di[v];
          store(a.gx, t, i, gx);
        }
        float w[V];
        unpack<DT>(w1[i], w);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          if (a.gg) sg[i * V + v] += di[v] * yn[v];
          if (a.gate) di[v] *= gate[v];
          if (a.w1) {
            s1[i * V + v] += di[v] * y[v];
            di[v] *= w[v] + a.offset;
            m1 = __builtin_fmaf(di[v], y[v], m1);
          }
        }
      }
    }
    if constexpr (BLOCK) {
      if (a.w1) m1 = block_sum(m1, red[2 + odd]) / (float)H;
      if (a.gy) {
#pragma unroll
        for (int i = 0; i < CPL; ++i) {
          float* di = d + i * V;
          if (a.w1) {
            float y[V];
            unpack<DT>(r.y[i], y);
#pragma unroll
            for (int v = 0; v < V; ++v) di[v] = r.r1 * (di[v] - y[v] * r.r1 * m1);
          }
          store(a.gy, t, i, di);
        }
      }
      if (a.gg && a.parts == 1 && (t + 1) % a.group == 0) {  // the gate's last token
#pragma unroll
        for (int i = 0; i < CPL; ++i) store(a.gg, t / a.group, i, sg + i * V);
#pragma unroll
        for (int i = 0; i < N; ++i) sg[i] = 0.f;
      }
    }
    if constexpr (!kAhead) {
      if (t + 1 < t1) fetch(t + 1, row);
    }
  }
  if (a.part1) partial(a.part1, s1);
  if (a.part2) partial(a.part2, s2);
  if (a.gg && a.parts > 1) partial(a.partg, sg);
}

// Wide rows after a block, in two kernels: the two means of every row first, then, with
// those known, a wave for 64 chunks of the columns of a run, which needs no other wave.
// The rows are read twice, but nothing stays in registers but a chunk and its sums (2048
// rows of 16384 bfloat16: 79 + 85 us, 65 are what the bytes of one reading take).
template <int DT>
__global__ __launch_bounds__(1024) void norm_means_kernel(NormBwdArgs a) {
  constexpr int V = Elems<DT>::kPerChunk;
  __shared__ float red[2][kMaxWaves];
  const int t = row_of_block(), H = a.nch * V;
  if (t >= a.T) return;  // uniform
  const u32x4 zero = {0, 0, 0, 0};
  auto chunk = [&](const void* p, int row, int j) {
    return p ? static_cast<const u32x4*>(p)[(size_t)row * a.nch + j] : zero;
  };
  const float r1 = a.rstd[2 * (size_t)t], r2 = a.rstd[2 * (size_t)t + 1];
  const int group = t / a.group;
  float m2 = 0.f, m1 = 0.f;
  if (a.gn) {
    for (int j = threadIdx.x; j < a.nch; j += blockDim.x) {
      float y[V], yn[V], gate[V], z[V], gn[V], gw[V];
      block_chunk<DT>(a, chunk(a.y, t, j), chunk(a.w1, 0, j), chunk(a.gate, group, j), r1, y, yn, gate);
      next_chunk<DT, true>(a, chunk(a.x, t, j), chunk(a.gn, t, j), chunk(a.w2, 0, j), r2, yn, gate, z, gn, gw);
#pragma unroll
      for (int v = 0; v < V; ++v) m2 = __builtin_fmaf(gw[v], z[v], m2);
    }
    m2 = block_sum(m2, red[0]) / (float)H;
  }
  if (a.w1) {
    for (int j = threadIdx.x; j < a.nch; j += blockDim.x) {  // the row again, from the caches
      float y[V], yn[V], gate[V], w[V], d[V];
      const u32x4 wc = chunk(a.w1, 0, j);
      block_chunk<DT>(a, chunk(a.y, t, j), wc, chunk(a.gate, group, j), r1, y, yn, gate);
      unpack<DT>(wc, w);
      unpack<DT>(chunk(a.g, t, j), d);
      if (a.gn) {
        float z[V], gn[V], gw[V];
        next_chunk<DT, true>(a, chunk(a.x, t, j), chunk(a.gn, t, j), chunk(a.w2, 0, j), r2, yn, gate, z, gn, gw);
#pragma unroll
        for (int v = 0; v < V; ++v) d[v] += r2 * (gw[v] - z[v] * m2);
      }
#pragma unroll
      for (int v = 0; v < V; ++v) m1 = __builtin_fmaf(d[v] * gate[v] * (w[v] + a.offset), y[v], m1);
    }
    m1 = block_sum(m1, red[1]) / (float)H;
  }
  if (threadIdx.x == 0) *reinterpret_cast<float2*>(a.means + 2 * (size_t)t) = make_float2(m1, m2);
}

template <int DT>
__global__ __launch_bounds__(256) void norm_columns_kernel(NormBwdArgs a) {
  constexpr int V = Elems<DT>::kPerChunk;
  const int columns = (a.nch + blockDim.x - 1) / blockDim.x;  // workgroups of a run
  const int run = blockIdx.x / columns, H = a.nch * V, j = blockIdx.x % columns * blockDim.x + threadIdx.x;
  if (j >= a.nch) return;
  int t0, t1;
  tokens_of_run(a, run, t0, t1);
  const u32x4 zero = {0, 0, 0, 0};
  auto chunk = [&](const void* p, int row) { return p ? static_cast<const u32x4*>(p)[(size_t)row * a.nch + j] : zero; };
  auto store = [&](void* p, int row, const float(&from)[V]) { static_cast<u32x4*>(p)[(size_t)row * a.nch + j] = pack<DT>(from); };
  struct Row {
    u32x4 g, gn, x, y;
    float2 r, m;
  };
  auto fetch = [&](int t, Row& r) {
    r.g = chunk(a.g, t);
    r.gn = chunk(a.gn, t);
    r.x = chunk(a.gn ? a.x : nullptr, t);
    r.y = chunk(a.y, t);
    r.r = *reinterpret_cast<const float2*>(a.rstd + 2 * (size_t)t);
    r.m = a.means ? *reinterpret_cast<const float2*>(a.means + 2 * (size_t)t) : make_float2(0.f, 0.f);
  };
  float s1[V], s2[V], sg[V];  // sums over the run
#pragma unroll
  for (int v = 0; v < V; ++v) s1[v] = s2[v] = sg[v] = 0.f;
  const u32x4 w1 = chunk(a.w1, 0), w2 = chunk(a.w2, 0);
  Row row;
  if (t0 < t1) fetch(t0, row);
  for (int t = t0; t < t1; ++t) {
    const Row r = row;
    if (t + 1 < t1) fetch(t + 1, row);
    float y[V], yn[V], gate[V], d[V], w[V];
    block_chunk<DT>(a, r.y, w1, chunk(a.gate, t / a.group), r.r.x, y, yn, gate);
    unpack<DT>(r.g, d);
    if (a.gn) {
      float z[V], gn[V], gw[V];
      next_chunk<DT, true>(a, r.x, r.gn, w2, r.r.y, yn, gate, z, gn, gw);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        s2[v] += gn[v] * z[v];
        d[v] += r.r.y * (gw[v] - z[v] * r.m.y);
      }
    }
    if (a.gx) {
      float gx[V];
#pragma unroll
      for (int v = 0; v < V; ++v) gx[v] = a.residual * d[v];
      store(a.gx, t, gx);
    }
    unpack<DT>(w1, w);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (a.gg) sg[v] += d[v] * yn[v];
      if (a.gate) d[v] *= gate[v];
      if (a.w1) {
        s1[v] += d[v] * y[v];
        d[v] = r.r.x * (d[v] * (w[v] + a.offset) - y[v] * r.m.x);
      }
    }
    if (a.gy) store(a.gy, t, d);
    if (a.gg && a.parts == 1 && (t + 1) % a.group == 0) {  // the gate's last token
      store(a.gg, t / a.group, sg);
#pragma unroll
      for (int v = 0; v < V; ++v) sg[v] = 0.f;
    }
  }
  auto partial = [&](float* p, const float(&from)[V]) {
#pragma unroll
    for (int v = 0; v < V; v += 4)
      *reinterpret_cast<float4*>(p + (size_t)run * H + (size_t)j * V + v) = make_float4(from[v], from[v + 1], from[v + 2], from[v + 3]);
  };
  if (a.part1) partial(a.part1, s1);
  if (a.part2) partial(a.part2, s2);
  if (a.gg && a.parts > 1) partial(a.partg, sg);
}

// Adds partials: blockIdx.y 0 the next norm's weight, 1 the post-norm's, from 2 on the gates
// (a grid's second dimension may hold fewer).  64 columns a workgroup, four a thread; a
// sixteenth of the partials each.
constexpr int kGateRows = 32768;  // of the grid

template <int DT>
__global__ __launch_bounds__(256) void norm_join_kernel(NormBwdArgs a) {
  __shared__ double sum[16][64], four[4][64];
  const int H = a.nch * Elems<DT>::kPerChunk;
  const int tid = threadIdx.x, q = tid % 16, k = tid / 16, col = blockIdx.x * 64 + 4 * q;
  const bool gates = blockIdx.y >= 2;
  void* to = gates ? a.gg : blockIdx.y == 1 ? a.gw1 : a.gw2;
  if (!to) return;  // uniform
  const int n = gates ? a.parts : a.runs;
  for (int64_t row = gates ? blockIdx.y - 2 : 0; row < (gates ? a.gates : 1); row += kGateRows) {
    const float* from = gates ? a.partg + row * n * H : blockIdx.y == 1 ? a.part1 : a.part2;
    double s[4] = {0.0, 0.0, 0.0, 0.0};
    if (col < H)
      for (int i0 = k; i0 < n; i0 += 16 * 8) {
        float4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = *reinterpret_cast<const float4*>(from + (size_t)min(i0 + 16 * u, n - 1) * H + col);
        __builtin_amdgcn_sched_barrier(0);  // all on their way before the first is added
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const bool there = i0 + 16 * u < n;
          s[0] += there ? v[u].x : 0.f;
          s[1] += there ? v[u].y : 0.f;
          s[2] += there ? v[u].z : 0.f;
          s[3] += there ? v[u].w : 0.f;
        }
      }
#pragma unroll
    for (int v = 0; v < 4; ++v) sum[k][4 * q + v] = s[v];
    __syncthreads();
    const int c = tid % 64, g = tid / 64 * 4;
    four[tid / 64][c] = ((sum[g][c] + sum[g + 1][c]) + sum[g + 2][c]) + sum[g + 3][c];
    __syncthreads();
    if (k == 0 && col < H) {
      float f[4];
#pragma unroll
      for (int v = 0; v < 4; ++v)
        f[v] = (float)(((four[0][4 * q + v] + four[1][4 * q + v]) + four[2][4 * q + v]) + four[3][4 * q + v]);
      if constexpr (DT == kF32)
        *reinterpret_cast<float4*>(static_cast<float*>(to) + row * H + col) = make_float4(f[0], f[1], f[2], f[3]);
      else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(to) + row * H + col) =
            make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
    }
  }
}

int threads(int nch, int cpl) { return ((nch + cpl - 1) / cpl + kWave - 1) / kWave * kWave; }

template <int DT, int SRC>
hipError_t launch_norm_typed(const NormArgs& a, hipStream_t s) {
  // two chunks a lane: fewer waves meet at a row's sums (4096 x 2048 bfloat16: 16.5 us, one
  // a lane 18.9, four 16.9; 8192 x 2816 with its combine: 100, 125, 201)
  const int cpl = a.nch <= kWave ? 1 : a.nch <= 1024 ? 2 : 4, n = threads(a.nch, cpl);
  if (cpl == 1) norm_kernel<DT, 1, SRC><<<row_grid(a.T), n, 0, s>>>(a);
  else if (cpl == 2) norm_kernel<DT, 2, SRC><<<row_grid(a.T), n, 0, s>>>(a);
  else norm_kernel<DT, 4, SRC><<<row_grid(a.T), n, 0, s>>>(a);
  return hipGetLastError();
}

template <int DT, bool BLOCK>
hipError_t launch_norm_bwd_typed(const NormBwdArgs& a, hipStream_t s) {
  if (a.runs > 0) {
    // a run's sums of two chunks of eight numbers a lane do not fit beside a row: rows of
    // more than 8192 after a block in two kernels (4096 x 8200 bfloat16: 178 us, in one 817;
    // 8192: 167 against 122; float32, 8196: 327, 8192: 295 against 254)
    if (BLOCK && a.nch * Elems<DT>::kPerChunk > kNormWide) {
      if (a.means) norm_means_kernel<DT><<<row_grid(a.T), a.nch >= 1024 ? 1024 : 512, 0, s>>>(a);
      norm_columns_kernel<DT><<<(a.nch + 255) / 256 * a.runs, 256, 0, s>>>(a);
    } else if (a.nch <= 512) norm_bwd_kernel<DT, 1, BLOCK, true, 512><<<a.runs, threads(a.nch, 1), 0, s>>>(a);
    else if (a.nch <= 1024) norm_bwd_kernel<DT, 2, BLOCK, false, 512><<<a.runs, threads(a.nch, 2), 0, s>>>(a);
    else if constexpr (!BLOCK || DT == kF32) {
      if (a.nch <= 2048) norm_bwd_kernel<DT, 2, BLOCK, false, 1024><<<a.runs, threads(a.nch, 2), 0, s>>>(a);
      else if constexpr (!BLOCK) norm_bwd_kernel<DT, 4, BLOCK, false, 1024><<<a.runs, threads(a.nch, 4), 0, s>>>(a);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const bool gates = a.gg && a.parts != 1;  // no part (an empty batch): zeros
  if (!a.gw1 && !a.gw2 && !gates) return hipSuccess;
  const int H = a.nch * Elems<DT>::kPerChunk;
  const int rows = !gates ? 0 : a.gates < kGateRows ? a.gates : kGateRows;
  norm_join_kernel<DT><<<dim3((H + 63) / 64, 2 + rows), 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
  const int src = !a.y ? kBefore : a.recv_pos ? kGather : kRows;
  if (a.dtype == kF32)
    return src == kBefore ? launch_norm_typed<kF32, kBefore>(a, s)
           : src == kRows ? launch_norm_typed<kF32, kRows>(a, s) : launch_norm_typed<kF32, kGather>(a, s);
  return src == kBefore ? launch_norm_typed<kBF16, kBefore>(a, s)
         : src == kRows ? launch_norm_typed<kBF16, kRows>(a, s) : launch_norm_typed<kBF16, kGather>(a, s);
}

template <int DT>
hipError_t launch_quant_typed(const NormArgs& a, hipStream_t s) {
  const int cpl = a.nch <= kWave ? 1 : a.nch <= 2 * kWave ? 2 : 4;
  const int64_t rows = 4 * (4 / cpl);  // of a workgroup
  const unsigned grid = (unsigned)((a.T + rows - 1) / rows);
  if (a.nch > 4 * kWave) quant_block_kernel<DT><<<row_grid(a.T), a.nch >= 1024 ? 1024 : 512, 0, s>>>(a);
  else if (cpl == 1) quant_wave_kernel<DT, 1><<<grid, 256, 0, s>>>(a);
  else if (cpl == 2) quant_wave_kernel<DT, 2><<<grid, 256, 0, s>>>(a);
  else quant_wave_kernel<DT, 4><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_quant(const NormArgs& a, hipStream_t s) {
  return a.dtype == kF32 ? launch_quant_typed<kF32>(a, s) : launch_quant_typed<kBF16>(a, s);
}

// Rows of a run, runs that share a gate, and runs in all: about 2048 waves (4096 x 2048
// bfloat16, four waves a row: 34 us with 512 runs, 44 with 256, 36 with 1024; 7168, eight
// waves: 110 with 256, 116 with 512).  Wide rows in two kernels have a wave for every 64
// chunks of a run: 128 runs (4096 x 8200: 178 us, 219 with 64, 183 with 512; 2048 x 16384:
// 168, 156, 170; 4096 x 12288: 227, 255, 246).  A run has at most 256 rows, more runs instead
// of longer ones past that, because its sums are in 32 bits (2^21 rows of 4 float32 alike in
// 1024 runs were off by 518 u of themselves, u = 2^-24; 2^18 x 2048 after a block: 1450 us so,
// 1310 with 512 runs, 2^19 x 2048 2660 both, 2^20 x 256 1080 and 1650).
void norm_bwd_plan(int64_t T, int64_t group, int nch, bool wide, int* rows, int* parts, int* runs) {
  if (T == 0) {
    *rows = *parts = *runs = 0;
    return;
  }
  const int waves = (nch + kWave - 1) / kWave, most = wide ? 128 : waves <= 2 ? 1024 : waves <= 4 ? 512 : 256;
  int64_t r = std::min<int64_t>((T + most - 1) / most, 256);
  if (group >= r) {
    *parts = (int)((group + r - 1) / r);
    if (*parts == 1) r = group;
    *runs = (int)(T / group * *parts);
  } else {
    r = r / group * group;  // whole gates
    *parts = 1;
    *runs = (int)((T + r - 1) / r);
  }
  *rows = (int)r;
}

hipError_t launch_norm_bwd(const NormBwdArgs& a, hipStream_t s) {
  const bool block = a.block;
  if (a.dtype == kF32) return block ? launch_norm_bwd_typed<kF32, true>(a, s) : launch_norm_bwd_typed<kF32, false>(a, s);
  return block ? launch_norm_bwd_typed<kBF16, true>(a, s) : launch_norm_bwd_typed<kBF16, false>(a, s);
}

}  // namespace moe
