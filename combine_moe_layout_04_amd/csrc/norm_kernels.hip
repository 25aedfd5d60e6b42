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
// once.  Sums over a row: each wave's by lane moves, then the waves' in order through
// LDS.  Sums over tokens: a workgroup's run in registers, one partial for each run,
// the partials added in the order of the runs by a second kernel, so that results do
// not depend on timing.
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
  for (int i = 0; i < N; ++i) ss += f[i] * f[i];
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

template <int DT, int CPL, int SRC>
__global__ __launch_bounds__(Block<CPL>::kMax) void norm_kernel(NormArgs a) {
  constexpr int V = Elems<DT>::kPerChunk;
  __shared__ float red[7][kMaxWaves];
  const int t = blockIdx.x, tid = threadIdx.x, H = a.nch * V;
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
  load(a.x, row, c);
  floats(c, x);
  float r1 = 1.f, r2 = 1.f;
  if constexpr (SRC != kBefore) {
    if constexpr (SRC == kRows) {
      load(a.y, row, c);
      floats(c, f);
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
      load(a.w1, 0, c);
      float w[CPL * V];
      floats(c, w);
#pragma unroll
      for (int i = 0; i < CPL * V; ++i) f[i] = f[i] * r1 * (w[i] + a.offset);
    }
    if (a.gate) {
      load(a.gate, (size_t)(t / a.group) * a.nch, c);
      float w[CPL * V];
      floats(c, w);
#pragma unroll
      for (int i = 0; i < CPL * V; ++i) f[i] *= w[i];
    }
#pragma unroll
    for (int i = 0; i < CPL * V; ++i) x[i] = a.residual * x[i] + f[i];
    store(a.out, x);
  }
  if (a.w2) {
    r2 = block_rstd(x, H, a.eps, red[3], red[4], red[5]);
    load(a.w2, 0, c);
    float w[CPL * V];
    floats(c, w);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < CPL * V; ++i) {
      x[i] = x[i] * r2 * (w[i] + a.offset);
      top = max(top, abs_bits(x[i]));
    }
    if (a.q) {
      const float s = quant_scale(block_max(top, red[6])), inv = 1.f / s;
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

// A wave per row where a row has at most 256 chunks (4 a lane), else a workgroup.
template <int DT>
__global__ __launch_bounds__(256) void quant_wave_kernel(NormArgs a) {
  constexpr int V = Elems<DT>::kPerChunk, CPL = 4;
  const int64_t t = (int64_t)blockIdx.x * 4 + threadIdx.x / kWave;
  if (t >= a.T) return;  // wave-uniform
  const int lane = lane_id();
  const u32x4* p = static_cast<const u32x4*>(a.x) + (size_t)t * a.nch;
  u32x4 c[CPL];
#pragma unroll
  for (int i = 0; i < CPL; ++i) {
    const int j = lane + i * kWave;
    c[i] = j < a.nch ? p[j] : u32x4{0, 0, 0, 0};
  }
  float f[CPL * V];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < CPL; ++i) unpack<DT>(c[i], f + i * V);
#pragma unroll
  for (int i = 0; i < CPL * V; ++i) top = max(top, abs_bits(f[i]));
  const float s = quant_scale(wave_max(top)), inv = 1.f / s;
#pragma unroll
  for (int i = 0; i < CPL; ++i) {
    const int j = lane + i * kWave;
    if (j < a.nch) store_quant<V>(a.q + (size_t)t * a.nch * V, j, f + i * V, s, inv);
  }
  if (lane == 0) a.scale[t] = s;
}

template <int DT>
__global__ __launch_bounds__(1024) void quant_block_kernel(NormArgs a) {
  constexpr int V = Elems<DT>::kPerChunk;
  __shared__ float red[kMaxWaves];
  const size_t t = blockIdx.x;
  const u32x4* p = static_cast<const u32x4*>(a.x) + t * a.nch;
  uint32_t top = 0;
  for (int j = threadIdx.x; j < a.nch; j += blockDim.x) {
    float f[V];
    unpack<DT>(p[j], f);
#pragma unroll
    for (int i = 0; i < V; ++i) top = max(top, abs_bits(f[i]));
  }
  const float s = quant_scale(block_max(top, red)), inv = 1.f / s;
  for (int j = threadIdx.x; j < a.nch; j += blockDim.x) {  // the row again, from the caches
    float f[V];
    unpack<DT>(p[j], f);
    store_quant<V>(a.q + t * a.nch * V, j, f, s, inv);
  }
  if (threadIdx.x == 0) a.scale[t] = s;
}

// ---- backward ---------------------------------------------------------------------

template <int DT, int CPL, bool BLOCK>
__global__ __launch_bounds__(Block<CPL>::kMax) void norm_bwd_kernel(NormBwdArgs a) {
  constexpr int V = Elems<DT>::kPerChunk, N = CPL * V;
  __shared__ float red[4][kMaxWaves];
  const int tid = threadIdx.x, run = blockIdx.x, H = a.nch * V;
  // the run's rows: a part of one gate's tokens, or whole gates
  int64_t t0, t1;
  if (a.parts > 1) {
    const int64_t group = run / a.parts, part = run % a.parts;
    t0 = group * a.group + part * a.rows;
    t1 = min(t0 + a.rows, (group + 1) * a.group);
  } else {
    t0 = (int64_t)run * a.rows;
    t1 = min(t0 + a.rows, (int64_t)a.T);
  }
  const u32x4 zero = {0, 0, 0, 0};
  auto chunks = [&](const void* p, size_t row, u32x4(&to)[CPL]) {
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      const int j = tid + i * blockDim.x;
      to[i] = p && j < a.nch ? static_cast<const u32x4*>(p)[row * a.nch + j] : zero;
    }
  };
  auto floats = [&](const u32x4(&from)[CPL], float(&to)[N]) {
#pragma unroll
    for (int i = 0; i < CPL; ++i) unpack<DT>(from[i], to + i * V);
  };
  auto store = [&](void* p, size_t row, const float(&from)[N]) {
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      const int j = tid + i * blockDim.x;
      if (j < a.nch) static_cast<u32x4*>(p)[row * a.nch + j] = pack<DT>(from + i * V);
    }
  };
  auto partial = [&](float* p, size_t at, const float(&from)[N]) {
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      const int j = tid + i * blockDim.x;
      if (j < a.nch)
#pragma unroll
        for (int v = 0; v < V; v += 4)
          *reinterpret_cast<float4*>(p + at * H + (size_t)j * V + v) =
              make_float4(from[i * V + v], from[i * V + v + 1], from[i * V + v + 2], from[i * V + v + 3]);
    }
  };
  // What a row reads: asked for a row ahead, so that it arrives during the sums of the
  // row before it.
  struct Row {
    u32x4 g[CPL], gn[CPL], x[CPL], y[CPL], gate[CPL];
    float r1, r2;
  };
  auto fetch = [&](int64_t t, Row& r) {
    chunks(a.g, t, r.g);
    chunks(a.gn, t, r.gn);
    chunks(a.gn ? a.x : nullptr, t, r.x);
    r.r1 = 1.f;
    if constexpr (BLOCK) {
      chunks(a.y, t, r.y);
      chunks(a.gate, t / a.group, r.gate);
      r.r1 = a.rstd[2 * t];
      r.r2 = a.rstd[2 * t + 1];
    } else {
      r.r2 = a.rstd[t];
    }
  };
  float s1[N], s2[N], sg[N];  // sums over the run
#pragma unroll
  for (int i = 0; i < N; ++i) s1[i] = s2[i] = sg[i] = 0.f;
  float w1[N], w2[N];
  u32x4 c[CPL];
  chunks(BLOCK ? a.w1 : nullptr, 0, c);
  floats(c, w1);
  chunks(a.w2, 0, c);
  floats(c, w2);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    w1[i] += a.offset;
    w2[i] += a.offset;
  }
  Row next;
  if (t0 < t1) fetch(t0, next);
  for (int64_t t = t0; t < t1; ++t) {
    const Row r = next;
    if (t + 1 < t1) fetch(t + 1, next);
    const int odd = (int)(t - t0) & 1;  // two rows' sums lie apart: one barrier a sum
    float d[N], y[N], o[N], g[N];
    floats(r.g, d);
    if constexpr (BLOCK) {
      floats(r.y, y);
      floats(r.gate, g);
#pragma unroll
      for (int i = 0; i < N; ++i) y[i] *= r.r1;
    }
    if (a.gn) {
      float gn[N];
      floats(r.gn, gn);
      floats(r.x, o);
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if constexpr (BLOCK) {  // z again, as the forward pass had it
          float f = a.w1 ? y[i] * w1[i] : y[i];
          if (a.gate) f *= g[i];
          o[i] = a.residual * o[i] + f;
        }
        o[i] *= r.r2;
        s2[i] += gn[i] * o[i];
        gn[i] *= w2[i];
        dot += gn[i] * o[i];
      }
      dot = block_sum(dot, red[odd]) / (float)H;
#pragma unroll
      for (int i = 0; i < N; ++i) d[i] += r.r2 * (gn[i] - o[i] * dot);
    }
    if constexpr (!BLOCK) {
      if (a.gx) store(a.gx, t, d);
      continue;
    }
    if (a.gx) {
      float gx[N];
#pragma unroll
      for (int i = 0; i < N; ++i) gx[i] = a.residual * d[i];
      store(a.gx, t, gx);
    }
    if (a.gate) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (a.gg) sg[i] += d[i] * (a.w1 ? y[i] * w1[i] : y[i]);
        d[i] *= g[i];
      }
    }
    if (a.w1) {
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        s1[i] += d[i] * y[i];
        d[i] *= w1[i];
        dot += d[i] * y[i];
      }
      dot = block_sum(dot, red[2 + odd]) / (float)H;
#pragma unroll
      for (int i = 0; i < N; ++i) d[i] = r.r1 * (d[i] - y[i] * dot);
    }
    if (a.gy) store(a.gy, t, d);
    if (a.gg && a.parts == 1 && (t + 1) % a.group == 0) {  // the gate's last token
      store(a.gg, t / a.group, sg);
#pragma unroll
      for (int i = 0; i < N; ++i) sg[i] = 0.f;
    }
  }
  if (a.part1) partial(a.part1, run, s1);
  if (a.part2) partial(a.part2, run, s2);
  if (a.gg && a.parts > 1) partial(a.partg, run, sg);
}

// Adds partials: blockIdx.y 0 the next norm's weight, 1 the post-norm's, 2.. the gates.
// 64 columns a workgroup, four a thread; a sixteenth of the partials each.
template <int DT>
__global__ __launch_bounds__(256) void norm_join_kernel(NormBwdArgs a) {
  __shared__ float4 sum[16][16];
  const int H = a.nch * Elems<DT>::kPerChunk;
  const int q = threadIdx.x % 16, k = threadIdx.x / 16, col = blockIdx.x * 64 + 4 * q;
  const float* from;
  void* to;
  int n = a.runs;
  size_t row = 0;
  if (blockIdx.y == 0) {
    from = a.part2;
    to = a.gw2;
  } else if (blockIdx.y == 1) {
    from = a.part1;
    to = a.gw1;
  } else {
    row = blockIdx.y - 2;
    from = a.partg + row * a.parts * H;
    to = a.gg;
    n = a.parts;
  }
  if (!to) return;  // uniform
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (col < H) {
#pragma unroll 8
    for (int i = k; i < n; i += 16) {
      const float4 v = *reinterpret_cast<const float4*>(from + (size_t)i * H + col);
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
  }
  sum[k][q] = s;
  __syncthreads();
  if (k != 0 || col >= H) return;
  for (int i = 1; i < 16; ++i) {
    const float4 v = sum[i][q];
    s.x += v.x;
    s.y += v.y;
    s.z += v.z;
    s.w += v.w;
  }
  if constexpr (DT == kF32)
    *reinterpret_cast<float4*>(static_cast<float*>(to) + row * H + col) = s;
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(to) + row * H + col) = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
}

int chunks_per_lane(int nch) { return nch <= 512 ? 1 : nch <= 1024 ? 2 : 4; }
int threads(int nch, int cpl) { return ((nch + cpl - 1) / cpl + kWave - 1) / kWave * kWave; }

template <int DT, int SRC>
hipError_t launch_norm_typed(const NormArgs& a, hipStream_t s) {
  const int cpl = chunks_per_lane(a.nch), n = threads(a.nch, cpl);
  if (cpl == 1) norm_kernel<DT, 1, SRC><<<a.T, n, 0, s>>>(a);
  else if (cpl == 2) norm_kernel<DT, 2, SRC><<<a.T, n, 0, s>>>(a);
  else norm_kernel<DT, 4, SRC><<<a.T, n, 0, s>>>(a);
  return hipGetLastError();
}

template <int DT, bool BLOCK>
hipError_t launch_norm_bwd_typed(const NormBwdArgs& a, hipStream_t s) {
  const int cpl = chunks_per_lane(a.nch), n = threads(a.nch, cpl);
  if (a.runs > 0) {
    if (cpl == 1) norm_bwd_kernel<DT, 1, BLOCK><<<a.runs, n, 0, s>>>(a);
    else if (cpl == 2) norm_bwd_kernel<DT, 2, BLOCK><<<a.runs, n, 0, s>>>(a);
    else norm_bwd_kernel<DT, 4, BLOCK><<<a.runs, n, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const bool gates = a.gg && a.parts != 1;  // no part (an empty batch): zeros
  if (!a.gw1 && !a.gw2 && !gates) return hipSuccess;
  const int H = a.nch * Elems<DT>::kPerChunk;
  norm_join_kernel<DT><<<dim3((H + 63) / 64, gates ? 2 + a.gates : 2), 256, 0, s>>>(a);
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

hipError_t launch_quant(const NormArgs& a, hipStream_t s) {
  if (a.nch <= 4 * kWave) {
    const unsigned grid = (unsigned)(((int64_t)a.T + 3) / 4);
    if (a.dtype == kF32) quant_wave_kernel<kF32><<<grid, 256, 0, s>>>(a);
    else quant_wave_kernel<kBF16><<<grid, 256, 0, s>>>(a);
  } else {
    const int n = a.nch >= 1024 ? 1024 : 512;
    if (a.dtype == kF32) quant_block_kernel<kF32><<<a.T, n, 0, s>>>(a);
    else quant_block_kernel<kBF16><<<a.T, n, 0, s>>>(a);
  }
  return hipGetLastError();
}

// Rows of a run, runs that share a gate, and runs in all.
void norm_bwd_plan(int64_t T, int64_t group, int* rows, int* parts, int* runs) {
  if (T == 0) {
    *rows = *parts = *runs = 0;
    return;
  }
  int64_t r = (T + 511) / 512;
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
