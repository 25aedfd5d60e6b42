// The balance loss and the z loss of a router, per-expert counts, and the
// gradient back to the logits.
//
//   s = softmax(z), or sigmoid(z) divided by the token's sum of them;
//   c[q,e] = pairs of sequence q's tokens with expert e, P[q,e] = sum of s[t,e],
//   n_q = its counted tokens, S' = sequences with any, n = all counted tokens:
//   balance = 1/S' sum_q E / (K n_q^2) sum_e c[q,e] P[q,e]
//   z       = 1/n sum_t lse(z_t)^2
//   a_e = g0 E / (S' K n_q^2) c[q,e]  (the counts have no gradient):
//   dz_j = s_j (1 - sigmoid(z_j) where the scores are sigmoids) (a_j - sum_m s_m a_m)
//          + g1 2/n lse softmax(z)_j
//
// One wavefront per token, its E values in registers (lane-strided), as in the
// router.  A workgroup takes a run of tokens; a run that meets several sequences
// leaves one partial for each.  Run w and sequence q use slot w + q: from one
// meeting to the next w or q grows, so no two share a slot and W + S slots are
// enough, without knowing on the host how long the sequences are.  The second
// kernel adds a sequence's slots in the order of the runs, so results do not
// depend on timing; whole numbers are counted with LDS atomics.  Its last
// workgroup to finish forms the losses.
//
// Sigmoid scores are formed relative to the largest one where all lie below
// 0.5: their share of the sum is right however small they are.  As in the router
// those below 2^-1022 (z < -708) count as zero.  A token whose scores are all
// zero (every logit -inf) has s = 0, no part in the z loss and no gradient.
#include "device_common.h"
#include "internal.h"
#include "../../include/moe_layout.h"

namespace moe {
namespace {

constexpr int kWaves = 4;          // of a workgroup of the first kernel and of the backward
constexpr int kCols = 32;          // experts of a workgroup of the second kernel
constexpr int kGroups = 32;        // slots it adds at once

template <int DT>
__device__ __forceinline__ float load_logit(const void* z, size_t i) {
  if constexpr (DT == kF32) return static_cast<const float*>(z)[i];
  return __uint_as_float((uint32_t)static_cast<const uint16_t*>(z)[i] << 16);
}

// Sequence q's tokens, inside [0, T) whatever the offsets hold.
__device__ __forceinline__ int seq_begin(const BalanceArgs& a, int q) {
  return a.seq ? min(max(a.seq[q], 0), a.T) : 0;
}
__device__ __forceinline__ int seq_end(const BalanceArgs& a, int q) {
  return a.seq ? min(max(a.seq[q + 1], 0), a.T) : a.T;
}

// Sequences that end at or before token t, S at most: 64 ends a step.
__device__ __forceinline__ int sequences_before(const BalanceArgs& a, int t) {
  if (!a.seq) return 0;
  int lo = 0, n = a.S;  // the answer lies in [lo, lo + n]
  while (n > 0) {
    const int step = (n + kWave - 1) / kWave;
    const int last = (lane_id() + 1) * step;  // this lane's block ends with the last-th of them
    const bool before = last <= n && seq_end(a, lo + last - 1) <= t;
    const int full = __popcll(__ballot(before)) * step;
    lo += full;
    n = min(step - 1, n - full);
  }
  return lo;
}

__device__ __forceinline__ float wave_maxf(float v) {  // a NaN among others is passed over
  v = fmaxf(v, __shfl_xor(v, 32, kWave));
#pragma unroll
  for (int s = 16; s >= 1; s >>= 1) v = fmaxf(v, __shfl_xor(v, s, kWave));
  return v;
}

// One token's softmax, its lse, and its scores (p is soft itself for softmax).
template <int VPL, bool SIG>
__device__ __forceinline__ void scores(const float (&z)[VPL], float (&soft)[VPL], float (&p)[VPL], float& lse) {
  float m = z[0];
#pragma unroll
  for (int v = 1; v < VPL; ++v) m = fmaxf(m, z[v]);
  m = wave_maxf(m);
  if (m == -INFINITY) m = 0.f;
  float sum = 0.f;
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    soft[v] = expf(z[v] - m);
    sum += soft[v];
  }
  sum = wave_sum(sum);
  lse = sum == 0.f ? 0.f : m + logf(sum);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  if constexpr (SIG) {
    float all = 0.f;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      // m > 0: the sigmoid itself; else relative to the largest logit
      const float top = m > 0.f ? expf(-fabsf(z[v])) : soft[v];
      const float bottom = m > 0.f ? top : expf(z[v]);
      p[v] = z[v] < -708.f ? 0.f : (m > 0.f && z[v] > 0.f ? 1.f : top) / (1.f + bottom);
      all += p[v];
    }
    all = wave_sum(all);
    const float share = all == 0.f ? 0.f : 1.f / all;
#pragma unroll
    for (int v = 0; v < VPL; ++v) p[v] *= share;
  }
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    soft[v] *= inv;
    if constexpr (!SIG) p[v] = soft[v];
  }
}

template <int DT, int VPL>
__device__ __forceinline__ void load_token(const BalanceArgs& a, int t, float (&z)[VPL]) {
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const int e = lane_id() + kWave * v;
    z[v] = e < a.E ? load_logit<DT>(a.z, (size_t)t * a.E + e) : -INFINITY;
  }
}

__device__ __forceinline__ bool counted(const BalanceArgs& a, int t) { return !a.mask || a.mask[t] != 0; }

template <int DT, int VPL, bool SIG>
__global__ __launch_bounds__(kWaves * kWave) void balance_kernel(BalanceArgs a) {
  __shared__ int hist[kWave * VPL];
  __shared__ float psum[kWaves][kWave * VPL];
  __shared__ float zsum[kWaves];
  __shared__ int nsum[kWaves];
  const int lane = lane_id(), wave = (int)(threadIdx.x / kWave);
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0u;
  const int t0 = blockIdx.x * a.tile, t1 = (int)min((int64_t)a.T, (int64_t)t0 + a.tile);
  for (int q = sequences_before(a, t0); q < a.S; ++q) {  // uniform over the workgroup
    const int begin = seq_begin(a, q);
    if (begin >= t1) break;
    const int lo = max(t0, begin), hi = min(t1, seq_end(a, q));
    if (lo >= hi) continue;
    for (int e = threadIdx.x; e < a.E; e += kWaves * kWave) hist[e] = 0;
    __syncthreads();
    float p[VPL], zz = 0.f;
    int n = 0;
#pragma unroll
    for (int v = 0; v < VPL; ++v) p[v] = 0.f;
    float z[VPL], next[VPL];
    if (lo + wave < hi) load_token<DT, VPL>(a, lo + wave, next);
    for (int t = lo + wave; t < hi; t += kWaves) {  // wave-uniform
#pragma unroll
      for (int v = 0; v < VPL; ++v) z[v] = next[v];
      if (t + kWaves < hi) load_token<DT, VPL>(a, t + kWaves, next);
      if (!counted(a, t)) continue;
      float soft[VPL], s[VPL], lse;
      scores<VPL, SIG>(z, soft, s, lse);
#pragma unroll
      for (int v = 0; v < VPL; ++v) p[v] += s[v];
      zz += lse * lse;
      ++n;
    }
    const int pairs = (hi - lo) * a.K;  // at most tile * K
    for (int i = threadIdx.x; i < pairs; i += kWaves * kWave) {
      const int t = lo + i / a.K;
      if (!counted(a, t)) continue;
      const size_t at = (size_t)lo * a.K + i;
      const int64_t e = a.itype == MOE_I32 ? (int64_t) static_cast<const int32_t*>(a.idx)[at]
                                           : static_cast<const int64_t*>(a.idx)[at];
      if (e >= 0 && e < a.E) atomicAdd(&hist[(int)e], 1);
    }
#pragma unroll
    for (int v = 0; v < VPL; ++v) psum[wave][lane + kWave * v] = p[v];
    if (lane == 0) {
      zsum[wave] = zz;
      nsum[wave] = n;
    }
    __syncthreads();
    const size_t slot = (size_t)blockIdx.x + q;
    for (int e = threadIdx.x; e < a.E; e += kWaves * kWave) {
      float s = psum[0][e];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) s += psum[w][e];
      a.part_p[slot * a.E + e] = s;
      a.part_c[slot * a.E + e] = hist[e];
    }
    if (threadIdx.x == 0) {
      float s = zsum[0];
      int c = nsum[0];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) {
        s += zsum[w];
        c += nsum[w];
      }
      a.part_z[slot] = s;
      a.part_n[slot] = c;
    }
    __syncthreads();
  }
}

// Sum over the workgroup of 1024 threads, in a fixed order, in every thread.
__device__ __forceinline__ double block_sum(double v, double* shared) {
#pragma unroll
  for (int s = 32; s >= 1; s >>= 1) v += __shfl_xor(v, s, kWave);
  __syncthreads();
  if (lane_id() == 0) shared[threadIdx.x / kWave] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int w = 0; w < 16; ++w) v += shared[w];
  return v;
}

// Sequence blockIdx.y, experts from blockIdx.x * kCols on.
__global__ __launch_bounds__(1024) void balance_finish_kernel(BalanceArgs a) {
  __shared__ double sp[kGroups][kCols];
  __shared__ int sc[kGroups][kCols];
  __shared__ double sums[16];
  __shared__ bool last;
  const int q = blockIdx.y, col = threadIdx.x % kCols, g = threadIdx.x / kCols;
  const int e = blockIdx.x * kCols + col;
  const int lo = seq_begin(a, q), hi = seq_end(a, q);
  const int w0 = lo < hi ? lo / a.tile : 0, w1 = lo < hi ? (hi - 1) / a.tile : -1;
  double p = 0.0;
  int c = 0;
  if (e < a.E)
    for (int w = w0 + g; w <= w1; w += kGroups) {
      const size_t at = (size_t)(w + q) * a.E + e;
      p += a.part_p[at];
      c += a.part_c[at];
    }
  sp[g][col] = p;
  sc[g][col] = c;
  __syncthreads();
  double product = 0.0;
  if (g == 0) {
    for (int k = 1; k < kGroups; ++k) {
      p += sp[k][col];
      c += sc[k][col];
    }
    if (e < a.E) {
      a.probs[(size_t)q * a.E + e] = (float)p;
      a.counts[(size_t)q * a.E + e] = c;
      product = p * c;
    }
  }
  product = block_sum(product, sums);
  double z = 0.0, n = 0.0;
  if (blockIdx.x == 0) {  // uniform
    for (int w = w0 + (int)threadIdx.x; w <= w1; w += 1024) {
      z += a.part_z[w + q];
      n += a.part_n[w + q];
    }
    z = block_sum(z, sums);
    n = block_sum(n, sums);  // whole numbers: exact
  }
  if (threadIdx.x == 0) {
    a.seq_sum[(size_t)q * gridDim.x + blockIdx.x] = product;
    if (blockIdx.x == 0) {
      a.seq_z[q] = z;
      a.tokens[q] = (int)n;
    }
    __threadfence();
    last = atomicAdd(a.ticket, 1u) == gridDim.x * gridDim.y - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  double sum = 0.0, all = 0.0, some = 0.0, zz = 0.0;
  for (int r = threadIdx.x; r < a.S; r += 1024) {
    const double nq = a.tokens[r];
    if (nq <= 0) continue;
    double s = 0.0;
    for (unsigned b = 0; b < gridDim.x; ++b) s += a.seq_sum[(size_t)r * gridDim.x + b];
    sum += s / (nq * nq);
    zz += a.seq_z[r];
    all += nq;
    some += 1.0;
  }
  sum = block_sum(sum, sums);
  zz = block_sum(zz, sums);
  all = block_sum(all, sums);
  some = block_sum(some, sums);
  if (threadIdx.x == 0) {
    a.loss[0] = some > 0 ? (float)(sum * a.E / (a.K * some)) : 0.f;
    a.loss[1] = all > 0 ? (float)(zz / all) : 0.f;
  }
}

template <int DT, int VPL, bool SIG>
__global__ __launch_bounds__(kWaves * kWave) void balance_bwd_kernel(BalanceArgs a) {
  const int lane = lane_id();
  const int64_t first = ((int64_t)blockIdx.x * kWaves + threadIdx.x / kWave) * a.tile;  // tile: tokens of a wave
  const int t0 = (int)min((int64_t)a.T, first), t1 = (int)min((int64_t)a.T, first + a.tile);
  if (t0 >= t1) return;
  int all = 0, some = 0;
  for (int q = lane; q < a.S; q += kWave) {
    const int n = a.tokens[q];
    all += n;
    some += n > 0;
  }
  all = read_lane_i((int)wave_scan((uint32_t)all), 63);
  some = read_lane_i((int)wave_scan((uint32_t)some), 63);
  const float g0 = a.grad_loss[0], g1 = all > 0 ? a.grad_loss[1] * (float)(2.0 / all) : 0.f;
  int q = sequences_before(a, t0), at = -1;
  int begin = q < a.S ? seq_begin(a, q) : a.T, end = q < a.S ? seq_end(a, q) : a.T;
  float c[VPL];  // the gradient of P of the sequence `at`
  float z[VPL], next[VPL];
  load_token<DT, VPL>(a, t0, next);
  for (int t = t0; t < t1; ++t) {
#pragma unroll
    for (int v = 0; v < VPL; ++v) z[v] = next[v];
    if (t + 1 < t1) load_token<DT, VPL>(a, t + 1, next);
    while (q < a.S && end <= t) {
      ++q;
      begin = q < a.S ? seq_begin(a, q) : a.T;
      end = q < a.S ? seq_end(a, q) : a.T;
    }
    float d[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) d[v] = 0.f;
    if (q < a.S && begin <= t && counted(a, t)) {  // wave-uniform
      if (q != at) {
        at = q;
        const double n = a.tokens[q];
        const float f = n > 0 ? (float)((double)a.E / ((double)a.K * some * n * n)) : 0.f;
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
          const int e = lane + kWave * v;
          c[v] = e < a.E ? g0 * (f * (float)a.counts[(size_t)q * a.E + e]) : 0.f;
        }
      }
      float soft[VPL], p[VPL], lse, dot = 0.f;
      scores<VPL, SIG>(z, soft, p, lse);
#pragma unroll
      for (int v = 0; v < VPL; ++v) dot += p[v] * c[v];
      dot = wave_sum(dot);
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        float s = p[v];
        if constexpr (SIG) {  // 1 - sigmoid(z)
          const float e = expf(-fabsf(z[v]));
          s *= (z[v] > 0.f ? e : 1.f) / (1.f + e);
        }
        d[v] = s * (c[v] - dot) + g1 * lse * soft[v];
      }
    }
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int e = lane + kWave * v;
      if (e < a.E) {
        const size_t i = (size_t)t * a.E + e;
        if (a.grad_base) d[v] += load_logit<DT>(a.grad_base, i);
        if constexpr (DT == kF32) static_cast<float*>(a.grad_z)[i] = d[v];
        else static_cast<uint16_t*>(a.grad_z)[i] = (uint16_t)f32_to_bf16(d[v]);
      }
    }
  }
}

template <int DT, int VPL, bool SIG>
hipError_t launch_one(const BalanceArgs& a, bool backward, dim3 grid, hipStream_t s) {
  if (backward) balance_bwd_kernel<DT, VPL, SIG><<<grid, kWaves * kWave, 0, s>>>(a);
  else balance_kernel<DT, VPL, SIG><<<grid, kWaves * kWave, 0, s>>>(a);
  return hipGetLastError();
}

template <int DT, bool SIG>
hipError_t launch_width(const BalanceArgs& a, bool backward, dim3 grid, hipStream_t s) {
  if (a.E <= 64) return launch_one<DT, 1, SIG>(a, backward, grid, s);
  if (a.E <= 128) return launch_one<DT, 2, SIG>(a, backward, grid, s);
  if (a.E <= 256) return launch_one<DT, 4, SIG>(a, backward, grid, s);
  if (a.E <= 512) return launch_one<DT, 8, SIG>(a, backward, grid, s);
  return launch_one<DT, 16, SIG>(a, backward, grid, s);
}

hipError_t launch_typed(const BalanceArgs& a, bool backward, dim3 grid, hipStream_t s) {
  const bool sig = a.score == MOE_SCORE_SIGMOID;
  if (a.dtype == kF32) return sig ? launch_width<kF32, true>(a, backward, grid, s) : launch_width<kF32, false>(a, backward, grid, s);
  return sig ? launch_width<kBF16, true>(a, backward, grid, s) : launch_width<kBF16, false>(a, backward, grid, s);
}

}  // namespace

int balance_tile(int64_t T) {
  const int64_t t = (T + 511) / 512;
  return (int)(t < 4 ? 4 : t);
}
int balance_runs(int64_t T) { return T > 0 ? (int)((T + balance_tile(T) - 1) / balance_tile(T)) : 1; }
int balance_columns(int E) { return (E + kCols - 1) / kCols; }

hipError_t launch_balance(BalanceArgs a, hipStream_t s) {
  a.tile = balance_tile(a.T);
  const hipError_t e = launch_typed(a, false, dim3(balance_runs(a.T)), s);
  if (e != hipSuccess) return e;
  balance_finish_kernel<<<dim3(balance_columns(a.E), a.S), 1024, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_balance_bwd(BalanceArgs a, hipStream_t s) {
  const int64_t most = 2048 * kWaves;  // waves
  a.tile = (int)((a.T + most - 1) / most);
  const int64_t waves = ((int64_t)a.T + a.tile - 1) / a.tile;
  return launch_typed(a, true, dim3((unsigned)((waves + kWaves - 1) / kWaves)), s);
}

}  // namespace moe
