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
// depend on timing (whole numbers are counted with LDS atomics), and a third the
// sequences' losses; where there is one sequence of few partials the second does
// that too.  (The last workgroup of the second kernel forming them, by a counter,
// took 18 us against 4: its fences write back and drop the L2s.)
//
// Sigmoid scores are formed relative to the largest one where all lie below
// 0.5: their share of the sum is right however small they are.  As in the router
// those below 2^-1022 (z < -708) count as zero.  A token whose scores are all
// zero (every logit -inf) has s = 0, no part in the z loss and no gradient.
//
// Bound by latency and instruction issue, not by its bytes.  Measured (MI355X, kernels):
// 4096 tokens of 128 experts 5.8 + 6.0 us forward, 5.3 backward (1.1 MB read by each);
// 16384 tokens of 256 experts in 24 sequences, sigmoid, float32: 14.2 + 5.1 + 4.5 forward
// (17 MB read), 16.2 backward (34 MB).  A run works through the sequences that it meets one by
// one, about 2 us each: 65535 tokens, each a sequence, 548 + 64 + 47 and 51.
#include "device_common.h"
#include "internal.h"
#include "../../include/moe_layout.h"

namespace moe {
namespace {

constexpr int kWaves = 4;     // of a workgroup of the backward
constexpr int kRuns = 256;    // workgroups of the first kernel: one a CU
constexpr int kAdded = 128;   // tokens that a wave adds in 32 bits at most
constexpr int kCols = 32;     // experts of a workgroup of the second kernel, if there is more than one
constexpr int kDirect = 1 << 15;  // values of a kind that one workgroup adds by itself

// Waves of a workgroup of the first kernel; the sums of all of them lie in LDS, 68 KiB of it
// with 1024 experts.  (Forward kernels with 16 waves and with 4: 16384 tokens of 320 experts
// 23.7 and 42.1 us, of 768 35.6 and 76.7, of 1024 in float32 28.7 and 33.0; 100 tokens of 320
// 11.3 and 15.8.)
constexpr int kRunWaves = 16;

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

// exp(x) for x <= 0 to 3 u of itself (u = 2^-24), below 2^-126 zero: the product with
// log2(e) in two parts, of which the hardware's exponential takes the first.  (That one
// alone is off by (|x| + 2) u.  16384 tokens of 256 experts, sigmoid, forward and backward
// kernels: 23.5 + 15.5 us; with expf and divisions 25.4 + 17.4; the first part alone 21.7 +
// 13.8.)
__device__ __forceinline__ float exp_below(float x) {
  x = x < -200.f ? -200.f : x;  // -inf has no second part
  float t;
  const float rest = exp_parts(x, t), e = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(e, rest, e);
}

// One token's softmax, its lse, its scores (p is soft itself for softmax) and, for
// sigmoids, 1 - sigmoid in rest.
template <int VPL, bool SIG>
__device__ __forceinline__ void scores(const float (&z)[VPL], float (&soft)[VPL], float (&p)[VPL], float (&rest)[VPL],
                                       float& lse) {
  float m = z[0];
#pragma unroll
  for (int v = 1; v < VPL; ++v) m = fmaxf(m, z[v]);
  m = wave_max(m);
  if (m == -INFINITY) m = 0.f;
  float sum = 0.f;
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    soft[v] = exp_below(z[v] - m);
    sum += soft[v];
  }
  sum = wave_sum(sum);
  lse = sum == 0.f ? 0.f : m + logf(sum);
  if (m == INFINITY) {  // its differences are NaN; the same in every lane
    bool nan = false;
#pragma unroll
    for (int v = 0; v < VPL; ++v) nan |= z[v] != z[v];
    if (!__any(nan)) lse = m;
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  if constexpr (SIG) {
    float all = 0.f;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      // above 0 the sigmoid itself; where all lie below, relative to the largest logit
      const float e = exp_below(-fabsf(z[v])), d = 1.f + e;  // 1 / d: about, and one step nearer
      const float near = __builtin_amdgcn_rcpf(d);
      const float q = __builtin_fmaf(__builtin_fmaf(-d, near, 1.f), near, near);
      const bool positive = z[v] > 0.f;
      const float top = m > 0.f ? (positive ? 1.f : e) : soft[v];
      p[v] = z[v] < -708.f ? 0.f : top * q;
      rest[v] = (positive ? e : 1.f) * q;
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
    if constexpr (!SIG) {
      p[v] = soft[v];
      rest[v] = 1.f;
    }
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
__global__ __launch_bounds__(kRunWaves * kWave) void balance_kernel(BalanceArgs a) {
  constexpr int kWaves = kRunWaves;
  __shared__ int hist[kWave * VPL];
  __shared__ float psum[kWaves][kWave * VPL];
  __shared__ float zsum[kWaves];
  __shared__ int nsum[kWaves];
  const int lane = lane_id(), wave = (int)(threadIdx.x / kWave);
  const int t0 = blockIdx.x * a.tile, t1 = (int)min((int64_t)a.T, (int64_t)t0 + a.tile);
  for (int q = sequences_before(a, t0); q < a.S; ++q) {  // uniform over the workgroup
    const int begin = seq_begin(a, q);
    if (begin >= t1) break;
    const int lo = max(t0, begin), hi = min(t1, seq_end(a, q));
    if (lo >= hi) {  // empty, as any number after it may be
      q = max(q, sequences_before(a, lo) - 1);
      continue;
    }
    for (int e = threadIdx.x; e < a.E; e += kWaves * kWave) hist[e] = 0;
    __syncthreads();
    float p[VPL], zz = 0.f;
    int n = 0;
#pragma unroll
    for (int v = 0; v < VPL; ++v) p[v] = 0.f;
    float z[VPL], next[VPL];
    bool there = false, there_next = false;
    if (lo + wave < hi) {
      load_token<DT, VPL>(a, lo + wave, next);
      there_next = counted(a, lo + wave);
    }
    // this thread's first pair, on its way during the tokens (-1: none)
    const int pairs = (hi - lo) * a.K;  // at most tile * K
    auto expert_of = [&](int i) -> int {
      if (!counted(a, lo + i / a.K)) return -1;
      const size_t at = (size_t)lo * a.K + i;
      const int64_t e = a.itype == MOE_I32 ? (int64_t) static_cast<const int32_t*>(a.idx)[at]
                                           : static_cast<const int64_t*>(a.idx)[at];
      return e >= 0 && e < a.E ? (int)e : -1;
    };
    const int pair = (int)threadIdx.x < pairs ? expert_of(threadIdx.x) : -1;
    for (int t = lo + wave; t < hi; t += kWaves) {  // wave-uniform
#pragma unroll
      for (int v = 0; v < VPL; ++v) z[v] = next[v];
      there = there_next;
      if (t + kWaves < hi) {
        load_token<DT, VPL>(a, t + kWaves, next);
        there_next = counted(a, t + kWaves);
      }
      if (!there) continue;
      float soft[VPL], s[VPL], rest[VPL], lse;
      scores<VPL, SIG>(z, soft, s, rest, lse);
#pragma unroll
      for (int v = 0; v < VPL; ++v) p[v] += s[v];
      zz += lse * lse;
      ++n;
    }
    if (pair >= 0) atomicAdd(&hist[pair], 1);
    for (int i = threadIdx.x + kWaves * kWave; i < pairs; i += kWaves * kWave) {
      const int e = expert_of(i);
      if (e >= 0) atomicAdd(&hist[e], 1);
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

// Three sums over the workgroup, in a fixed order, in every thread.
template <int WAVES>
__device__ __forceinline__ void block_sums(double (&v)[3], double (&shared)[3][WAVES]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) v[i] = wave_sum(v[i]);
  if (lane_id() == 0)
#pragma unroll
    for (int i = 0; i < 3; ++i) shared[i][threadIdx.x / kWave] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    v[i] = 0.0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) v[i] += shared[i][w];
  }
}

__device__ __forceinline__ void write_loss(const BalanceArgs& a, double sum, double z, double all, double some) {
  a.loss[0] = some > 0 ? (float)(sum * a.E / (a.K * some)) : 0.f;
  a.loss[1] = all > 0 ? (float)(z / all) : 0.f;
}

// Sequence blockIdx.y, a.cols experts from blockIdx.x * a.cols on.
template <int THREADS>
__global__ __launch_bounds__(THREADS) void balance_finish_kernel(BalanceArgs a) {
  __shared__ double sp[THREADS];
  __shared__ int sc[THREADS];
  __shared__ double sums[3][THREADS / kWave];
  const int q = blockIdx.y, wide = (a.cols + kCols - 1) / kCols * kCols, groups = THREADS / wide;
  const int col = threadIdx.x % wide, g = threadIdx.x / wide;
  const int e = blockIdx.x * a.cols + col;
  const bool mine = g < groups && col < a.cols && e < a.E;
  const int lo = seq_begin(a, q), hi = seq_end(a, q);
  const int w0 = lo < hi ? lo / a.tile : 0, w1 = lo < hi ? (hi - 1) / a.tile : -1;
  double v[3] = {0.0, 0.0, 0.0};  // counts times probabilities, z, tokens
  if (blockIdx.x == 0)
    for (int w = w0 + (int)threadIdx.x; w <= w1; w += THREADS) {
      v[1] += a.part_z[w + q];
      v[2] += a.part_n[w + q];
    }
  double p = 0.0;
  int c = 0;
  if (mine) {
    const float* pp = a.part_p + e;
    const int* pc = a.part_c + e;
#pragma unroll 8
    for (int w = w0 + g; w <= w1; w += groups) {
      p += pp[(size_t)(w + q) * a.E];
      c += pc[(size_t)(w + q) * a.E];
    }
  }
  sp[threadIdx.x] = p;
  sc[threadIdx.x] = c;
  __syncthreads();
  if (mine && g == 0) {
    for (int k = 1; k < groups; ++k) {
      p += sp[k * wide + col];
      c += sc[k * wide + col];
    }
    a.probs[(size_t)q * a.E + e] = (float)p;
    a.counts[(size_t)q * a.E + e] = c;
    v[0] = p * c;
  }
  block_sums(v, sums);
  if (threadIdx.x != 0) return;
  const double n = v[2];
  if (blockIdx.x == 0) a.tokens[q] = (int)n;  // whole numbers: exact
  if (gridDim.x * gridDim.y == 1) {
    write_loss(a, n > 0 ? v[0] / (n * n) : 0.0, v[1], n, n > 0 ? 1.0 : 0.0);
  } else {
    a.seq_sum[(size_t)q * gridDim.x + blockIdx.x] = v[0];
    if (blockIdx.x == 0) a.seq_z[q] = v[1];
  }
}

// The losses from the sums of the sequences' columns.
__global__ __launch_bounds__(1024) void balance_loss_kernel(BalanceArgs a, int columns) {
  __shared__ double sums[3][16], more[3][16];
  double v[3] = {0.0, 0.0, 0.0}, some[3] = {0.0, 0.0, 0.0};
  for (int q = threadIdx.x; q < a.S; q += 1024) {
    const double n = a.tokens[q], z = a.seq_z[q];  // zeros of a sequence without tokens
    double s = 0.0;
    for (int b = 0; b < columns; ++b) s += a.seq_sum[(size_t)q * columns + b];
    v[0] += n > 0 ? s / (n * n) : 0.0;
    v[1] += z;
    v[2] += n;
    some[0] += n > 0 ? 1.0 : 0.0;
  }
  block_sums(v, sums);
  block_sums(some, more);
  if (threadIdx.x == 0) write_loss(a, v[0], v[1], v[2], some[0]);
}

template <int DT, int VPL, bool SIG>
__global__ __launch_bounds__(kWaves * kWave) void balance_bwd_kernel(BalanceArgs a) {
  __shared__ int sums[2][kWaves];
  const int lane = lane_id();
  const int64_t first = ((int64_t)blockIdx.x * kWaves + threadIdx.x / kWave) * a.tile;  // tile: tokens of a wave
  const int t0 = (int)min((int64_t)a.T, first), t1 = (int)min((int64_t)a.T, first + a.tile);
  const bool mine = t0 < t1;  // wave-uniform
  // everything a wave begins with is asked for before any of it is used
  float z[VPL], next[VPL];
  bool there, there_next = false;
  if (mine) {
    load_token<DT, VPL>(a, t0, next);
    there_next = counted(a, t0);
  }
  const float given0 = a.grad_loss[0], given1 = a.grad_loss[1];
  int q = sequences_before(a, t0);
  int begin, end, count[VPL];
  float n;
  auto enter = [&](int s) {  // sequence s
    const bool in = s < a.S;
    begin = in ? seq_begin(a, s) : a.T;
    end = in ? seq_end(a, s) : a.T;
    n = in ? (float)a.tokens[s] : 0.f;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int e = lane + kWave * v;
      count[v] = in && e < a.E ? a.counts[(size_t)s * a.E + e] : 0;
    }
  };
  enter(q);
  // all sequences' tokens: a wave by itself where it has one each lane, else the workgroup
  const bool alone = a.S <= kWave;
  int all = 0, some = 0;
  auto add = [&](int s) {
    const int m = a.tokens[s];
    all += m;
    some += m > 0;
  };
  if (alone) {
    if (lane < a.S) add(lane);
  } else {
#pragma unroll 8
    for (int s = threadIdx.x; s < a.S; s += kWaves * kWave) add(s);
  }
  all = read_lane_i((int)wave_scan((uint32_t)all), 63);
  some = read_lane_i((int)wave_scan((uint32_t)some), 63);
  if (!alone) {
    sums[0][threadIdx.x / kWave] = all;
    sums[1][threadIdx.x / kWave] = some;
    __syncthreads();
    all = some = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      all += sums[0][w];
      some += sums[1][w];
    }
  }
  const float g0 = given0, g1 = all > 0 ? given1 * (2.f / (float)all) : 0.f;
  const float even = (float)a.E / ((float)a.K * (float)some);
  float c[VPL];  // the gradient of the sequence's P
  auto weigh = [&]() {
    const float f = n > 0.f ? even / n / n : 0.f;
#pragma unroll
    for (int v = 0; v < VPL; ++v) c[v] = g0 * (f * (float)count[v]);
  };
  weigh();
  for (int t = t0; t < t1; ++t) {
#pragma unroll
    for (int v = 0; v < VPL; ++v) z[v] = next[v];
    there = there_next;
    if (t + 1 < t1) {
      load_token<DT, VPL>(a, t + 1, next);
      there_next = counted(a, t + 1);
    }
    if (q < a.S && end <= t) {
      enter(++q);
      if (end <= t && q < a.S) enter(q = max(q, sequences_before(a, t)));  // that one was empty
      weigh();
    }
    float d[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) d[v] = 0.f;
    if (q < a.S && begin <= t && there) {  // wave-uniform
      float soft[VPL], p[VPL], rest[VPL], lse, dot = 0.f;
      scores<VPL, SIG>(z, soft, p, rest, lse);
#pragma unroll
      for (int v = 0; v < VPL; ++v) dot += p[v] * c[v];
      dot = wave_sum(dot);
#pragma unroll
      for (int v = 0; v < VPL; ++v) d[v] = p[v] * rest[v] * (c[v] - dot) + g1 * lse * soft[v];
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
  else balance_kernel<DT, VPL, SIG><<<grid, kRunWaves * kWave, 0, s>>>(a);
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

// Tokens of a run: enough runs for the CUs, two tokens or more for each wave.  Past 2^19
// tokens there are more runs instead of longer ones: sums over a run are in 32 bits, those
// of the runs in 64, so a result is as near with 2^26 tokens as with 2^19 (2^23 tokens of 13
// experts alike: off by 432 u of itself with 256 runs, u = 2^-24).
int balance_tile(int64_t T) {
  const int64_t t = (T + kRuns - 1) / kRuns;
  return (int)(t < 2 * kRunWaves ? 2 * kRunWaves : t > kAdded * kRunWaves ? kAdded * kRunWaves : t);
}
int balance_runs(int64_t T) { return T > 0 ? (int)((T + balance_tile(T) - 1) / balance_tile(T)) : 1; }
int balance_columns(int E) { return (E + kCols - 1) / kCols; }

hipError_t launch_balance(BalanceArgs a, hipStream_t s) {
  a.tile = balance_tile(a.T);
  const int runs = balance_runs(a.T);
  hipError_t e = launch_typed(a, false, dim3(runs), s);
  if (e != hipSuccess) return e;
  // one sequence of few partials is one workgroup's work, losses included
  const bool direct = a.S == 1 && (int64_t)runs * a.E <= kDirect;
  // Sequences of a few partials on average: a wave for 64 experts of each, not 1024 threads
  // for 32.  (Forward kernels of 16384 tokens, 256 runs, 128 experts: 1024 sequences 34 us and
  // 81, 64 20.2 and 20.4, 24 20.3 and 19.8, 2 27 and 20; 320 experts: 64 29 and 35, 24 28.6
  // and 27.7.)
  const bool few = !direct && 4 * (int64_t)a.S >= runs;
  a.cols = direct ? a.E : few ? kWave : kCols;
  const int columns = (a.E + a.cols - 1) / a.cols;
  if (few) balance_finish_kernel<kWave><<<dim3(columns, a.S), kWave, 0, s>>>(a);
  else balance_finish_kernel<1024><<<dim3(columns, a.S), 1024, 0, s>>>(a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (columns * a.S == 1) return hipSuccess;
  balance_loss_kernel<<<1, 1024, 0, s>>>(a, columns);
  return hipGetLastError();
}

hipError_t launch_balance_bwd(BalanceArgs a, hipStream_t s) {
  const int64_t most = 2048 * kWaves;  // waves
  a.tile = (int)((a.T + most - 1) / most);
  const int64_t waves = ((int64_t)a.T + a.tile - 1) / a.tile;
  return launch_typed(a, true, dim3((unsigned)((waves + kWaves - 1) / kWaves)), s);
}

}  // namespace moe
