// The router: from a token's expert scores to its K experts and their weights,
// and the gradient back to the scores.
//
//   s = softmax(z) or sigmoid(z) over the E experts of a token;
//   c = s + bias (a bias moves the choice, never the weight); without a bias
//       and without groups c is z itself, because both scores grow with z;
//   group limit: a group's value is the sum of its two largest c, and only the
//       topk_groups best groups take part;
//   the K largest c win; equal ones go to the lower expert (group) id;
//   w = scale * s, divided by the sum of the K chosen s when renormalised.
//
// One wavefront per token.  Its E values lie in registers (lane-strided, or
// by group: L lanes per group), the choice is K rounds of a wave-wide maximum
// over each lane's best remaining value, on integer keys that order like the
// numbers.  The plain top-k compares the logits themselves, which rounds
// nothing.  Values that have to be compared after arithmetic (bias, group
// sums) are formed in 32 bits first; a token whose choice hangs on a difference
// that the rounding could have turned is chosen again in 64 bits, so that a
// choice next to a border is the definition's (16384 tokens, 256 experts: 28 us
// in 64 bits throughout, 21 so).
//
// Renormalised weights need the chosen scores only up to a factor, and are formed
// from such, relative to the largest chosen logit where their sum is small.  So no
// sum is too small for 32 bits, however far below zero the logits lie or below the
// others a bias takes the choice.  Sigmoids below 2^-1022 (z < -708), where 64 bits
// begin to lose them, count as zero: masks of the type's lowest value get no weight.
//
// Logits that are NaN count as -inf in the choice and spread to the weights
// as the formulas say.  A sum of scores that is zero (every expert masked by
// -inf) gives zero weights, not 0/0.
#include "device_common.h"
#include "internal.h"
#include "../../include/moe_layout.h"

namespace moe {
namespace {

// ---- keys: unsigned integers in the order of the numbers ----------------------
// Every number's key is above 0, which marks "nothing to choose".

__device__ __forceinline__ uint32_t key_of(float f) {
  if (f != f) f = -INFINITY;
  const uint32_t b = __float_as_uint(f + 0.f);  // -0 and +0 are one value
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float float_of(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

__device__ __forceinline__ uint64_t key_of(double f) {
  if (f != f) f = -INFINITY;
  const uint64_t b = (uint64_t)__double_as_longlong(f + 0.0);
  return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

template <typename R>
struct Key;
template <>
struct Key<float> {
  typedef uint32_t T;
};
template <>
struct Key<double> {
  typedef uint64_t T;
};

template <int DT>
__device__ __forceinline__ float load_logit(const void* z, size_t i) {
  if constexpr (DT == kF32) return static_cast<const float*>(z)[i];
  return __uint_as_float((uint32_t)static_cast<const uint16_t*>(z)[i] << 16);
}

template <int DT>
__device__ __forceinline__ void store_elem(void* p, size_t i, float v) {
  if constexpr (DT == kF32) static_cast<float*>(p)[i] = v;
  else static_cast<uint16_t*>(p)[i] = (uint16_t)f32_to_bf16(v);
}

__device__ __forceinline__ float sigmoid(float z) {  // for small ones as exact as for large ones
  const float e = expf(-fabsf(z));
  return (z > 0.f ? 1.f : e) / (1.f + e);
}
__device__ __forceinline__ double sigmoid(double z) { return 1.0 / (1.0 + exp(-z)); }

// The largest chosen logit, of lanes with `mine`; 0 where there is none above -inf.
__device__ __forceinline__ float largest_chosen(float z, bool mine) {
  const float m = float_of(wave_max(mine ? key_of(z) : 1u));
  return m >= -3.402823466e38f ? m : 0.f;
}

// The scores of the chosen experts (lanes with `mine`, logits z) up to a common
// factor, and their sum: a softmax's relative to m, a sigmoid's as they are.  Where
// that sum is small, relative to the largest chosen logit.
__device__ __forceinline__ float chosen_scores(bool softmax, float z, bool mine, float m, float& total) {
  float s = mine ? softmax ? expf(z - m) : sigmoid(z) : 0.f;
  total = wave_sum(s);
  if (total < 0x1p-20f) {  // wave-uniform; above it 32 bits hold every share that is not below 2^-106
    const float top = largest_chosen(z, mine);
    s = mine ? expf(z - top) : 0.f;
    if (!softmax) s = z < -708.f ? 0.f : s / (1.f + expf(z));
    total = wave_sum(s);
  }
  return s;
}

// ---- forward ----------------------------------------------------------------------

// The choice itself: K rounds; lane k ends with the k-th chosen expert.
// key[v] belongs to expert base + step*v, so a lane's experts ascend with v.
// Up to 4 values a lane keeps them sorted (largest first, the lower id first
// among equals) and a winning lane shifts; more are searched again each round.
// each(m) sees the winning keys in their order.
template <int VPL, typename KEY, typename F>
__device__ __forceinline__ int choose(KEY (&key)[VPL], int base, int step, int K, F each) {
  const int lane = lane_id();
  int id[VPL];
#pragma unroll
  for (int v = 0; v < VPL; ++v) id[v] = base + step * v;
  constexpr bool kSorted = VPL <= 4;
  if constexpr (kSorted) {
#pragma unroll
    for (int i = 1; i < VPL; ++i)
#pragma unroll
      for (int j = i; j > 0; --j) {  // neighbours only: equal keys keep their order
        const bool up = key[j] > key[j - 1];
        const KEY a = key[j - 1], b = key[j];
        const int p = id[j - 1], q = id[j];
        key[j - 1] = up ? b : a;
        key[j] = up ? a : b;
        id[j - 1] = up ? q : p;
        id[j] = up ? p : q;
      }
  }
  int mine = 0;
  for (int k = 0; k < K; ++k) {
    KEY head = key[0];
    int hid = id[0];
    if constexpr (!kSorted) {
#pragma unroll
      for (int v = 1; v < VPL; ++v)
        if (key[v] > head) {
          head = key[v];
          hid = id[v];
        }
    }
    const KEY m = wave_max(head);
    each(m);
    const uint64_t with = __ballot(head == m);
    const int e = __popcll(with) == 1 ? read_lane_i(hid, __builtin_ctzll(with))
                                      : (int)wave_min(head == m ? (uint32_t)hid : 0xFFFFFFFFu);
    if (lane == k) mine = e;
    const bool won = head == m && hid == e;
    if constexpr (kSorted) {
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        const KEY next = v + 1 < VPL ? key[v + 1 < VPL ? v + 1 : v] : (KEY)0;
        const int nid = v + 1 < VPL ? id[v + 1 < VPL ? v + 1 : v] : id[v];
        key[v] = won ? next : key[v];
        id[v] = won ? nid : id[v];
      }
    } else {
#pragma unroll
      for (int v = 0; v < VPL; ++v)
        if (won && id[v] == e) key[v] = 0;
    }
  }
  return mine;
}

template <int DT, int VPL>
__global__ __launch_bounds__(256) void route_kernel(RouteArgs a) {
  const int lane = lane_id();
  const int t = blockIdx.x * (256 / kWave) + (int)(threadIdx.x / kWave);
  if (t >= a.T) return;  // wave-uniform
  const size_t row = (size_t)t * a.E;
  uint32_t key[VPL];
  bool nan = false;
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const int e = lane + kWave * v;
    key[v] = 0u;
    if (e < a.E) {
      const float z = load_logit<DT>(a.z, row + e);
      key[v] = key_of(z);
      nan |= z != z;
    }
  }
  // softmax over all experts: only when the weights are not renormalised
  // (the common factor drops out of a renormalised weight)
  float m = 0.f, total = 1.f;
  const bool softmax = a.score == MOE_SCORE_SOFTMAX;
  bool bad = false;  // a NaN anywhere in the row reaches every softmax weight
  if (softmax) {
    uint32_t top = key[0];
#pragma unroll
    for (int v = 1; v < VPL; ++v) top = max(top, key[v]);
    m = float_of(wave_max(top));
    if (m == -INFINITY) m = 0.f;
    bad = __ballot(nan) != 0;
    if (!a.renorm) {
      float sum = 0.f;
#pragma unroll
      for (int v = 0; v < VPL; ++v)
        if (lane + kWave * v < a.E) sum += expf(float_of(key[v]) - m);
      total = wave_sum(sum);
    }
  }
  const int e = choose<VPL>(key, lane, kWave, a.K, [](uint32_t) {});
  const bool mine = lane < a.K;
  const float z = mine ? load_logit<DT>(a.z, row + e) : -INFINITY;
  float s = a.renorm ? chosen_scores(softmax, z, mine, m, total) : softmax ? expf(z - m) : sigmoid(z);
  if (bad) s = NAN;
  if (mine) {
    a.idx[(size_t)t * a.K + lane] = e;
    a.w[(size_t)t * a.K + lane] = total == 0.f && !bad ? 0.f : s / total * a.scale;
  }
}

// The choice with a bias or a group limit, formed in R (float or double); lane
// k gets the k-th expert.  L lanes (a power of two) hold one group's experts, g
// and l are the lane's group and place.  In float, `sure` says whether every
// comparison that the choice hangs on was of values further apart than their
// errors (u = 2^-24; a bias adds u times the largest value, `far`):
//   softmax: scores within 41 u of the largest one, 1 / all (the numerator within
//     0.37 u from the rounded difference and 2 u of itself, a sum of at most 32
//     terms a lane within 38 u of itself, the division), so two values are told
//     apart from 2^-17 / all + 2^-22 far on;
//   sigmoid: within 4 u (the fast exponential of -z within (2 + |z|) u of itself,
//     the reciprocal and the sum before it within 3 u; s (1 - s) |z| is at most
//     0.23), so two values with their biases are off by less than 10 u times
//     the larger of far and 1, and told apart from 2^-20 times it on.
// Group sums count twice that.
template <typename R, int VPL>
__device__ __forceinline__ int choose_scored(const RouteArgs& a, const float (&z)[VPL], const float (&bias)[VPL], int g,
                                             int l, bool& sure, R& m, R& all) {
  constexpr bool kExact = sizeof(R) == 8;
  const bool softmax = a.score == MOE_SCORE_SOFTMAX;
  R c[VPL];
  bool there[VPL];
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    there[v] = g < a.groups && l + a.L * v < a.per;
    c[v] = (R)z[v];
  }
  m = 0;
  all = 1;
  if (softmax) {
    m = -INFINITY;
#pragma unroll
    for (int v = 0; v < VPL; ++v) m = max(m, c[v]);
#pragma unroll
    for (int s = 32; s >= 1; s >>= 1) m = max(m, __shfl_xor(m, s, kWave));
    if (m == -INFINITY) m = 0;
    R sum = 0;
#pragma unroll
    for (int v = 0; v < VPL; ++v)
      if (there[v]) {
        c[v] = exp(c[v] - m);
        sum += c[v];
      }
    all = wave_sum(sum);
    if (all == 0) all = 1;
#pragma unroll
    for (int v = 0; v < VPL; ++v) c[v] /= all;
  } else {
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      if constexpr (kExact) c[v] = sigmoid(c[v]);
      else c[v] = __builtin_amdgcn_rcpf(1.f + __expf(-c[v]));
    }
  }
  R far = softmax ? 0 : 1;  // the size that a bias's rounding goes by
#pragma unroll
  for (int v = 0; v < VPL; ++v)
    if (there[v]) {
      c[v] += (R)bias[v];
      if (c[v] != c[v]) c[v] = -INFINITY;
      const R size = fabs(c[v]);
      if (!kExact && size > far && size < INFINITY) far = size;
    } else {
      c[v] = -INFINITY;
    }
  R near = 0;  // two values closer than this are not told apart
  if constexpr (!kExact) {
    far = __uint_as_float(wave_max(__float_as_uint((float)far)));  // not below 0: ordered like its bits
    near = softmax ? 0x1p-17f / all + 0x1p-22f * far : 0x1p-20f * far;
  }
  sure = true;
  bool open = g < a.groups;
  if (a.topk_groups < a.groups) {
    R b1 = -INFINITY, b2 = -INFINITY;  // this lane's two largest, then its group's
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      b2 = max(b2, min(b1, c[v]));
      b1 = max(b1, c[v]);
    }
    for (int s = 1; s < a.L; s <<= 1) {
      const R o1 = __shfl_xor(b1, s, kWave), o2 = __shfl_xor(b2, s, kWave);
      b2 = max(min(b1, o1), max(b2, o2));
      b1 = max(b1, o1);
    }
    // (a value of +inf, as a bias can give, is not to meet a -inf)
    const R value = a.per > 1 && b1 < INFINITY ? b1 + b2 : b1;
    int better = 0;
    bool close = false;
    for (int i = 0; i < a.groups; ++i) {
      const R other = __shfl(value, i * a.L, kWave);
      better += other > value || (other == value && i < g);
      if (!kExact) close |= i != g && !(fabs(other - value) > 2 * near);  // also where both are infinite
    }
    if (!kExact) sure = !__ballot(open && close);
    open = open && better < a.topk_groups;
  }
  typename Key<R>::T key[VPL];
#pragma unroll
  for (int v = 0; v < VPL; ++v) key[v] = open && there[v] ? key_of(c[v]) : 0;
  if constexpr (kExact) {
    return choose<VPL>(key, g * a.per + l, a.L, a.K, [](uint64_t) {});
  } else {
    // one round more: the first that is not chosen counts too
    float last = INFINITY;
    return choose<VPL>(key, g * a.per + l, a.L, a.K + 1, [&](uint32_t k) {
      if (k == 0) return;  // nothing is left
      const float v = float_of(k);
      sure = sure && last - v > near;
      last = v;
    });
  }
}

template <int DT, int VPL>
__global__ __launch_bounds__(256) void route_scored_kernel(RouteArgs a) {
  const int lane = lane_id();
  const int t = blockIdx.x * (256 / kWave) + (int)(threadIdx.x / kWave);
  if (t >= a.T) return;  // wave-uniform
  const size_t row = (size_t)t * a.E;
  const int g = lane / a.L, l = lane & (a.L - 1);
  const bool softmax = a.score == MOE_SCORE_SOFTMAX;
  float z[VPL], bias[VPL];
  bool nan = false;
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const int j = l + a.L * v;
    const bool there = g < a.groups && j < a.per;
    z[v] = there ? load_logit<DT>(a.z, row + g * a.per + j) : -INFINITY;
    bias[v] = a.bias && there ? a.bias[g * a.per + j] : 0.f;
    nan |= z[v] != z[v];
    if (z[v] != z[v]) z[v] = -INFINITY;
  }
  bool bad = softmax && __ballot(nan) != 0;  // a NaN anywhere reaches every softmax weight
  bool sure;
  float m, all;
  int e = choose_scored<float, VPL>(a, z, bias, g, l, sure, m, all);
  if (!sure) {  // wave-uniform
    double m64, all64;
    e = choose_scored<double, VPL>(a, z, bias, g, l, sure, m64, all64);
  }
  bad = bad || all != all;  // +inf among the logits, chosen or not
  const bool mine = lane < a.K;
  const float x = mine ? load_logit<DT>(a.z, row + e) : -INFINITY;
  float total = 1.f;
  float s = a.renorm ? chosen_scores(softmax, x, mine, m, total) : softmax ? expf(x - m) / all : sigmoid(x);
  if (bad) s = NAN;
  if (mine) {
    a.idx[(size_t)t * a.K + lane] = e;
    a.w[(size_t)t * a.K + lane] = total == 0.f && !bad ? 0.f : s / total * a.scale;
  }
}

// ---- backward ---------------------------------------------------------------------
//
// With G_k = scale * grad_w[t,k]:
//   softmax               dz_j = p_j (sum_k [idx_k = j] G_k - sum_k p_k G_k)
//   softmax renormalised  q_k = p_k / sum p:  dz_k = q_k (G_k - sum_m q_m G_m)
//   sigmoid               dz_k = G_k s_k (1 - s_k)
//   sigmoid renormalised  dz_k = (G_k - sum_m q_m G_m) / sum s * s_k (1 - s_k)
// Only the dense softmax needs the row's other logits.  An id that repeats
// adds up, one outside [0, E) has no expert and no part in any sum.
template <int DT, int VPL>
__global__ __launch_bounds__(256) void route_bwd_kernel(RouteBwdArgs a) {
  const int lane = lane_id();
  const int t = blockIdx.x * (256 / kWave) + (int)(threadIdx.x / kWave);
  if (t >= a.T) return;  // wave-uniform
  const size_t row = (size_t)t * a.E;
  const bool softmax = a.score == MOE_SCORE_SOFTMAX;
  const bool dense = softmax && !a.renorm;

  int id = -1;
  float G = 0.f, z = -INFINITY;
  if (lane < a.K) {
    id = a.idx[(size_t)t * a.K + lane];
    if ((unsigned)id < (unsigned)a.E) {
      G = a.scale * a.grad_w[(size_t)t * a.K + lane];
      z = load_logit<DT>(a.z, row + id);
    } else {
      id = -1;
    }
  }
  float p[VPL];
  float d = 0.f;  // this lane's pair: its gradient, or G_k in the dense form
  float dot = 0.f;
  if (dense) {
    uint32_t top = 0u;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int e = lane + kWave * v;
      p[v] = e < a.E ? load_logit<DT>(a.z, row + e) : -INFINITY;
      if (e < a.E) top = max(top, key_of(p[v]));
    }
    float m = float_of(wave_max(top));
    if (m == -INFINITY) m = 0.f;
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      p[v] = expf(p[v] - m);
      sum += p[v];
    }
    float total = wave_sum(sum);
    if (total == 0.f) total = 1.f;
    const float inv = 1.f / total;
#pragma unroll
    for (int v = 0; v < VPL; ++v) p[v] *= inv;
    dot = wave_sum(id >= 0 ? expf(z - m) * inv * G : 0.f);
    d = G;
  } else {
    float s = 0.f;
    float total = 1.f;
    const float m = softmax ? largest_chosen(z, id >= 0) : 0.f;
    if (a.renorm) s = chosen_scores(softmax, z, id >= 0, m, total);
    else if (id >= 0) s = sigmoid(z);
    if (total == 0.f) total = 1.f;
    const float q = s / total;  // s itself when not renormalised
    const float mean = a.renorm ? wave_sum(id >= 0 ? q * G : 0.f) : 0.f;
    if (id >= 0) d = softmax ? q * (G - mean) : (G - mean) * q * sigmoid(-z);  // 1 - s
  }
  float acc[VPL];
#pragma unroll
  for (int v = 0; v < VPL; ++v) acc[v] = 0.f;
  for (int k = 0; k < a.K; ++k) {
    const int e = read_lane_i(id, k);
    const float x = read_lane_f(d, k);
#pragma unroll
    for (int v = 0; v < VPL; ++v) acc[v] += e == lane + kWave * v ? x : 0.f;
  }
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const int e = lane + kWave * v;
    if (e < a.E) store_elem<DT>(a.grad_z, row + e, dense ? p[v] * (acc[v] - dot) : acc[v]);
  }
}

template <typename F, typename A>
hipError_t launch_rows(F kernel, int T, hipStream_t s, const A& a) {
  hipLaunchKernelGGL(kernel, dim3((T + 3) / 4), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const RouteArgs& args, hipStream_t s) {
  RouteArgs a = args;
  if (!a.bias && a.groups == a.topk_groups) {  // no arithmetic before the comparison
    const int need = (a.E + kWave - 1) / kWave;
#define MOE_ROUTE(V) \
  return a.dtype == MOE_F32 ? launch_rows(route_kernel<kF32, V>, a.T, s, a) : launch_rows(route_kernel<kBF16, V>, a.T, s, a)
    if (need <= 1) MOE_ROUTE(1);
    if (need <= 2) MOE_ROUTE(2);
    if (need <= 4) MOE_ROUTE(4);
    if (need <= 8) MOE_ROUTE(8);
    MOE_ROUTE(16);
#undef MOE_ROUTE
  }
  if (a.groups == a.topk_groups) a.groups = a.topk_groups = 1;  // no limit: one group of all
  a.per = a.E / a.groups;
  a.L = 1;
  while (a.L * 2 * a.groups <= kWave) a.L *= 2;
  const int need = (a.per + a.L - 1) / a.L;
#define MOE_ROUTE(V)                                                                \
  return a.dtype == MOE_F32 ? launch_rows(route_scored_kernel<kF32, V>, a.T, s, a)  \
                            : launch_rows(route_scored_kernel<kBF16, V>, a.T, s, a)
  if (need <= 1) MOE_ROUTE(1);
  if (need <= 2) MOE_ROUTE(2);
  if (need <= 4) MOE_ROUTE(4);
  if (need <= 8) MOE_ROUTE(8);
  if (need <= 16) MOE_ROUTE(16);
  if (need <= 32) MOE_ROUTE(32);
#undef MOE_ROUTE
  return hipErrorInvalidValue;  // cannot happen: E <= 1024 and groups <= 64 need at most 32 a lane
}

hipError_t launch_route_bwd(const RouteBwdArgs& a, hipStream_t s) {
  const int need = (a.E + kWave - 1) / kWave;
#define MOE_ROUTE(V)                                                             \
  return a.dtype == MOE_F32 ? launch_rows(route_bwd_kernel<kF32, V>, a.T, s, a)  \
                            : launch_rows(route_bwd_kernel<kBF16, V>, a.T, s, a)
  if (need <= 1) MOE_ROUTE(1);
  if (need <= 2) MOE_ROUTE(2);
  if (need <= 4) MOE_ROUTE(4);
  if (need <= 8) MOE_ROUTE(8);
  MOE_ROUTE(16);
#undef MOE_ROUTE
}

}  // namespace moe
