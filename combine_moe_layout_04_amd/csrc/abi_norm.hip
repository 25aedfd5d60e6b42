// C ABI of the norms around a block (moe_prenorm, moe_postnorm and their
// backward passes): host-side validation and launches, under the same rules as
// abi.hip.
#include <math.h>

#include "handle.h"

namespace {

static_assert(moe::kNormWide == MOE_NORM_WIDE, "one limit");

int check_norm(int dtype, int64_t T, int64_t H) {
  if (T < 0) return MOE_ERR_INVALID_ARG;
  if (H < 1) return MOE_ERR_SHAPE;
  const int eb = moe::elem_bytes(dtype);
  if (eb == 0 || T > (int64_t(1) << 26) || H > (int64_t(1) << 20)) return MOE_ERR_UNSUPPORTED;
  if ((H * eb) % 16 != 0) return MOE_ERR_SHAPE;
  if (H * eb > MOE_MAX_NORM_BYTES) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int check_gates(int64_t T, int64_t gates) {
  if (gates < 0) return MOE_ERR_INVALID_ARG;
  if (gates > 0 && T % gates != 0) return MOE_ERR_SHAPE;
  return T == 0 && gates > 65533 ? MOE_ERR_UNSUPPORTED : MOE_OK;  // zeros for each, in a grid of so many
}

bool bad_eps(float eps) { return !(eps > 0.f) || !isfinite(eps); }

template <typename... P>
bool all_aligned(size_t n, P... p) {
  return (moe::aligned(p, n) && ...);
}

moe::NormBwdArgs bwd_args(int dtype, int64_t T, int64_t H, int64_t gates, bool block) {
  moe::NormBwdArgs a{};
  a.block = block;
  a.T = (int)T;
  a.nch = (int)(H * moe::elem_bytes(dtype) / 16);
  a.gates = (int)gates;
  a.group = (int)(T > 0 ? T / gates : 1);
  a.dtype = dtype;
  moe::norm_bwd_plan(T, a.group, a.nch, block && H > moe::kNormWide, &a.rows, &a.parts, &a.runs);
  return a;
}

// Partials of one kind of sum over tokens.
size_t part_bytes(const moe::NormBwdArgs& a, int64_t H) { return (size_t)a.runs * H * sizeof(float); }

// A wide row's means.
size_t means_bytes(int64_t T, int64_t H) { return H > moe::kNormWide ? (size_t)T * 2 * sizeof(float) : 0; }

}  // namespace

extern "C" {

int moe_prenorm(const void* x, int dtype, int64_t T, int64_t H, const void* weight, float offset, float eps, void* n,
                int8_t* q, float* scale, float* rstd, hipStream_t stream) {
  const int st = check_norm(dtype, T, H);
  if (st != MOE_OK) return st;
  if (bad_eps(eps) || !isfinite(offset)) return MOE_ERR_INVALID_ARG;
  if ((n != nullptr) + (q != nullptr) > 1) return MOE_ERR_INVALID_ARG;
  if (q && H % 16 != 0) return MOE_ERR_SHAPE;
  if (T == 0) return MOE_OK;  // nothing to read or write; empty arrays may be NULL
  if (!x || !weight || (!n && !q) || (q && !scale)) return MOE_ERR_INVALID_ARG;
  if (!all_aligned(16, x, weight, n, q) || !all_aligned(4, scale, rstd)) return MOE_ERR_ALIGNMENT;
  moe::NormArgs a{};
  a.x = x;
  a.w2 = weight;
  a.n = n;
  a.q = q;
  a.scale = scale;
  a.rstd = rstd;
  a.eps = eps;
  a.offset = offset;
  a.T = (int)T;
  a.nch = (int)(H * moe::elem_bytes(dtype) / 16);
  a.group = 1;
  a.dtype = dtype;
  return moe::hip_status(moe::launch_norm(a, stream));
}

int moe_postnorm(moe_handle_t h, const void* x, const void* y, int dtype, int64_t T, int64_t H,
                 const float* topk_weights, const void* weight, const void* gate, int64_t gates, float residual_scale,
                 const void* next_weight, float offset, float eps, void* out, void* n, float* rstd,
                 hipStream_t stream) {
  if (h) {
    if (!moe::valid_handle(h)) return MOE_ERR_INVALID_ARG;
    if (!h->has_layout) return MOE_ERR_HANDLE;
    if (T != h->T) return MOE_ERR_SHAPE;
  } else if (topk_weights) {
    return MOE_ERR_INVALID_ARG;  // weights of pairs need their layout
  }
  const int st = check_norm(dtype, T, H);
  if (st != MOE_OK) return st;
  if (bad_eps(eps) || !isfinite(offset) || !isfinite(residual_scale)) return MOE_ERR_INVALID_ARG;
  const int gs = check_gates(T, gates);
  if (gs != MOE_OK) return gs;
  if (T == 0) return MOE_OK;
  if (!x || !y || !out || (gate != nullptr) != (gates > 0) || (next_weight != nullptr) != (n != nullptr))
    return MOE_ERR_INVALID_ARG;
  if (!all_aligned(16, x, y, weight, gate, next_weight, out, n) || !all_aligned(8, rstd) || !all_aligned(4, topk_weights))
    return MOE_ERR_ALIGNMENT;
  moe::NormArgs a{};
  a.x = x;
  a.y = y;
  a.w1 = weight;
  a.gate = gate;
  a.w2 = next_weight;
  a.out = out;
  a.n = n;
  a.rstd = rstd;
  a.residual = residual_scale;
  a.eps = eps;
  a.offset = offset;
  a.T = (int)T;
  a.nch = (int)(H * moe::elem_bytes(dtype) / 16);
  a.group = (int)(gates > 0 ? T / gates : T);
  a.dtype = dtype;
  if (h) {
    a.recv_pos = moe::ws_ptr<int>(h, h->plan.recv_pos);
    a.status = moe::ws_ptr<int>(h, h->plan.status);
    a.w = topk_weights;
    a.K = h->K;
    a.R = (int)h->R;
  }
  return moe::hip_status(moe::launch_norm(a, stream));
}

int moe_norm_bwd_workspace_size(int dtype, int64_t T, int64_t H, int64_t gates, size_t* bytes) {
  if (!bytes) return MOE_ERR_INVALID_ARG;
  const int st = check_norm(dtype, T, H);
  if (st != MOE_OK) return st;
  const int gs = check_gates(T, gates);
  if (gs != MOE_OK) return gs;
  const size_t before = part_bytes(bwd_args(dtype, T, H, 1, false), H);
  const size_t after = 3 * part_bytes(bwd_args(dtype, T, H, gates > 0 ? gates : 1, true), H) + means_bytes(T, H);
  *bytes = before > after ? before : after;
  return MOE_OK;
}

int moe_prenorm_bwd(const void* grad_n, const void* x, int dtype, int64_t T, int64_t H, const void* weight, float offset,
                    const float* rstd, const void* grad_base, void* grad_x, void* grad_weight, void* workspace,
                    size_t workspace_bytes, hipStream_t stream) {
  const int st = check_norm(dtype, T, H);
  if (st != MOE_OK) return st;
  if (!isfinite(offset) || (!grad_x && !grad_weight && T > 0)) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!grad_n || !x || !weight || !rstd || (grad_weight && !workspace))) return MOE_ERR_INVALID_ARG;
  if (!all_aligned(16, grad_n, x, weight, grad_base, grad_x, grad_weight, workspace) || !all_aligned(4, rstd))
    return MOE_ERR_ALIGNMENT;
  moe::NormBwdArgs a = bwd_args(dtype, T, H, 1, false);
  if (grad_weight && workspace_bytes < part_bytes(a, H)) return MOE_ERR_WORKSPACE;
  a.g = grad_base;
  a.gn = grad_n;
  a.x = x;
  a.w2 = weight;
  a.rstd = rstd;
  a.gx = grad_x;
  a.gw2 = grad_weight;
  a.part2 = grad_weight ? static_cast<float*>(workspace) : nullptr;
  a.offset = offset;
  return moe::hip_status(moe::launch_norm_bwd(a, stream));
}

int moe_postnorm_bwd(const void* grad_out, const void* grad_n, const void* x, const void* y, int dtype, int64_t T,
                     int64_t H, const float* rstd, const void* weight, const void* gate, int64_t gates,
                     float residual_scale, const void* next_weight, float offset, void* grad_x, void* grad_y,
                     void* grad_weight, void* grad_gate, void* grad_next_weight, void* workspace,
                     size_t workspace_bytes, hipStream_t stream) {
  const int st = check_norm(dtype, T, H);
  if (st != MOE_OK) return st;
  if (!isfinite(offset) || !isfinite(residual_scale)) return MOE_ERR_INVALID_ARG;
  const int gs = check_gates(T, gates);
  if (gs != MOE_OK) return gs;
  if (grad_gate && gates < 1) return MOE_ERR_INVALID_ARG;
  const bool sums = grad_weight || grad_gate || grad_next_weight;
  if (T > 0) {
    if (!grad_out && !grad_n) return MOE_ERR_INVALID_ARG;
    if ((gate != nullptr) != (gates > 0)) return MOE_ERR_INVALID_ARG;
    if (grad_n && (!next_weight || !x || !y)) return MOE_ERR_INVALID_ARG;
    if ((weight || grad_gate) && !y) return MOE_ERR_INVALID_ARG;
    if ((grad_weight && !weight) || (grad_next_weight && !next_weight)) return MOE_ERR_INVALID_ARG;
    if (!grad_x && !grad_y && !sums) return MOE_ERR_INVALID_ARG;
    if (!rstd || ((sums || H > moe::kNormWide) && !workspace)) return MOE_ERR_INVALID_ARG;
  }
  if (!all_aligned(16, grad_out, grad_n, x, y, weight, gate, next_weight, grad_x, grad_y, grad_weight, grad_gate,
                   grad_next_weight, workspace) ||
      !all_aligned(8, rstd))
    return MOE_ERR_ALIGNMENT;
  moe::NormBwdArgs a = bwd_args(dtype, T, H, gates > 0 ? gates : 1, true);
  const size_t part = part_bytes(a, H), means = means_bytes(T, H);
  if ((sums || means) && workspace_bytes < 3 * part + means) return MOE_ERR_WORKSPACE;
  float* ws = static_cast<float*>(workspace);
  a.g = grad_out;
  a.gn = grad_n;
  a.x = x;
  a.y = (weight || grad_gate || grad_n) ? y : nullptr;
  a.w1 = weight;
  a.gate = gate;
  a.w2 = next_weight;
  a.rstd = rstd;
  a.gx = grad_x;
  a.gy = grad_y;
  a.gw1 = grad_weight;
  a.gg = grad_gate;
  a.gw2 = grad_next_weight;
  a.part1 = grad_weight ? ws : nullptr;
  a.part2 = grad_next_weight ? ws + part / sizeof(float) : nullptr;
  a.partg = grad_gate ? ws + 2 * (part / sizeof(float)) : nullptr;
  a.means = means && (weight || grad_n) ? ws + 3 * (part / sizeof(float)) : nullptr;
  a.residual = residual_scale;
  a.offset = offset;
  return moe::hip_status(moe::launch_norm_bwd(a, stream));
}

}  // extern "C"
