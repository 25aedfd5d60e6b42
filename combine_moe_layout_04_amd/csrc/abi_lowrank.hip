// C ABI of the low-rank adapters (moe_lowrank, moe_lowrank_bwd): host-side
// validation and launches, under the same rules as abi.hip.
#include "handle.h"

namespace {

int check_lowrank(const moe_handle_s* h, int dtype, int64_t H, int64_t N, int A, int r) {
  if (!moe::valid_handle(h)) return MOE_ERR_INVALID_ARG;
  if (!h->has_layout) return MOE_ERR_HANDLE;
  const int eb = moe::elem_bytes(dtype);
  if (eb == 0) return MOE_ERR_UNSUPPORTED;
  if (h->K != 1 || A < 1 || A > h->E || r < 1 || H < 1 || N < 1) return MOE_ERR_SHAPE;
  if (r > MOE_MAX_RANK || H > (int64_t(1) << 20) || N > (int64_t(1) << 20)) return MOE_ERR_UNSUPPORTED;
  if (h->R > (int64_t(1) << 26)) return MOE_ERR_UNSUPPORTED;  // 32 threads a row: a grid has fewer than 2^32
  if ((H * eb) % 16 != 0 || (N * eb) % 16 != 0 || (r * eb) % 16 != 0) return MOE_ERR_SHAPE;
  return MOE_OK;
}

moe::LowrankArgs lowrank_args(const moe_handle_s* h, int dtype, int A, int r) {
  moe::LowrankArgs a{};
  a.expert_offset = moe::ws_ptr<int>(h, h->plan.expert_offset);
  a.recv_token = moe::ws_ptr<int>(h, h->plan.recv_token);
  a.T = (int)h->T;
  a.E = h->E;
  a.A = A;
  a.R = (int)h->R;
  a.r = r;
  a.dtype = dtype;
  return a;
}

// Bytes of the backward's workspace: gu, then the parts of grad_a and grad_b.
size_t gu_bytes(const moe_handle_s* h, int r) { return (size_t)h->R * r * sizeof(float); }

size_t parts_bytes(int64_t H, int64_t N, int A, int r, int splits) {
  return splits > 1 ? (size_t)splits * A * r * (H + N) * sizeof(float) : 0;
}

}  // namespace

extern "C" {

int moe_lowrank_bwd_workspace_size(moe_handle_t h, int dtype, int64_t H, int64_t N, int num_adapters, int rank,
                                   size_t* bytes) {
  const int st = check_lowrank(h, dtype, H, N, num_adapters, rank);
  if (st != MOE_OK) return st;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  const int es = moe::elem_bytes(dtype);
  const int splits = moe::lowrank_wgrad_splits(h->R, num_adapters, rank, (int)(H * es / 16), (int)(N * es / 16), dtype);
  *bytes = gu_bytes(h, rank) + parts_bytes(H, N, num_adapters, rank, splits);
  return MOE_OK;
}

int moe_lowrank(moe_handle_t h, const void* x, int dtype, int64_t H, const void* a, const void* b,
                int num_adapters, int rank, int64_t N, const float* topk_weights, const void* base, void* out,
                float* u, hipStream_t stream) {
  const int st = check_lowrank(h, dtype, H, N, num_adapters, rank);
  if (st != MOE_OK) return st;
  if (h->T == 0) return MOE_OK;  // nothing to read or write; empty arrays may be NULL
  if (!x || !a || !b || !out || !u) return MOE_ERR_INVALID_ARG;
  if (!moe::aligned(x, 16) || !moe::aligned(a, 16) || !moe::aligned(b, 16) || !moe::aligned(out, 16) ||
      !moe::aligned(u, 16) || (base && !moe::aligned(base, 16)) || (topk_weights && !moe::aligned(topk_weights, 4)))
    return MOE_ERR_ALIGNMENT;
  const int es = moe::elem_bytes(dtype);
  moe::LowrankArgs k = lowrank_args(h, dtype, num_adapters, rank);
  k.rows = x;
  k.bank = a;
  k.u = u;
  k.wch = (int)(H * es / 16);
  moe::LowrankArgs wide = k;
  wide.bank = b;
  wide.w = topk_weights;
  wide.base = base;
  wide.out = out;
  wide.wch = (int)(N * es / 16);
  return moe::hip_status(moe::launch_lowrank_pass(k, wide, stream));
}

int moe_lowrank_bwd(moe_handle_t h, const void* grad_out, int dtype, int64_t H, const void* x, const void* a,
                    const void* b, int num_adapters, int rank, int64_t N, const float* topk_weights,
                    const float* u, const void* grad_base, void* grad_x, void* grad_a, void* grad_b,
                    float* grad_w, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  int st = check_lowrank(h, dtype, H, N, num_adapters, rank);
  if (st != MOE_OK) return st;
  if (!grad_x && !grad_a && !grad_b && !grad_w) return MOE_ERR_INVALID_ARG;
  const bool through = grad_x || grad_a || grad_w;  // gradients that pass through the rank's space
  if (h->T > 0) {
    if (!grad_out || (through && (!b || !workspace))) return MOE_ERR_INVALID_ARG;
    if ((grad_x && !a) || (grad_a && !x) || ((grad_b || grad_w) && !u)) return MOE_ERR_INVALID_ARG;
  }
  if (!moe::aligned(grad_out, 16) || !moe::aligned(x, 16) || !moe::aligned(a, 16) || !moe::aligned(b, 16) ||
      !moe::aligned(u, 16) || !moe::aligned(grad_base, 16) || !moe::aligned(grad_x, 16) ||
      !moe::aligned(grad_a, 16) || !moe::aligned(grad_b, 16) || !moe::aligned(topk_weights, 4) ||
      !moe::aligned(grad_w, 4) || !moe::aligned(workspace, 16))
    return MOE_ERR_ALIGNMENT;
  if (through && workspace_bytes < gu_bytes(h, rank)) return MOE_ERR_WORKSPACE;
  const int es = moe::elem_bytes(dtype);
  const int hch = (int)(H * es / 16), nch = (int)(N * es / 16);
  moe::LowrankArgs k = lowrank_args(h, dtype, num_adapters, rank);
  float* gu = static_cast<float*>(workspace);
  if (through && h->T > 0) {
    k.rows = grad_out;
    k.bank = b;
    k.w = topk_weights;
    k.u = gu;
    k.saved = u;
    k.dot = grad_w;
    k.wch = nch;
    k.backward = true;
    if (grad_x) {
      moe::LowrankArgs wide = k;
      wide.bank = a;
      wide.w = nullptr;  // gu holds the weight
      wide.base = grad_base;
      wide.out = grad_x;
      wide.wch = hch;
      st = moe::hip_status(moe::launch_lowrank_pass(k, wide, stream));
    } else {
      st = moe::hip_status(moe::launch_lowrank_shrink(k, stream));
    }
    if (st != MOE_OK) return st;
  }
  if (grad_a || grad_b) {  // also for an empty batch: zeros
    moe::LowrankArgs ga = k, gb = k;
    ga.rows = x;
    ga.w = nullptr;  // gu holds the weight
    ga.u = gu;
    ga.out = grad_a;
    ga.wch = hch;
    gb.rows = grad_out;
    gb.w = topk_weights;
    gb.u = const_cast<float*>(u);
    gb.out = grad_b;
    gb.wch = nch;
    int splits = moe::lowrank_wgrad_splits(h->R, num_adapters, rank, hch, nch, dtype);
    if (!workspace || workspace_bytes < gu_bytes(h, rank) + parts_bytes(H, N, num_adapters, rank, splits)) splits = 1;
    float* parts = splits > 1 ? gu + (size_t)h->R * rank : nullptr;
    if ((st = moe::hip_status(moe::launch_lowrank_wgrad(ga, gb, parts, splits, stream))) != MOE_OK) return st;
  }
  return MOE_OK;
}

}  // extern "C"
