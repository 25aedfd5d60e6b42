// C ABI of the router (moe_route, moe_route_bwd): host-side validation and
// launches, under the same rules as abi.hip.
#include <math.h>

#include "handle.h"

namespace {

int check_route(int dtype, int64_t T, int E, int K, const moe_route_options* o) {
  if (!o || T < 0) return MOE_ERR_INVALID_ARG;
  if (o->score != MOE_SCORE_SOFTMAX && o->score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if ((o->renormalize != 0 && o->renormalize != 1) || !isfinite(o->scale)) return MOE_ERR_INVALID_ARG;
  if (K < 1 || E < 1 || K > E) return MOE_ERR_SHAPE;
  if (K > MOE_MAX_K || E > MOE_MAX_E) return MOE_ERR_UNSUPPORTED;
  if (T > (int64_t(1) << 26) - 4) return MOE_ERR_UNSUPPORTED;  // four tokens a workgroup of 256: a grid has fewer than 2^32
  if (moe::elem_bytes(dtype) == 0) return MOE_ERR_UNSUPPORTED;
  if (o->num_groups < 1 || o->topk_groups < 1 || o->topk_groups > o->num_groups) return MOE_ERR_SHAPE;
  if (E % o->num_groups != 0 || K > o->topk_groups * (E / o->num_groups)) return MOE_ERR_SHAPE;
  if (o->num_groups > MOE_MAX_P) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace

extern "C" {

int moe_route(const void* logits, int dtype, int64_t T, int E, int K, const moe_route_options* options,
              const float* bias, int32_t* topk_idx, float* topk_weights, hipStream_t stream) {
  const int st = check_route(dtype, T, E, K, options);
  if (st != MOE_OK) return st;
  if (T == 0) return MOE_OK;  // nothing to read or write; empty arrays may be NULL
  if (!logits || !topk_idx || !topk_weights) return MOE_ERR_INVALID_ARG;
  if (!moe::aligned(logits, moe::elem_bytes(dtype)) || !moe::aligned(topk_idx, 4) ||
      !moe::aligned(topk_weights, 4) || (bias && !moe::aligned(bias, 4)))
    return MOE_ERR_ALIGNMENT;
  moe::RouteArgs a{};
  a.z = logits;
  a.bias = bias;
  a.idx = topk_idx;
  a.w = topk_weights;
  a.T = (int)T;
  a.E = E;
  a.K = K;
  a.dtype = dtype;
  a.score = options->score;
  a.renorm = options->renormalize != 0;
  a.scale = options->scale;
  a.groups = options->num_groups;
  a.topk_groups = options->topk_groups;
  return moe::hip_status(moe::launch_route(a, stream));
}

int moe_route_bwd(const void* logits, int dtype, int64_t T, int E, int K, const moe_route_options* options,
                  const int32_t* topk_idx, const float* grad_weights, void* grad_logits,
                  hipStream_t stream) {
  const int st = check_route(dtype, T, E, K, options);
  if (st != MOE_OK) return st;
  if (T == 0) return MOE_OK;
  if (!logits || !topk_idx || !grad_weights || !grad_logits) return MOE_ERR_INVALID_ARG;
  if (!moe::aligned(logits, moe::elem_bytes(dtype)) || !moe::aligned(grad_logits, moe::elem_bytes(dtype)) ||
      !moe::aligned(topk_idx, 4) || !moe::aligned(grad_weights, 4))
    return MOE_ERR_ALIGNMENT;
  moe::RouteBwdArgs a{};
  a.z = logits;
  a.idx = topk_idx;
  a.grad_w = grad_weights;
  a.grad_z = grad_logits;
  a.T = (int)T;
  a.E = E;
  a.K = K;
  a.dtype = dtype;
  a.score = options->score;
  a.renorm = options->renormalize != 0;
  a.scale = options->scale;
  return moe::hip_status(moe::launch_route_bwd(a, stream));
}

}  // extern "C"
