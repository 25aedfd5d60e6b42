// C ABI of the expert layer for a few tokens (moe_few): host-side validation
// and launches, under the same rules as abi.hip.
#include "handle.h"

namespace {

int check_few(int dtype, int64_t T, int K, int E, int64_t H, int64_t I) {
  if (T < 0) return MOE_ERR_INVALID_ARG;
  if (K < 1 || E < 1 || H < 1 || I < 1) return MOE_ERR_SHAPE;
  const int eb = moe::elem_bytes(dtype);
  if (eb == 0) return MOE_ERR_UNSUPPORTED;
  if (K > MOE_MAX_K || E > MOE_MAX_E) return MOE_ERR_UNSUPPORTED;
  if (T > MOE_FEW_MAX_PAIRS || T * K > MOE_FEW_MAX_PAIRS) return MOE_ERR_UNSUPPORTED;
  if (H > (int64_t(1) << 18) || I > (int64_t(1) << 18)) return MOE_ERR_UNSUPPORTED;
  if ((H * eb) % 16 != 0 || (I * eb) % 16 != 0) return MOE_ERR_SHAPE;
  return MOE_OK;
}

}  // namespace

extern "C" {

int moe_few_workspace_size(int dtype, int64_t T, int K, int64_t I, size_t* bytes) {
  if (!bytes) return MOE_ERR_INVALID_ARG;
  const int st = check_few(dtype, T, K, K, 16, I);
  if (st != MOE_OK) return st;
  *bytes = (size_t)T * K * I * sizeof(float);
  return MOE_OK;
}

int moe_few(const void* x, int dtype, int64_t T, int64_t H, const void* topk_idx, int itype, int K,
            const float* topk_weights, const void* w13, const void* w2, int E, int64_t I, int activation,
            void* out, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const int st = check_few(dtype, T, K, E, H, I);
  if (st != MOE_OK) return st;
  if (itype != MOE_I32 && itype != MOE_I64) return MOE_ERR_UNSUPPORTED;
  if (activation != MOE_ACT_SILU && activation != MOE_ACT_GELU_TANH) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;  // nothing to read or write; empty arrays may be NULL
  if (!x || !topk_idx || !w13 || !w2 || !out || !workspace) return MOE_ERR_INVALID_ARG;
  if (!moe::aligned(x, 16) || !moe::aligned(w13, 16) || !moe::aligned(w2, 16) || !moe::aligned(out, 16) ||
      !moe::aligned(workspace, 256))
    return MOE_ERR_ALIGNMENT;
  if (!moe::aligned(topk_idx, itype == MOE_I32 ? 4 : 8) || (topk_weights && !moe::aligned(topk_weights, 4)))
    return MOE_ERR_ALIGNMENT;
  const size_t es = moe::elem_bytes(dtype);
  if (workspace_bytes < (size_t)T * K * I * sizeof(float)) return MOE_ERR_WORKSPACE;
  moe::FewArgs a{};
  a.x = x;
  a.idx = topk_idx;
  a.w = topk_weights;
  a.w13 = w13;
  a.w2 = w2;
  a.mid = static_cast<float*>(workspace);
  a.out = out;
  a.T = (int)T;
  a.K = K;
  a.E = E;
  a.H = (int)H;
  a.I = (int)I;
  a.itype = itype;
  a.dtype = dtype;
  a.act = activation;
  a.pairs = (int)(T * K);
  a.hch = (int)(H * es / 16);
  a.ich = (int)(I * es / 16);
  return moe::hip_status(moe::launch_few(a, stream));
}

}  // extern "C"
