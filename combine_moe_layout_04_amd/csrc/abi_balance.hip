// C ABI of the router's balance loss (moe_balance, moe_balance_bwd): host-side
// validation and launches, under the same rules as abi.hip.
#include "handle.h"

namespace {

int check_balance(int dtype, int64_t T, int E, int K, int64_t S, bool seq, int score) {
  if (T < 0 || S < 0) return MOE_ERR_INVALID_ARG;
  if (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (K < 1 || E < 1 || S < 1 || (!seq && S != 1)) return MOE_ERR_SHAPE;
  if (K > MOE_MAX_K || E > MOE_MAX_E || S > MOE_MAX_SEQUENCES) return MOE_ERR_UNSUPPORTED;
  if (T > (int64_t(1) << 26) - 4) return MOE_ERR_UNSUPPORTED;
  if (moe::elem_bytes(dtype) == 0) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// The workspace's sections in order; returns their total.
size_t place(moe::BalanceArgs* a, char* ws, int64_t T, int E, int64_t S) {
  const size_t slots = (size_t)moe::balance_runs(T) + S;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* p = ws + at;
    at += up256(bytes);
    return p;
  };
  char* seq_sum = take((size_t)S * moe::balance_columns(E) * sizeof(double));
  char* seq_z = take((size_t)S * sizeof(double));
  char* part_z = take(slots * sizeof(float));
  char* part_n = take(slots * sizeof(int));
  char* part_p = take(slots * E * sizeof(float));
  char* part_c = take(slots * E * sizeof(int));
  if (a) {
    a->seq_sum = reinterpret_cast<double*>(seq_sum);
    a->seq_z = reinterpret_cast<double*>(seq_z);
    a->part_z = reinterpret_cast<float*>(part_z);
    a->part_n = reinterpret_cast<int*>(part_n);
    a->part_p = reinterpret_cast<float*>(part_p);
    a->part_c = reinterpret_cast<int*>(part_c);
  }
  return at;
}

}  // namespace

extern "C" {

int moe_balance_workspace_size(int64_t T, int E, int64_t S, size_t* bytes) {
  if (!bytes) return MOE_ERR_INVALID_ARG;
  const int st = check_balance(MOE_F32, T, E, 1, S, true, MOE_SCORE_SOFTMAX);
  if (st != MOE_OK) return st;
  *bytes = place(nullptr, nullptr, T, E, S);
  return MOE_OK;
}

int moe_balance(const void* logits, int dtype, int64_t T, int E, const void* topk_idx, int itype, int K,
                const int32_t* seq_offset, int64_t S, const uint8_t* token_mask, int score, float* loss,
                int32_t* counts, float* probs, int32_t* tokens, void* workspace, size_t workspace_bytes,
                hipStream_t stream) {
  const int st = check_balance(dtype, T, E, K, S, seq_offset != nullptr, score);
  if (st != MOE_OK) return st;
  if (itype != MOE_I32 && itype != MOE_I64) return MOE_ERR_UNSUPPORTED;
  if (!loss || !counts || !probs || !tokens || !workspace) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!logits || !topk_idx)) return MOE_ERR_INVALID_ARG;
  if (!moe::aligned(logits, moe::elem_bytes(dtype)) || !moe::aligned(topk_idx, itype == MOE_I32 ? 4 : 8) ||
      !moe::aligned(seq_offset, 4) || !moe::aligned(loss, 4) || !moe::aligned(counts, 4) || !moe::aligned(probs, 4) ||
      !moe::aligned(tokens, 4) || !moe::aligned(workspace, 256))
    return MOE_ERR_ALIGNMENT;
  moe::BalanceArgs a{};
  if (workspace_bytes < place(&a, static_cast<char*>(workspace), T, E, S)) return MOE_ERR_WORKSPACE;
  a.z = logits;
  a.idx = topk_idx;
  a.seq = seq_offset;
  a.mask = token_mask;
  a.loss = loss;
  a.counts = counts;
  a.probs = probs;
  a.tokens = tokens;
  a.T = (int)T;
  a.E = E;
  a.K = K;
  a.S = (int)S;
  a.dtype = dtype;
  a.itype = itype;
  a.score = score;
  return moe::hip_status(moe::launch_balance(a, stream));
}

int moe_balance_bwd(const void* logits, int dtype, int64_t T, int E, int K, const int32_t* seq_offset, int64_t S,
                    const uint8_t* token_mask, int score, const int32_t* counts, const int32_t* tokens,
                    const float* grad_loss, const void* grad_base, void* grad_logits, hipStream_t stream) {
  const int st = check_balance(dtype, T, E, K, S, seq_offset != nullptr, score);
  if (st != MOE_OK) return st;
  if (T == 0) return MOE_OK;  // nothing to read or write; empty arrays may be NULL
  if (!logits || !counts || !tokens || !grad_loss || !grad_logits) return MOE_ERR_INVALID_ARG;
  if (!moe::aligned(logits, moe::elem_bytes(dtype)) || !moe::aligned(grad_logits, moe::elem_bytes(dtype)) ||
      !moe::aligned(grad_base, moe::elem_bytes(dtype)) || !moe::aligned(seq_offset, 4) || !moe::aligned(counts, 4) ||
      !moe::aligned(tokens, 4) || !moe::aligned(grad_loss, 4))
    return MOE_ERR_ALIGNMENT;
  moe::BalanceArgs a{};
  a.z = logits;
  a.seq = seq_offset;
  a.mask = token_mask;
  a.counts = const_cast<int32_t*>(counts);
  a.tokens = const_cast<int32_t*>(tokens);
  a.grad_loss = grad_loss;
  a.grad_base = grad_base;
  a.grad_z = grad_logits;
  a.T = (int)T;
  a.E = E;
  a.K = K;
  a.S = (int)S;
  a.dtype = dtype;
  a.score = score;
  return moe::hip_status(moe::launch_balance_bwd(a, stream));
}

}  // extern "C"
