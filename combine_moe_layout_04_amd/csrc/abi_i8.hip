// C ABI of the products in 8-bit integers (moe_quant_rows, moe_matmul_i8):
// host-side validation and launches, under the same rules as abi.hip.
#include "handle.h"

extern "C" {

int moe_quant_rows(const void* x, int dtype, int64_t rows, int64_t width, int8_t* q, float* scale,
                   hipStream_t stream) {
  if (rows < 0) return MOE_ERR_INVALID_ARG;
  if (width < 1 || width % 16 != 0) return MOE_ERR_SHAPE;
  const int eb = moe::elem_bytes(dtype);
  if (eb == 0 || width > MOE_MAX_I8_WIDTH || rows > (int64_t(1) << 26) - 4) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;  // nothing to read or write; empty arrays may be NULL
  if (!x || !q || !scale) return MOE_ERR_INVALID_ARG;
  if (!moe::aligned(x, 16) || !moe::aligned(q, 16) || !moe::aligned(scale, 4)) return MOE_ERR_ALIGNMENT;
  moe::NormArgs a{};
  a.x = x;
  a.q = q;
  a.scale = scale;
  a.T = (int)rows;
  a.nch = (int)(width * eb / 16);
  a.dtype = dtype;
  return moe::hip_status(moe::launch_quant(a, stream));
}

int moe_matmul_i8(moe_handle_t h, const int8_t* q, const float* scale, int64_t rows, int64_t width, int tokens,
                  const int8_t* w, const float* w_scale, int num_experts, int first_expert, int64_t N, int activation,
                  void* out, int out_dtype, hipStream_t stream) {
  if (h) {
    if (!moe::valid_handle(h)) return MOE_ERR_INVALID_ARG;
    if (!h->has_layout) return MOE_ERR_HANDLE;
  }
  if (rows < 0 || (tokens != 0 && tokens != 1)) return MOE_ERR_INVALID_ARG;
  if (activation != MOE_ACT_NONE && activation != MOE_ACT_SILU && activation != MOE_ACT_GELU_TANH)
    return MOE_ERR_INVALID_ARG;
  const int eb = moe::elem_bytes(out_dtype);
  if (eb == 0) return MOE_ERR_UNSUPPORTED;
  if (num_experts < 1 || first_expert < 0 || width < 1 || N < 1) return MOE_ERR_SHAPE;
  if (h) {
    if ((int64_t)first_expert + num_experts > h->E || rows != (tokens ? h->T : h->R)) return MOE_ERR_SHAPE;
  } else {
    if (num_experts != 1 || first_expert != 0) return MOE_ERR_SHAPE;
    if (tokens) return MOE_ERR_INVALID_ARG;  // token rows need their layout
  }
  if (width > MOE_MAX_I8_WIDTH || N > (int64_t(1) << 20) || N * width >= (int64_t(1) << 31)) return MOE_ERR_UNSUPPORTED;
  const int64_t R = h ? h->R : rows;
  if (R > (int64_t(1) << 26) || (tokens && rows * width > 0xFFFFFFE0LL)) return MOE_ERR_UNSUPPORTED;
  const bool gated = activation != MOE_ACT_NONE;
  if (width % 16 != 0 || (gated && N % 2 != 0)) return MOE_ERR_SHAPE;
  const int64_t cols = gated ? N / 2 : N;
  if ((cols * eb) % 16 != 0) return MOE_ERR_SHAPE;
  if (rows == 0) return MOE_OK;  // nothing to read or write; empty arrays may be NULL
  if (!q || !scale || !w || !w_scale || !out) return MOE_ERR_INVALID_ARG;
  if (!moe::aligned(q, 16) || !moe::aligned(w, 16) || !moe::aligned(out, 16) || !moe::aligned(scale, 4) ||
      !moe::aligned(w_scale, 4))
    return MOE_ERR_ALIGNMENT;
  moe::I8Args a{};
  a.q = q;
  a.qs = scale;
  a.w = w;
  a.ws = w_scale;
  a.out = out;
  a.M = (int)rows;
  a.R = (int)R;
  a.E = num_experts;
  a.N = (int)N;
  a.kch = (int)(width / 16);
  a.act = activation;
  a.dtype = out_dtype;
  if (h) {
    a.offset = moe::ws_ptr<int>(h, h->plan.expert_offset) + first_expert;
    a.recv_token = tokens ? moe::ws_ptr<int>(h, h->plan.recv_token) : nullptr;
  }
  return moe::hip_status(moe::launch_i8(a, stream));
}

}  // extern "C"
