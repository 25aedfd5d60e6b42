// The opaque layout handle and the host-side helpers shared by the files that
// implement the C ABI.
#pragma once

#include "internal.h"
#include "../../include/moe_layout.h"

struct moe_handle_s {
  static constexpr uint32_t kMagic = 0x4D4F454Cu;  // "MOEL"
  uint32_t magic = kMagic;
  bool has_layout = false;
  int64_t T = 0;
  int K = 0, E = 0, P = 0;
  int pad = 1;     // expert segments padded to a multiple of this (fixed at creation)
  int64_t R = 0;   // receive rows of the current layout: T*K + E*(pad-1)
  char* ws = nullptr;
  moe::WsLayout plan{};
  moe::Tuning tune{};
  hipEvent_t ev_start = nullptr;  // moe_time_next_kernel: for the next kernel launch only
  hipEvent_t ev_stop = nullptr;
};

namespace moe {

inline bool valid_handle(const moe_handle_s* h) { return h && h->magic == moe_handle_s::kMagic; }

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline int elem_bytes(int dtype) { return dtype == MOE_F32 ? 4 : dtype == MOE_BF16 ? 2 : 0; }

inline int hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

template <typename T>
T* ws_ptr(const moe_handle_s* h, size_t off) {
  return reinterpret_cast<T*>(h->ws + off);
}

}  // namespace moe
