// The handle of the block operators and the argument checks that their C entry
// points share (host side).
#pragma once

#include <cuda_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "block.h"

namespace tpo {

inline tpo_status fail(tpo_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  set_last_error(buf);
  return s;
}

inline tpo_status cuda_fail(cudaError_t e, const char* what) {
  return fail(TPO_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorString(e), cudaGetErrorName(e));
}

constexpr int64_t kMaxSize = 1ll << 30;
constexpr size_t kErrBytes = 256;  // the error words ahead of the workspace

inline int64_t round_up(int64_t v, int64_t q) { return (v + q - 1) / q * q; }

// Pitch of a bf16 workspace matrix: whole 128-byte lines.
inline int64_t ws_pitch(int64_t m) { return round_up(m, 64); }

}  // namespace tpo

struct tpo_block {
  int device = 0;
  uint8_t* mem = nullptr;  // error words, then the workspace
  int64_t ws_bytes = 0;
  tpo::Machine machine{};
  int64_t path = 0, split = 0, wait_timeout_ms = 2000;  // options
  uint32_t* err() const { return reinterpret_cast<uint32_t*>(mem); }
  tpo::Watch watch() const { return {err(), static_cast<unsigned long long>(wait_timeout_ms) * 1000000ull}; }
  uint8_t* ws() const { return mem + tpo::kErrBytes; }
};

namespace tpo {

inline tpo_status check_vec(const char* name, const void* p, int elem) {
  if (reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(elem))
    return fail(TPO_ERR_INVALID_ARG, "%s must be aligned to its elements", name);
  return TPO_OK;
}

// The handle, checked last so that the other argument errors need no GPU.
inline tpo_status check_block(const tpo_block* b, int64_t need) {
  if (!b) return fail(TPO_ERR_INVALID_ARG, "NULL block handle");
  if (need > b->ws_bytes)
    return fail(TPO_ERR_INVALID_ARG, "the call needs %lld bytes of workspace, the handle has %lld", (long long)need,
                (long long)b->ws_bytes);
  int dev = -1;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "no usable CUDA device");
  if (dev != b->device)
    return fail(TPO_ERR_INVALID_ARG, "the handle is of device %d, the current device is %d", b->device, dev);
  return TPO_OK;
}

inline tpo_status launched(cudaError_t e) { return e == cudaSuccess ? TPO_OK : cuda_fail(e, "kernel launch"); }

}  // namespace tpo
