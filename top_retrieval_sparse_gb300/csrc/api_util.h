// api_util.h -- host helpers of the C ABI's translation units: errors, checks
// that several of them make, launches.
#pragma once

#include <cuda_runtime.h>

#include <cstdarg>
#include <cstdio>

#include "../../include/tsa.h"

namespace tsa {

// Defined in api.cu: this thread's error message, the host checks of a bf16 cache, the
// count of launches, the current device's SMs.
int report_error(int code, const char* msg);
int report_ok();
int validate_kv(const tsa_kv* kv);
cudaError_t count_launch(cudaError_t e);
int num_sms();

constexpr size_t kAlign = 256;

inline int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return report_error(code, buf);
}

inline int launched(cudaError_t e, const char* what) {
  if (count_launch(e) != cudaSuccess)
    return fail(TSA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  return report_ok();
}

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline size_t round_up(size_t n) { return (n + kAlign - 1) / kAlign * kAlign; }

inline int check_workspace(const void* ws, size_t bytes, size_t need) {
  if (!ws || !aligned(ws, kAlign))
    return fail(TSA_ERR_WORKSPACE, "workspace NULL or not 256-byte aligned");
  if (bytes < need)
    return fail(TSA_ERR_WORKSPACE, "workspace too small: %zu bytes, %zu needed", bytes, need);
  return TSA_OK;
}

}  // namespace tsa
