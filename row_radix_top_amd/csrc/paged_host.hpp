// What the host files of the paged cache's entry points share: argument checks
// and launches.  No allocation, no memset and no synchronisation.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdio>

#include "paged_internal.h"
#include "topk_internal.h"

namespace {

using rrt::set_error;

// Every check that fails names the argument; nothing has been launched then.
#define REQUIRE(cond, text) \
  do {                      \
    if (!(cond)) return set_error(TOPK_EINVAL, text); \
  } while (0)

[[maybe_unused]] bool aligned(const void* p, uintptr_t by) { return reinterpret_cast<uintptr_t>(p) % by == 0; }

[[maybe_unused]] int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

[[maybe_unused]] int launch(const void* fn, int64_t grid, int block, void* params, hipStream_t stream, const char* what,
                            size_t lds = 0) {
  char buf[192];
  if (fn == nullptr) {
    std::snprintf(buf, sizeof(buf), "%s: no kernel instance for these arguments", what);
    return set_error(TOPK_EINVAL, buf);
  }
  if (grid * block > (int64_t)UINT32_MAX) {  // threads of a launch are counted in 32 bits
    std::snprintf(buf, sizeof(buf), "%s: %lld workgroups are more than one launch takes", what, (long long)grid);
    return set_error(TOPK_EINVAL, buf);
  }
  void* args[] = {params};
  hipError_t e = hipLaunchKernel(fn, dim3((unsigned)grid), dim3((unsigned)block), args, lds, stream);
  if (e == hipSuccess) e = hipGetLastError();
  if (e != hipSuccess) {
    std::snprintf(buf, sizeof(buf), "%s: launch failed: %s", what, hipGetErrorString(e));
    return set_error(TOPK_ELAUNCH, buf);
  }
  return TOPK_OK;
}

[[maybe_unused]] int check_types(paged_dtype dtype, paged_dtype store) {
  REQUIRE(dtype == PAGED_BF16 || dtype == PAGED_FP16, "dtype must be PAGED_BF16 or PAGED_FP16");
  REQUIRE(store == dtype || store == PAGED_E4M3, "store must be dtype or PAGED_E4M3");
  return TOPK_OK;
}

// The sizes of a workspace and whether it was given.
[[maybe_unused]] int check_workspace(const void* workspace, size_t bytes) {
  if (bytes == 0) return TOPK_OK;
  if (workspace == nullptr) {
    char buf[96];
    std::snprintf(buf, sizeof(buf), "this launch needs a workspace of %zu bytes", bytes);
    return set_error(TOPK_EWORKSPACE, buf);
  }
  REQUIRE(aligned(workspace, 16), "workspace must be 16-byte aligned");
  return TOPK_OK;
}

}  // namespace
