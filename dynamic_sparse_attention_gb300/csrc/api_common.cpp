// Error reporting and version entry points of the C ABI.
#include "api_common.h"

#include <atomic>
#include <cstring>
#include <thread>

#include "launch.h"

namespace dsa {

namespace {
thread_local char g_msg[512] = "";
}

const char *last_error() { return g_msg; }

void clear_error() { g_msg[0] = '\0'; }

int fail(int status, const char *fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(g_msg, sizeof(g_msg), fmt, ap);
  va_end(ap);
  return status;
}

int cuda_fail(cudaError_t e, const char *what) {
  return fail(DSA_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorString(e), cudaGetErrorName(e));
}

namespace {
// The largest limit that each kernel has been given on each device; places are found by hashing and never
// given up.  (Set anew by every call, as a context that was torn down and made again has forgotten it.)
struct SharedLimit {
  const void *kern;
  int dev;
  size_t bytes;
};
constexpr int kLimits = 1024;   // kernels times devices; where no place is left, a call's own size is set
SharedLimit g_limit[kLimits];
std::atomic_flag g_limit_lock = ATOMIC_FLAG_INIT;
}  // namespace

cudaError_t allow_shared(const void *kern, size_t bytes) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  while (g_limit_lock.test_and_set(std::memory_order_acquire)) std::this_thread::yield();
  SharedLimit *at = nullptr;
  for (size_t i = 0, h = reinterpret_cast<uintptr_t>(kern) / 16 + static_cast<size_t>(dev) * 31; i < kLimits; ++i) {
    SharedLimit &l = g_limit[(h + i) % kLimits];
    if (l.kern && (l.kern != kern || l.dev != dev)) continue;
    at = &l;
    break;
  }
  const size_t most = at && at->bytes > bytes ? at->bytes : bytes;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most));
  if (e == cudaSuccess && at) *at = SharedLimit{kern, dev, most};
  g_limit_lock.clear(std::memory_order_release);
  return e;
}

}  // namespace dsa

extern "C" {

const char *dsa_last_error(void) { return dsa::last_error(); }

const char *dsa_strerror(int status) {
  switch (status) {
    case DSA_OK: return "ok";
    case DSA_ERR_INVALID_ARG: return "invalid argument";
    case DSA_ERR_UNSUPPORTED: return "unsupported configuration";
    case DSA_ERR_WORKSPACE: return "workspace missing or too small";
    case DSA_ERR_ALIGNMENT: return "null or misaligned pointer";
    case DSA_ERR_CUDA: return "CUDA launch error";
    case DSA_ERR_DEVICE_CHECK: return "device-side check failed";
    default: return "unknown status";
  }
}

int dsa_version(void) { return DSA_VERSION; }

}  // extern "C"
