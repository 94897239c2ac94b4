// Per-device launch settings shared by the kernel launchers: the dynamic
// shared-memory limit of each kernel, the widest cluster that fits, and the SM
// count.  All are looked up once and reused; a process may drive several devices
// from several host threads, so the caches are keyed on the context (attributes,
// clusters) or the device (the SM count) and safe to use concurrently.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <mutex>
#include <vector>

#include "mla_launch.h"

namespace mla {
namespace {

using CtxGetCurrentFn = CUresult (*)(CUcontext*);

// cuCtxGetCurrent through the runtime's driver entry point (the library does
// not link the driver API directly).
CtxGetCurrentFn ctx_get_current_fn() {
  static CtxGetCurrentFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<CtxGetCurrentFn>(p);
  });
  return fn;
}

CUcontext current_context() {
  CUcontext ctx = nullptr;
  const CtxGetCurrentFn get = ctx_get_current_fn();
  if (!get || get(&ctx) != CUDA_SUCCESS) return nullptr;
  return ctx;
}

bool set_attribute(const void* func, cudaFuncAttribute attr, int value) {
  // An attribute belongs to the function as loaded in one context: remember
  // the (function, attribute, context) triples it was set for.  A context made
  // after a device reset is a new one and gets the attribute again.
  struct Done {
    const void* func;
    cudaFuncAttribute attr;
    CUcontext ctx;
  };
  static std::mutex mu;
  static std::vector<Done> done;
  CUcontext ctx = current_context();   // null before the device's first runtime call: set it then
  if (ctx) {
    std::lock_guard<std::mutex> lock(mu);
    for (const auto& e : done)
      if (e.func == func && e.attr == attr && e.ctx == ctx) return true;
  }
  if (cudaFuncSetAttribute(func, attr, value) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  ctx = current_context();             // the call above made a context current if none was
  if (ctx) {
    std::lock_guard<std::mutex> lock(mu);
    done.push_back({func, attr, ctx});
  }
  return true;
}

}  // namespace

bool set_smem_limit(const void* func, int bytes) {
  return set_attribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

int widest_cluster(const void* func, int threads, int wide) {
  struct Found {
    const void* func;
    CUcontext ctx;
    int ctas;
  };
  static std::mutex mu;
  static std::vector<Found> found;
  // (sets the attribute in every context; a call without a context makes one)
  const bool allowed = set_attribute(func, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  const CUcontext ctx = current_context();
  if (ctx) {
    std::lock_guard<std::mutex> lock(mu);
    for (const auto& e : found)
      if (e.func == func && e.ctx == ctx) return e.ctas;
  }
  auto fits = [&](int ctas) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(ctas);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, func, &cfg) == cudaSuccess) return n > 0;
    cudaGetLastError();
    return false;
  };
  int ctas = allowed ? wide : 8;
  while (ctas > 0 && !fits(ctas)) ctas /= 2;
  if (ctx && ctas > 0) {
    std::lock_guard<std::mutex> lock(mu);
    found.push_back({func, ctx, ctas});
  }
  return ctas;
}

int device_sm_count() {
  // queried once per device ordinal; a race only repeats the query
  static std::atomic<int> sms_of[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  const int cached = (dev >= 0 && dev < 64) ? sms_of[dev].load(std::memory_order_relaxed) : 0;
  if (cached > 0) return cached;
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) {
    cudaGetLastError();
    return 0;
  }
  if (dev >= 0 && dev < 64) sms_of[dev].store(n, std::memory_order_relaxed);
  return n;
}

}  // namespace mla
