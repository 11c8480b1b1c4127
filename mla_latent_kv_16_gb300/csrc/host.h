// What the launchers set up on the host, once per process or device. Calls come from any
// thread (the bindings let go of the interpreter's lock), so nothing here is seen half done.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstddef>
#include <cstdint>

namespace mla {

// cuTensorMapEncodeTiled of the driver; nullptr where there is none.
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

// Opts kernels into `bytes` of dynamic shared memory on the current device. A static one
// per launcher remembers the devices where that is done; two threads that come first may
// both do it, to the same effect.
class SmemOptIn {
 public:
  template <typename... Kernels>
  cudaError_t operator()(size_t bytes, Kernels... kernels) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (e != cudaSuccess || (done_.load(std::memory_order_acquire) & bit) != 0) return e;
    for (const void* k : {reinterpret_cast<const void*>(kernels)...})
      if (e == cudaSuccess)
        e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
    if (e == cudaSuccess) done_.fetch_or(bit, std::memory_order_release);
    return e;
  }

 private:
  std::atomic<uint64_t> done_{0};
};

}  // namespace mla
