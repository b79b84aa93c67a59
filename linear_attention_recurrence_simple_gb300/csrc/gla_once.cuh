// What a kernel needs once on each device before its first launch there (its shared memory allowed, its
// register count checked).  Written over the runtime's call for the current device, so that it runs without a GPU.
#pragma once

#include <atomic>

namespace gla {

// once(f) runs f() unless it has succeeded on the current device before; any thread, any device.  (Two
// threads may both run it the first time; devices past the 64th run it every time.)
template <class Api>
class OncePerDevice {
 public:
  template <class F>
  typename Api::Error operator()(F f) {
    int dev = 0;
    typename Api::Error e = Api::device(dev);
    if (e != Api::kSuccess) return e;
    const bool kept = dev >= 0 && dev < kMaxDevices;
    if (kept && done_[dev].load()) return Api::kSuccess;
    e = f();
    if (e == Api::kSuccess && kept) done_[dev].store(true);
    return e;
  }

 private:
  static constexpr int kMaxDevices = 64;
  std::atomic<bool> done_[kMaxDevices] = {};
};

#ifdef __CUDACC__
struct CudaDeviceApi {
  using Error = cudaError_t;
  static constexpr Error kSuccess = cudaSuccess;
  static Error device(int& dev) { return cudaGetDevice(&dev); }
};
#endif

}  // namespace gla
