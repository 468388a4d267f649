// kernel_attrs.h -- the dynamic shared memory that each kernel has been allowed on each
// device.  No CUDA here: the caller passes the call that sets the limit.
#pragma once

namespace attn {

// A kernel's limit holds on the device that was current when it was set, and kernels whose
// launches differ in size (pages.cu) ask for more or less from call to call: the limit is
// kept per (kernel, device) and only ever raised.  Not locked.
class SharedMemoryLimits {
 public:
  static constexpr int kMaxDevices = 64;
  static constexpr int kMaxKernels = 64;  // instantiations that set their size

  // Let `kernel` use `bytes` on device `dev`: set(kernel, bytes) returns 0 on success,
  // and is not called where the limit is that high already.
  template <typename Set>
  auto allow(const void* kernel, int dev, int bytes, Set set) -> decltype(set(kernel, bytes)) {
    int i = 0;
    while (i < n_ && entries_[i].kernel != kernel) ++i;
    if (i < n_ && entries_[i].bytes[dev] >= bytes) return {};
    const auto err = set(kernel, bytes);
    if (err != decltype(err){}) return err;
    if (i == n_) {
      if (n_ == kMaxKernels) return {};  // table full: set again next time
      entries_[n_++].kernel = kernel;
    }
    entries_[i].bytes[dev] = bytes;
    return {};
  }

 private:
  struct Entry {
    const void* kernel;
    int bytes[kMaxDevices];
  };
  Entry entries_[kMaxKernels] = {};
  int n_ = 0;
};

}  // namespace attn
