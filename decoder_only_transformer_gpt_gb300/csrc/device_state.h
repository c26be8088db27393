// What the library keeps per device, asked or made once (each question costs the host about half a microsecond, which
// counts where a whole step takes ten). Plain C++ over the runtime's C functions; every part may be used from several host
// threads at once.
#pragma once

#include <cuda_runtime_api.h>

#include <atomic>
#include <mutex>

namespace gptgb {

constexpr int kMaxLaunchDevices = 64;

// The current device's number and its SM count.
inline cudaError_t device_sms(int* dev, int* sms) {
  static std::atomic<int> known[kMaxLaunchDevices];
  cudaError_t e = cudaGetDevice(dev);
  if (e != cudaSuccess) return e;
  if (*dev < 0 || *dev >= kMaxLaunchDevices) return cudaErrorInvalidDevice;
  *sms = known[*dev].load(std::memory_order_relaxed);
  if (*sms > 0) return cudaSuccess;
  e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *dev);
  if (e == cudaSuccess) known[*dev].store(*sms, std::memory_order_relaxed);
  return e;
}

// Largest dynamic shared memory that a kernel has been allowed on each device. It only grows: callers that want more take
// turns, so a smaller limit is never set behind a larger one, and `bytes` is what the device has been told.
struct SmemLimit {
  std::atomic<int> bytes[kMaxLaunchDevices];
  std::mutex mu;
  template <typename K>
  cudaError_t raise(K* kernel, int dev, int want) {
    if (want <= bytes[dev].load(std::memory_order_acquire)) return cudaSuccess;
    std::lock_guard<std::mutex> lk(mu);
    if (want <= bytes[dev].load(std::memory_order_relaxed)) return cudaSuccess;
    const cudaError_t e =
        cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize, want);
    if (e == cudaSuccess) bytes[dev].store(want, std::memory_order_release);
    return e;
  }
};

// One int of device memory per device, 0 when it is made, which the kernels launched there may write. The first caller on
// a device makes it; nullptr (and no CUDA error left behind) where that fails.
struct DeviceWord {
  std::atomic<int*> word[kMaxLaunchDevices];
  std::mutex mu;
  int* get() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return failed();
    if (dev < 0 || dev >= kMaxLaunchDevices) return nullptr;
    if (int* p = word[dev].load(std::memory_order_acquire)) return p;
    std::lock_guard<std::mutex> lk(mu);
    if (int* p = word[dev].load(std::memory_order_relaxed)) return p;
    void* p = nullptr;
    if (cudaMalloc(&p, sizeof(int)) != cudaSuccess) return failed();
    if (cudaMemset(p, 0, sizeof(int)) != cudaSuccess) {
      cudaFree(p);
      return failed();
    }
    word[dev].store(static_cast<int*>(p), std::memory_order_release);
    return static_cast<int*>(p);
  }

 private:
  static int* failed() {
    cudaGetLastError();
    return nullptr;
  }
};

}  // namespace gptgb
