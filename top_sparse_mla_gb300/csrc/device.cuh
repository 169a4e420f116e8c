// The device that a call is for.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

#include "dsa_sparse_attn.h"

namespace dsa {

// SMs of the current device, which has to be of compute capability 10.3.  These are properties of the device,
// asked for once.
inline int gb300_sms(int* sms) {
  constexpr int DEVICES = 64;
  static std::atomic<int> known[DEVICES];   // SMs; 0: not asked for, -1: another architecture
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DSA_ERR_CUDA;
  int n = dev < DEVICES ? known[dev].load(std::memory_order_relaxed) : 0;
  if (n == 0) {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return DSA_ERR_CUDA;
    if (major != 10 || minor != 3) n = -1;
    if (dev < DEVICES) known[dev].store(n, std::memory_order_relaxed);
  }
  if (n < 0) return DSA_ERR_UNSUPPORTED_DEVICE;
  *sms = n;
  return DSA_OK;
}

// SMs of the current device, of whatever capability: for sizes of workspaces.
inline int current_sms(int* sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DSA_ERR_CUDA;
  return cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace dsa
