// qk_host.h -- host-side helpers shared by the translation units of the C ABI.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/qk.h"

namespace qk {

constexpr uint64_t kWaitTimeoutNs = 1000000000ull;  // 1 s bound on any in-kernel wait

// What a launch needs to know of the calling thread's current device.
struct CurrentDevice {
  int index;
  int sms;
  int smem_optin;
  int* status;  // device address of the status word
};
// Facts of the current device, looked up once per device (qk_api.cu).
qk_status current_device(CurrentDevice* out);

inline int elem_size(int dt) { return dt == QK_F32 ? 4 : 2; }
inline bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }
inline bool aligned_to(const void* ptr, size_t n) { return (reinterpret_cast<uintptr_t>(ptr) % n) == 0; }

// [a, a+na) and [b, b+nb) share a byte.
inline bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  if (a == nullptr || b == nullptr || na <= 0 || nb <= 0) return false;
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
  return pa < pb + uintptr_t(nb) && pb < pa + uintptr_t(na);
}

// A launch with programmatic stream serialisation: every kernel of the library
// waits for the previous grid before its first global access.
template <typename... P, typename... A>
qk_status launch_pdl(void (*kernel)(P...), dim3 grid, int threads, size_t smem, void* stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = grid;
  cfg.blockDim = dim3(unsigned(threads), 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, P(args)...) != cudaSuccess) {
    cudaGetLastError();
    return QK_ERR_LAUNCH;
  }
  return QK_OK;
}

}  // namespace qk
