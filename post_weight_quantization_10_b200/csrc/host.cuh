// host.cuh -- host-side helpers shared by the library's translation units:
// the launch counter, device queries and the tensor-map encoder.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <stdint.h>

#include "../../include/admmq.h"

#define CK(x)                                      \
  do {                                             \
    cudaError_t e_ = (x);                          \
    if (e_ != cudaSuccess) return ADMMQ_ERR_CUDA;  \
  } while (0)

namespace admmq {

inline unsigned long long g_launches = 0;  // kernels launched by this library
inline void count_launch() { __atomic_fetch_add(&g_launches, 1ull, __ATOMIC_RELAXED); }

inline int num_sms() {
  int dev = 0, n = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n > 0 ? n : 1;
}

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }
  return fn;
}

// Whether the current device is one of those that the library is built for.  Its
// context becomes the calling thread's (cudaSetDevice does that, cudaGetDevice
// does not): a thread whose first use of the GPU is a call of this library
// could not encode a tensor map without one.
inline int device_ok() {
  int dev = 0, major = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaSetDevice(dev) != cudaSuccess) return ADMMQ_ERR_CUDA;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess)
    return ADMMQ_ERR_CUDA;
  return major == 10 ? ADMMQ_OK : ADMMQ_ERR_UNSUPPORTED;
}

// Shared memory that a block may ask for at launch beyond its static variables.
// Kernels whose plans differ from call to call are allowed the most that any
// plan asks for, not their own: the limit belongs to the kernel, and another
// thread could set its own between this thread's setting and launch.
constexpr int kMaxSmem = 227 * 1024;

inline int cdiv(long long a, long long b) { return (int)((a + b - 1) / b); }

}  // namespace admmq
