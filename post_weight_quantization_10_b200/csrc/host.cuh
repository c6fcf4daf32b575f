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

// Encodes a tiled tensor map (arguments as for cuTensorMapEncodeTiled).  That
// takes a current context, which a thread whose first use of the GPU is a call of
// this library has not got (cudaGetDevice sets none): the call is then made again
// with the device's context current.  (To make it current in front of every call
// would cost each 0.3 us.)
template <typename... Args>
bool encode_tiled(CUtensorMap* m, Args... args) {
  auto fn = encode_fn();
  if (!fn) return false;
  if (fn(m, args...) == CUDA_SUCCESS) return true;
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess &&
         fn(m, args...) == CUDA_SUCCESS;
}

inline int device_ok() {
  int dev = 0, major = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ADMMQ_ERR_CUDA;
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
