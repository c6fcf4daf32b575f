// async.cuh -- further PTX wrappers of the quantised-weight products: bulk
// copies and reads of a cluster's shared memory.
#pragma once
#include <stdint.h>

namespace admmq {

// Position in a ring of n buffers: the buffer and the parity of its use.  (A
// role is one thread or a few warps: a division per step would be most of its
// time.)
struct Ring {
  int i = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int n) {
    if (++i == n) {
      i = 0;
      phase ^= 1u;
    }
  }
};

// True for one lane of the (converged) warp.  A role that issues tcgen05
// instructions runs on its whole warp and elects a lane for the issue alone:
// descriptors and loop state then stay in uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// Untiled asynchronous copy global -> shared (16-byte aligned, size a multiple
// of 16), completing on an mbarrier.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// A float in the shared memory of a CTA of the cluster.
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr_cluster) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr_cluster) : "memory");
  return v;
}

}  // namespace admmq
