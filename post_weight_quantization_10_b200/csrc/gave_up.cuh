// gave_up.cuh -- the operators' bounded waits that gave up, told to the host.
//
// A kernel whose wait gives up (see ptx.cuh) ends with NaN in the outputs that
// it could not compute and sets a device word, which admmq_operators_check reads
// and clears.  Every translation unit with such kernels has a word of its own
// (device code is not linked across them) and hands out these functions.
#pragma once
#include "host.cuh"
#include "ptx.cuh"

namespace admmq {

static __device__ int g_gave_up;

// At a kernel's end, after a barrier of the block: abort_flag is what its waits set.
static __device__ __forceinline__ void report_gave_up(int abort_flag) {
  if (threadIdx.x == 0 && abort_flag) atomicExch(&g_gave_up, 1);
}

// Test hook: waits for a barrier that nothing completes.
static __global__ void k_give_up() {
  __shared__ uint64_t bar;
  __shared__ int abort_flag;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&bar), 1);
    abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  mbar_wait(smem_u32(&bar), 0, &abort_flag, nullptr);
  __syncthreads();
  report_gave_up(abort_flag);
}

struct GaveUp {
  int (*take)(int* any, cudaStream_t st);  // reads the word (after the stream) and clears it
  int (*give_up)(cudaStream_t st);         // launches the test hook
};

static int take_gave_up(int* any, cudaStream_t st) {
  int word = 0;
  CK(cudaMemcpyFromSymbolAsync(&word, g_gave_up, sizeof(int), 0, cudaMemcpyDeviceToHost, st));
  CK(cudaStreamSynchronize(st));
  if (word != 0) {
    const int zero = 0;
    CK(cudaMemcpyToSymbolAsync(g_gave_up, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, st));
    CK(cudaStreamSynchronize(st));
    *any = 1;
  }
  return ADMMQ_OK;
}

static int launch_give_up(cudaStream_t st) {
  count_launch();
  k_give_up<<<1, 32, 0, st>>>();
  CK(cudaGetLastError());
  return ADMMQ_OK;
}

}  // namespace admmq
