// product.cuh -- out[m][n] = g sum_k A(m, k) B(n, k) in fp32 on the CUDA
// cores, the elements of A and B given by functors.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "host.cuh"

namespace admmq {

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(__half* p, float v) { *p = __float2half_rn(v); }

// 64 x 64 outputs a block of 256 threads, 4 x 4 each, 32 of K at a time.
template <typename T, class A, class B>
__global__ void __launch_bounds__(256)
    k_product(A a, B b, int m, int n, int k, const float* __restrict__ ga,
              const float* __restrict__ gb, T* __restrict__ out) {
  __shared__ float sa[32][65], sb[32][65];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const long long m0 = (long long)blockIdx.y * 64;
  const int n0 = blockIdx.x * 64;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < k; k0 += 32) {
    for (int i = threadIdx.x; i < 64 * 32; i += 256) {
      const int r = i >> 5, c = i & 31;
      sa[c][r] = m0 + r < m ? a(m0 + r, k0 + c) : 0.f;
      sb[c][r] = n0 + r < n ? b(n0 + r, k0 + c) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < 32; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] += sa[c][ty * 4 + i] * sb[c][tx * 4 + j];
    __syncthreads();
  }
  const float g = (ga ? *ga : 1.f) * (gb ? *gb : 1.f);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const long long r = m0 + ty * 4 + i;
      const int c = n0 + tx * 4 + j;
      if (r < m && c < n) put(out + r * n + c, acc[i][j] * g);
    }
}

template <typename T, class A, class B>
void launch_product(A a, B b, int m, int n, int k, const float* ga, const float* gb, T* out,
                    cudaStream_t st) {
  count_launch();
  k_product<T><<<dim3(cdiv(n, 64), cdiv(m, 64)), 256, 0, st>>>(a, b, m, n, k, ga, gb, out);
}

}  // namespace admmq
