// packed.cu -- product of activations with the packed b-bit codes of a solved
// layer: out[m][n] = sum over groups G of s[n][G] sum_{k in G} (c[n][k] - z[n][G]) x[m][k].
#include "host.cuh"
#include "packed_few.cuh"
#include "product.cuh"

using namespace admmq;

namespace {

template <typename T>
struct DenseElement {
  const T* x;
  long long ld;
  __device__ __forceinline__ float operator()(long long row, int k) const {
    return (float)x[row * ld + k];
  }
};

struct PackedElement {
  const uint32_t* packed;
  const float *scale, *zero;
  int words, bits, group, groups;
  __device__ __forceinline__ float operator()(long long row, int k) const {
    const int pos = k * bits, w = pos >> 5, sh = pos & 31;
    const uint32_t* p = packed + row * words;
    uint32_t c = p[w] >> sh;
    if (sh + bits > 32) c |= p[w + 1] << (32 - sh);
    c &= (1u << bits) - 1u;
    const long long g = row * groups + k / group;
    return ((float)c - zero[g]) * scale[g];
  }
};

// Tokens up to which the weights go straight into registers.
constexpr int kFewTokens = 16;

template <typename X>
const void* few_kernel(int m, int bits) {
  static const void* const one[8] = {
      (const void*)k_packed_few<X, 1, 1>, (const void*)k_packed_few<X, 1, 2>,
      (const void*)k_packed_few<X, 1, 3>, (const void*)k_packed_few<X, 1, 4>,
      (const void*)k_packed_few<X, 1, 5>, (const void*)k_packed_few<X, 1, 6>,
      (const void*)k_packed_few<X, 1, 7>, (const void*)k_packed_few<X, 1, 8>};
  static const void* const two[8] = {
      (const void*)k_packed_few<X, 2, 1>, (const void*)k_packed_few<X, 2, 2>,
      (const void*)k_packed_few<X, 2, 3>, (const void*)k_packed_few<X, 2, 4>,
      (const void*)k_packed_few<X, 2, 5>, (const void*)k_packed_few<X, 2, 6>,
      (const void*)k_packed_few<X, 2, 7>, (const void*)k_packed_few<X, 2, 8>};
  return (m <= 8 ? one : two)[bits - 1];
}

template <typename X>
int launch_few(const PackedArgs& p, cudaStream_t st) {
  const int blocks = cdiv(p.n, kFewRows), spans = cdiv(p.k, 128);
  // enough blocks for three on each SM, each with a span for every warp
  int ranks = 1;
  while (ranks < 8 && blocks * 2 * ranks <= 3 * num_sms() && spans >= 16 * ranks) ranks *= 2;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)(blocks * ranks));
  lc.blockDim = dim3(kFewThreads);
  lc.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  count_launch();
  const void* kern = few_kernel<X>(p.m, p.bits);
  PackedArgs args = p;
  void* argv[] = {&args};
  CK(cudaLaunchKernelExC(&lc, kern, argv));
  return ADMMQ_OK;
}

}  // namespace

extern "C" int admmq_packed_matmul(const void* x, int x_dtype, int64_t m, int64_t ldx,
                                   const uint32_t* packed, const float* scale, const float* zero,
                                   int d_in, int d_out, int bits, int group, void* out,
                                   int out_dtype, void* stream) {
  if (m < 0 || m > (1ll << 30) || d_in <= 0 || d_out <= 0 || d_in % 32 != 0 ||
      (group != 32 && group != 64 && group != 128) || d_in % group != 0 || bits < 1 || bits > 8 ||
      ldx < d_in || (x_dtype != ADMMQ_DTYPE_BF16 && x_dtype != ADMMQ_DTYPE_F16) ||
      out_dtype < ADMMQ_DTYPE_F32 || out_dtype > ADMMQ_DTYPE_F16)
    return ADMMQ_ERR_INVALID_ARG;
  if (m == 0) return ADMMQ_OK;
  if (!x || !packed || !scale || !zero || !out || ((uintptr_t)x & 15) || ((uintptr_t)packed & 15) ||
      ((uintptr_t)scale & 3) || ((uintptr_t)zero & 3) || ((uintptr_t)out & 15) || ldx % 8 != 0)
    return ADMMQ_ERR_INVALID_ARG;
  int rc = device_ok();
  if (rc) return rc;
  const PackedElement w{packed, scale, zero, d_in / 32 * bits, bits, group, d_in / group};
  cudaStream_t st = (cudaStream_t)stream;
  if (m <= kFewTokens) {
    const PackedArgs p{x,        packed, scale, zero, out,       ldx, (int)m,
                       d_out,    d_in,   bits,  group, d_in / 32 * bits, d_in / group, out_dtype};
    return x_dtype == ADMMQ_DTYPE_BF16 ? launch_few<__nv_bfloat16>(p, st) : launch_few<__half>(p, st);
  }
#define PACKED_T(X, T)                                                                          \
  launch_product<T>(DenseElement<X>{(const X*)x, ldx}, w, (int)m, d_out, d_in, nullptr, nullptr, \
                    (T*)out, st)
#define PACKED_X(X)                         \
  if (out_dtype == ADMMQ_DTYPE_F32) {       \
    PACKED_T(X, float);                     \
  } else if (out_dtype == ADMMQ_DTYPE_BF16) { \
    PACKED_T(X, __nv_bfloat16);             \
  } else {                                  \
    PACKED_T(X, __half);                    \
  }
  if (x_dtype == ADMMQ_DTYPE_BF16) {
    PACKED_X(__nv_bfloat16)
  } else {
    PACKED_X(__half)
  }
#undef PACKED_X
#undef PACKED_T
  CK(cudaGetLastError());
  return ADMMQ_OK;
}
