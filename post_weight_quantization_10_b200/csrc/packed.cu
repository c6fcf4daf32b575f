// packed.cu -- product of activations with the packed b-bit codes of a solved
// layer: out[m][n] = sum over groups G of s[n][G] sum_{k in G} (c[n][k] - z[n][G]) x[m][k].
#include "host.cuh"
#include "packed_few.cuh"

using namespace admmq;

namespace admmq {
int packed_gemm_bf16(const PackedArgs& p, cudaStream_t st);  // packed_gemm_bf16.cu
int packed_gemm_fp16(const PackedArgs& p, cudaStream_t st);  // packed_gemm_fp16.cu
}  // namespace admmq

namespace {

// Tokens that the mma.sync kernel takes: up to there it is the faster one for
// most layers, beyond it the tensor-memory kernel.  In us, mma.sync against
// tcgen05: 9 to 12 tokens of 4096 -> 4096 (4 bits) 11.0 / 13.3, 4096 -> 6144 (3)
// 13.5 / 18.1, 4096 -> 24576 (4) 40 / 55, 12288 -> 4096 (2) 24.1 / 22.7; 16 tokens
// 13.1 / 13.2, 16.1 / 18.3, 52 / 48, 24.4 / 22.9.
constexpr int kFewTokens = 12;

template <typename X, int NT, int RT>
const void* few_kernel(int bits) {
  static const void* const table[8] = {
      (const void*)k_packed_few<X, NT, RT, 1>, (const void*)k_packed_few<X, NT, RT, 2>,
      (const void*)k_packed_few<X, NT, RT, 3>, (const void*)k_packed_few<X, NT, RT, 4>,
      (const void*)k_packed_few<X, NT, RT, 5>, (const void*)k_packed_few<X, NT, RT, 6>,
      (const void*)k_packed_few<X, NT, RT, 7>, (const void*)k_packed_few<X, NT, RT, 8>};
  return table[bits - 1];
}

template <typename X>
int launch_few(PackedArgs p, cudaStream_t st) {
  const int spans = cdiv(p.k, 128);
  // all activations next to two stages in half of the shared memory? (8 tokens of
  // 4096 -> 24576 at 3 bits: 28.9 us against 31.6 staged, 6 tokens 24.5 / 31.0; 2 of
  // 12288 -> 4096 13.3 / 12.6)
  const bool one = p.m <= 8 && (long long)p.m * (spans * 256 + 64) <= 70 * 1024;
  const int rows = one ? 16 : 64, blocks = cdiv(p.n, rows);
  // ranks, as long as all blocks run at once, three on an SM (a fourth block's
  // worth: 4 tokens of 12288 -> 4096 20.9 us instead of 14.6)
  int ranks = 1, shift = 0;
  if (!one)
    while (ranks < 8 && blocks * 2 * ranks <= 3 * num_sms() && spans >= 4 * ranks) ranks *= 2, ++shift;
  const int range = cdiv(spans, ranks), most = one ? 32 : 8;
  int per = 1;
  while (per < most && per < range) per *= 2;
  FewPlan plan(rows, per, range, p.bits, p.group, p.m, !one);
  while (plan.smem > (one ? 110 : 72) * 1024 && per > 1) {
    per /= 2;
    plan = FewPlan(rows, per, range, p.bits, p.group, p.m, !one);
  }
  plan.blocks = blocks;
  plan.rank_shift = shift;
  const void* kern = one         ? few_kernel<X, 1, 1>(p.bits)
                     : p.m <= 8  ? few_kernel<X, 1, 4>(p.bits)
                                 : few_kernel<X, 2, 4>(p.bits);
  CK(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, plan.smem));
  const int once = few_blocks(1) * num_sms(), grid = one && blocks > once ? once : blocks;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)(grid * ranks));
  lc.blockDim = dim3(kFewThreads);
  lc.dynamicSmemBytes = plan.smem;
  lc.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  void* argv[] = {&p, &plan};
  count_launch();
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
  const PackedArgs p{x,     packed, scale, zero,  out,               ldx,           (int)m,
                     d_out, d_in,   bits,  group, d_in / 32 * bits, d_in / group, out_dtype};
  const bool bf16 = x_dtype == ADMMQ_DTYPE_BF16, few = m <= kFewTokens;
  cudaStream_t st = (cudaStream_t)stream;
  if (few) return bf16 ? launch_few<__nv_bfloat16>(p, st) : launch_few<__half>(p, st);
  return bf16 ? packed_gemm_bf16(p, st) : packed_gemm_fp16(p, st);
}
