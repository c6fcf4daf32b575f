// packed.cu -- product of activations with the packed b-bit codes of a solved
// layer: out[m][n] = sum over groups G of s[n][G] sum_{k in G} (c[n][k] - z[n][G]) x[m][k].
#include "host.cuh"
#include "packed_few.cuh"
#include "packed_gemm.cuh"
#include "tmem_fair.cuh"

using namespace admmq;

namespace {

// Tokens that the mma.sync kernel takes.
constexpr int kFewTokens = 32;

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
  // all activations next to two stages in a third of the shared memory?
  const bool one = p.m <= 8 && (long long)p.m * (spans * 256 + 64) <= 34 * 1024;
  const int rows = one ? 16 : 64, blocks = cdiv(p.n, rows);
  int ranks = 1, shift = 0;
  if (!one)
    while (ranks < 8 && blocks * 2 * ranks <= 4 * num_sms() && spans >= 4 * ranks) ranks *= 2, ++shift;
  const int range = cdiv(spans, ranks), most = one ? 32 : 8;
  int per = 1;
  while (per < most && per < range) per *= 2;
  FewPlan plan(rows, per, range, p.bits, p.group, p.m, !one);
  while (plan.smem > 72 * 1024 && per > 1) {
    per /= 2;
    plan = FewPlan(rows, per, range, p.bits, p.group, p.m, !one);
  }
  plan.blocks = blocks;
  plan.rank_shift = shift;
  const void* kern = one         ? few_kernel<X, 1, 1>(p.bits)
                     : p.m <= 8  ? few_kernel<X, 1, 4>(p.bits)
                     : p.m <= 16 ? few_kernel<X, 2, 4>(p.bits)
                                 : few_kernel<X, 4, 4>(p.bits);
  CK(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, plan.smem));
  const int grid = one && blocks > 3 * num_sms() ? 3 * num_sms() : blocks;
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

bool make_x_map(CUtensorMap* m, const PackedArgs& p, bool bf16, int box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)p.k, (cuuint64_t)p.m};
  cuuint64_t strides[1] = {(cuuint64_t)p.ldx * 2};
  cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
            const_cast<void*>(p.x), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Packed rows as bytes, boxes of a 128-code chunk (16 b bytes).
bool make_w_map(CUtensorMap* m, const PackedArgs& p, int box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)p.words * 4, (cuuint64_t)p.n};
  cuuint64_t strides[1] = {(cuuint64_t)p.words * 4};
  cuuint32_t box[2] = {(cuuint32_t)(16 * p.bits), (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  const CUtensorMapSwizzle sw = p.bits == 2   ? CU_TENSOR_MAP_SWIZZLE_32B
                                : p.bits == 4 ? CU_TENSOR_MAP_SWIZZLE_64B
                                : p.bits == 8 ? CU_TENSOR_MAP_SWIZZLE_128B
                                              : CU_TENSOR_MAP_SWIZZLE_NONE;
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint32_t*>(p.packed), dims, strides,
            box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename X, int TN, int C>
int launch_gemm(const PackedArgs& p, cudaStream_t st) {
  using Cfg = PackedCfg<TN, C>;
  PackedGemmArgs a;
  a.p = p;
  a.tiles_m = cdiv(p.m, TN * C);
  const long long tiles = (long long)a.tiles_m * cdiv(p.n, 128);
  if (tiles > (1 << 28)) return ADMMQ_ERR_UNSUPPORTED;
  a.tiles = (int)tiles;
  a.chunks = cdiv(p.k, 128);
  a.passes = 128 / p.group;
  a.w_tma = p.words % 4 == 0;
  int ranks = C;
  if (C == 1)
    while (ranks < 8 && a.chunks >= 4 * ranks && tiles * 2 * ranks <= num_sms()) ranks *= 2;
  a.range = C == 1 ? cdiv(a.chunks, ranks) : a.chunks;
  const int room = 226 * 1024, wbytes = 16 * Cfg::ROWS * p.bits;
  a.stages = 4;
  a.wbufs = (room - 1024 - a.stages * Cfg::STAGE - 512) / wbytes;
  if (a.wbufs > 4) a.wbufs = 4;
  if (!make_x_map(&a.x, p, __is_same(X, __nv_bfloat16), TN)) return ADMMQ_ERR_CUDA;
  if (a.w_tma && !make_w_map(&a.w, p, Cfg::ROWS)) return ADMMQ_ERR_CUDA;
  int smem = a.stages * Cfg::STAGE + a.wbufs * wbytes + 1024 + 512;
  smem = tmem_fair_smem(smem, Cfg::TMEM_COLS);
  auto kern = k_packed_gemm<X, TN, C>;
  CK(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
  const int most = C == 1 && ranks > 1 ? a.tiles : num_sms() / ranks;
  const int clusters = a.tiles < most ? a.tiles : most;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)(clusters * ranks));
  lc.blockDim = dim3(kPackedThreads);
  lc.dynamicSmemBytes = smem;
  lc.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  count_launch();
  CK(cudaLaunchKernelEx(&lc, kern, a));
  return ADMMQ_OK;
}

template <typename X>
int launch_packed(const PackedArgs& p, cudaStream_t st) {
  if (p.m <= kFewTokens) return launch_few<X>(p, st);
  if (p.m <= 64) return launch_gemm<X, 64, 1>(p, st);
  if (p.m <= 128) return launch_gemm<X, 128, 1>(p, st);
  if (p.m <= 256) return launch_gemm<X, 256, 1>(p, st);
  return launch_gemm<X, 256, 2>(p, st);
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
  return x_dtype == ADMMQ_DTYPE_BF16 ? launch_packed<__nv_bfloat16>(p, (cudaStream_t)stream)
                                     : launch_packed<__half>(p, (cudaStream_t)stream);
}
