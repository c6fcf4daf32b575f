// packed.cu -- product of activations with the packed b-bit codes of a solved
// layer: out[m][n] = sum over groups G of s[n][G] sum_{k in G} (c[n][k] - z[n][G]) x[m][k].
#include "host.cuh"
#include "packed_few.cuh"
#include "packed_gemm_launch.cuh"

using namespace admmq;

namespace admmq {
int packed_gemm_bf16(const PackedArgs& p, cudaStream_t st);  // packed_gemm_bf16.cu
int packed_gemm_fp16(const PackedArgs& p, cudaStream_t st);  // packed_gemm_fp16.cu
extern const GaveUp mx_gave_up, packed_bf16_gave_up, packed_fp16_gave_up;  // mx.cu and these
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

// Shared memory of a block at most: half of an SM's, or a third (one stage of one
// span takes less than either).
constexpr int few_smem(bool one) { return (one ? 110 : 72) * 1024; }

// How a call is laid out.
struct FewLaunch {
  FewPlan plan;
  bool one;         // RT = 1, activations resident
  int ranks, grid;  // CTAs of a cluster; clusters
};

FewLaunch plan_few(const PackedArgs& p, int sms) {
  const int spans = cdiv(p.k, 128);
  // all activations next to two stages in half of the shared memory? (8 tokens of
  // 4096 -> 24576 at 3 bits: 28.9 us against 31.6 staged, 6 tokens 24.5 / 31.0; 2 of
  // 12288 -> 4096 13.3 / 12.6)
  const bool one = p.m <= 8 && p.m * (spans * 256ll + 64) <= 70 * 1024;
  const int rows = one ? 16 : 64, blocks = cdiv(p.n, rows);
  // ranks, as long as all blocks run at once, three on an SM (a fourth block's
  // worth: 4 tokens of 12288 -> 4096 20.9 us instead of 14.6)
  int ranks = 1, shift = 0;
  if (!one)
    while (ranks < 8 && blocks * 2 * ranks <= 3 * sms && spans >= 4 * ranks) ranks *= 2, ++shift;
  const int range = cdiv(spans, ranks), most = one ? 32 : 8;
  int per = 1;
  while (per < most && per < range) per *= 2;
  FewPlan plan(rows, per, range, p.bits, p.group, p.m, !one);
  while (plan.smem > few_smem(one) && per > 1) {
    per /= 2;
    plan = FewPlan(rows, per, range, p.bits, p.group, p.m, !one);
  }
  plan.blocks = blocks;
  plan.rank_shift = shift;
  // 16 bytes of scales at a time where a row, a stage and a rank's range each begin
  // on a whole piece of 4 groups.  (Ranges rounded up to whole pieces instead leave
  // the last ranks short: 10 tokens of 2560 -> 4096 11.0 us against 9.9 with 4-byte
  // copies, 12 of 2560 -> 6144 14.0 / 12.3, but 2 of 25600 -> 5120 40.6 / 43.3.)
  const int rank_groups = ranks > 1 ? range * (128 / p.group) : 0;
  plan.vec_scales = ((p.groups | plan.groups | rank_groups) & 3) == 0;
  const int once = few_blocks(1) * sms;
  return {plan, one, ranks, one && blocks > once ? once : blocks};
}

template <typename X>
int launch_few(PackedArgs p, cudaStream_t st) {
  FewLaunch l = plan_few(p, num_sms());
  const void* kern = l.one       ? few_kernel<X, 1, 1>(p.bits)
                     : p.m <= 8  ? few_kernel<X, 1, 4>(p.bits)
                                 : few_kernel<X, 2, 4>(p.bits);
  CK(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, few_smem(l.one)));
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)(l.grid * l.ranks));
  lc.blockDim = dim3(kFewThreads);
  lc.dynamicSmemBytes = l.plan.smem;
  lc.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = l.ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  void* argv[] = {&p, &l.plan};
  count_launch();
  CK(cudaLaunchKernelExC(&lc, kern, argv));
  return ADMMQ_OK;
}

// Sizes that the product takes.  (Rows up to 2^30 columns: the kernels count
// columns, also those of a stage or two past the last, in 32 bits.)
bool packed_shape_ok(int64_t m, int d_in, int d_out, int bits, int group) {
  return m >= 0 && m <= (1ll << 30) && d_in > 0 && d_in <= (1 << 30) && d_out > 0 &&
         d_in % 32 == 0 &&
         (group == 32 || group == 64 || group == 128) && d_in % group == 0 && bits >= 1 && bits <= 8;
}

PackedArgs packed_args(int64_t m, int d_in, int d_out, int bits, int group) {
  PackedArgs p = {};
  p.m = (int)m;
  p.n = d_out;
  p.k = d_in;
  p.bits = bits;
  p.group = group;
  p.words = d_in / 32 * bits;
  p.groups = d_in / group;
  return p;
}

}  // namespace

extern "C" int admmq_packed_matmul(const void* x, int x_dtype, int64_t m, int64_t ldx,
                                   const uint32_t* packed, const float* scale, const float* zero,
                                   int d_in, int d_out, int bits, int group, void* out,
                                   int out_dtype, void* stream) {
  if (!packed_shape_ok(m, d_in, d_out, bits, group) || ldx < d_in || (x_dtype != ADMMQ_DTYPE_BF16 && x_dtype != ADMMQ_DTYPE_F16) ||
      out_dtype < ADMMQ_DTYPE_F32 || out_dtype > ADMMQ_DTYPE_F16)
    return ADMMQ_ERR_INVALID_ARG;
  if (m == 0) return ADMMQ_OK;
  if (!x || !packed || !scale || !zero || !out || ((uintptr_t)x & 15) || ((uintptr_t)packed & 15) ||
      ((uintptr_t)scale & 3) || ((uintptr_t)zero & 3) || ((uintptr_t)out & 15) || ldx % 8 != 0)
    return ADMMQ_ERR_INVALID_ARG;
  int rc = device_ok();
  if (rc) return rc;
  PackedArgs p = packed_args(m, d_in, d_out, bits, group);
  p.x = x;
  p.packed = packed;
  p.scale = scale;
  p.zero = zero;
  p.out = out;
  p.ldx = ldx;
  p.out_dtype = out_dtype;
  const bool bf16 = x_dtype == ADMMQ_DTYPE_BF16, few = m <= kFewTokens;
  cudaStream_t st = (cudaStream_t)stream;
  if (few) return bf16 ? launch_few<__nv_bfloat16>(p, st) : launch_few<__half>(p, st);
  return bf16 ? packed_gemm_bf16(p, st) : packed_gemm_fp16(p, st);
}

extern "C" int admmq_debug_packed_plan(int64_t m, int d_in, int d_out, int bits, int group, int sms,
                                       int* plan) {
  if (!packed_shape_ok(m, d_in, d_out, bits, group) || m == 0 || !plan) return ADMMQ_ERR_INVALID_ARG;
  const PackedArgs p = packed_args(m, d_in, d_out, bits, group);
  if (sms <= 0) sms = num_sms();
  if (m <= kFewTokens) {
    const FewLaunch l = plan_few(p, sms);
    const int v[10] = {l.one || m <= 8 ? 8 : 16, l.one ? 16 : 64, l.plan.blocks, l.grid, l.ranks, l.plan.range,
                       l.plan.spans, l.plan.groups, l.plan.x_staged, l.plan.vec_scales};
    for (int i = 0; i < 10; ++i) plan[i] = v[i];
    return ADMMQ_OK;
  }
  PackedGemmPlan g;
  const int tile = packed_tile(p, sms);
  const int rc = tile == 64    ? plan_gemm<64, 1>(p, sms, g)
                 : tile == 128 ? plan_gemm<128, 1>(p, sms, g)
                               : plan_gemm<256, 2>(p, sms, g);
  if (rc) return rc;
  const int v[10] = {tile, 128, g.a.tiles, g.clusters, g.ranks, g.a.range, g.a.stages, g.a.wbufs, 0, 0};
  for (int i = 0; i < 10; ++i) plan[i] = v[i];
  return ADMMQ_OK;
}

// The words of all units with operator kernels: mx, few tokens, many in bf16 and in fp16.
static const GaveUp* gave_up_unit(int i) {
  static const GaveUp few = {take_gave_up, launch_give_up};
  const GaveUp* const units[] = {&mx_gave_up, &few, &packed_bf16_gave_up, &packed_fp16_gave_up};
  return i >= 0 && i < 4 ? units[i] : nullptr;
}

extern "C" int admmq_operators_check(void* stream) {
  int rc = device_ok(), any = 0;
  for (int i = 0; rc == ADMMQ_OK && gave_up_unit(i); ++i)
    rc = gave_up_unit(i)->take(&any, (cudaStream_t)stream);
  return rc ? rc : any ? ADMMQ_ERR_TIMEOUT : ADMMQ_OK;
}

extern "C" int admmq_debug_give_up(int unit, void* stream) {
  if (!gave_up_unit(unit)) return ADMMQ_ERR_INVALID_ARG;
  const int rc = device_ok();
  return rc ? rc : gave_up_unit(unit)->give_up((cudaStream_t)stream);
}
