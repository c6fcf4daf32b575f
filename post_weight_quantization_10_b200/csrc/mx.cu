// mx.cu -- microscaled 4-bit floating point matrices (mxfp4, nvfp4):
// quantisation, dequantisation and the product of two of them.
#include "host.cuh"
#include "async.cuh"
#include "mx.cuh"
#include "mx_gemm.cuh"
#include "tmem_fair.cuh"

namespace admmq {
extern const GaveUp mx_gave_up = {take_gave_up, launch_give_up};
}

using namespace admmq;

namespace {

// A block of threads takes 128 rows x SPAN columns: the scale tiles it fills (or
// reads) are whole and lie next to each other.  A lane takes 16 elements: an
// nvfp4 block, or half of an mxfp4 one, whose two lanes share its largest
// magnitude.  With 512 columns a warp's accesses are a row's next kilobyte;
// with 128 it takes four rows at a time, and there are four times the blocks:
// for matrices of less than four blocks an SM (there and back, 512 against 128
// columns: 48 x 12288 8.1 / 5.0 us to quantise, 2047 x 12288 37.7 / 35.0; but
// 24576 x 4096 85.5 / 89.0, 25600 x 5120 dequantised 60 / 64).
// What bounds them: HBM for 16-bit to mxfp4 (24576 x 4096 in about 40 us, 6.2 TB/s)
// and for dequantisation (25600 x 5120 nvfp4 to bf16 57 us, 5.9 TB/s of 6.5); for
// nvfp4 instructions: 21 an element, which is rounded twice (see quantize16), 64 %
// of the issue slots and 52 % of the ALU (no other pipe above 31 %), the rest of
// the slots lost to loads, results and the tile's barriers: 2047 x 12288 in 23 us,
// HBM would need 10.
constexpr int kMxThreads = 256;
constexpr int kMxWarps = kMxThreads / 32;

template <int FMT, typename T, int SPAN>
__global__ void __launch_bounds__(kMxThreads)
    k_mx_quantize(const T* __restrict__ x, long long rows, int k, long long ld, int spans,
                  const float* __restrict__ tensor_scale, uint8_t* __restrict__ codes,
                  uint8_t* __restrict__ scale) {
  constexpr int TILE_K = MxFormat<FMT>::TILE_K;
  constexpr int LANES = MxFormat<FMT>::BLOCK / 16;  // lanes that share a block
  constexpr int TILES = SPAN / TILE_K;
  constexpr int ROW_LANES = SPAN / 16, ROWS = 32 / ROW_LANES;  // of a warp: lanes of a row, rows
  __shared__ __align__(16) uint8_t tile[TILES * kScaleTile];
  let_next_kernel_start();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long row_tile = blockIdx.x / spans;
  const int span = (int)(blockIdx.x - row_tile * spans);
  const int col = span * SPAN + (lane % ROW_LANES) * 16, row0 = warp * ROWS + lane / ROW_LANES;
  const float g = FMT == MX_NVFP4 && tensor_scale ? *tensor_scale : 1.f;
  const float r6g = 1.f / (6.f * g);
  const int col_tiles = (k + TILE_K - 1) / TILE_K;
  const int here = min(TILES, col_tiles - span * TILES);
  const int last = rows - row_tile * 128 < 128 ? (int)(rows - row_tile * 128) : 128;
  // bytes of blocks or rows that do not exist are zero (blocks: in a row's last tile)
  if (last < 128 || (k % TILE_K != 0 && span == spans - 1))
    for (int i = threadIdx.x; i < TILES * kScaleTile / 16; i += kMxThreads)
      reinterpret_cast<uint4*>(tile)[i] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  const T* src = x + (row_tile * 128 + row0) * ld + col;
  uint8_t* dst = codes + ((row_tile * 128 + row0) * k + col) / 2;
  constexpr int STEP = kMxWarps * ROWS;  // rows from one of a lane's to its next
  const long long src_step = ld * STEP, dst_step = (long long)(k / 2) * STEP;
  const int c = lane % ROW_LANES / LANES;
  uint8_t* to = tile + (c >> 2) * kScaleTile + (c & 3);
  // rows of the warp's first lane, and of this one; a block's lanes are inside
  // or outside together, all stay for the shuffle
  const int n = (last - warp * ROWS + STEP - 1) / STEP;
  const int mine = col < k ? (last - row0 + STEP - 1) / STEP : 0;
  const bool wide = (((uintptr_t)x | (uintptr_t)(ld * sizeof(T))) & 31) == 0;
  // a few rows' loads go out before the first is used (the rare exact path's
  // branch would keep the compiler from doing so itself)
  constexpr int AHEAD = 4;
  for (int j0 = 0; j0 < n; j0 += AHEAD) {
    Raw16<T> raw[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
#pragma unroll
      for (int i = 0; i < (int)(4 * sizeof(T)); ++i) raw[j].w[i] = 0u;
      if (j0 + j < mine) load_raw(src + j * src_step, wide, raw[j]);
    }
    src += AHEAD * src_step;
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      if (j0 + j >= n) break;
      float v[16];
      values_of(raw[j], v);
      uint32_t amax = amax_of(raw[j]);
      if (LANES == 2) amax = max(amax, __shfl_xor_sync(~0u, amax, 1));
      const uint32_t byte = block_scale<FMT>(amax, g, r6g);
      const uint2 out = quantize16<FMT>(v, byte, g);
      if (j0 + j < mine) {
        *reinterpret_cast<uint2*>(dst) = out;
        if (lane % LANES == 0) to[scale_at((j0 + j) * STEP + row0, 0)] = (uint8_t)byte;
      }
      dst += dst_step;
    }
  }
  __syncthreads();
  uint4* out = reinterpret_cast<uint4*>(scale + (row_tile * col_tiles + span * TILES) * kScaleTile);
  for (int i = threadIdx.x; i < here * kScaleTile / 16; i += kMxThreads)
    out[i] = reinterpret_cast<const uint4*>(tile)[i];
}

template <int FMT, typename T, int SPAN>
__global__ void __launch_bounds__(kMxThreads)
    k_mx_dequantize(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scale,
                    long long rows, int k, int spans, const float* __restrict__ tensor_scale,
                    T* __restrict__ out, long long ld) {
  constexpr int TILE_K = MxFormat<FMT>::TILE_K;
  constexpr int LANES = MxFormat<FMT>::BLOCK / 16;
  constexpr int TILES = SPAN / TILE_K;
  constexpr int ROW_LANES = SPAN / 16, ROWS = 32 / ROW_LANES;  // of a warp: lanes of a row, rows
  __shared__ __align__(16) uint8_t tile[TILES * kScaleTile];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long row_tile = blockIdx.x / spans;
  const int span = (int)(blockIdx.x - row_tile * spans);
  const int col = span * SPAN + (lane % ROW_LANES) * 16, row0 = warp * ROWS + lane / ROW_LANES;
  const float g = FMT == MX_NVFP4 && tensor_scale ? *tensor_scale : 1.f;
  const int col_tiles = (k + TILE_K - 1) / TILE_K;
  const int here = min(TILES, col_tiles - span * TILES);
  const uint4* in =
      reinterpret_cast<const uint4*>(scale + (row_tile * col_tiles + span * TILES) * kScaleTile);
  for (int i = threadIdx.x; i < here * kScaleTile / 16; i += kMxThreads)
    reinterpret_cast<uint4*>(tile)[i] = __ldg(in + i);
  __syncthreads();
  if (col >= k) return;
  const int last = rows - row_tile * 128 < 128 ? (int)(rows - row_tile * 128) : 128;
  constexpr int STEP = kMxWarps * ROWS;
  const int n = (last - row0 + STEP - 1) / STEP;
  const uint8_t* src = codes + ((row_tile * 128 + row0) * k + col) / 2;
  T* dst = out + (row_tile * 128 + row0) * ld + col;
  const long long src_step = (long long)(k / 2) * STEP, dst_step = ld * STEP;
  const int c = lane % ROW_LANES / LANES;
  const uint8_t* from = tile + (c >> 2) * kScaleTile + (c & 3);
  const bool wide = (((uintptr_t)out | (uintptr_t)(ld * sizeof(T))) & 31) == 0;
  constexpr int AHEAD = 8;
  for (int j0 = 0; j0 < n; j0 += AHEAD) {
    uint2 w[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j)
      w[j] = j0 + j < n ? __ldg(reinterpret_cast<const uint2*>(src + j * src_step)) : make_uint2(0, 0);
    src += AHEAD * src_step;
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      if (j0 + j >= n) break;
      const float t = block_step<FMT>(from[scale_at((j0 + j) * STEP + row0, 0)], g);
      float v[16];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 f = e2m1x2_values(((i < 4 ? w[j].x : w[j].y) >> (8 * (i & 3))) & 0xFFu);
        v[2 * i] = f.x * t;
        v[2 * i + 1] = f.y * t;
      }
      Raw16<T> r;
      raw_of(v, r);
      store_raw(dst, wide, r);
      dst += dst_step;
    }
  }
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }
int mx_tile_k(int fmt) { return fmt == ADMMQ_MX_MXFP4 ? 128 : 64; }
bool mx_shape_ok(int64_t rows, int k, int fmt) {
  return rows >= 0 && rows <= (1ll << 30) && k > 0 && k % 32 == 0 && k <= (1 << 24) &&
         (fmt == ADMMQ_MX_MXFP4 || fmt == ADMMQ_MX_NVFP4);
}
int dtype_size(int dtype) { return dtype == ADMMQ_DTYPE_F32 ? 4 : 2; }
// Codes [rows][k / 2] in boxes of 128 bytes x box_rows, 128-byte swizzle,
// bytes out of range read as zero (the code of 0).
bool make_codes_map(CUtensorMap* m, const void* ptr, int k, int64_t rows, int box_rows) {
  cuuint64_t dims[2] = {(cuuint64_t)k / 2, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)k / 2};
  cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  return encode_tiled(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

// Scale tiles as rows of 128 words, boxes of `tiles` rows; rows out of range
// read as zero.
bool make_scales_map(CUtensorMap* m, const void* ptr, int64_t tiles, int box_rows) {
  cuuint64_t dims[2] = {kScaleTile / 4, (cuuint64_t)tiles};
  cuuint64_t strides[1] = {kScaleTile};
  cuuint32_t box[2] = {kScaleTile / 4, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  return encode_tiled(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(ptr), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

template <int FMT, typename T>
int launch_pair(const uint8_t* w_codes, const uint8_t* x_codes, const MxArgs& q, cudaStream_t st) {
  using Cfg = MxPairCfg<FMT>;
  MxPairArgs p;
  p.gw = q.gw;
  p.gx = q.gx;
  p.out = q.out;
  p.m = q.m;
  p.n = q.n;
  p.k = q.k;
  p.tiles_m = cdiv(q.m, 256);
  const long long tiles = (long long)p.tiles_m * cdiv(q.n, 256);
  if (tiles > (1 << 28)) return ADMMQ_ERR_UNSUPPORTED;
  p.tiles = (int)tiles;
  p.kblocks = q.kblocks;
  p.col_tiles = q.col_tiles;
  p.stages = (226 * 1024 - 1024) / (Cfg::STAGE + 16);
  if (!make_codes_map(&p.w, w_codes, q.k, q.n, 128) || !make_codes_map(&p.x, x_codes, q.k, q.m, 128) ||
      !make_scales_map(&p.ws, q.w_scale, (int64_t)cdiv(q.n, 128) * q.col_tiles, Cfg::NSF) ||
      !make_scales_map(&p.xs, q.x_scale, (int64_t)cdiv(q.m, 128) * q.col_tiles, Cfg::NSF))
    return ADMMQ_ERR_CUDA;
  const int smem = tmem_fair_smem(p.stages * (Cfg::STAGE + 16) + 1024 + 64, 512);
  auto kern = k_mx_pair<FMT, T>;
  CK(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
  const int pairs = num_sms() / 2;
  count_launch();
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)(2 * (p.tiles < pairs ? p.tiles : pairs)));
  lc.blockDim = dim3(kMxPairThreads);
  lc.dynamicSmemBytes = smem;
  lc.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = q.overlap ? 1 : 0;
  CK(cudaLaunchKernelEx(&lc, kern, p));
  return ADMMQ_OK;
}

// How k_mx_tile's work is laid out: ranks of a cluster (returned), stages.
// `fits`: every stage of a block is resident at once.
int plan_tile(MxArgs& p, int fmt, bool& fits) {
  const int nsf = kMxBK / mx_tile_k(fmt);
  const int tiles = p.tiles_n, sms = num_sms();
  int ranks = 1;
  while (ranks < 8 && 2 * ranks <= p.kblocks && tiles * 2 * ranks <= cluster_ctas(2 * ranks, sms)) ranks *= 2;
  p.stage_bytes = 128 * 128 + ((p.tn * 128 + 1023) & ~1023) + ((2 * nsf * kScaleTile + 1023) & ~1023);
  p.part_bytes = ranks > 1 ? ranks * cdiv(p.tn, ranks) * 512 : 0;
  // everything that a block reads on its way at once, or half of an SM's
  // shared memory where the blocks are more than the SMs
  const int blocks = cdiv(p.kblocks, ranks), room = tiles * ranks > sms ? 108 * 1024 : 216 * 1024;
  p.stages = (room - p.part_bytes) / p.stage_bytes;
  fits = p.stages >= blocks;
  if (fits) p.stages = blocks;
  return ranks;
}

// Tokens that k_mx_tile quantises itself, where all of a block's stages are
// resident: every block repeats the work for its part of k, which takes up to 8
// tokens no longer than a launch of its own (4096 -> 4096: 1 token 5.6 us device
// time against 6.0, 8 tokens 6.6 against 6.5, 16 tokens 8.6 against 7.2) and
// saves the host a launch and a workspace.
constexpr int kFusedTokens = 8;

template <int FMT, typename T>
int launch_tile(MxArgs& p, bool fused, cudaStream_t st) {
  constexpr int NSF = kMxBK / MxFormat<FMT>::TILE_K;
  bool fits;
  const int ranks = plan_tile(p, FMT, fits);
  const int tiles = p.tiles_n, cols = ((p.tn + 31) & ~31) + 8 * NSF;
  p.tmem_cols = 32;
  while (p.tmem_cols < cols) p.tmem_cols *= 2;
  const int smem = tmem_fair_smem(p.stages * p.stage_bytes + p.part_bytes + 1024 + 16 * p.stages + 64, p.tmem_cols);
  auto kern = fused ? k_mx_tile<FMT, T, true> : k_mx_tile<FMT, T, false>;
  CK(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem));
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)(tiles * ranks));
  lc.blockDim = dim3(kMxTileThreads);
  lc.dynamicSmemBytes = smem;
  lc.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = p.overlap ? 2 : 1;
  count_launch();
  CK(cudaLaunchKernelEx(&lc, kern, p));
  return ADMMQ_OK;
}

bool dtype_ok(int dtype) { return dtype >= ADMMQ_DTYPE_F32 && dtype <= ADMMQ_DTYPE_F16; }

}  // namespace

// Calls BODY(FMT, T) with the format and element type of the arguments.
#define MX_DISPATCH_T(FMT, dtype, BODY)                  \
  if ((dtype) == ADMMQ_DTYPE_F32) {                      \
    BODY(FMT, float);                                    \
  } else if ((dtype) == ADMMQ_DTYPE_BF16) {              \
    BODY(FMT, __nv_bfloat16);                            \
  } else {                                               \
    BODY(FMT, __half);                                   \
  }
#define MX_DISPATCH(fmt, dtype, BODY)                    \
  if ((fmt) == ADMMQ_MX_MXFP4) {                         \
    MX_DISPATCH_T(MX_MXFP4, dtype, BODY)                 \
  } else {                                               \
    MX_DISPATCH_T(MX_NVFP4, dtype, BODY)                 \
  }

namespace {

MxArgs mx_args(const uint8_t* a_scale, const float* a_tensor_scale, const uint8_t* b_scale,
               const float* b_tensor_scale, int64_t m, int n, int k, int fmt, void* out) {
  MxArgs p;
  p.w_scale = b_scale;
  p.x_scale = a_scale;
  p.gw = b_tensor_scale;
  p.gx = a_tensor_scale;
  p.out = out;
  p.m = (int)m;
  p.n = n;
  p.k = k;
  p.tn = m <= 128 ? ((int)m + 15) / 16 * 16 : 0;  // (k_mx_pair has its own)
  p.tiles_n = cdiv(n, 128);
  p.kblocks = cdiv(k, kMxBK);
  p.col_tiles = cdiv(k, mx_tile_k(fmt));
  p.raw = nullptr;
  p.overlap = 0;
  return p;
}

// Whether admmq_mx_linear quantises inside the product.
bool mx_linear_fused(int64_t m, int n, int k, int fmt) {
  if (m > kFusedTokens) return false;
  MxArgs p = mx_args(nullptr, nullptr, nullptr, nullptr, m, n, k, fmt, nullptr);
  bool fits;
  plan_tile(p, fmt, fits);
  return fits;
}

// The product of two MX matrices; check_only: its argument checks alone.
int mx_product(const uint8_t* a_codes, const uint8_t* a_scale, const float* a_tensor_scale,
                    const uint8_t* b_codes, const uint8_t* b_scale, const float* b_tensor_scale,
                    int64_t m, int n, int k, int fmt, void* out, int out_dtype, void* stream, bool check_only, bool overlap) {
  if (!mx_shape_ok(m, k, fmt) || !mx_shape_ok(n, k, fmt) || n < 1 || !dtype_ok(out_dtype))
    return ADMMQ_ERR_INVALID_ARG;
  if (fmt == ADMMQ_MX_MXFP4 && (a_tensor_scale || b_tensor_scale)) return ADMMQ_ERR_INVALID_ARG;
  if ((((uintptr_t)a_tensor_scale | (uintptr_t)b_tensor_scale) & 3) != 0)
    return ADMMQ_ERR_INVALID_ARG;
  if (m == 0) return ADMMQ_OK;
  if (!a_codes || !a_scale || !b_codes || !b_scale || !out || !aligned16(a_codes) ||
      !aligned16(a_scale) || !aligned16(b_codes) || !aligned16(b_scale) || !aligned16(out))
    return ADMMQ_ERR_INVALID_ARG;
  int rc = device_ok();
  if (rc || check_only) return rc;
  MxArgs p = mx_args(a_scale, a_tensor_scale, b_scale, b_tensor_scale, m, n, k, fmt, out);
  p.overlap = overlap;
  const bool pair = m > 128;
  if (!pair && (!make_codes_map(&p.w, b_codes, k, n, 128) || !make_codes_map(&p.x, a_codes, k, m, p.tn)))
    return ADMMQ_ERR_CUDA;
#define PRODUCT(FMT, T)                                                            \
  rc = pair ? launch_pair<FMT, T>(b_codes, a_codes, p, (cudaStream_t)stream)       \
            : launch_tile<FMT, T>(p, false, (cudaStream_t)stream)
  MX_DISPATCH(fmt, out_dtype, PRODUCT)
#undef PRODUCT
  return rc;
}

}  // namespace

extern "C" {

size_t admmq_mx_scale_bytes(int64_t rows, int k, int fmt) {
  if (!mx_shape_ok(rows, k, fmt)) return 0;
  return (size_t)((rows + 127) / 128) * (size_t)cdiv(k, mx_tile_k(fmt)) * kScaleTile;
}

int admmq_mx_quantize(const void* x, int x_dtype, int64_t rows, int k, int64_t ld, int fmt,
                      const float* tensor_scale, uint8_t* codes, uint8_t* scale, void* stream) {
  if (!mx_shape_ok(rows, k, fmt) || !dtype_ok(x_dtype) || ld < k) return ADMMQ_ERR_INVALID_ARG;
  if (fmt == ADMMQ_MX_MXFP4 && tensor_scale) return ADMMQ_ERR_INVALID_ARG;
  if (((uintptr_t)tensor_scale & 3) != 0) return ADMMQ_ERR_INVALID_ARG;
  if (rows == 0) return ADMMQ_OK;
  if (!x || !codes || !scale || !aligned16(x) || !aligned16(codes) || !aligned16(scale) ||
      ld * dtype_size(x_dtype) % 16 != 0)
    return ADMMQ_ERR_INVALID_ARG;
  int rc = device_ok();
  if (rc) return rc;
  const long long row_tiles = (rows + 127) / 128;
  const bool small = row_tiles * cdiv(k, 512) < 4 * num_sms();
  const int spans = cdiv(k, small ? 128 : 512);
  const long long grid = row_tiles * spans;
  if (grid > 0x7FFFFFFFll) return ADMMQ_ERR_UNSUPPORTED;
#define QUANTIZE(FMT, T)                                                                        \
  auto kern = small ? k_mx_quantize<FMT, T, 128> : k_mx_quantize<FMT, T, 512>;                  \
  count_launch(), kern<<<(unsigned)grid, kMxThreads, 0, (cudaStream_t)stream>>>(                \
                      (const T*)x, rows, k, ld, spans, tensor_scale, codes, scale)
  MX_DISPATCH(fmt, x_dtype, QUANTIZE)
#undef QUANTIZE
  CK(cudaGetLastError());
  return ADMMQ_OK;
}

int admmq_mx_dequantize(const uint8_t* codes, const uint8_t* scale, int64_t rows, int k, int fmt,
                        const float* tensor_scale, void* out, int out_dtype, int64_t ld,
                        void* stream) {
  if (!mx_shape_ok(rows, k, fmt) || !dtype_ok(out_dtype) || ld < k) return ADMMQ_ERR_INVALID_ARG;
  if (fmt == ADMMQ_MX_MXFP4 && tensor_scale) return ADMMQ_ERR_INVALID_ARG;
  if (((uintptr_t)tensor_scale & 3) != 0) return ADMMQ_ERR_INVALID_ARG;
  if (rows == 0) return ADMMQ_OK;
  if (!out || !codes || !scale || !aligned16(out) || !aligned16(codes) || !aligned16(scale) ||
      ld * dtype_size(out_dtype) % 16 != 0)
    return ADMMQ_ERR_INVALID_ARG;
  int rc = device_ok();
  if (rc) return rc;
  const long long row_tiles = (rows + 127) / 128;
  const bool small = row_tiles * cdiv(k, 512) < 4 * num_sms();
  const int spans = cdiv(k, small ? 128 : 512);
  const long long grid = row_tiles * spans;
  if (grid > 0x7FFFFFFFll) return ADMMQ_ERR_UNSUPPORTED;
#define DEQUANTIZE(FMT, T)                                                                      \
  auto kern = small ? k_mx_dequantize<FMT, T, 128> : k_mx_dequantize<FMT, T, 512>;              \
  count_launch(), kern<<<(unsigned)grid, kMxThreads, 0, (cudaStream_t)stream>>>(                \
                      codes, scale, rows, k, spans, tensor_scale, (T*)out, ld)
  MX_DISPATCH(fmt, out_dtype, DEQUANTIZE)
#undef DEQUANTIZE
  CK(cudaGetLastError());
  return ADMMQ_OK;
}

int admmq_mx_matmul(const uint8_t* a_codes, const uint8_t* a_scale, const float* a_tensor_scale,
                    const uint8_t* b_codes, const uint8_t* b_scale, const float* b_tensor_scale,
                    int64_t m, int n, int k, int fmt, void* out, int out_dtype, void* stream) {
  return mx_product(a_codes, a_scale, a_tensor_scale, b_codes, b_scale, b_tensor_scale, m, n, k, fmt,
                    out, out_dtype, stream, false, false);
}

size_t admmq_mx_linear_workspace_bytes(int64_t m, int n, int k, int fmt) {
  if (!mx_shape_ok(m, k, fmt) || !mx_shape_ok(n, k, fmt) || n < 1 || m == 0 ||
      mx_linear_fused(m, n, k, fmt))
    return 0;
  return (((size_t)m * (k / 2) + 255) & ~(size_t)255) + admmq_mx_scale_bytes(m, k, fmt);
}

int admmq_mx_linear(const void* x, int x_dtype, int64_t m, int64_t ldx, const float* x_tensor_scale,
                    const uint8_t* w_codes, const uint8_t* w_scale, const float* w_tensor_scale,
                    int n, int k, int fmt, void* out, int out_dtype, void* ws, size_t ws_bytes,
                    void* stream) {
  if (!mx_shape_ok(m, k, fmt) || !dtype_ok(x_dtype) || !dtype_ok(out_dtype) || n < 1 || ldx < k)
    return ADMMQ_ERR_INVALID_ARG;
  if (m == 0) return ADMMQ_OK;
  if (!x || !aligned16(x) || ldx * dtype_size(x_dtype) % 16 != 0) return ADMMQ_ERR_INVALID_ARG;
  const bool fused = mx_linear_fused(m, n, k, fmt);
  if (!fused && (!ws || ((uintptr_t)ws & 255))) return ADMMQ_ERR_INVALID_ARG;
  if (ws_bytes < admmq_mx_linear_workspace_bytes(m, n, k, fmt)) return ADMMQ_ERR_WORKSPACE;
  uint8_t* codes = fused ? (uint8_t*)w_codes : (uint8_t*)ws;  // (fused: checked, not used)
  uint8_t* scale = fused ? (uint8_t*)w_scale : codes + (((size_t)m * (k / 2) + 255) & ~(size_t)255);
  // the product's arguments first: nothing is launched when they are refused
  int rc = mx_product(codes, scale, x_tensor_scale, w_codes, w_scale, w_tensor_scale, m, n, k, fmt,
                      out, out_dtype, stream, true, false);
  if (rc) return rc;
  if (fused) {
    MxArgs p = mx_args(nullptr, x_tensor_scale, w_scale, w_tensor_scale, m, n, k, fmt, out);
    p.raw = x;
    p.ld = ldx;
    p.raw_dtype = x_dtype;
    if (!make_codes_map(&p.w, w_codes, k, n, 128)) return ADMMQ_ERR_CUDA;
    p.x = p.w;  // not used
#define FUSED(FMT, T) rc = launch_tile<FMT, T>(p, true, (cudaStream_t)stream)
    MX_DISPATCH(fmt, out_dtype, FUSED)
#undef FUSED
    return rc;
  }
  rc = admmq_mx_quantize(x, x_dtype, m, k, ldx, fmt, x_tensor_scale, codes, scale, stream);
  if (rc) return rc;
  // The product starts while the quantisation in front of it runs (an ordinary
  // launch, so everything before it is done): it reads the weights at once and
  // the activations when they are there.
  return mx_product(codes, scale, x_tensor_scale, w_codes, w_scale, w_tensor_scale, m, n, k, fmt,
                    out, out_dtype, stream, false, true);
}

}  // extern "C"
