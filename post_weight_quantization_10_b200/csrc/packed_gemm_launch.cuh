// packed_gemm_launch.cuh -- host side of packed_gemm.cuh, compiled once for each
// activation type (packed_gemm_bf16.cu, packed_gemm_fp16.cu).
#pragma once
#include "host.cuh"
#include "packed_gemm.cuh"
#include "tmem_fair.cuh"

namespace admmq {

inline bool make_x_map(CUtensorMap* m, const PackedArgs& p, bool bf16, int box_rows) {
  cuuint64_t dims[2] = {(cuuint64_t)p.k, (cuuint64_t)p.m};
  cuuint64_t strides[1] = {(cuuint64_t)p.ldx * 2};
  cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  return encode_tiled(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
            const_cast<void*>(p.x), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

// Packed rows as bytes, boxes of a 128-code chunk (16 b bytes).
inline bool make_w_map(CUtensorMap* m, const PackedArgs& p, int box_rows) {
  cuuint64_t dims[2] = {(cuuint64_t)p.words * 4, (cuuint64_t)p.n};
  cuuint64_t strides[1] = {(cuuint64_t)p.words * 4};
  cuuint32_t box[2] = {(cuuint32_t)(16 * p.bits), (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  const CUtensorMapSwizzle sw = p.bits == 2   ? CU_TENSOR_MAP_SWIZZLE_32B
                                : p.bits == 4 ? CU_TENSOR_MAP_SWIZZLE_64B
                                : p.bits == 8 ? CU_TENSOR_MAP_SWIZZLE_128B
                                              : CU_TENSOR_MAP_SWIZZLE_NONE;
  return encode_tiled(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint32_t*>(p.packed), dims, strides,
            box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

// Ranks that share the reduction of a tile, where the tiles are too few.
inline int split_ranks(long long tiles, int chunks, int sms) {
  int ranks = 1;
  while (ranks < 8 && chunks >= 4 * ranks && 2 * ranks * tiles <= cluster_ctas(2 * ranks, sms)) ranks *= 2;
  return ranks;
}

// About how long a tile shape takes: rounds of tiles x chunks of a rank x a
// chunk's time, plus what adding partial tiles takes.
inline double tile_time(const PackedArgs& p, int tokens, int ctas, double chunk_us, int sms) {
  const int chunks = cdiv(p.k, 128);
  const long long tiles = (long long)cdiv(p.m, tokens) * cdiv(p.n, 128);
  const int ranks = ctas == 1 ? split_ranks(tiles, chunks, sms) : 1;
  const int at_once = ranks > 1 ? cluster_ctas(ranks, sms) / ranks : sms / ctas;
  return (double)((tiles + at_once - 1) / at_once) * cdiv(chunks, ranks) * chunk_us + (ranks > 1 ? 3.0 : 0.0);
}

// The tile shape that is estimated to take least: tokens of a tile, 64, 128 or
// 512 (two CTAs).  A chunk's times are measured (33 tokens of 4096 -> 24576: 47 us
// in two rounds of 32 chunks; 256: 96 us in three; 4096: 890 us in 21): 64 tokens
// cost as much as the decoding that they share, 512 a cluster's MMAs.
inline int packed_tile(const PackedArgs& p, int sms) {
  const double t64 = tile_time(p, 64, 1, 0.74, sms), t128 = tile_time(p, 128, 1, 1.0, sms),
               t512 = tile_time(p, 512, 2, 1.32, sms);
  return t64 <= t128 && t64 <= t512 ? 64 : t128 <= t512 ? 128 : 512;
}

// How a call is laid out (all but the tensor maps of `a`).
struct PackedGemmPlan {
  PackedGemmArgs a;
  int ranks, clusters, smem;
};

template <int TN, int C>
int plan_gemm(const PackedArgs& p, int sms, PackedGemmPlan& plan) {
  using Cfg = PackedCfg<TN, C>;
  PackedGemmArgs& a = plan.a;
  a.p = p;
  a.tiles_m = cdiv(p.m, TN * C);
  const long long tiles = (long long)a.tiles_m * cdiv(p.n, 128);
  if (tiles > (1 << 28)) return ADMMQ_ERR_UNSUPPORTED;
  a.tiles = (int)tiles;
  a.chunks = cdiv(p.k, 128);
  a.passes = 128 / p.group;
  a.w_tma = p.words % 4 == 0;
  int ranks = C == 1 ? split_ranks(tiles, a.chunks, sms) : C;
  // Shared memory: the ranks' partial tiles; packed chunks, which come from HBM,
  // a long way off (a third of the rings, at most 16); operand stages the rest.
  // A decoder group may wait for a buffer that others have yet to use once:
  // with a buffer for each group no wait is more than one use ahead, which is
  // as far as a barrier's parity tells uses apart.
  const int wbytes = 16 * Cfg::ROWS * p.bits;
  constexpr int least_w = Cfg::DG < 2 ? 2 : Cfg::DG, least_s = 2 * (Cfg::DG < 2 ? 2 : Cfg::DG);
  for (;; ranks /= 2) {
    a.part_bytes = C == 1 && ranks > 1 ? ranks * cdiv(TN, ranks) * 512 : 0;
    const int room = 225 * 1024 - a.part_bytes;
    a.wbufs = room / 3 / wbytes;
    a.wbufs = a.wbufs < least_w ? least_w : a.wbufs > 16 ? 16 : a.wbufs;
    a.stages = (room - a.wbufs * wbytes) / Cfg::STAGE & ~1;
    if (a.stages < least_s) a.stages = least_s;
    if (a.stages > 8) a.stages = 8;
    a.wbufs = (room - a.stages * Cfg::STAGE) / wbytes;
    if (a.wbufs > 16) a.wbufs = 16;
    if (a.wbufs >= least_w) break;
    if (ranks == C) return ADMMQ_ERR_UNSUPPORTED;
  }
  a.range = C == 1 ? cdiv(a.chunks, ranks) : a.chunks;
  plan.smem = tmem_fair_smem(a.stages * Cfg::STAGE + a.wbufs * wbytes + a.part_bytes + 2048, Cfg::TMEM_COLS);
  const int most = C == 1 && ranks > 1 ? a.tiles : sms / ranks;
  plan.ranks = ranks;
  plan.clusters = a.tiles < most ? a.tiles : most;
  return ADMMQ_OK;
}

template <typename X, int TN, int C, bool BY_BITS>
int launch_gemm(const PackedArgs& p, int sms, cudaStream_t st) {
  using Cfg = PackedCfg<TN, C>;
  PackedGemmPlan plan;
  int rc = plan_gemm<TN, C>(p, sms, plan);
  if (rc) return rc;
  PackedGemmArgs& a = plan.a;
  if (!make_x_map(&a.x, p, __is_same(X, __nv_bfloat16), TN)) return ADMMQ_ERR_CUDA;
  if (a.w_tma && !make_w_map(&a.w, p, Cfg::ROWS)) return ADMMQ_ERR_CUDA;
  const void* kern;
  if constexpr (BY_BITS) {
    static const void* const table[8] = {
        (const void*)k_packed_gemm<X, TN, C, 1>, (const void*)k_packed_gemm<X, TN, C, 2>,
        (const void*)k_packed_gemm<X, TN, C, 3>, (const void*)k_packed_gemm<X, TN, C, 4>,
        (const void*)k_packed_gemm<X, TN, C, 5>, (const void*)k_packed_gemm<X, TN, C, 6>,
        (const void*)k_packed_gemm<X, TN, C, 7>, (const void*)k_packed_gemm<X, TN, C, 8>};
    kern = table[p.bits - 1];
  } else {
    kern = (const void*)k_packed_gemm<X, TN, C, 0>;
  }
  CK(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem));
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)(plan.clusters * plan.ranks));
  lc.blockDim = dim3(Cfg::THREADS);
  lc.dynamicSmemBytes = plan.smem;
  lc.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = plan.ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  count_launch();
  void* argv[] = {&a};
  CK(cudaLaunchKernelExC(&lc, kern, argv));
  return ADMMQ_OK;
}

template <typename X>
int packed_gemm(const PackedArgs& p, cudaStream_t st) {
  const int sms = num_sms();
  switch (packed_tile(p, sms)) {
    case 64: return launch_gemm<X, 64, 1, true>(p, sms, st);
    case 128: return launch_gemm<X, 128, 1, true>(p, sms, st);
    default: return launch_gemm<X, 256, 2, false>(p, sms, st);
  }
}

}  // namespace admmq
