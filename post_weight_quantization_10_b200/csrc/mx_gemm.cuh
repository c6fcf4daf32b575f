// mx_gemm.cuh -- product of two microscaled 4-bit matrices on the block-scaled
// tensor cores: out[i][j] = g_a g_b sum_k a[i][k] b[j][k].
//
// The weights b are the MMA's first operand (128 output columns j on the 128
// tensor-memory lanes), the activations a its second (up to 256 tokens i): few
// tokens then cost few columns, and a warp's lanes hold neighbouring columns j
// of one token, which out stores next to each other.
#pragma once
#include "async.cuh"
#include "../../include/admmq.h"
#include "gave_up.cuh"
#include "mx.cuh"
#include "ptx.cuh"

namespace admmq {

// ------------------------------------------------------------- PTX wrappers

// One scale tile (512 bytes: 32 rows of 16 bytes) from shared memory to four
// tensor-memory columns, repeated in the four lane quarters.
__device__ __forceinline__ void tmem_copy_scales(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
               : "memory");
}
// Its descriptor: no swizzle, groups of 8 rows 128 bytes apart.
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
}

// D[tmem] (+)= A[smem] B[smem], e2m1 elements, K = 64: scales per 32 (e8m0) or
// per 16 elements (e4m3) from tensor memory.
template <int FMT>
__device__ __forceinline__ void mma_mx(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                       uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                       uint32_t accumulate) {
  if (FMT == MX_MXFP4)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], "
        "[%5], p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, "
        "[%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// Instruction descriptor: e2m1 x e2m1, scale type, M rows and N columns; sf:
// which byte pair of the scale words the K = 64 step takes (mxfp4: 0 or 2).
template <int FMT>
__device__ __forceinline__ uint32_t idesc_mx(int M, int N, uint32_t sf) {
  return (sf << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) |
         (FMT == MX_MXFP4 ? 1u << 23 : 0u) | ((uint32_t)(M >> 7) << 27) | (sf << 29);
}

// The tensor scales as two factors of a sum, applied one after the other: their
// product and 1, or, where the product alone leaves fp32's normal range and the
// sum may bring it back, the larger and the smaller.
__device__ __forceinline__ float2 output_factors(const float* gw, const float* gx) {
  const float a = gw ? *gw : 1.f, b = gx ? *gx : 1.f, g = a * b;
  const bool left = (g < 0x1p-126f && a > 0.f && b > 0.f) || g == __int_as_float(0x7F800000);
  return left ? make_float2(fmaxf(a, b), fminf(a, b)) : make_float2(g, 1.f);
}

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(__half* p, float v) { *p = __float2half_rn(v); }

// ------------------------------------------------------------------- kernel

struct MxArgs {
  CUtensorMap w, x;            // codes of the weights and of the activations
  const uint8_t *w_scale, *x_scale;
  const float *gw, *gx;        // tensor scales or null
  void* out;
  int m, n, k;                 // tokens, output columns, reduction
  int tn;                      // tokens of a tile: a multiple of 16 up to 128 that holds all
  int tiles_n;                 // 128-column tiles
  int kblocks, col_tiles;      // 256-element stages; scale tiles along k
  int stages, stage_bytes, part_bytes;  // part_bytes: the ranks' partial tiles
  const void* raw;             // k_mx_tile<..., true>: the activations themselves,
  long long ld;                // their row distance
  int raw_dtype;               // and type
  int overlap;                 // launched to overlap with the kernel in front
  int tmem_cols;
};

constexpr int kMxBK = 256;  // elements of K per stage: 128-byte rows
constexpr int kMxTileThreads = 192;

// Quantises a block's part of the activations, tokens x 256-column stages from
// kb0 on, as k_mx_quantize does, into the stages' swizzled code rows and scale
// tiles.  Half a warp takes a token's stage (16 columns a lane) and loads a few
// of them before it uses the first.  What lies behind the last column is zero
// (codes and scales).
template <int FMT, typename X>
__device__ __forceinline__ void quantize_stages(const X* x, long long ld, int tokens, int k, int kb0,
                                                int stages, const float* tensor_scale, uint8_t* smem,
                                                int stage_bytes, int x_off, int sx_off, int warp) {
  constexpr int LANES = MxFormat<FMT>::BLOCK / 16, AHEAD = 8 / (int)sizeof(X);
  const float g = tensor_scale ? *tensor_scale : 1.f, r6g = 1.f / (6.f * g);
  const int half = (threadIdx.x >> 4) & 1, lane = threadIdx.x & 15, items = tokens * stages;
  for (int i0 = 2 * warp; i0 < items; i0 += 8 * AHEAD) {
    Raw16<X> raw[AHEAD];
    int token[AHEAD], stage[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const int i = i0 + 8 * j + half;
      stage[j] = i / tokens;
      token[j] = i - stage[j] * tokens;
      const int col = (kb0 + stage[j]) * kMxBK + 16 * lane;
#pragma unroll
      for (int w = 0; w < (int)(4 * sizeof(X)); ++w) raw[j].w[w] = 0u;
      if (i < items && col < k) load_raw(x + token[j] * ld + col, false, raw[j]);
    }
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      if (i0 + 8 * j >= items) break;
      const int row = token[j];
      const bool in = (kb0 + stage[j]) * kMxBK + 16 * lane < k;
      float v[16];
      values_of(raw[j], v);
      uint32_t amax = amax_of(raw[j]);
      if (LANES == 2) amax = max(amax, __shfl_xor_sync(~0u, amax, 1));
      const uint32_t byte = in ? block_scale<FMT>(amax, g, r6g) : 0u;
      const uint2 out = quantize16<FMT>(v, byte, g);
      if (i0 + 8 * j + half < items) {
        uint8_t *codes = smem + stage[j] * stage_bytes + x_off, *scales = smem + stage[j] * stage_bytes + sx_off;
        *reinterpret_cast<uint2*>(codes + row * 128 + (((lane >> 1) ^ (row & 7)) << 4) + 8 * (lane & 1)) = out;
        const int c = lane / LANES;
        if (lane % LANES == 0) scales[(c >> 2) * kScaleTile + scale_at(row, c & 3)] = (uint8_t)byte;
      }
      __syncwarp();
    }
  }
}

// One output tile of 128 columns x tn tokens per cluster; the cluster's CTAs
// share the reduction (contiguous ranges of stages); each rank sums a share of
// the tokens, from partial tiles that all ranks store into its shared memory,
// in rank order.
// FUSED (a few tokens, every stage of a block resident): the activations are
// quantised here, by the epilogue's warps while the weights are on their way,
// instead of by a launch of their own.
// What bounds it: up to 128 tokens the weights (0.53 bytes each) are all that
// counts, and a layer's 9 to 30 MB are so little that the chain load - MMA -
// cluster sum shows: 1 token of 4096 -> 4096 5.6 us device time where HBM needs
// 1.4, 48 tokens of 12288 -> 4096 15.6 us (quantisation included) of 4.6.  The
// cluster's share of k was worth most (48 tokens: 36 to 24 us), then having all
// of a block's stages in flight at once, then overlapping with the quantisation
// in front (24 to 19) or, for a few tokens, doing it here (1 token: 9.3 to 5.6).
//   warp 0  TMA producer    warp 1  MMA issuer    warps 2-5  epilogue
template <int FMT, typename T, bool FUSED>
__global__ void __launch_bounds__(kMxTileThreads)
    k_mx_tile(const __grid_constant__ MxArgs p) {
  constexpr int NSF = kMxBK / MxFormat<FMT>::TILE_K;  // scale tiles per stage and 128 rows
  extern __shared__ uint8_t smem_raw[];
  // (an offset, not a cast: the compiler has to see shared memory behind it)
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const int x_bytes = p.tn * 128;
  const int x_off = 128 * 128, sw_off = x_off + ((x_bytes + 1023) & ~1023),
            sx_off = sw_off + NSF * kScaleTile;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + p.stages * p.stage_bytes + p.part_bytes);
  uint64_t* empty = full + p.stages;
  uint64_t* done = empty + p.stages;
  uint64_t* quantised = done + 1;  // FUSED: the activations' codes and scales are there
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(quantised + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t rank, ranks;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
  const int tn_tile = blockIdx.x / ranks;
  const int kb0 = (int)((long long)rank * p.kblocks / ranks);
  const int kb1 = (int)((long long)(rank + 1) * p.kblocks / ranks);

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    mbar_init(smem_u32(done), 1);
    mbar_init(smem_u32(quantised), 4);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc(smem_u32(tmem_slot), p.tmem_cols);
  __syncthreads();
  // awaited before anything is stored into another rank
  if (ranks > 1) asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      bool ok = true;
      Ring r;
      int loads = 0;
      const uint8_t* ws = p.w_scale + (long long)tn_tile * p.col_tiles * kScaleTile;
      auto load_w = [&](int kb, uint32_t st, uint32_t bar) {
        const int sf = min(NSF, p.col_tiles - kb * NSF) * kScaleTile;  // scale bytes of this stage
        mbar_arrive_expect_tx(bar, 128 * 128 + sf + (FUSED ? 0 : x_bytes + sf));
        tma_load_2d(st, &p.w, kb * 128, tn_tile * 128, bar);
        bulk_load(st + sw_off, ws + kb * NSF * kScaleTile, sf, bar);
      };
      auto load_x = [&](int kb, uint32_t st, uint32_t bar) {
        const int sf = min(NSF, p.col_tiles - kb * NSF) * kScaleTile;
        tma_load_2d(st + x_off, &p.x, kb * 128, 0, bar);
        bulk_load(st + sx_off, p.x_scale + (long long)kb * NSF * kScaleTile, sf, bar);
      };
      // the weights of every stage before the first activation, which the
      // kernel in front may still be writing
      const int first = min(p.stages, kb1 - kb0);
      const uint32_t st0 = smem_u32(smem), bar0 = smem_u32(full);
      for (int s = 0; s < first; ++s) load_w(kb0 + s, st0 + s * p.stage_bytes, bar0 + 8 * s);
      if (!FUSED) {
        wait_for_previous_kernel();
        for (int s = 0; s < first; ++s) load_x(kb0 + s, st0 + s * p.stage_bytes, bar0 + 8 * s);
      }
      loads = first;
      r.phase = 1;  // the ring's second round
      for (int kb = kb0 + first; kb < kb1; ++kb, ++loads) {
        if (!mbar_wait(smem_u32(&empty[r.i]), r.phase ^ 1u, abort_flag, nullptr)) {
          ok = false;
          break;
        }
        const uint32_t bar = bar0 + 8 * r.i, st = st0 + r.i * p.stage_bytes;
        load_w(kb, st, bar);
        if (!FUSED) load_x(kb, st, bar);
        r.next(p.stages);
      }
      if (!ok)
        for (int j = max(0, loads - p.stages); j < loads; ++j)
          mbar_wait_drain(smem_u32(&full[j % p.stages]), (uint32_t)(j / p.stages) & 1u);
    }
  } else if (warp == 1) {
    const uint32_t sfw = tmem + ((p.tn + 31) & ~31), sfx = sfw + 4 * NSF;
    const uint64_t dw0 = smem_desc_sw128(smem_u32(smem), 16, 1024);
    const uint64_t dx0 = smem_desc_sw128(smem_u32(smem) + x_off, 16, 1024);
    const uint64_t dsw0 = scale_desc(smem_u32(smem) + sw_off), dsx0 = scale_desc(smem_u32(smem) + sx_off);
    if (elect_one()) {
      Ring r;
      bool ok = !FUSED || mbar_wait(smem_u32(quantised), 0, abort_flag, nullptr);
      for (int kb = kb0; kb < kb1 && ok; ++kb) {
        ok = mbar_wait(smem_u32(&full[r.i]), r.phase, abort_flag, nullptr);
        if (!ok) break;
        tc_fence_after();
        const uint32_t at = r.i * (p.stage_bytes >> 4);
        const int steps = min(4, (p.k - kb * kMxBK + 63) >> 6);
        const int tiles = min(NSF, p.col_tiles - kb * NSF);
#pragma unroll
        for (int i = 0; i < NSF; ++i) {
          if (i < tiles) {
            tmem_copy_scales(sfw + 4 * i, dsw0 + at + i * (kScaleTile >> 4));
            tmem_copy_scales(sfx + 4 * i, dsx0 + at + i * (kScaleTile >> 4));
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j < steps) {
            const int t = FMT == MX_MXFP4 ? j >> 1 : j;
            const uint32_t sf = FMT == MX_MXFP4 ? 2u * (j & 1) : 0u;
            mma_mx<FMT>(tmem, dw0 + at + 2 * j, dx0 + at + 2 * j, idesc_mx<FMT>(128, p.tn, sf),
                        sfw + 4 * t, sfx + 4 * t, (kb > kb0 || j > 0) ? 1u : 0u);
          }
        }
        mma_commit(smem_u32(&empty[r.i]));
        r.next(p.stages);
      }
      mma_commit(smem_u32(done));
    }
  }
  __syncwarp();
  // ------------------------------------------------------------- epilogue
  const int row = (warp & 3) * 32 + lane;  // column of the output tile
  const uint32_t ta = tmem + ((uint32_t)((warp & 3) * 32) << 16);
  bool ok = true;
  const long long col = (long long)tn_tile * 128 + row;
  const int tokens = p.m;
  const float2 g = output_factors(p.gw, p.gx);
  T* out = reinterpret_cast<T*>(p.out) + col;
  const int per = (tokens + (int)ranks - 1) / (int)ranks;  // tokens that a rank sums
  const uint32_t part = smem_u32(smem) + p.stages * p.stage_bytes;  // [ranks][per][128]
  if (FUSED && warp >= 2) {
    auto quantise = [&](auto* x) {
      quantize_stages<FMT>(x, p.ld, p.m, p.k, kb0, kb1 - kb0, p.gx, smem, p.stage_bytes, x_off, sx_off, warp - 2);
    };
    if (p.raw_dtype == ADMMQ_DTYPE_BF16)
      quantise((const __nv_bfloat16*)p.raw);
    else if (p.raw_dtype == ADMMQ_DTYPE_F16)
      quantise((const __half*)p.raw);
    else
      quantise((const float*)p.raw);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(quantised));
  }
  if (warp >= 2) {
    ok = mbar_wait(smem_u32(done), 0, abort_flag, nullptr);
    ok = __all_sync(~0u, ok) && !*abort_flag;
    tc_fence_after();
    if (ranks > 1) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    int owner = 0, at = 0;  // of the next token
    for (int c = 0; c < tokens; c += 16) {
      float v[16];
      tmem_ld16(ta + c, v);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (c + i >= tokens) break;
        if (!ok) v[i] = __int_as_float(0x7FFFFFFF);
        if (ranks > 1) {
          st_cluster_f32(cluster_addr(part + (((int)rank * per + at) * 128 + row) * 4, owner), v[i]);
          if (++at == per) {
            at = 0;
            ++owner;
          }
        } else if (col < p.n) {
          put(out + (long long)(c + i) * p.n, v[i] * g.x * g.y);
        }
      }
    }
    tc_fence_before();
  } else if (ranks > 1) {
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
  }
  if (ranks > 1) {
    __syncwarp();
    cluster_sync();  // all partial tiles have arrived
    if (warp >= 2 && col < p.n) {
      const int c0 = (int)rank * per, c1 = min(c0 + per, tokens);
      for (int c = c0; c < c1; ++c) {
        float v = 0.f;
        for (uint32_t r = 0; r < ranks; ++r)
          v += ld_shared_f32(part + (((int)r * per + c - c0) * 128 + row) * 4);
        put(out + (long long)c * p.n, v * g.x * g.y);
      }
    }
  }
  __syncthreads();
  report_gave_up(*abort_flag);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, p.tmem_cols);
  }
}

// --------------------------------------------------------------- many tokens

__device__ __forceinline__ void tmem_copy_scales_pair(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
               : "memory");
}
template <int FMT>
__device__ __forceinline__ void mma_mx_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                            uint32_t accumulate) {
  if (FMT == MX_MXFP4)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], "
        "[%5], p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, "
        "[%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

struct MxPairArgs {
  CUtensorMap w, x, ws, xs;    // codes and scale tiles (512-byte rows)
  const float *gw, *gx;
  void* out;
  int m, n, k;
  int tiles_m, tiles;          // 256-token tiles; all tiles (token tiles of 256 columns in turn)
  int kblocks, col_tiles, stages;
};

constexpr int kMxPairThreads = 320;

template <int FMT>
struct MxPairCfg {
  static constexpr int NSF = kMxBK / MxFormat<FMT>::TILE_K;  // scale tiles per stage and 128 rows
  static constexpr int CODES = 128 * 128;                    // bytes of 128 rows of a stage
  static constexpr int X_OFF = CODES, SW_OFF = 2 * CODES, SX_OFF = SW_OFF + NSF * kScaleTile;
  static constexpr int BYTES = SX_OFF + 2 * NSF * kScaleTile;  // loaded per CTA and stage
  static constexpr int STAGE = (BYTES + 1023) & ~1023;
};

// Pairs of CTAs (2-SM MMAs) go from tile to tile of 256 output columns x 256
// tokens.  Each CTA stages its 128 weight rows, its 128 of the tokens, the
// scales of those weight rows and of all the tokens; the leader issues the
// scale copies and MMAs for both; each CTA's tensor memory holds its 128
// columns' accumulators for the 256 tokens (256 of its 512 tensor-memory
// columns; a second accumulator would leave no room for the scales).  The
// epilogue takes the whole accumulator into registers, frees it for the next
// tile's MMAs and stores from there.
// What bounds it: the tensor cores under the power limit.  4096 tokens of
// 4096 -> 24576 in mxfp4: 173 us with the quantisation, 4.8 PFLOP/s (1.58 GHz at
// 985 W); single CTAs with 128 x 256 tiles took 581 us.
//   warp 0  TMA producer    warp 1  MMA issuer    warps 2-9  epilogue
template <int FMT, typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kMxPairThreads, 1)
    k_mx_pair(const __grid_constant__ MxPairArgs p) {
  using Cfg = MxPairCfg<FMT>;
  constexpr int NSF = Cfg::NSF;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const int S = p.stages;
  const uint32_t base = smem_u32(smem);
  const uint32_t full = base + S * Cfg::STAGE, empty = full + 8 * S, dfull = empty + 8 * S,
                 dempty = dfull + 8, drain = dempty + 8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S * Cfg::STAGE + 16 * S + 24);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair0 = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full + 8 * s, 1);
      mbar_init(empty + 8 * s, 1);
    }
    mbar_init(dfull, 1);
    mbar_init(dempty, 16);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc_pair(smem_u32(tmem_slot), 512);
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      bool ok = true;
      Ring r;
      int loads = 0;
      const uint32_t full0 = cluster_addr(full, 0);
      wait_for_previous_kernel();
      for (int tile = pair0; tile < p.tiles && ok; tile += pairs) {
        const int tn = tile / p.tiles_m, tm = tile - tn * p.tiles_m;
        const int w_row = tn * 256 + (int)rank * 128, x_row = tm * 256 + (int)rank * 128;
        int ws = (tn * 2 + (int)rank) * p.col_tiles, xs0 = tm * 2 * p.col_tiles;
        for (int kb = 0; kb < p.kblocks; ++kb, ++loads) {
          if (!mbar_wait(empty + 8 * r.i, r.phase ^ 1u, abort_flag, nullptr)) {
            ok = false;
            break;
          }
          const uint32_t st = base + r.i * Cfg::STAGE, bar = full0 + 8 * r.i;
          if (rank == 0) mbar_arrive_expect_tx(full + 8 * r.i, 2 * Cfg::BYTES);
          tma_load_2d_pair(st, &p.w, kb * 128, w_row, bar);
          tma_load_2d_pair(st + Cfg::X_OFF, &p.x, kb * 128, x_row, bar);
          tma_load_2d_pair(st + Cfg::SW_OFF, &p.ws, 0, ws, bar);
          tma_load_2d_pair(st + Cfg::SX_OFF, &p.xs, 0, xs0, bar);
          tma_load_2d_pair(st + Cfg::SX_OFF + NSF * kScaleTile, &p.xs, 0, xs0 + p.col_tiles, bar);
          ws += NSF;
          xs0 += NSF;
          r.next(S);
        }
      }
      if (!ok) {
        // copies in flight land before the CTA retires; the member's count on
        // the leader's barriers, so it waits a fixed ~1 ms instead
        if (rank == 0) {
          for (int j = max(0, loads - S); j < loads; ++j)
            mbar_wait_drain(full + 8 * (j % S), (uint32_t)(j / S) & 1u);
        } else {
          const long long t0 = clock64();
          while (clock64() - t0 < 2000000LL) {
          }
        }
      }
    }
  } else if (warp == 1) {
    if (rank == 0) {
      const uint32_t sfw = tmem + 256, sfx = sfw + 4 * NSF;
      const uint64_t dw0 = smem_desc_sw128(base, 16, 1024);
      const uint64_t dx0 = smem_desc_sw128(base + Cfg::X_OFF, 16, 1024);
      const uint64_t dsw0 = scale_desc(base + Cfg::SW_OFF), dsx0 = scale_desc(base + Cfg::SX_OFF);
      const uint32_t peer = cluster_addr(base, 1) - base;
      const uint32_t self = cluster_addr(base, 0) - base;
      if (elect_one()) {
        Ring r, d;
        bool ok = true;
        for (int tile = pair0; tile < p.tiles && ok; tile += pairs) {
          ok = mbar_wait_cluster(dempty, d.phase ^ 1u, abort_flag, nullptr);
          d.next(1);
          for (int kb = 0; kb < p.kblocks; ++kb) {
            ok = ok && mbar_wait(full + 8 * r.i, r.phase, abort_flag, nullptr);
            if (!ok) break;
            tc_fence_after();
            const uint32_t at = r.i * (Cfg::STAGE >> 4);
            const int steps = min(4, (p.k - kb * kMxBK + 63) >> 6);
#pragma unroll
            for (int i = 0; i < NSF; ++i) {
              tmem_copy_scales_pair(sfw + 4 * i, dsw0 + at + i * (kScaleTile >> 4));
              tmem_copy_scales_pair(sfx + 8 * i, dsx0 + at + i * (kScaleTile >> 4));
              tmem_copy_scales_pair(sfx + 8 * i + 4, dsx0 + at + (NSF + i) * (kScaleTile >> 4));
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (j < steps) {
                const int t = FMT == MX_MXFP4 ? j >> 1 : j;
                const uint32_t sf = FMT == MX_MXFP4 ? 2u * (j & 1) : 0u;
                mma_mx_pair<FMT>(tmem, dw0 + at + 2 * j, dx0 + at + 2 * j,
                                 idesc_mx<FMT>(256, 256, sf), sfw + 4 * t, sfx + 8 * t,
                                 (kb > 0 || j > 0) ? 1u : 0u);
              }
            }
            mma_commit_pair(empty + self + 8 * r.i);
            mma_commit_pair(empty + peer + 8 * r.i);
            r.next(S);
          }
          if (ok) {
            mma_commit_pair(dfull + self);
            mma_commit_pair(dfull + peer);
          }
        }
        mma_commit_pair(drain + self);
      }
      __syncwarp();
      mbar_wait_drain(drain, 0);
    }
  } else {
    const int half = (warp - 2) >> 2, quarter = warp & 3;
    const uint32_t ta = tmem + ((uint32_t)(quarter * 32) << 16) + half * 128;
    const float2 g = output_factors(p.gw, p.gx);
    const uint32_t dempty0 = cluster_addr(dempty, 0);
    Ring d;
    bool ok = true;
    for (int tile = pair0; tile < p.tiles; tile += pairs) {
      const int tn = tile / p.tiles_m, tm = tile - tn * p.tiles_m;
      const long long col = (long long)tn * 256 + rank * 128 + quarter * 32 + lane;
      if (ok) ok = mbar_wait(dfull, d.phase, abort_flag, nullptr);
      ok = __all_sync(~0u, ok);
      d.next(1);
      float v[128];
      if (ok) {
        tc_fence_after();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float u[32];
          tmem_ld32(ta + 32 * j, u);
#pragma unroll
          for (int i = 0; i < 32; ++i) v[32 * j + i] = u[i];
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(dempty0);
      } else {
#pragma unroll
        for (int i = 0; i < 128; ++i) v[i] = __int_as_float(0x7FFFFFFF);
      }
      if (col < p.n) {
        const int token0 = tm * 256 + half * 128, tokens = p.m - token0;
        T* out = reinterpret_cast<T*>(p.out) + (long long)token0 * p.n + col;
#pragma unroll
        for (int i = 0; i < 128; ++i) {
          if (i < tokens) put(out, v[i] * g.x * g.y);
          out += p.n;
        }
      }
    }
  }
  __syncthreads();
  report_gave_up(*abort_flag);
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

}  // namespace admmq
