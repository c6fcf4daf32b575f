// packed_gemm.cuh -- product of many tokens with packed b-bit codes on the
// tensor cores:
//   out[i][j] = sum over groups G of s[j][G] sum_{k in G} (c[j][k] - z[j][G]) x[i][k].
//
// The weights are the MMA's first operand: 128 output columns j on the 128
// tensor-memory lanes, up to 256 tokens along the accumulator's columns.  Four
// warps turn codes into bf16 or fp16 integers c - z (exact) in the swizzled
// shared-memory tile that the MMA reads.  Each group is accumulated by itself
// in one of two tensor-memory slots, and eight warps add s times a finished
// group to fp32 registers while the next group's MMAs run: the scales never
// touch a 16-bit number, and the tensor core's own accumulator, which rounds
// to one side, never sums more than a group.
#pragma once
#include "async.cuh"
#include "packed.cuh"
#include "ptx.cuh"

namespace admmq {

struct PackedGemmArgs {
  CUtensorMap x, w;    // activations [m][k]; packed rows in bytes
  PackedArgs p;
  int tiles_m, tiles;  // token tiles; all tiles (token tiles of 128 columns in turn)
  int chunks, range;   // 128-column chunks of k; of them, a rank's
  int w_tma;           // rows of packed words start on 16 bytes: TMA brings them
  int stages, wbufs;   // ring depths: operand stages (64 of k), packed chunks
  int passes;          // groups of a chunk
};

constexpr int kPackedThreads = 512;

// Thread roles, four warpgroups:
//   0  warp 0: TMA producer, warp 1: MMA issuer
//   1  decoders
//   2, 3  consumers: thread = accumulator row, half of the tile's tokens each
// One output tile of 128 x TN per cluster and turn; a cluster's CTAs share the
// reduction (contiguous ranges of chunks) and add their tiles in rank order
// through distributed shared memory.  A cluster of one goes on to further tiles.
template <int TN>
struct PackedCfg {
  static constexpr int HALF = TN / 2;
  static constexpr int X_BYTES = TN * 128, A_BYTES = 128 * 128, STAGE = X_BYTES + A_BYTES;
  static constexpr int TMEM_COLS = 2 * TN;
};

// Words of unit q (32 codes) of a row of a packed chunk in shared memory.  TMA
// left rows of 16 B bytes, swizzled where their pitch is 32, 64 or 128 bytes:
// the eight rows that a phase of the warp reads then lie in different banks.
template <int B>
__device__ __forceinline__ void chunk_words(const uint8_t* buf, int row, int q, uint32_t (&w)[B]) {
  const uint8_t* at = buf + row * (16 * B);
  if constexpr (B == 8) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint4 v = *reinterpret_cast<const uint4*>(at + (((2 * q + j) ^ (row & 7)) << 4));
      w[4 * j] = v.x; w[4 * j + 1] = v.y; w[4 * j + 2] = v.z; w[4 * j + 3] = v.w;
    }
  } else if constexpr (B == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(at + ((q ^ ((row >> 1) & 3)) << 4));
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  } else if constexpr (B == 2) {
    const uint2 v =
        *reinterpret_cast<const uint2*>(at + (((q >> 1) ^ ((row >> 2) & 1)) << 4) + 8 * (q & 1));
    w[0] = v.x; w[1] = v.y;
  } else if constexpr (B == 6) {
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      const uint2 v = reinterpret_cast<const uint2*>(at + 24 * q)[j];
      w[2 * j] = v.x; w[2 * j + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int j = 0; j < B; ++j) w[j] = reinterpret_cast<const uint32_t*>(at + 4 * B * q)[j];
  }
}

// One chunk (128 rows x 128 columns) by the four decoder warps into the
// operand tiles of its two stages.
template <typename X, int B>
__device__ __forceinline__ void decode_chunk(const PackedGemmArgs& a, const uint8_t* buf,
                                             uint8_t* tile0, uint8_t* tile1, long long row0,
                                             int chunk, const float (&zero)[4]) {
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3;
  const int q = lane >> 3;
  uint8_t* tile = q < 2 ? tile0 : tile1;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = warp * 32 + i * 8 + (lane & 7);
    uint32_t w[B], v[16];
    if (a.w_tma) {
      chunk_words<B>(buf, row, q, w);
    } else {
      const bool in = row0 + row < a.p.n && chunk * 128 + 32 * q < a.p.k;
      const uint32_t* src = a.p.packed + (row0 + row) * a.p.words + (chunk * 4 + q) * B;
#pragma unroll
      for (int j = 0; j < B; ++j) w[j] = in ? __ldg(src + j) : 0u;
    }
    decode32<X, B>(w, zero[i], v);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      // columns 8 c .. 8 c + 7 of the unit, in order again
      const int h = 4 * (c & 1);
      const uint32_t sel = c < 2 ? 0x5410 : 0x7632;
      uint4 o;
      o.x = __byte_perm(v[2 * h], v[2 * h + 1], sel);
      o.y = __byte_perm(v[2 * h + 2], v[2 * h + 3], sel);
      o.z = __byte_perm(v[2 * h + 4], v[2 * h + 5], sel);
      o.w = __byte_perm(v[2 * h + 6], v[2 * h + 7], sel);
      *reinterpret_cast<uint4*>(tile + row * 128 + ((((q & 1) * 4 + c) ^ (row & 7)) << 4)) = o;
    }
  }
}

// Shared-memory addresses of the barriers (arrays of 8-byte words).
struct PackedBars {
  uint32_t full_x, full_a, empty;  // [stages]: activations, decoded weights; stage read
  uint32_t wfull, wempty;          // [wbufs]: packed chunk there; decoded
  uint32_t rfull, rempty, drain;   // [2]: group finished; added; everything finished
  uint32_t end;
  __device__ PackedBars(uint32_t at, int stages, int wbufs) {
    full_x = at;
    full_a = full_x + 8 * stages;
    empty = full_a + 8 * stages;
    wfull = empty + 8 * stages;
    wempty = wfull + 8 * wbufs;
    rfull = wempty + 8 * wbufs;
    rempty = rfull + 16;
    drain = rempty + 16;
    end = drain + 8;
  }
};

// The MMA warp's loop: 8 MMAs of K = 16 per chunk, PASSES groups.
template <typename X, int TN, int PASSES>
__device__ __forceinline__ bool issue_mmas(const PackedGemmArgs& a, int ch0, int ch1, int tile0,
                                           int tile_step, uint32_t tmem, const uint8_t* smem,
                                           const PackedBars& bars, volatile int* abort_flag) {
  using Cfg = PackedCfg<TN>;
  constexpr uint32_t IDESC = idesc_f32acc(__is_same(X, __nv_bfloat16) ? 1 : 0, 128, TN, false, false);
  constexpr int PER = 8 / PASSES;  // MMAs of a group
  const uint64_t dx0 = smem_desc_sw128(smem_u32(smem), 16, 1024);
  const uint64_t dw0 = smem_desc_sw128(smem_u32(smem) + Cfg::X_BYTES, 16, 1024);
  Ring st, slot;
  for (int tile = tile0; tile < a.tiles; tile += tile_step) {
    for (int ch = ch0; ch < ch1; ++ch) {
      const int groups = min(PASSES, a.p.groups - ch * PASSES);  // of this chunk
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        bool ok = mbar_wait(bars.full_x + 8 * st.i, st.phase, abort_flag, nullptr) &&
                  mbar_wait(bars.full_a + 8 * st.i, st.phase, abort_flag, nullptr);
        const uint64_t dx = dx0 + (uint32_t)(st.i * (Cfg::STAGE >> 4));
        const uint64_t dw = dw0 + (uint32_t)(st.i * (Cfg::STAGE >> 4));
        // the half's MMAs, a group (or the half of one) at a time
#pragma unroll
        for (int j0 = 0; j0 < 4; j0 += PER < 4 ? PER : 4) {
          const int step = 4 * h + j0;
          if (step / PER < groups) {
            if (step % PER == 0)
              ok = ok && mbar_wait(bars.rempty + 8 * slot.i, slot.phase ^ 1u, abort_flag, nullptr);
            if (!__all_sync(~0u, ok)) return false;
            tc_fence_after();
            const bool ends = (step + (PER < 4 ? PER : 4)) % PER == 0;
            if (elect_one()) {
#pragma unroll
              for (int j = j0; j < j0 + (PER < 4 ? PER : 4); ++j)
                mma_f16(tmem + slot.i * TN, dw + 2 * j, dx + 2 * j, IDESC,
                        (4 * h + j) % PER == 0 ? 0u : 1u);
              if (ends) mma_commit(bars.rfull + 8 * slot.i);
            }
            __syncwarp();
            if (ends) slot.next(2);
          }
        }
        if (!__all_sync(~0u, ok)) return false;
        if (elect_one()) mma_commit(bars.empty + 8 * st.i);
        __syncwarp();
        st.next(a.stages);
      }
    }
  }
  return true;
}

template <typename X, int TN>
__global__ void __launch_bounds__(kPackedThreads, 1)
    k_packed_gemm(const __grid_constant__ PackedGemmArgs a) {
  using Cfg = PackedCfg<TN>;
  const PackedArgs& p = a.p;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int S = a.stages, NW = a.wbufs, wbytes = 2048 * p.bits;
  uint8_t* wring = smem + S * Cfg::STAGE;
  const PackedBars bars(smem_u32(wring + NW * wbytes), S, NW);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(wring + NW * wbytes + (bars.end - bars.full_x));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t rank, ranks;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
  const int tile0 = blockIdx.x / ranks, tile_step = gridDim.x / ranks;
  const int ch0 = rank * a.range, ch1 = min(ch0 + a.range, a.chunks);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(bars.full_x + 8 * s, 1);
      mbar_init(bars.full_a + 8 * s, 4);
      mbar_init(bars.empty + 8 * s, 1);
    }
    for (int i = 0; i < NW; ++i) {
      mbar_init(bars.wfull + 8 * i, 1);
      mbar_init(bars.wempty + 8 * i, 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bars.rfull + 8 * i, 1);
      mbar_init(bars.rempty + 8 * i, 8);
    }
    mbar_init(bars.drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc(smem_u32(tmem_slot), Cfg::TMEM_COLS);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int wg = warp >> 2;

  if (wg == 0) {
    if constexpr (TN == 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------------- producer
      bool ok = true;
      Ring x, w;  // a fresh ring's buffers count as emptied once: parity 1
      int loads = 0, chunks = 0;
      for (int tile = tile0; tile < a.tiles && ok; tile += tile_step) {
        const int tn = tile / a.tiles_m, tm = tile - tn * a.tiles_m;
        for (int ch = ch0; ch < ch1 && ok; ++ch) {
          if (a.w_tma) {
            const uint32_t bar = bars.wfull + 8 * w.i;
            if (!mbar_wait(bars.wempty + 8 * w.i, w.phase ^ 1u, abort_flag, nullptr)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(bar, wbytes);
            tma_load_2d(smem_u32(wring + w.i * wbytes), &a.w, ch * 16 * p.bits, tn * 128, bar);
            w.next(NW);
            ++chunks;
          }
          for (int h = 0; h < 2; ++h) {
            const uint32_t bar = bars.full_x + 8 * x.i;
            if (!mbar_wait(bars.empty + 8 * x.i, x.phase ^ 1u, abort_flag, nullptr)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(bar, Cfg::X_BYTES);
            tma_load_2d(smem_u32(smem + x.i * Cfg::STAGE), &a.x, ch * 128 + 64 * h, tm * TN, bar);
            x.next(S);
            ++loads;
          }
        }
      }
      if (!ok) {
        // the copies in flight land before the block retires
        for (int j = max(0, loads - S); j < loads; ++j)
          mbar_wait_drain(bars.full_x + 8 * (j % S), (uint32_t)(j / S) & 1u);
        for (int j = max(0, chunks - NW); j < chunks; ++j)
          mbar_wait_drain(bars.wfull + 8 * (j % NW), (uint32_t)(j / NW) & 1u);
      }
    } else if (warp == 1) {
      // -------------------------------------------------------- MMA issuer
      const bool ok = a.passes == 1   ? issue_mmas<X, TN, 1>(a, ch0, ch1, tile0, tile_step, tmem, smem, bars, abort_flag)
                      : a.passes == 2 ? issue_mmas<X, TN, 2>(a, ch0, ch1, tile0, tile_step, tmem, smem, bars, abort_flag)
                                      : issue_mmas<X, TN, 4>(a, ch0, ch1, tile0, tile_step, tmem, smem, bars, abort_flag);
      (void)ok;
      if (elect_one()) mma_commit(bars.drain);
      __syncwarp();
      mbar_wait_drain(bars.drain, 0);
    }
  } else if (wg == 1) {
    // -------------------------------------------------------------- decoders
    if constexpr (TN == 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    bool ok = true;
    Ring st, wr;
    const int q = lane >> 3;
    const int group_shift = __ffs(p.group) - 1;
    for (int tile = tile0; tile < a.tiles && ok; tile += tile_step) {
      const long long row0 = (long long)(tile / a.tiles_m) * 128;
      float next[4], zero[4];
      auto load_zeros = [&](int ch) {
        const int k = ch * 128 + 32 * q;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const long long row = row0 + (warp & 3) * 32 + i * 8 + (lane & 7);
          next[i] = row < p.n && k < p.k ? __ldg(p.zero + row * p.groups + (k >> group_shift)) : 0.f;
        }
      };
      load_zeros(ch0);
      for (int ch = ch0; ch < ch1; ++ch) {
#pragma unroll
        for (int i = 0; i < 4; ++i) zero[i] = next[i];
        if (ch + 1 < ch1) load_zeros(ch + 1);
        Ring st1 = st;
        st1.next(S);
        ok = (!a.w_tma || mbar_wait(bars.wfull + 8 * wr.i, wr.phase, abort_flag, nullptr)) &&
             mbar_wait(bars.empty + 8 * st.i, st.phase ^ 1u, abort_flag, nullptr) &&
             mbar_wait(bars.empty + 8 * st1.i, st1.phase ^ 1u, abort_flag, nullptr);
        if (!ok) break;
        const uint8_t* buf = wring + wr.i * wbytes;
        uint8_t* t0 = smem + st.i * Cfg::STAGE + Cfg::X_BYTES;
        uint8_t* t1 = smem + st1.i * Cfg::STAGE + Cfg::X_BYTES;
        switch (p.bits) {
          case 1: decode_chunk<X, 1>(a, buf, t0, t1, row0, ch, zero); break;
          case 2: decode_chunk<X, 2>(a, buf, t0, t1, row0, ch, zero); break;
          case 3: decode_chunk<X, 3>(a, buf, t0, t1, row0, ch, zero); break;
          case 4: decode_chunk<X, 4>(a, buf, t0, t1, row0, ch, zero); break;
          case 5: decode_chunk<X, 5>(a, buf, t0, t1, row0, ch, zero); break;
          case 6: decode_chunk<X, 6>(a, buf, t0, t1, row0, ch, zero); break;
          case 7: decode_chunk<X, 7>(a, buf, t0, t1, row0, ch, zero); break;
          default: decode_chunk<X, 8>(a, buf, t0, t1, row0, ch, zero); break;
        }
        // the MMA reads what these stores wrote through the async proxy
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bars.full_a + 8 * st.i);
          mbar_arrive(bars.full_a + 8 * st1.i);
          if (a.w_tma) mbar_arrive(bars.wempty + 8 * wr.i);
        }
        st = st1;
        st.next(S);
        wr.next(NW);
      }
    }
  } else {
    // ------------------------------------------------------------- consumers
    if constexpr (TN == 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    constexpr int HALF = Cfg::HALF;
    const int half = wg - 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t ta = tmem + ((uint32_t)((warp & 3) * 32) << 16) + half * HALF;
    bool ok = true;
    Ring slot;
    for (int tile = tile0; tile < a.tiles; tile += tile_step) {
      const int tn = tile / a.tiles_m, tm = tile - tn * a.tiles_m;
      const long long col = (long long)tn * 128 + row;
      float acc[HALF];
#pragma unroll
      for (int i = 0; i < HALF; ++i) acc[i] = 0.f;
      const int g0 = ch0 * a.passes, g1 = min(ch1 * a.passes, p.groups);
      const float* scale = p.scale + col * p.groups;
      float s = col < p.n && g0 < g1 ? __ldg(scale + g0) : 0.f;
      for (int g = g0; g < g1; ++g) {
        const float here = s;
        if (g + 1 < g1) s = col < p.n ? __ldg(scale + g + 1) : 0.f;
        if (ok) {
          ok = mbar_wait(bars.rfull + 8 * slot.i, slot.phase, abort_flag, nullptr);
          ok = __all_sync(~0u, ok);
        }
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int j = 0; j < HALF / 16; ++j) {
          float v[16];
          tmem_ld16(ta + slot.i * TN + 16 * j, v);
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[16 * j + i] += here * v[i];
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars.rempty + 8 * slot.i);
        slot.next(2);
      }
      if (!ok)
#pragma unroll
        for (int i = 0; i < HALF; ++i) acc[i] = __int_as_float(0x7FFFFFFF);
      if (ranks == 1) {
        const int token0 = tm * TN + half * HALF;
        if (col < p.n) {
#pragma unroll
          for (int i = 0; i < HALF; ++i)
            if (token0 + i < p.m) put_out(p, (long long)(token0 + i) * p.n + col, acc[i]);
        }
      } else {
        float* part = reinterpret_cast<float*>(smem);  // [TN][128], over the used stages
#pragma unroll
        for (int i = 0; i < HALF; ++i) part[(half * HALF + i) * 128 + row] = acc[i];
      }
    }
  }
  if (ranks > 1) {
    __syncwarp();
    cluster_sync();
    const int row = threadIdx.x & 127;
    const long long col = (long long)(tile0 / a.tiles_m) * 128 + row;
    const int token0 = tile0 % a.tiles_m * TN;
    const float* part = reinterpret_cast<const float*>(smem);
    if (col < p.n)
      for (int c = rank + ranks * (threadIdx.x >> 7); c < TN && token0 + c < p.m;
           c += ranks * (kPackedThreads / 128)) {
        float v = 0.f;
        for (uint32_t r = 0; r < ranks; ++r)
          v += ld_cluster_f32(cluster_addr(smem_u32(part + c * 128 + row), r));
        put_out(p, (long long)(token0 + c) * p.n + col, v);
      }
    cluster_sync();
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, Cfg::TMEM_COLS);
  }
}

}  // namespace admmq
