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
//
// What bounds it: at 33 tokens of 12288 -> 4096 (2 bits, 22.5 us; HBM needs 2.6) a
// chunk's chain of waits, decoding, stores and MMAs times the chunks of a rank;
// at 4096 tokens of 4096 -> 24576 (4 bits) the MMAs wait for decoders and
// group sums, the tensor pipe is active half of the cycles, and the power limit
// sets the clock (1.62 GHz): 790 us in a burst, 890 sustained, 1.04 and 0.93
// PFLOP/s, where a bf16 product of that size takes 503 and 592.  On the way there: 39 ms on the CUDA cores, 2.9 ms with one warp
// group for everything, 1.4 with no division in the single-thread loops, 1.08
// with a converged MMA warp, 0.91 with the decoding shared by two CTAs.
#pragma once
#include "async.cuh"
#include "gave_up.cuh"
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
  int part_bytes;      // room for the ranks' partial tiles
};

// Thread roles, by warpgroup:
//   0    warps 0 and 2: TMA producers, warp 1: MMA issuer, warp 3: copies
//   1..  DG groups of decoders, taking turns by the chunk
//   then CG groups of consumers: thread = accumulator row, a share of the tokens
// A chunk costs a decoder a chain of waits, loads, arithmetic, stores and a
// fence of about 2000 cycles, the MMAs of 64 tokens 256: fewer tokens, more
// groups.  256 tokens leave registers for one.
// Turning codes into operands takes about as many instructions as there are
// cycles in the MMAs that use them, so with C = 2 a cluster of two CTAs works
// on the same 128 weight rows and two token tiles: each decodes half of the
// rows and copies them into the other's shared memory.  Clusters go from tile
// to tile.  With C = 1 (one token tile) the CTAs of a cluster share the
// reduction instead (contiguous ranges of chunks) and add their tiles in rank
// order through distributed shared memory.
template <int TN, int C>
struct PackedCfg {
  static constexpr int CG = 2, DG = TN == 64 ? 3 : TN == 128 ? 2 : 1;
  // registers of a thread of each role; together no more than the launch's
  // (warpgroups x 80, 96 or 128)
  static constexpr int REGS0 = 40, REGS_D = TN == 256 ? 88 : 80,
                       REGS_C = TN == 64 ? 96 : TN == 128 ? 136 : 192;
  static constexpr int LAUNCH = 65536 / (128 * (1 + DG + CG)) / 8 * 8;
  static_assert(REGS0 + DG * REGS_D + CG * REGS_C <= (1 + DG + CG) * LAUNCH, "register split");
  static constexpr int THREADS = 128 * (1 + DG + CG);
  static constexpr int SHARE = TN / CG;        // tokens of a consumer group
  static constexpr int X_BYTES = TN * 128, A_BYTES = 128 * 128, STAGE = X_BYTES + A_BYTES;
  static constexpr int TMEM_COLS = 2 * TN;
  static constexpr int ROWS = 128 / C;         // weight rows that a CTA decodes
  static constexpr int STEPS = ROWS / 32;      // of 8 rows, per decoder warp
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

// A chunk's words of two of this lane's rows (unit q of rows row and row + 8)
// to 16-bit pairs in column order.
template <typename X, int B>
__device__ __forceinline__ void decode_chunk(const PackedGemmArgs& a, const uint8_t* buf, int row,
                                             int q, long long row0, int chunk, const float* zero,
                                             uint32_t (&v)[2][16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t w[B];
    if (a.w_tma) {
      chunk_words<B>(buf, row + 8 * i, q, w);
    } else {
      const bool in = row0 + row + 8 * i < a.p.n && chunk * 128 + 32 * q < a.p.k;
      const uint32_t* src = a.p.packed + (row0 + row + 8 * i) * a.p.words + (chunk * 4 + q) * B;
#pragma unroll
      for (int j = 0; j < B; ++j) w[j] = in ? __ldg(src + j) : 0u;
    }
    decode32_in_order<X, B>(w, zero[i], v[i]);
  }
}

// Shared-memory addresses of the barriers (arrays of 8-byte words).
struct PackedBars {
  uint32_t full, empty;            // [stages]: activations and decoded weights there; read
  uint32_t part;                   // [stages] (C > 1): the part decoded here is there
  uint32_t wfull, wempty;          // [wbufs]: packed chunk there; decoded
  uint32_t rfull, rempty, drain;   // [2]: group finished; added; everything finished
  uint32_t end;
  __device__ PackedBars(uint32_t at, int stages, int wbufs) {
    full = at;
    empty = full + 8 * stages;
    part = empty + 8 * stages;
    wfull = part + 8 * stages;
    wempty = wfull + 8 * wbufs;
    rfull = wempty + 8 * wbufs;
    rempty = rfull + 16;
    drain = rempty + 16;
    end = drain + 8;
  }
};

// The MMA thread's loop: 8 MMAs of K = 16 per chunk, PASSES groups.
template <typename X, int TN, int C, int PASSES>
__device__ __forceinline__ void issue_mmas(const PackedGemmArgs& a, int ch0, int ch1, int tile0,
                                           int tile_step, uint32_t tmem, const uint8_t* smem,
                                           const PackedBars& bars, volatile int* abort_flag) {
  using Cfg = PackedCfg<TN, C>;
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
        if (!mbar_wait(bars.full + 8 * st.i, st.phase, abort_flag, nullptr)) return;
        tc_fence_after();
        const uint64_t dx = dx0 + (uint32_t)(st.i * (Cfg::STAGE >> 4));
        const uint64_t dw = dw0 + (uint32_t)(st.i * (Cfg::STAGE >> 4));
        // the half's MMAs, a group (or the half of one) at a time
#pragma unroll
        for (int j0 = 0; j0 < 4; j0 += PER < 4 ? PER : 4) {
          const int step = 4 * h + j0;
          if (step / PER < groups) {
            if (step % PER == 0) {
              if (!mbar_wait(bars.rempty + 8 * slot.i, slot.phase ^ 1u, abort_flag, nullptr)) return;
              tc_fence_after();
            }
#pragma unroll
            for (int j = j0; j < j0 + (PER < 4 ? PER : 4); ++j)
              mma_f16(tmem + slot.i * TN, dw + 2 * j, dx + 2 * j, IDESC,
                      (4 * h + j) % PER == 0 ? 0u : 1u);
            if ((step + (PER < 4 ? PER : 4)) % PER == 0) {
              mma_commit(bars.rfull + 8 * slot.i);
              slot.next(2);
            }
          }
        }
        // a stage's decoders write to every CTA that uses it
        if (C == 1) mma_commit(bars.empty + 8 * st.i);
#pragma unroll
        for (int c = 0; c < (C > 1 ? C : 0); ++c) mma_commit(cluster_addr(bars.empty + 8 * st.i, c));
        st.next(a.stages);
      }
    }
  }
}

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(__half* p, float v) { *p = __float2half_rn(v); }

// Column `col` of the output, tokens token0 .. + SHARE - 1.
template <int SHARE, typename T>
__device__ __forceinline__ void store_column(T* out, const PackedArgs& p, int token0, long long col,
                                             const float2 (&acc)[SHARE / 2]) {
  T* at = out + (long long)token0 * p.n + col;
  const int tokens = p.m - token0;
#pragma unroll
  for (int i = 0; i < SHARE; ++i) {
    if (i < tokens) put(at, i & 1 ? acc[i / 2].y : acc[i / 2].x);
    at += p.n;
  }
}

// BITS: of a code, or 0 for p.bits (the largest tiles, which gain nothing from
// a kernel of their own for each width; at 33 tokens it saves a fifth).
template <typename X, int TN, int C, int BITS>
__global__ void __launch_bounds__(PackedCfg<TN, C>::THREADS, 1)
    k_packed_gemm(const __grid_constant__ PackedGemmArgs a) {
  using Cfg = PackedCfg<TN, C>;
  const PackedArgs& p = a.p;
  extern __shared__ uint8_t smem_raw[];
  // (an offset, not a cast: the compiler has to see shared memory behind it)
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const int S = a.stages, NW = a.wbufs, wbytes = 16 * Cfg::ROWS * p.bits;
  uint8_t* wring = smem + S * Cfg::STAGE;
  // C = 1: partial tiles of the cluster's ranks, behind the rings
  const uint32_t part = smem_u32(wring + NW * wbytes);
  const PackedBars bars(part + a.part_bytes, S, NW);
  uint32_t* tmem_slot =
      reinterpret_cast<uint32_t*>(wring + NW * wbytes + a.part_bytes + (bars.end - bars.full));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t rank, ranks;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
  // with C > 1 `tiles` counts clusters of tiles: C token tiles of 128 columns
  const int tile0 = blockIdx.x / ranks, tile_step = gridDim.x / ranks;
  const int ch0 = C > 1 ? 0 : rank * a.range, ch1 = min(ch0 + a.range, a.chunks);
  const int part0 = C > 1 ? rank * Cfg::ROWS : 0;  // first of the weight rows decoded here

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      // the activations' producer and four decoder warps, or the copying thread
      mbar_init(bars.full + 8 * s, C > 1 ? 2 : 5);
      mbar_init(bars.part + 8 * s, 4);
      mbar_init(bars.empty + 8 * s, C);
    }
    for (int i = 0; i < NW; ++i) {
      mbar_init(bars.wfull + 8 * i, 1);
      mbar_init(bars.wempty + 8 * i, 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bars.rfull + 8 * i, 1);
      mbar_init(bars.rempty + 8 * i, 4 * Cfg::CG);
    }
    mbar_init(bars.drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc(smem_u32(tmem_slot), Cfg::TMEM_COLS);
  __syncthreads();
  if (C > 1)
    cluster_sync();  // the peers' barriers exist
  else if (ranks > 1)
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");  // awaited before anything remote
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int wg = warp >> 2;

  if (wg == 0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg::REGS0));
    if (warp == 0 && lane == 0) {
      // ----------------------------------------------- activations' producer
      bool ok = true;
      Ring x;  // a fresh ring's buffers count as emptied once: parity 1
      int loads = 0;
      for (int tile = tile0; tile < a.tiles && ok; tile += tile_step) {
        const int tn = tile / a.tiles_m, tm = (tile - tn * a.tiles_m) * C + (C > 1 ? rank : 0);
        for (int k = ch0 * 128; k < ch1 * 128; k += 64, ++loads) {
          const uint32_t bar = bars.full + 8 * x.i;
          if (!mbar_wait(bars.empty + 8 * x.i, x.phase ^ 1u, abort_flag, nullptr)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(bar, Cfg::X_BYTES);
          tma_load_2d(smem_u32(smem + x.i * Cfg::STAGE), &a.x, k, tm * TN, bar);
          x.next(S);
        }
      }
      if (!ok)  // the copies in flight land before the block retires
        for (int j = max(0, loads - S); j < loads; ++j)
          mbar_wait_drain(bars.full + 8 * (j % S), (uint32_t)(j / S) & 1u);
    } else if (warp == 2 && lane == 0 && a.w_tma) {
      // ----------------------------------------------- packed codes' producer
      bool ok = true;
      Ring w;
      int chunks = 0;
      for (int tile = tile0; tile < a.tiles && ok; tile += tile_step)
        for (int ch = ch0; ch < ch1; ++ch, ++chunks) {
          const uint32_t bar = bars.wfull + 8 * w.i;
          if (!mbar_wait(bars.wempty + 8 * w.i, w.phase ^ 1u, abort_flag, nullptr)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(bar, wbytes);
          tma_load_2d(smem_u32(wring + w.i * wbytes), &a.w, ch * 16 * p.bits,
                      tile / a.tiles_m * 128 + part0, bar);
          w.next(NW);
        }
      if (!ok)
        for (int j = max(0, chunks - NW); j < chunks; ++j)
          mbar_wait_drain(bars.wfull + 8 * (j % NW), (uint32_t)(j / NW) & 1u);
    } else if (C > 1 && warp == 3 && lane == 0) {
      // ------------------- copies of the rows decoded here to the other CTA
      // (8 KB a stage; a decoder that issued them itself lost 800 cycles a chunk)
      constexpr uint32_t BYTES = Cfg::ROWS * 128;
      const uint32_t src0 = smem_u32(smem) + Cfg::X_BYTES + part0 * 128;
      const uint32_t peer = cluster_addr(smem_u32(smem), rank ^ 1) - smem_u32(smem);
      Ring st;
      bool ok = true;
      for (int tile = tile0; tile < a.tiles && ok; tile += tile_step)
        for (int h = 2 * ch0; h < 2 * ch1; ++h) {
          if (!mbar_wait(bars.part + 8 * st.i, st.phase, abort_flag, nullptr)) {
            ok = false;
            break;
          }
          const uint32_t src = src0 + st.i * Cfg::STAGE, bar = bars.full + 8 * st.i;
          bulk_copy_to_peer(src + peer, src, BYTES, bar + peer);
          mbar_arrive_expect_tx(bar, BYTES);  // the other CTA's rows
          st.next(S);
        }
    } else if (warp == 1) {
      // -------------------------------------------------------- MMA issuer
      if (elect_one()) {
        if (a.passes == 1)
          issue_mmas<X, TN, C, 1>(a, ch0, ch1, tile0, tile_step, tmem, smem, bars, abort_flag);
        else if (a.passes == 2)
          issue_mmas<X, TN, C, 2>(a, ch0, ch1, tile0, tile_step, tmem, smem, bars, abort_flag);
        else
          issue_mmas<X, TN, C, 4>(a, ch0, ch1, tile0, tile_step, tmem, smem, bars, abort_flag);
        mma_commit(bars.drain);
      }
      __syncwarp();
      mbar_wait_drain(bars.drain, 0);
    }
  } else if (wg <= Cfg::DG) {
    // -------------------------------------------------------------- decoders
    if constexpr (Cfg::REGS_D < Cfg::LAUNCH)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg::REGS_D));
    // The codes are decoded into registers while the MMAs still read the stage
    // that they will go to; what is left once it is free are the stores.
    Ring st, wr;
    bool ok = true;
    int turn = Cfg::DG - wg;  // chunks until this group's next one
    const int q = lane >> 3;
    const int row = (warp & 3) * Cfg::STEPS * 8 + (lane & 7);  // of the part decoded here
    const int group_shift = __ffs(p.group) - 1;
    uint32_t to[4];  // of this lane's four 16-byte pieces in a stage's operand tile
#pragma unroll
    for (int c = 0; c < 4; ++c)
      to[c] = smem_u32(smem) + Cfg::X_BYTES + (part0 + row) * 128 +
              ((((q & 1) * 4 + c) ^ (row & 7)) << 4);
    for (int tile = tile0; tile < a.tiles && ok; tile += tile_step) {
      const long long row0 = (long long)(tile / a.tiles_m) * 128 + part0;
      const float* zeros = p.zero + (row0 + row) * p.groups;
      float next[Cfg::STEPS], zero[Cfg::STEPS];
      auto load_zeros = [&](int ch) {
        const int k = ch * 128 + 32 * q;
#pragma unroll
        for (int i = 0; i < Cfg::STEPS; ++i)
          next[i] = load_ahead(zeros + 8 * i * p.groups + (k >> group_shift),
                               row0 + row + 8 * i < p.n && k < p.k);
      };
      load_zeros(ch0 + turn);
      for (int ch = ch0; ch < ch1; ++ch) {
        const Ring st0 = st, w = wr;
        Ring st1 = st;
        st1.next(S);
        st = st1;
        st.next(S);
        wr.next(NW);
        if (Cfg::DG > 1 && turn-- > 0) continue;
        turn = Cfg::DG - 1;
#pragma unroll
        for (int i = 0; i < Cfg::STEPS; ++i) zero[i] = next[i];
        load_zeros(ch + Cfg::DG);
        if (a.w_tma && !mbar_wait(bars.wfull + 8 * w.i, w.phase, abort_flag, nullptr)) {
          ok = false;
          break;
        }
        const uint8_t* buf = wring + w.i * wbytes;
        const Ring mine = q < 2 ? st0 : st1;  // units 0, 1 go to the first stage, 2, 3 to the second
        const uint32_t stage = mine.i * Cfg::STAGE;
#pragma unroll
        for (int i = 0; i < Cfg::STEPS; i += 2) {
          uint32_t v[2][16];
          const float* z = zero + i;
          switch (BITS ? BITS : p.bits) {
            case 1: decode_chunk<X, 1>(a, buf, row + 8 * i, q, row0, ch, z, v); break;
            case 2: decode_chunk<X, 2>(a, buf, row + 8 * i, q, row0, ch, z, v); break;
            case 3: decode_chunk<X, 3>(a, buf, row + 8 * i, q, row0, ch, z, v); break;
            case 4: decode_chunk<X, 4>(a, buf, row + 8 * i, q, row0, ch, z, v); break;
            case 5: decode_chunk<X, 5>(a, buf, row + 8 * i, q, row0, ch, z, v); break;
            case 6: decode_chunk<X, 6>(a, buf, row + 8 * i, q, row0, ch, z, v); break;
            case 7: decode_chunk<X, 7>(a, buf, row + 8 * i, q, row0, ch, z, v); break;
            default: decode_chunk<X, 8>(a, buf, row + 8 * i, q, row0, ch, z, v); break;
          }
          if (i == 0)
            ok = C > 1 ? mbar_wait_cluster(bars.empty + 8 * mine.i, mine.phase ^ 1u, abort_flag, nullptr)
                       : mbar_wait(bars.empty + 8 * mine.i, mine.phase ^ 1u, abort_flag, nullptr);
          if (!ok) break;
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              st_shared_v4(to[c] + stage + (i + j) * 8 * 128, v[j][4 * c], v[j][4 * c + 1],
                           v[j][4 * c + 2], v[j][4 * c + 3]);
        }
        if (!__all_sync(~0u, ok)) {
          ok = false;
          break;
        }
        // the MMA and the copies read what these stores wrote through the async proxy
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane < 2) {  // a lane for each of the two stages
          mbar_arrive((C > 1 ? bars.part : bars.full) + 8 * (lane ? st1.i : st0.i));
        } else if (lane == 2 && a.w_tma) {
          mbar_arrive(bars.wempty + 8 * w.i);
        }
      }
    }
  } else {
    // ------------------------------------------------------------- consumers
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Cfg::REGS_C));
    constexpr int SHARE = Cfg::SHARE;
    const int share = wg - 1 - Cfg::DG;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t ta = tmem + ((uint32_t)((warp & 3) * 32) << 16) + share * SHARE;
    bool ok = true;
    Ring slot;
    for (int tile = tile0; tile < a.tiles; tile += tile_step) {
      const int tn = tile / a.tiles_m, tm = (tile - tn * a.tiles_m) * C + (C > 1 ? rank : 0);
      const long long col = (long long)tn * 128 + row;
      float2 acc[SHARE / 2];
#pragma unroll
      for (int i = 0; i < SHARE / 2; ++i) acc[i] = make_float2(0.f, 0.f);
      const int g0 = ch0 * a.passes, g1 = min(ch1 * a.passes, p.groups);
      const float* scale = p.scale + col * p.groups;
      float s = load_ahead(scale + g0, col < p.n && g0 < g1);
      for (int g = g0; g < g1; ++g) {
        const float here = s;
        s = load_ahead(scale + g + 1, col < p.n && g + 1 < g1);
        if (ok) {
          ok = mbar_wait(bars.rfull + 8 * slot.i, slot.phase, abort_flag, nullptr);
          ok = __all_sync(~0u, ok);
        }
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int j = 0; j < SHARE / 16; ++j) {
          float v[16];
          tmem_ld16(ta + slot.i * TN + 16 * j, v);
#pragma unroll
          for (int i = 0; i < 8; ++i) fma_x2(acc[8 * j + i], here, v[2 * i], v[2 * i + 1]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars.rempty + 8 * slot.i);
        slot.next(2);
      }
      if (!ok)
#pragma unroll
        for (int i = 0; i < SHARE / 2; ++i)
          acc[i] = make_float2(__int_as_float(0x7FFFFFFF), __int_as_float(0x7FFFFFFF));
      if (C > 1 || ranks == 1) {
        const int token0 = tm * TN + share * SHARE;
        if (col < p.n) {
          if (p.out_dtype == ADMMQ_DTYPE_F32)
            store_column<SHARE>((float*)p.out, p, token0, col, acc);
          else if (p.out_dtype == ADMMQ_DTYPE_BF16)
            store_column<SHARE>((__nv_bfloat16*)p.out, p, token0, col, acc);
          else
            store_column<SHARE>((__half*)p.out, p, token0, col, acc);
        }
      } else {
        // to the rank that sums these tokens: slots [rank][TN / ranks][128]
        asm volatile("barrier.cluster.wait.acquire;" ::: "memory");  // every rank has begun
        const int per = (TN + ranks - 1) / ranks;
#pragma unroll
        for (int i = 0; i < SHARE; ++i) {
          const int token = share * SHARE + i, owner = token / per;
          st_cluster_f32(cluster_addr(part + ((rank * per + token - owner * per) * 128 + row) * 4, owner),
                         i & 1 ? acc[i / 2].y : acc[i / 2].x);
        }
      }
    }
  }
  __syncwarp();
  if (C > 1) {
    cluster_sync();  // no copy or arrival from here is under way to the other CTA
  } else if (ranks > 1) {
    if (wg <= Cfg::DG) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    __syncwarp();
    cluster_sync();  // all partial tiles have arrived
    const int per = (TN + ranks - 1) / ranks, row = threadIdx.x & 127;
    const long long col = (long long)(tile0 / a.tiles_m) * 128 + row;
    const int token0 = tile0 % a.tiles_m * TN + rank * per;
    if (col < p.n)
      for (int c = threadIdx.x >> 7; c < per && rank * per + c < TN && token0 + c < p.m;
           c += Cfg::THREADS / 128) {
        float v = 0.f;
        for (uint32_t r = 0; r < ranks; ++r) v += ld_shared_f32(part + ((r * per + c) * 128 + row) * 4);
        put_out(p, (long long)(token0 + c) * p.n + col, v);
      }
  }
  __syncthreads();
  report_gave_up(*abort_flag);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, Cfg::TMEM_COLS);
  }
}

}  // namespace admmq
