// packed_few.cuh -- product of a few tokens (at most 16, used up to 12) with
// packed b-bit codes, on mma.sync.  What bounds it is reading the weights once
// and turning each code into an operand: instruction issue (three or four a
// code of a lane, 4096 -> 24576 at 4 bits 21 us for 1 token where HBM needs 8, 62 %
// of the issue slots taken), which up to 8 tokens share, and for small layers the
// chain launch - load - decode - sum (1 token of 4096 -> 6144 at 3 bits: 7.6 us
// device time of 1.7, 43 % of the slots: warps wait for results, words and barriers).
//
// mma.m16n8k16 sums over k in an order that nothing depends on, so each of the
// four lanes that share a weight row takes 32 consecutive codes of a
// 128-column span (b whole words), and the lane that holds a token's
// activations the same 32 columns, in the pairs that decode32 gives.  Eight
// instructions use up a span of 16 rows.  The codes enter as code - zero, an
// integer that bf16 and fp16 hold exactly; a group's sum leaves the tensor
// core in fp32 and is scaled there.  A group of 64 or 32 columns is summed by
// itself by running the span's instructions once per group with the other
// groups' activations set to zero.
#pragma once
#include "async.cuh"
#include "gave_up.cuh"
#include "packed.cuh"
#include "ptx.cuh"

namespace admmq {

constexpr int kFewThreads = 256;
// Blocks on an SM.  With RT = 1 two: their longer stages and registers for two
// rows' codes are worth more than a third block (4096 -> 4096 at 4 bits: 1 token
// 5.7 us against 6.7, 4 tokens 6.6 / 7.9; 4096 -> 24576 22.3 / 24.3 and 23.6 /
// 26.0; only 384 row blocks, one round of three, lose: 4096 -> 6144 7.8 / 7.4).
// With RT = 4 three (8 tokens of 4096 -> 24576 36 us, with two 51).
constexpr int few_blocks(int rt) { return rt == 1 ? 2 : 3; }

template <typename X>
__device__ __forceinline__ void mma_m16n8k16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (__is_same(X, __nv_bfloat16))
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Asynchronous copies that write zeros where there is nothing to read.
__device__ __forceinline__ void cp_async4_or_zero(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
               "r"(there ? 4 : 0)
               : "memory");
}

// How a block's work is laid out (made on the host).  A stage of the pipeline
// holds `spans` spans (a power of two) of the block's 16 RT rows: packed rows,
// scales and zero points ([row][group]).  The activations lie behind the
// stages, for the whole range or (x_staged) for a stage each, and behind them
// 64 bytes of zeros that the lanes of tokens that do not exist read.  Rows of
// words are spaced so that the 32 lanes' words (B (4 row + lane % 4) apart)
// fall into different banks, tokens 64 bytes off a multiple of 128 for the
// same reason.
struct FewPlan {
  int spans, range;                // per stage; of a rank
  int blocks;                      // row blocks
  int rank_shift, passes, groups;  // log2 ranks; groups of a span; of a stage
  int x_staged;
  int vec_scales;                  // every stage's scales begin and end on whole 16-byte pieces
  int pitch, x_pitch;              // of a row in words, of a token in bytes
  int s_off, bytes;                // of a stage
  int x_off, x_bytes, smem;
  FewPlan(int rows, int spans_, int range_, int bits, int group, int tokens, bool staged) {
    spans = spans_;
    range = range_;
    x_staged = staged;
    passes = 128 / group;
    groups = spans * passes;
    pitch = spans * 4 * bits;
    pitch += (4 * bits - pitch) & 31;
    const int x_spans = staged || spans > range ? spans : range;
    x_pitch = x_spans * 256 + 64;
    s_off = rows * pitch * 4;
    bytes = (s_off + 2 * rows * groups * 4 + 127) & ~127;
    x_off = 2 * bytes;
    x_bytes = (tokens * x_pitch + 127) & ~127;
    smem = x_off + (staged ? 2 : 1) * x_bytes + 64;
  }
};

// A block takes 16 RT output columns and one of the cluster's ranges of spans
// (and, with RT = 1, further row blocks after that), a stage at a time: the
// next stage's words are on their way while one is used.  Its eight warps are
// RT row tiles of 16 by 8 / RT shares of the spans.  RT = 1 keeps all of the
// activations in shared memory, which few tokens allow; with more tokens RT = 4
// reads them from L2 a quarter as often.
template <typename X, int NT, int RT, int B>
__global__ void __launch_bounds__(kFewThreads, few_blocks(RT))
    k_packed_few(const __grid_constant__ PackedArgs p, const __grid_constant__ FewPlan st) {
  constexpr int ROWS = 16 * RT, KW = 8 / RT;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float sum[RT == 1 ? 8 : 1][8 * NT][ROWS];
  __shared__ uint64_t full[2];
  __shared__ int abort_flag;
  const int ranks = 1 << st.rank_shift, rank = blockIdx.x & (ranks - 1);
  const int block0 = blockIdx.x >> st.rank_shift, block_step = gridDim.x >> st.rank_shift;
  const int sp0 = rank * st.range, sp1 = min(sp0 + st.range, (p.k + 127) >> 7);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = lane >> 2, q = lane & 3, rt = RT == 1 ? 0 : warp & (RT - 1), kw = warp / RT;
  const int passes = st.passes;
  const bool vec = (p.words & 3) == 0;  // rows of words start on 16 bytes
  const bool vec_s = st.vec_scales &&
                     (((uintptr_t)p.scale | (uintptr_t)p.zero) & 15) == 0;  // so do a stage's scales

  // Words, scales and zero points of the spans from sp on into a stage.  The
  // words of a row are one bulk copy (rows that start on 16 bytes; others go
  // word by word).  What lies behind the last column or row is not read: such
  // codes meet activations and scales of zero, or outputs that do not exist.
  auto fetch = [&](int block, int sp, int buf) {
    const long long row0 = (long long)block * ROWS;
    const int rows = p.n - row0 < ROWS ? (int)(p.n - row0) : ROWS;
    const uint32_t base = smem_u32(smem) + buf * st.bytes, bar = smem_u32(&full[buf]);
    const int first = sp * 4 * B, words = min(min(st.spans, sp1 - sp) * 4 * B, p.words - first);
    const int g0 = sp * passes, groups = min(st.groups, p.groups - g0);
    const int t = threadIdx.x;
    if (t == 0)
      mbar_arrive_expect_tx(bar, rows * ((vec ? words * 4 : 0) + (vec_s && !st.x_staged ? groups * 8 : 0)));
    // (a row's copies are issued by a thread each, a few in every warp: one warp
    // that issued all of them would be late for the products)
    constexpr int MINE = ROWS / (kFewThreads / 32);
    const int row = warp * MINE + lane % MINE;
    if (vec) {
      if (lane < MINE && row < rows)
        bulk_load(base + row * st.pitch * 4, p.packed + (row0 + row) * p.words + first, words * 4, bar);
    } else {
      for (int row = warp; row < rows; row += kFewThreads / 32)
        for (int c = lane; c < words; c += 32)
          cp_async4_or_zero(base + (row * st.pitch + c) * 4,
                            p.packed + (row0 + row) * p.words + first + c, true);
    }
    const uint32_t s_dst = base + st.s_off, z_dst = s_dst + ROWS * st.groups * 4;
    if (vec_s && st.x_staged) {
      const int shift = __ffs(st.groups) - 3;  // of 16-byte pieces
      for (int i = t; i < ROWS << shift; i += kFewThreads) {
        const int r16 = i >> shift, c = (i & ((1 << shift) - 1)) * 4;
        if (r16 < rows && c < groups) {
          const long long at = (row0 + r16) * p.groups + g0 + c;
          cp_async16(s_dst + i * 16, p.scale + at);
          cp_async16(z_dst + i * 16, p.zero + at);
        }
      }
    } else if (vec_s) {
      if (lane >= MINE && lane < 3 * MINE && row < rows)
        bulk_load((lane < 2 * MINE ? s_dst : z_dst) + row * st.groups * 4,
                  (lane < 2 * MINE ? p.scale : p.zero) + (row0 + row) * p.groups + g0, groups * 4, bar);
    } else {
      const int shift = __ffs(st.groups) - 1;
      for (int i = t; i < ROWS << shift; i += kFewThreads) {
        const int row = i >> shift, c = i & (st.groups - 1);
        const bool ok = row < rows && c < groups;
        const long long at = ok ? (row0 + row) * p.groups + g0 + c : 0;
        cp_async4_or_zero(s_dst + i * 4, p.scale + at, ok);
        cp_async4_or_zero(z_dst + i * 4, p.zero + at, ok);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // Activations of n spans in the order the lanes read them: per token and
  // span four 16-byte pieces (pairs 4 i .. 4 i + 3) of each of the four lanes.
  auto fetch_x = [&](int sp, int n, int buf) {
    uint8_t* base = smem + st.x_off + buf * st.x_bytes;
    // 8 n half blocks of 16 columns (8 pairs) per token; 8 to 256 threads a token
    const int shift = n >= 32 ? 8 : 35 - __clz(2 * n - 1 >> 1);
    for (int token = threadIdx.x >> shift; token < p.m; token += kFewThreads >> shift)
      for (int c = threadIdx.x & ((1 << shift) - 1); c < 8 * n; c += 1 << shift) {
        const int block32 = c >> 1, half = c & 1;       // columns 8 half .. + 7 and 16 + 8 half ..
        const int k = sp * 128 + block32 * 32;
        uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
        if (k < p.k) {
          const X* src = (const X*)p.x + token * p.ldx + k + 8 * half;
          lo = __ldg(reinterpret_cast<const uint4*>(src));
          hi = __ldg(reinterpret_cast<const uint4*>(src + 16));
        }
        uint4 a, b;
        a.x = __byte_perm(lo.x, hi.x, 0x5410); a.y = __byte_perm(lo.x, hi.x, 0x7632);
        a.z = __byte_perm(lo.y, hi.y, 0x5410); a.w = __byte_perm(lo.y, hi.y, 0x7632);
        b.x = __byte_perm(lo.z, hi.z, 0x5410); b.y = __byte_perm(lo.z, hi.z, 0x7632);
        b.z = __byte_perm(lo.w, hi.w, 0x5410); b.w = __byte_perm(lo.w, hi.w, 0x7632);
        uint4* dst = reinterpret_cast<uint4*>(base + token * st.x_pitch + (block32 >> 2) * 256);
        dst[(2 * half) * 4 + (block32 & 3)] = a;
        dst[(2 * half + 1) * 4 + (block32 & 3)] = b;
      }
  };

  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&full[0]), 1);
    mbar_init(smem_u32(&full[1]), 1);
    abort_flag = 0;
    fence_barrier_init();
  }
  uint8_t* nothing = smem + st.x_off + (st.x_staged ? 2 : 1) * st.x_bytes;
  if (threadIdx.x < 16) reinterpret_cast<uint32_t*>(nothing)[threadIdx.x] = 0u;
  __syncthreads();
  // the items of this block, (row block, stage) in turn: the next one to fetch
  int f_block = block0, f_sp = sp0;
  auto fetch_next = [&](int buf) {
    if (f_block < st.blocks && f_sp < sp1) {
      fetch(f_block, f_sp, buf);
      f_sp += st.spans;
      if (f_sp >= sp1) {
        f_sp = sp0;
        f_block += block_step;
      }
    } else {
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  };
  fetch_next(0);
  fetch_next(1);
  if (!st.x_staged) fetch_x(sp0, sp1 - sp0, 0);
  const bool by_threads = !vec || !vec_s || st.x_staged;
  if (!by_threads) __syncthreads();
  bool ok = true;
  int buf = 0;
  uint32_t phase = 0;
  for (int block = block0; block < st.blocks; block += block_step) {
    const long long row0 = (long long)block * ROWS;
    float acc[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[t][j] = 0.f;
    for (int sp = sp0; sp < sp1; sp += st.spans) {
      const int there = min(st.spans, sp1 - sp);
      if (st.x_staged) fetch_x(sp, there, buf);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      ok = mbar_wait(smem_u32(&full[buf]), phase, &abort_flag, nullptr) && ok;
      // what threads stored or copied themselves, unlike bulk copies, waits for all
      if (by_threads) __syncthreads();
      const uint8_t* base = smem + buf * st.bytes;
      const uint32_t* src =
          reinterpret_cast<const uint32_t*>(base) + (rt * 16 + r) * st.pitch + (4 * kw + q) * B;
      const int low = 8 * st.pitch;      // to the lane's second row
      const float* scales =
          reinterpret_cast<const float*>(base + st.s_off) + (rt * 16 + r) * st.groups + kw * passes;
      const float* zeros = scales + ROWS * st.groups + (q * passes >> 2);
      const int low_s = 8 * st.groups;
      const uint8_t* xs[NT];
      int x_step[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const bool token = t * 8 + r < p.m;
        xs[t] = token ? smem + st.x_off + (st.x_staged ? buf * st.x_bytes : (sp - sp0) * 256) +
                            (t * 8 + r) * st.x_pitch + kw * 256 + q * 16
                      : nothing;
        x_step[t] = token ? 64 : 0;
      }
      for (int i = kw; i < there; i += KW) {
        uint32_t w0[B], w1[B], a0[16], a1[16];
        if constexpr (B % 4 == 0) {
#pragma unroll
          for (int j = 0; j < B / 4; ++j) {
            const uint4 u = reinterpret_cast<const uint4*>(src)[j];
            const uint4 v = reinterpret_cast<const uint4*>(src + low)[j];
            w0[4 * j] = u.x; w0[4 * j + 1] = u.y; w0[4 * j + 2] = u.z; w0[4 * j + 3] = u.w;
            w1[4 * j] = v.x; w1[4 * j + 1] = v.y; w1[4 * j + 2] = v.z; w1[4 * j + 3] = v.w;
          }
        } else if constexpr (B % 2 == 0) {
#pragma unroll
          for (int j = 0; j < B / 2; ++j) {
            const uint2 u = reinterpret_cast<const uint2*>(src)[j];
            const uint2 v = reinterpret_cast<const uint2*>(src + low)[j];
            w0[2 * j] = u.x; w0[2 * j + 1] = u.y;
            w1[2 * j] = v.x; w1[2 * j + 1] = v.y;
          }
        } else {
#pragma unroll
          for (int j = 0; j < B; ++j) {
            w0[j] = src[j];
            w1[j] = src[low + j];
          }
        }
        decode32<X, B>(w0, zeros[0], a0);
        decode32<X, B>(w1, zeros[low_s], a1);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          uint32_t x[16];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 v = *reinterpret_cast<const uint4*>(xs[t] + j * x_step[t]);
            x[4 * j] = v.x; x[4 * j + 1] = v.y; x[4 * j + 2] = v.z; x[4 * j + 3] = v.w;
          }
          xs[t] += 4 * KW * x_step[t];
          if (passes == 1) {
            float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 8; ++j)
              mma_m16n8k16<X>(d, a0[2 * j], a1[2 * j], a0[2 * j + 1], a1[2 * j + 1], x[2 * j],
                              x[2 * j + 1]);
            const float s0 = scales[0], s1 = scales[low_s];
            acc[t][0] += s0 * d[0];
            acc[t][1] += s0 * d[1];
            acc[t][2] += s1 * d[2];
            acc[t][3] += s1 * d[3];
          } else {
            for (int g = 0; g < passes; ++g) {
              const bool mine = q * passes >> 2 == g;
              float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int j = 0; j < 8; ++j)
                mma_m16n8k16<X>(d, a0[2 * j], a1[2 * j], a0[2 * j + 1], a1[2 * j + 1],
                                mine ? x[2 * j] : 0u, mine ? x[2 * j + 1] : 0u);
              // no scale is read for a group behind the last column
              const bool there_g = (sp + i) * passes + g < p.groups;
              const float s0 = there_g ? scales[g] : 0.f, s1 = there_g ? scales[low_s + g] : 0.f;
              acc[t][0] += s0 * d[0];
              acc[t][1] += s0 * d[1];
              acc[t][2] += s1 * d[2];
              acc[t][3] += s1 * d[3];
            }
          }
        }
        src += 4 * KW * B;
        scales += KW * passes;
        zeros += KW * passes;
      }
      __syncthreads();
      fetch_next(buf);
      buf ^= 1;
      if (buf == 0) phase ^= 1;
    }
    // a wait that gave up leaves no number behind
    if (!ok)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[t][j] = __int_as_float(0x7FFFFFFF);
    // the shares' sums, then the cluster's, each in a fixed order
    if (RT == 1) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          sum[RT == 1 ? kw : 0][t * 8 + 2 * q + (j & 1)][r + 8 * (j >> 1)] = acc[t][j];
      __syncthreads();
    } else {
#pragma unroll
      for (int share = 0; share < KW; ++share) {
        if (kw == share) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float& at = sum[0][t * 8 + 2 * q + (j & 1)][rt * 16 + r + 8 * (j >> 1)];
              at = share ? at + acc[t][j] : acc[t][j];
            }
        }
        __syncthreads();
      }
    }
    if (ranks > 1) cluster_sync();
    for (int i = rank * kFewThreads + threadIdx.x; i < p.m * ROWS; i += ranks * kFewThreads) {
      const int token = i / ROWS, c = i % ROWS;
      if (row0 + c >= p.n) continue;
      float v = 0.f;
      if (ranks > 1) {
        for (int k = 0; k < ranks; ++k)
          v += ld_cluster_f32(cluster_addr(smem_u32(&sum[0][token][c]), k));
      } else {
#pragma unroll
        for (int w = 0; w < (RT == 1 ? 8 : 1); ++w) v += sum[w][token][c];
      }
      put_out(p, (long long)token * p.n + row0 + c, v);
    }
    if (ranks > 1) cluster_sync();  // the sums stay until every rank has read them
  }
  __syncthreads();
  report_gave_up(abort_flag);
  if (!ok) {  // copies in flight land before the block retires (about 1 ms)
    const long long t0 = clock64();
    while (clock64() - t0 < 2000000LL) {
    }
  }
}

}  // namespace admmq
