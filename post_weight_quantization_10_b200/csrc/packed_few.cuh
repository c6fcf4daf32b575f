// packed_few.cuh -- product of a few tokens (at most 16) with packed b-bit
// codes.  The weights are read once, straight into the registers that feed
// the matrix instructions.
//
// mma.m16n8k16 sums over k in an order that nothing depends on, so each of the
// four lanes that share a weight row takes 32 consecutive codes of a
// 128-column span (b whole words) and the lane that holds the activations of a
// token reads the same 32 columns.  Eight instructions use up a span.  The
// codes enter as code - zero, an integer of at most 8 bits and exact in bf16
// and fp16; a group's sum leaves the tensor core in fp32 and is scaled there.
// A group of 64 or 32 columns is summed by itself by running the span's
// instructions once per group with the other groups' activations set to zero:
// the matrix pipe has room for it, and the decoded codes stay in registers.
#pragma once
#include "packed.cuh"
#include "ptx.cuh"

namespace admmq {

constexpr int kFewRows = 64;      // output columns (weight rows) of a block
constexpr int kFewThreads = 256;

template <typename X>
__device__ __forceinline__ void mma_m16n8k16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma_m16n8k16<__nv_bfloat16>(float (&d)[4], uint32_t a0, uint32_t a1,
                                                            uint32_t a2, uint32_t a3, uint32_t b0,
                                                            uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma_m16n8k16<__half>(float (&d)[4], uint32_t a0, uint32_t a1,
                                                     uint32_t a2, uint32_t a3, uint32_t b0,
                                                     uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A block takes 64 output columns and one of the cluster's ranges of spans;
// its warps take spans in turn.
template <typename X, int NT, int B>
__device__ __forceinline__ void packed_few(const PackedArgs& p, float (&acc)[4][NT][4], int block,
                                           int sp0, int sp1) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = lane >> 2, q = lane & 3;
  const int passes = 128 / p.group;
  const bool vec = p.words % 4 == 0;  // rows start on 16 bytes
  for (int sp = sp0 + warp; sp < sp1; sp += kFewThreads / 32) {
    const int k = sp * 128 + 32 * q;   // this lane's 32 columns
    const bool in = k < p.k;
    uint32_t w[8][B];
    float z[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const long long row = (long long)block * kFewRows + i * 8 + r;
      if (in && row < p.n) {
        load_words<B>(p.packed + row * p.words + (sp * 4 + q) * B, vec, w[i]);
        z[i] = __ldg(p.zero + row * p.groups + k / p.group);
      } else {
#pragma unroll
        for (int j = 0; j < B; ++j) w[i][j] = 0u;
        z[i] = 0.f;
      }
    }
    uint32_t x[NT][16];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int token = t * 8 + r;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (in && token < p.m)
          v = __ldg(reinterpret_cast<const uint4*>((const X*)p.x + token * p.ldx + k) + i);
        x[t][4 * i] = v.x; x[t][4 * i + 1] = v.y; x[t][4 * i + 2] = v.z; x[t][4 * i + 3] = v.w;
      }
    }
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
      uint32_t a[2][16];
      decode32<X, B>(w[2 * rt], z[2 * rt], a[0]);
      decode32<X, B>(w[2 * rt + 1], z[2 * rt + 1], a[1]);
      const long long row = (long long)block * kFewRows + rt * 16 + r;
      for (int g = 0; g < passes; ++g) {
        const int gi = sp * passes + g;
        const bool mine = passes == 1 || q * passes / 4 == g;
        const bool there = gi < p.groups;
        const float s0 = there && row < p.n ? __ldg(p.scale + row * p.groups + gi) : 0.f;
        const float s1 = there && row + 8 < p.n ? __ldg(p.scale + (row + 8) * p.groups + gi) : 0.f;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < 8; ++j)
            mma_m16n8k16<X>(d, a[0][2 * j], a[1][2 * j], a[0][2 * j + 1], a[1][2 * j + 1],
                            mine ? x[t][2 * j] : 0u, mine ? x[t][2 * j + 1] : 0u);
          acc[rt][t][0] += s0 * d[0];
          acc[rt][t][1] += s0 * d[1];
          acc[rt][t][2] += s1 * d[2];
          acc[rt][t][3] += s1 * d[3];
        }
      }
    }
  }
}

template <typename X, int NT, int B>
__global__ void __launch_bounds__(kFewThreads) k_packed_few(const PackedArgs p) {
  __shared__ float part[kFewThreads / 32][8 * NT][kFewRows];
  __shared__ float sum[8 * NT][kFewRows];
  uint32_t rank, ranks;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
  const int block = blockIdx.x / ranks;
  const int spans = (p.k + 127) / 128;
  const int sp0 = (int)((long long)rank * spans / ranks), sp1 = (int)((long long)(rank + 1) * spans / ranks);
  float acc[4][NT][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][t][j] = 0.f;
  packed_few<X, NT, B>(p, acc, block, sp0, sp1);
  // the warps' sums, then the cluster's, each in a fixed order
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int rt = 0; rt < 4; ++rt)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        part[warp][t * 8 + 2 * (lane & 3) + (j & 1)][rt * 16 + (lane >> 2) + 8 * (j >> 1)] =
            acc[rt][t][j];
  __syncthreads();
  constexpr int OUT = 8 * NT * kFewRows;
  for (int i = threadIdx.x; i < OUT; i += kFewThreads) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kFewThreads / 32; ++w) v += part[w][i / kFewRows][i % kFewRows];
    sum[i / kFewRows][i % kFewRows] = v;
  }
  if (ranks > 1)
    cluster_sync();
  else
    __syncthreads();
  for (int i = rank * kFewThreads + threadIdx.x; i < OUT; i += ranks * kFewThreads) {
    const int token = i / kFewRows;
    const long long col = (long long)block * kFewRows + i % kFewRows;
    if (token >= p.m || col >= p.n) continue;
    float v = 0.f;
    if (ranks > 1) {
      for (uint32_t c = 0; c < ranks; ++c) {
        float f;
        asm volatile("ld.shared::cluster.f32 %0, [%1];"
                     : "=f"(f)
                     : "r"(cluster_addr(smem_u32(&sum[token][i % kFewRows]), c))
                     : "memory");
        v += f;
      }
    } else {
      v = sum[token][i % kFewRows];
    }
    put_out(p, (long long)token * p.n + col, v);
  }
  if (ranks > 1) cluster_sync();  // the sums stay until every rank has read them
}

}  // namespace admmq
