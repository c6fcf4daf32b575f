// packed.cuh -- packed b-bit codes: loading and decoding 32 of them (b words)
// into 16-bit floating point.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "../../include/admmq.h"

namespace admmq {

struct PackedArgs {
  const void* x;
  const uint32_t* packed;
  const float *scale, *zero;
  void* out;
  long long ldx;
  int m, n, k;               // tokens, output columns, reduction
  int bits, group;
  int words, groups;         // words and groups of a weight row
  int out_dtype;
};

__device__ __forceinline__ void put_out(const PackedArgs& p, long long i, float v) {
  if (p.out_dtype == ADMMQ_DTYPE_F32)
    ((float*)p.out)[i] = v;
  else if (p.out_dtype == ADMMQ_DTYPE_BF16)
    ((__nv_bfloat16*)p.out)[i] = __float2bfloat16_rn(v);
  else
    ((__half*)p.out)[i] = __float2half_rn(v);
}

// The b words of 32 codes; vec: they start on b words' natural alignment (16
// bytes for 4 and 8 bits, 8 for 2 and 6).
template <int B>
__device__ __forceinline__ void load_words(const uint32_t* p, bool vec, uint32_t (&w)[B]) {
  if (B % 4 == 0 && vec) {
#pragma unroll
    for (int i = 0; i < B / 4; ++i) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
      w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
    }
  } else if (B % 2 == 0 && vec) {
#pragma unroll
    for (int i = 0; i < B / 2; ++i) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(p) + i);
      w[2 * i] = v.x; w[2 * i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < B; ++i) w[i] = __ldg(p + i);
  }
}

// Bits [at, at + 32) of the word array (what lies past it reads as zero).
template <int B>
__device__ __forceinline__ uint32_t bits_at(const uint32_t (&w)[B], int at) {
  const int i = at >> 5, s = at & 31;
  const uint32_t lo = w[i < B ? i : B - 1];
  if (s == 0) return lo;
  const uint32_t hi = i + 1 < B ? w[i + 1 < B ? i + 1 : B - 1] : 0u;
  return __funnelshift_r(lo, hi, s);
}

// 32 codes minus their zero point, as 16 pairs of X in column order.  A code
// goes into the low mantissa bits of 128 (bf16) or 1024 (fp16), where one
// step is 1; subtracting 128 + zero (1024 + zero) is exact.  Eight bits do not
// fit behind bf16's 128: they go through fp32's 2^23 instead.
template <typename X, int B>
__device__ __forceinline__ void decode32(const uint32_t (&w)[B], float zero, uint32_t (&out)[16]) {
  constexpr bool BF = sizeof(X) == 2 && __is_same(X, __nv_bfloat16);
  constexpr uint32_t MASK = (1u << B) - 1u;
  if constexpr (BF && B == 8) {
    const float zz = 8388608.f + zero;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t v = w[i >> 1];
      const float lo = __uint_as_float(__byte_perm(v, 0x4B000000u, 0x7650 + (i & 1 ? 2 : 0))) - zz;
      const float hi = __uint_as_float(__byte_perm(v, 0x4B000000u, 0x7651 + (i & 1 ? 2 : 0))) - zz;
      const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
      out[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  } else {
    constexpr uint32_t MAGIC = BF ? 0x43004300u : 0x64006400u;
    X z1;
    if constexpr (BF)
      z1 = __float2bfloat16_rn(128.f + zero);
    else
      z1 = __float2half_rn(1024.f + zero);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      // code 2i at bit 0 and code 2i + 1 at bit 16
      const uint32_t lo = bits_at<B>(w, 2 * i * B) & MASK;
      const uint32_t t = (2 * i + 1) * B >= 16 ? bits_at<B>(w, (2 * i + 1) * B - 16)
                                               : w[0] << (16 - (2 * i + 1) * B);
      const uint32_t v = lo | (t & (MASK << 16)) | MAGIC;
      if constexpr (BF) {
        const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v),
                                         __halves2bfloat162(z1, z1));
        out[i] = *reinterpret_cast<const uint32_t*>(&d);
      } else {
        const __half2 d =
            __hsub2(*reinterpret_cast<const __half2*>(&v), __halves2half2(z1, z1));
        out[i] = *reinterpret_cast<const uint32_t*>(&d);
      }
    }
  }
}

}  // namespace admmq
