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

// Bits [at, at + 32) of the word array (what lies past it reads as zero).
template <int B>
__device__ __forceinline__ uint32_t bits_at(const uint32_t (&w)[B], int at) {
  const int i = at >> 5, s = at & 31;
  const uint32_t lo = w[i < B ? i : B - 1];
  if (s == 0) return lo;
  const uint32_t hi = i + 1 < B ? w[i + 1 < B ? i + 1 : B - 1] : 0u;
  return __funnelshift_r(lo, hi, s);
}

// (a & b) | c
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// 32 codes minus their zero point as 16 pairs of X: pair i holds codes i and
// i + 16.  (The two are 16 b bits apart, so one window of 16 bits from each
// half of the block, side by side in a word, gives 16 / b pairs by a mask.)  A
// masked code at bit p goes into the mantissa of 128 (bf16) or 1024 (fp16),
// whose last bit is worth 1: 128 + 2^p code.  One multiply-add by 2^-p and
// -(128 2^-p + zero) leaves code - zero; every value on the way is exact.
// Eight bits do not fit behind bf16's 128: they go through fp32's 2^23.
template <typename X, int B>
__device__ __forceinline__ void decode32(const uint32_t (&w)[B], float zero, uint32_t (&out)[16]) {
  constexpr bool BF = __is_same(X, __nv_bfloat16);
  if constexpr (BF && B == 8) {
    const float zz = 8388608.f + zero;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t sel = 0x7650u + (i & 3);  // byte i % 4, then the three upper bytes of 2^23
      const float lo = __uint_as_float(__byte_perm(w[i >> 2], 0x4B000000u, sel)) - zz;
      const float hi = __uint_as_float(__byte_perm(w[4 + (i >> 2)], 0x4B000000u, sel)) - zz;
      const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
      out[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  } else {
    constexpr uint32_t MASK = (1u << B) - 1u;
    constexpr int MANTISSA = BF ? 7 : 10;
    constexpr int PER = 16 / B;             // codes of a 16-bit window
    constexpr int FIT = MANTISSA / B;       // of them, without a shift
    constexpr uint32_t MAGIC = BF ? 0x43004300u : 0x64006400u;
    constexpr float BASE = BF ? 128.f : 1024.f;
    X minus[FIT];
#pragma unroll
    for (int f = 0; f < FIT; ++f) {
      const float c = -(BASE / (float)(1 << (f * B)) + zero);
      if constexpr (BF)
        minus[f] = __float2bfloat16_rn(c);
      else
        minus[f] = __float2half_rn(c);
    }
#pragma unroll
    for (int c0 = 0; c0 < 16; c0 += PER) {
      // (a window that ends with its word is that word's upper half)
      const bool upper = (B * c0 & 31) == 16 && (B * 16 & 31) == 0;
      const uint32_t t = upper ? __byte_perm(w[B * c0 >> 5], w[B * (c0 + 16) >> 5], 0x7632)
                               : __byte_perm(bits_at<B>(w, B * c0), bits_at<B>(w, B * (c0 + 16)), 0x5410);
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (c0 + i >= 16) break;
        const int f = i % FIT;
        const uint32_t m = (MASK | (MASK << 16)) << (f * B);
        const uint32_t v = and_or(t >> ((i - f) * B), m, MAGIC);
        if constexpr (BF) {
          const X up = __float2bfloat16_rn(1.f / (float)(1 << (f * B)));
          const __nv_bfloat162 d = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&v),
                                           __halves2bfloat162(up, up),
                                           __halves2bfloat162(minus[f], minus[f]));
          out[c0 + i] = *reinterpret_cast<const uint32_t*>(&d);
        } else {
          const X up = __float2half_rn(1.f / (float)(1 << (f * B)));
          const __half2 d = __hfma2(*reinterpret_cast<const __half2*>(&v), __halves2half2(up, up),
                                    __halves2half2(minus[f], minus[f]));
          out[c0 + i] = *reinterpret_cast<const uint32_t*>(&d);
        }
      }
    }
  }
}

// As decode32, but in column order: out[j] holds codes 2 j and 2 j + 1.  Two
// windows of the bit stream, one code apart, side by side: a mask then takes
// neighbouring codes from the two halves.  (For 2 and 4 bits a byte of the
// word and of the word shifted by one code serve as the windows.)
template <typename X, int B>
__device__ __forceinline__ void decode32_in_order(const uint32_t (&w)[B], float zero,
                                                  uint32_t (&out)[16]) {
  constexpr bool BF = __is_same(X, __nv_bfloat16);
  if constexpr (BF && B == 8) {
    const float zz = 8388608.f + zero;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const uint32_t sel = 0x7650u + 2 * (j & 1);
      const float lo = __uint_as_float(__byte_perm(w[j >> 1], 0x4B000000u, sel)) - zz;
      const float hi = __uint_as_float(__byte_perm(w[j >> 1], 0x4B000000u, sel + 1)) - zz;
      const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
      out[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
  } else {
    constexpr uint32_t MASK = (1u << B) - 1u;
    constexpr int MANTISSA = BF ? 7 : 10;
    constexpr bool BYTES = B == 2 || B == 4 || B == 8;
    constexpr int PER = BYTES ? 8 / B : 16 / B;        // codes of a window
    constexpr int PAIRS = (PER + 1) / 2;               // pairs (even code, next one) of two windows
    constexpr int FIT = (MANTISSA - B) / (2 * B) + 1;  // of them, without a shift
    constexpr uint32_t MAGIC = BF ? 0x43004300u : 0x64006400u;
    constexpr float BASE = BF ? 128.f : 1024.f;
    X minus[FIT];
#pragma unroll
    for (int f = 0; f < FIT; ++f) {
      const float c = -(BASE / (float)(1 << (2 * f * B)) + zero);
      if constexpr (BF)
        minus[f] = __float2bfloat16_rn(c);
      else
        minus[f] = __float2half_rn(c);
    }
#pragma unroll
    for (int j0 = 0; j0 < 16; j0 += PAIRS) {
      uint32_t t;
      if constexpr (B == 8) {
        t = __byte_perm(w[j0 >> 1], 0u, j0 & 1 ? 0x4342 : 0x4140);
      } else if constexpr (BYTES) {
        const uint32_t v = w[2 * j0 * B / 32];
        const int byte = 2 * j0 * B / 8 % 4;
        t = __byte_perm(v, v >> B, byte | (byte << 4) | ((byte + 4) << 8) | ((byte + 4) << 12));
      } else {
        t = __byte_perm(bits_at<B>(w, 2 * j0 * B), bits_at<B>(w, (2 * j0 + 1) * B), 0x5410);
      }
#pragma unroll
      for (int i = 0; i < PAIRS; ++i) {
        if (j0 + i >= 16) break;
        const int f = i % FIT;
        const uint32_t m = (MASK | (MASK << 16)) << (2 * f * B);
        const uint32_t v = and_or(t >> (2 * (i - f) * B), m, MAGIC);
        if constexpr (BF) {
          const X up = __float2bfloat16_rn(1.f / (float)(1 << (2 * f * B)));
          const __nv_bfloat162 d = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&v),
                                           __halves2bfloat162(up, up),
                                           __halves2bfloat162(minus[f], minus[f]));
          out[j0 + i] = *reinterpret_cast<const uint32_t*>(&d);
        } else {
          const X up = __float2half_rn(1.f / (float)(1 << (2 * f * B)));
          const __half2 d = __hfma2(*reinterpret_cast<const __half2*>(&v), __halves2half2(up, up),
                                    __halves2half2(minus[f], minus[f]));
          out[j0 + i] = *reinterpret_cast<const uint32_t*>(&d);
        }
      }
    }
  }
}

}  // namespace admmq
