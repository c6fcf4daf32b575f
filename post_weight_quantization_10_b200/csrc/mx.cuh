// mx.cuh -- microscaled 4-bit floating point: element and scale conversions
// and the layout of the stored scales.
//
// An element is e2m1 (sign, 2 exponent bits, 1 mantissa bit: 0, 1/2, 1, 3/2,
// 2, 3, 4, 6), two to a byte, element 2i in the low nibble.  A block of a row
// shares a step t, the value of the element code 1.0:
//   mxfp4  32 elements, t = 2^(byte - 127) (e8m0; byte 255 is NaN);
//   nvfp4  16 elements, t = fl32(e4m3(byte) g), g the tensor's fp32 scale.
// Scale bytes lie as the tensor cores read them: tiles of 128 rows x 4 blocks,
// 512 bytes, [ceil(rows / 128)][ceil(blocks / 4)][32][4][4]: row r, block c of
// a tile at byte 16 (r % 32) + 4 (r / 32) + c.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace admmq {

enum { MX_MXFP4 = 0, MX_NVFP4 = 1 };

template <int FMT>
struct MxFormat {
  static constexpr int BLOCK = FMT == MX_MXFP4 ? 32 : 16;  // elements that share a scale
  static constexpr int TILE_K = 4 * BLOCK;                 // elements of a row in a scale tile
};

constexpr int kScaleTile = 512;

// Byte of row r (of 128) and block c (of 4) inside a scale tile.
__device__ __forceinline__ int scale_at(int r, int c) { return 16 * (r & 31) + 4 * (r >> 5) + c; }

// Two fp32 values to e2m1, nearest-even, saturating at 6; lo in the low nibble.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 b;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\t"
      "cvt.u32.u8 %0, b;\n\t}"
      : "=r"(r)
      : "f"(hi), "f"(lo));
  return r;
}

// The two elements of a byte, exact in fp16.
__device__ __forceinline__ float2 e2m1x2_values(uint32_t byte) {
  uint32_t r;
  asm("{\n\t.reg .b8 b;\n\t"
      "cvt.u8.u32 b, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b;\n\t}"
      : "=r"(r)
      : "r"(byte));
  return __half22float2(*reinterpret_cast<__half2*>(&r));
}

// e8m0 byte to its power of two (2^-127 is an fp32 subnormal; 255 is NaN).
__device__ __forceinline__ float e8m0_value(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7FFFFFFFu : byte << 23);
}

// e4m3 byte (sign clear) to fp32, exact; 0x7F is NaN.
__device__ __forceinline__ float e4m3_value(uint32_t byte) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)byte));
  return __low2float(*reinterpret_cast<__half2*>(&r));
}

// fp32 >= 0 to e4m3, nearest-even, saturating at 448; NaN to 0x7F.
__device__ __forceinline__ uint32_t e4m3_byte(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
  return r & 0xFFu;
}

// Step of a block from its scale byte (g: the tensor scale, 1 for mxfp4).
template <int FMT>
__device__ __forceinline__ float block_step(uint32_t byte, float g) {
  return FMT == MX_MXFP4 ? e8m0_value(byte) : __fmul_rn(e4m3_value(byte), g);
}

// Scale byte of a block from the largest magnitude in it (bit pattern, so that
// infinities and NaN stay on top).  A block that holds one is NaN as a whole.
template <int FMT>
__device__ __forceinline__ uint32_t block_scale(uint32_t amax_bits, float g) {
  if (FMT == MX_MXFP4) {
    // 2^(floor(log2 amax) - 2), not below 2^-127: the largest element lands
    // in [4, 8) and saturates at 6
    if (amax_bits >= 0x7F800000u) return 0xFFu;
    const uint32_t e = amax_bits >> 23;
    return e > 2 ? e - 2 : 0;
  }
  if (amax_bits == 0u) return 0u;  // whatever g is (0 too, from a matrix of zeros)
  if (amax_bits >= 0x7F800000u) return 0x7Fu;
  // e4m3(amax / (6 g)), nearest-even.  6 g and the comparison against any
  // rounding border need 32 bits, so the float64 quotient is on the right
  // side of it; its tail goes into the float's last bit (round to odd), which
  // a second rounding to 4 bits respects.
  const double q = (double)__uint_as_float(amax_bits) / (6.0 * (double)g);
  float f = __double2float_rz(q);
  if ((double)f != q) f = __uint_as_float(__float_as_uint(f) | 1u);
  return e4m3_byte(f);
}

// 1 / step for mxfp4 (a power of two, exact; byte <= 252).
__device__ __forceinline__ float e8m0_inverse(uint32_t byte) {
  return __uint_as_float((254u - byte) << 23);
}

// x / t for one element, good enough to be rounded to e2m1 as the exact
// quotient would be: the quotient is corrected once by its residual, and the
// sign of what remains goes into the last bit, so that a value next to a
// rounding border stays on its side of it.  2^-100 <= t, r = 1 / t.
__device__ __forceinline__ float quotient_to_odd(float x, float t, float r) {
  const float a = fminf(fabsf(x), 8.f * t);  // above 6 t everything saturates
  float y = __fmul_rn(a, r);
  y = __fmaf_rn(__fmaf_rn(-y, t, a), r, y);
  const float e = __fmaf_rn(-y, t, a);
  uint32_t b = __float_as_uint(y);
  if (e < 0.f) b -= 1u;
  if (e != 0.f) b |= 1u;
  return __uint_as_float(b | (__float_as_uint(x) & 0x80000000u));
}

}  // namespace admmq
