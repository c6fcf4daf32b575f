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

// Eight fp32 values to e2m1, nearest-even, saturating at 6; the first in the
// lowest nibble.
__device__ __forceinline__ uint32_t e2m1x8(const float* v) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
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
// g: the tensor scale, r6g = 1 / (6 g) (nvfp4).
template <int FMT>
__device__ __forceinline__ uint32_t block_scale(uint32_t amax_bits, float g, float r6g) {
  if (FMT == MX_MXFP4) {
    // 2^(floor(log2 amax) - 2), not below 2^-127: the largest element lands
    // in [4, 8) and saturates at 6
    if (amax_bits >= 0x7F800000u) return 0xFFu;
    const uint32_t e = amax_bits >> 23;
    return e > 2 ? e - 2 : 0;
  }
  if (amax_bits == 0u) return 0u;  // whatever g is (0 too, from a matrix of zeros)
  if (amax_bits >= 0x7F800000u) return 0x7Fu;
  // e4m3(amax / (6 g)), nearest-even.  The fp32 product is within 2^-21 of the
  // quotient: where both ends of that range round to one value, so does it.
  const float q32 = __uint_as_float(amax_bits) * r6g;
  if (q32 >= 0x1p-20f && q32 < 0x1p20f) {
    const uint32_t lo = e4m3_byte(q32 * (1.f - 0x1p-20f)), hi = e4m3_byte(q32 * (1.f + 0x1p-20f));
    if (lo == hi) return lo;
  }
  // Else by float64: 6 g and a comparison against any rounding border need 32
  // bits, so its quotient is on the right side of the border; its tail goes
  // into the float's last bit (round to odd), which a second rounding to 4
  // bits respects.
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

// Two products by one factor.
__device__ __forceinline__ void mul_x2(float& a, float& b, float x, float y, float f) {
  uint64_t p, q;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(x), "f"(y));
  asm("mov.b64 %0, {%1, %1};" : "=l"(q) : "f"(f));
  asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(p) : "l"(q));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}

// nvfp4 elements next to a rounding border of their block's grid: exactly.
// (Rare, and kept out of the way of the common path's code.)
__device__ __noinline__ uint2 quantize_exactly(const float* v, float t) {
  // tiny steps: both sides times 2^64, so that 1 / t is finite
  const float up = t < 0x1p-64f ? 0x1p64f : 1.f, tt = t * up, r = __frcp_rn(tt);
  uint32_t out[2];
#pragma unroll 1
  for (int j = 0; j < 2; ++j) {
    float u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = quotient_to_odd(v[8 * j + i] * up, tt, r);
    out[j] = e2m1x8(u);
  }
  return make_uint2(out[0], out[1]);
}

// Sixteen elements of a block with scale byte `byte` to e2m1, two to a byte.
template <int FMT>
__device__ __forceinline__ uint2 quantize16(const float (&v)[16], uint32_t byte, float g) {
  uint32_t out[2];
  float u[16];
  if (FMT == MX_MXFP4) {
    const float inv = e8m0_inverse(byte == 0xFFu ? 127u : byte);
#pragma unroll
    for (int i = 0; i < 16; i += 2) mul_x2(u[i], u[i + 1], v[i], v[i + 1], inv);
    const bool nan = byte == 0xFFu;
    return make_uint2(nan ? 0u : e2m1x8(u), nan ? 0u : e2m1x8(u + 8));
  }
  const float t = block_step<FMT>(byte, g);
  if (!(t > 0.f)) return make_uint2(0u, 0u);  // zero or NaN
  // x times 1 / t is within 2^-21 of the quotient; where both ends of that
  // range round to one code, so does the quotient
  const float r = __frcp_rn(t), lo = r * (1.f - 0x1p-20f), hi = r * (1.f + 0x1p-20f);
#pragma unroll
  for (int i = 0; i < 16; i += 2) mul_x2(u[i], u[i + 1], v[i], v[i + 1], lo);
  out[0] = e2m1x8(u);
  out[1] = e2m1x8(u + 8);
#pragma unroll
  for (int i = 0; i < 16; i += 2) mul_x2(u[i], u[i + 1], v[i], v[i + 1], hi);
  if ((out[0] ^ e2m1x8(u)) | (out[1] ^ e2m1x8(u + 8)) | (uint32_t)(t < 0x1p-100f)) {
    float w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = v[i];
    return quantize_exactly(w, t);
  }
  return make_uint2(out[0], out[1]);
}

// Sixteen consecutive elements of a row in registers, and as fp32.  Rows on 32
// bytes (wide) move by 256-bit accesses, whole sectors of a lane's own; others
// by 128-bit ones.
template <typename T>
struct Raw16 {
  uint32_t w[4 * sizeof(T)];
};
template <typename T>
__device__ __forceinline__ void load_raw(const T* p, bool wide, Raw16<T>& r) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
    uint32_t(&w)[8] = *reinterpret_cast<uint32_t(*)[8]>(r.w + 8 * i);
    const uint4* q = reinterpret_cast<const uint4*>(p) + 2 * i;
    if (wide) {
      asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                     "=r"(w[6]), "=r"(w[7])
                   : "l"(q));
    } else {
      const uint4 a = __ldg(q), b = __ldg(q + 1);
      w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
      w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    }
  }
}
__device__ __forceinline__ void values_of(const Raw16<float>& r, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r.w[i]);
}
__device__ __forceinline__ void values_of(const Raw16<__nv_bfloat16>& r, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[2 * i] = __uint_as_float(r.w[i] << 16);
    v[2 * i + 1] = __uint_as_float(r.w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void values_of(const Raw16<__half>& r, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r.w[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
// Largest magnitude as an fp32 bit pattern; NaN stays on top.
__device__ __forceinline__ uint32_t amax_of(const Raw16<float>& r) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(__uint_as_float(r.w[i]))));
  return __float_as_uint(m) & 0x7FFFFFFFu;
}
template <typename T2, typename T>
__device__ __forceinline__ T2 amax_pairs(const Raw16<T>& r) {
  T2 m[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) m[i] = __habs2(*reinterpret_cast<const T2*>(&r.w[i]));
#pragma unroll
  for (int n = 4; n > 0; n >>= 1)
#pragma unroll
    for (int i = 0; i < n; ++i) m[i] = __hmax2_nan(m[i], m[i + n]);
  return m[0];
}
__device__ __forceinline__ uint32_t amax_of(const Raw16<__nv_bfloat16>& r) {
  const __nv_bfloat162 m = amax_pairs<__nv_bfloat162>(r);
  const uint32_t w = *reinterpret_cast<const uint32_t*>(&m);
  return max(w << 16, w & 0xFFFF0000u);  // magnitudes: ordered as integers
}
__device__ __forceinline__ uint32_t amax_of(const Raw16<__half>& r) {
  const __half2 m = amax_pairs<__half2>(r);
  const uint32_t w = *reinterpret_cast<const uint32_t*>(&m);
  return __float_as_uint(__half2float(__ushort_as_half((unsigned short)max(w & 0xFFFFu, w >> 16)))) & 0x7FFFFFFFu;
}
// The other way: rounded to T and stored.
__device__ __forceinline__ void raw_of(const float (&v)[16], Raw16<float>& r) {
#pragma unroll
  for (int i = 0; i < 16; ++i) r.w[i] = __float_as_uint(v[i]);
}
__device__ __forceinline__ void raw_of(const float (&v)[16], Raw16<__nv_bfloat16>& r) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    r.w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
}
__device__ __forceinline__ void raw_of(const float (&v)[16], Raw16<__half>& r) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    r.w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
}
template <typename T>
__device__ __forceinline__ void store_raw(T* p, bool wide, const Raw16<T>& r) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
    const uint32_t* w = r.w + 8 * i;
    uint4* q = reinterpret_cast<uint4*>(p) + 2 * i;
    if (wide) {
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(q), "r"(w[0]),
                   "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                   : "memory");
    } else {
      q[0] = make_uint4(w[0], w[1], w[2], w[3]);
      q[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
}

}  // namespace admmq
