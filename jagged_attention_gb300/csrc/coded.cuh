// coded.cuh -- how a cache of 8 or 4 bits holds a row of a head, and the arithmetic
// between its codes and their values.
//
// 8 bits: e4m3 codes and one byte c for the row's head, value = code * 2^(c - 127).  A
// power of two: codes have the same 3 mantissa bits anywhere in their range, so a finer
// scale would gain nothing, and this one multiplies and divides exactly.  The range of
// c keeps weights times scales far within fp32 (decode_coded.cuh).
// 4 bits: e2m1 codes, the first value of two in the lower nibble, and a byte for each
// 16 values, their scale as bits 14 .. 7 of the fp16 number (5 exponent bits, 3 of the
// mantissa, no sign): a code has 2 mantissa bits, its product with a scale 6, exact in
// fp16 and bf16.
// A byte of 255 is NaN in both: what it belongs to held a value that is not finite.
#pragma once
#include <cstdint>
#include <cuda_fp16.h>

#include "sm103_ptx.cuh"

namespace jfa {

constexpr int kBlock = 16;                        // values of a scale, 4 bits
constexpr int kLeastPower = 79, kMostPower = 175;  // bytes of 2^-48 and 2^48, 8 bits
constexpr int kNanScale = 255;
constexpr float kMostScale = 10240.f;  // 4 bits: 6 * 11264, the next scale's largest, is beyond fp16

template <int kBits>
__host__ __device__ constexpr int scale_bytes(int D) {
  return kBits == 8 ? 1 : D / kBlock;
}

// ---- values to codes.  `top`: the largest magnitude of bf16 values, as its bits.

__device__ __forceinline__ uint32_t top_of(uint32_t a, uint32_t b) { return __vmaxu2(a & 0x7fff7fffu, b & 0x7fff7fffu); }
__device__ __forceinline__ uint32_t top_of(const uint4& w) {
  const uint32_t t = __vmaxu2(top_of(w.x, w.y), top_of(w.z, w.w));
  return max(t & 0xffffu, t >> 16);
}
// The byte of the least power of two that takes `top` to 448 = 1.75 * 2^8 at most: its
// exponent less 8, one more from a mantissa of 97/128 on.
__device__ __forceinline__ int power_of(uint32_t top) {
  if (top >= 0x7f80u) return kNanScale;
  return min(max(static_cast<int>((top + 31) >> 7) - 8, kLeastPower), kMostPower);
}
// The byte of a block's scale, top / 6 to nearest even.  The quotient's rounding to
// fp32 moves no value over or onto a border between two scales: a border has 5 bits,
// six times it 7 or fewer, as bf16 has 8.
__device__ __forceinline__ int scale_of(uint32_t top) {
  if (top >= 0x7f80u) return kNanScale;
  const float s = fminf(__fdiv_rn(__uint_as_float(top << 16), 6.f), kMostScale);
  if (s < 0x1p-14f) return __float2int_rn(s * 0x1p17f);
  const uint32_t bits = __float_as_uint(s);
  return static_cast<int>((bits + 0x7ffffu + ((bits >> 20) & 1)) >> 20) - (112 << 3);
}
__device__ __forceinline__ float scale_value(int byte) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(byte << 7)));
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{.reg .b16 x, y;\n\tcvt.rn.satfinite.e4m3x2.f32 x, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 y, %4, %3;\n\t"
      "mov.b32 %0, {x, y};}" : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
__device__ __forceinline__ uint32_t e2m1x8(const float (&x)[8]) {
  uint32_t r;
  asm("{.reg .b8 a, b, c, d;\n\tcvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\tmov.b32 %0, {a, b, c, d};}"
      : "=r"(r) : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}
// 8 bf16 values as e4m3 codes of a row with power byte c.
__device__ __forceinline__ uint2 code8(const float (&x)[8], int c) {
  const float by = __uint_as_float(static_cast<uint32_t>(254 - c) << 23);  // c = 255: whatever, all is NaN
  return make_uint2(e4m3x4(x[0] * by, x[1] * by, x[2] * by, x[3] * by), e4m3x4(x[4] * by, x[5] * by, x[6] * by, x[7] * by));
}
// 8 bf16 values as e2m1 codes of a block with scale byte c.  x / s is a value half way
// between two codes or at least 2^-11 from it (8 bits of x, 4 of s); x times the rounded
// 1 / s is off by 2^-21, and rounded to a multiple of 2^-14 it is that value again, or on
// the right side of it.
__device__ __forceinline__ uint32_t code4(const float (&x)[8], int c) {
  const float s = scale_value(c);
  const float by = s > 0.f ? __frcp_rn(s) : 0.f;  // 0 for NaN
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)  // zero keeps the sign
    y[i] = copysignf(__fsub_rn(__fadd_rn(__fmul_rn(x[i], by), 768.f), 768.f), x[i]);
  return e2m1x8(y);
}

// ---- codes to values

// A power byte of a row as it counts: NaN, or a power of two.
__device__ __forceinline__ float power_value(int c) {
  return c == kNanScale ? __uint_as_float(0x7fffffffu)
                        : __uint_as_float(static_cast<uint32_t>(min(max(c, kLeastPower), kMostPower)) << 23);
}
__device__ __forceinline__ void halves_of_e4m3x4(uint32_t w, uint32_t& a, uint32_t& b) {
  asm("{.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\tcvt.rn.f16x2.e4m3x2 %1, y;}"
      : "=r"(a), "=r"(b) : "r"(w));
}
__device__ __forceinline__ void halves_of_e2m1x8(uint32_t w, uint32_t (&r)[4]) {
  asm("{.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(w));
}
__device__ __forceinline__ float2 floats_of(uint32_t h2) { return __half22float2(*reinterpret_cast<__half2*>(&h2)); }
// A pair of fp16 values times a factor, as bf16: exact for codes and their scales.
__device__ __forceinline__ uint32_t bf16_of(uint32_t h2, float by) {
  const float2 f = floats_of(h2);
  return pack_bf16x2(f.x * by, f.y * by);
}

}  // namespace jfa
