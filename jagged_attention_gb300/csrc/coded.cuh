// coded.cuh -- how a cache of 8 or 4 bits holds a row of a head, and the arithmetic
// between its codes and their values.
//
// 8 bits: e4m3 codes and one byte c for the row's head, value = code * 2^(c - 127).  A
// power of two: codes have the same 3 mantissa bits anywhere in their range, so a finer
// scale would gain nothing, and this one multiplies and divides exactly.  The range of
// c keeps weights times scales far within fp32 (decode_kernel.cuh).
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

// The larger magnitudes of two pairs of bf16 values, as their bits; NaN is the largest.
// Sign bits may be set.
__device__ __forceinline__ uint32_t max_of(uint32_t a, uint32_t b) {
  uint32_t m;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
  return m;
}
__device__ __forceinline__ uint32_t top_of(uint32_t pair) { return max(pair & 0x7fffu, (pair >> 16) & 0x7fffu); }
__device__ __forceinline__ uint32_t max_of(const uint4& w) { return max_of(max_of(w.x, w.y), max_of(w.z, w.w)); }
// The byte of the least power of two that takes `top` to 448 = 1.75 * 2^8 at most: its
// exponent less 8, one more from a mantissa of 97/128 on.
__device__ __forceinline__ int power_of(uint32_t top) {
  if (top >= 0x7f80u) return kNanScale;
  return min(max(static_cast<int>((top + 31) >> 7) - 8, kLeastPower), kMostPower);
}
// The byte of a block's scale, top / 6 to nearest even.  Half way between two scales lie
// numbers of 5 bits; six times one has 7, so that top, of 8 bits, is that or 2^-9 off it.
// top times the rounded 1/6 is off by 2^-23, and rounded to 12 bits it is the number
// again, or on the right side of it.
__device__ __forceinline__ int scale_of(uint32_t top) {
  if (top >= 0x7f80u) return kNanScale;
  const float s = fminf(__uint_as_float(top << 16) * (1.f / 6.f), kMostScale);
  const uint32_t bits = (__float_as_uint(s) + 0x800u) & 0xfffff000u;
  const int byte = static_cast<int>((bits + 0x7ffffu + ((bits >> 20) & 1)) >> 20) - (112 << 3);
  return s < 0x1p-14f ? __float2int_rn(__uint_as_float(bits) * 0x1p17f) : byte;
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
// Codes of 8 numbers, by way of fp16.
__device__ __forceinline__ uint32_t e2m1x8(const float (&x)[8]) {
  uint32_t r;
  asm("{.reg .b8 a, b, c, d;\n\t.reg .b32 s, t, u, v;\n\tcvt.rn.f16x2.f32 s, %2, %1;\n\tcvt.rn.f16x2.f32 t, %4, %3;\n\t"
      "cvt.rn.f16x2.f32 u, %6, %5;\n\tcvt.rn.f16x2.f32 v, %8, %7;\n\tcvt.rn.satfinite.e2m1x2.f16x2 a, s;\n\t"
      "cvt.rn.satfinite.e2m1x2.f16x2 b, t;\n\tcvt.rn.satfinite.e2m1x2.f16x2 c, u;\n\t"
      "cvt.rn.satfinite.e2m1x2.f16x2 d, v;\n\tmov.b32 %0, {a, b, c, d};}"
      : "=r"(r) : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}
// 8 bf16 values as e4m3 codes of a row with power byte c.
__device__ __forceinline__ uint2 code8(const float (&x)[8], int c) {
  const float by = __uint_as_float(static_cast<uint32_t>(254 - c) << 23);  // c = 255: whatever, all is NaN
  const uint64_t by2 = f2_pack(by, by);
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; i += 2) f2_unpack(f2_mul(f2_pack(x[i], x[i + 1]), by2), y[i], y[i + 1]);
  return make_uint2(e4m3x4(y[0], y[1], y[2], y[3]), e4m3x4(y[4], y[5], y[6], y[7]));
}
// 1 / s for a block with scale byte c; 0 where s is 0, and all codes are 0, or NaN, and they do not matter.
__device__ __forceinline__ float inverse_scale(int c) {
  const float s = scale_value(c);
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));  // a unit in the last place
  return s > 0.f ? r : 0.f;
}
// 8 bf16 values as e2m1 codes of a block with that inverse scale.  x / s is a value half way
// between two codes, of 3 bits, or at least 2^-8 of itself from it (8 bits of x, 4 of s); x
// times 1 / s as the hardware has it is off by 2^-21, and rounded to the 11 bits of fp16 it
// is that value again, or on the right side of it.
__device__ __forceinline__ uint32_t code4(const float (&x)[8], float by) {
  const uint64_t by2 = f2_pack(by, by);
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; i += 2) f2_unpack(f2_mul(f2_pack(x[i], x[i + 1]), by2), y[i], y[i + 1]);
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
