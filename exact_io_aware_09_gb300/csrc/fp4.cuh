// The 4-bit format of the cache: blocks of sixteen values of a row, each a scale byte and sixteen codes.
//
// A code is E2M1: a sign and 0, 1/2, 1, 3/2, 2, 3, 4 or 6.  A scale byte is E5M3, unsigned: fp16's exponent
// and its first three mantissa bits, so that the byte shifted left by seven is the scale in fp16.  Against
// E4M3, the usual type for such scales, it spends the sign's bit on range: blocks of 2^-17 to 61,440 need no
// second scale over them, and it converts with a shift.  A product code * scale has at most six significant
// bits, none below 2^-18, and is at most 61,440: exact in fp16, and in bf16.  A scale of all ones is a NaN
// in fp16 too, and makes the block's values NaN.
#pragma once
#include <cstdint>

namespace attn {

constexpr int kFp4Block = 16;
constexpr uint32_t kFp4MaxScale = 0xe2;  // 10,240: the largest whose product with 6 fp16 holds
constexpr uint32_t kFp4Nan = 0xff;

// Two codes (byte B of w, the low four bits first) -> an f16 pair.
template <int B>
__device__ __forceinline__ uint32_t e2m1x2_f16x2(uint32_t w) {
  uint32_t r;
  if constexpr (B == 0)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(r) : "r"(w));
  else if constexpr (B == 1)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(r) : "r"(w));
  else if constexpr (B == 2)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}" : "=r"(r) : "r"(w));
  else
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, d;\n\t}" : "=r"(r) : "r"(w));
  return r;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// A scale byte as an f16 pair of twice the same, and two as a pair.
__device__ __forceinline__ uint32_t fp4_scale_pair(uint32_t s) { return s * 0x00800080u; }
__device__ __forceinline__ uint32_t fp4_scale_pair(uint32_t lo, uint32_t hi) {
  return lo * 0x80u + hi * 0x800000u;
}

// A scale byte's value (not the NaN's).
__device__ __forceinline__ float fp4_scale(uint32_t s) {
  float f;
  asm("{\n\t.reg .b16 a;\n\tcvt.u16.u32 a, %1;\n\tcvt.f32.f16 %0, a;\n\t}" : "=f"(f) : "r"(s << 7));
  return f;
}

// Eight codes (a word, low bits first) times a scale pair -> four f16 pairs.
__device__ __forceinline__ void fp4_values8(uint32_t w, uint32_t scale, uint32_t (&v)[4]) {
  v[0] = mul_f16x2(e2m1x2_f16x2<0>(w), scale);
  v[1] = mul_f16x2(e2m1x2_f16x2<1>(w), scale);
  v[2] = mul_f16x2(e2m1x2_f16x2<2>(w), scale);
  v[3] = mul_f16x2(e2m1x2_f16x2<3>(w), scale);
}

// Eight values -> eight codes (a word, low bits first), nearest even, at most 6 in magnitude.
__device__ __forceinline__ uint32_t fp4_codes8(const float* v) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// The scale byte of a block whose largest magnitude is amax (finite): amax / 6 rounded to E5M3, nearest
// even; at least the smallest one where amax is not zero, at most kFp4MaxScale.
__device__ __forceinline__ uint32_t fp4_scale_byte(float amax) {
  // amax is a 16-bit number.  Half way between two scales (amax = 6 m, m of five bits) the product with the
  // rounded 1/6, 2^-25 too large, rounds to m itself: half of fp32's step there is more.  Elsewhere amax / 6 is
  // 2^-12 or more away from half way.
  const float t = amax * (1.0f / 6.0f);
  uint32_t b;
  if (t >= 6.103515625e-05f) {  // 2^-14, the smallest normal number
    const uint32_t u = __float_as_uint(t);
    b = ((u + 0x7ffffu + ((u >> 20) & 1u)) >> 20) - ((127 - 15) << 3);
  } else {
    b = static_cast<uint32_t>(__float2int_rn(t * 131072.0f));  // in units of 2^-17
  }
  if (amax > 0.0f && b == 0) b = 1;
  return b < kFp4MaxScale ? b : kFp4MaxScale;
}

}  // namespace attn
