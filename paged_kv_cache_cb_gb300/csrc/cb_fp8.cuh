// The 8-bit KV cache format and its conversions.
//
// A row x (one token, one KV head, A values) is stored as A e4m3 values and one
// exponent byte b = e + 127:
//     e = the least integer >= -126 with max|x| <= 448 * 2^e     (448: e4m3's largest)
//     stored value = round_e4m3(x * 2^-e)  (nearest, ties to even; never saturates)
// and stands for value * 2^e.  A row with a NaN or an infinity is stored as
// zeros with b = 255 and stands for NaNs, so no stored value is ever a NaN
// pattern and a bad row poisons only what its own (token, KV head) reaches.
// The scale is a power of two so that reading back is exact: an e4m3 value has 4
// significant bits, and times 2^e it is a bf16 number (8 bits, the exponents of
// fp32).  A free scale would cost a second rounding there, and it gains nothing:
// e4m3's relative step does not depend on where in its range a value falls.
#pragma once
#include "cb_common.cuh"

namespace cb {

constexpr uint32_t kExpNan = 255;      // exponent byte of a row that is not finite

// Exponent byte of a row whose largest magnitude has the bf16 bits `amax` (sign
// cleared): with amax = (1 + m / 128) 2^(E - 127), 448 = 1.75 * 2^8 gives
// e = E - 127 - 8 + (m > 96).
__device__ __forceinline__ uint32_t row_exp(uint32_t amax) {
  if (amax >= 0x7F80u) return kExpNan;
  return (uint32_t)max(1, (int)(amax >> 7) - 8 + ((amax & 127u) > 96u));
}
// 2^e of an exponent byte (NaN for 255); 2^-e of a finite one (1 .. 253).
__device__ __forceinline__ float exp_scale(uint32_t b) {
  return __uint_as_float(b == kExpNan ? 0x7FC00000u : b << 23);
}
__device__ __forceinline__ float exp_inverse(uint32_t b) { return __uint_as_float((254u - b) << 23); }

// Two floats -> two e4m3 in the low 16 bits (first one lowest), rounded to nearest even.
__device__ __forceinline__ uint32_t pack_e4m3(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two e4m3 (low 16 bits of w) -> two halves packed in a word; exact.
__device__ __forceinline__ uint32_t e4m3_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)w));
  return r;
}
// Two e4m3 (low 16 bits of w) -> two floats; exact.
__device__ __forceinline__ void e4m3_to_f32(uint32_t w, float& lo, float& hi) {
  const uint32_t h = e4m3_to_f16x2(w);
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
}

}  // namespace cb
