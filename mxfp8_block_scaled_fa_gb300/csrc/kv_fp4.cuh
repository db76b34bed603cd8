// kv_fp4.cuh -- arithmetic of the 4-bit cache shared by its kernels: E2M1 codes and
// block scales as binary16, and packing.
#pragma once
#include "mx_ptx.cuh"

namespace mxfa {

// Eight E2M1 codes -> four pairs of binary16 (exact).  One conversion per byte; the
// byte is chosen within the instruction.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t* h) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// A pair of E8M0 bytes -> binary16 pair 2^(b - 127); 0xFF gives Inf, which times
// the code 0 it comes with is NaN; 0 gives 0.
__device__ __forceinline__ uint32_t e8m0_pair(uint32_t lo, uint32_t hi) {
  return pack_f16(__uint_as_float(lo << 23), __uint_as_float(hi << 23));
}
// Two E4M3 bytes -> binary16 pair (exact, NaN stays NaN).
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(uint16_t(two)));
  return r;
}

// The power of two that brings a query row whose largest |bf16| pattern is `mx`
// to [2^14, 2^15) (at most 2^126; 1 for a row of zeros), and its inverse.  For a row with
// Inf or NaN, whose scores are all infinite or NaN and so its results NaN, the first is NaN:
// scores of -inf alone would look like a row that sees no key.
__device__ __forceinline__ float2 q_row_scale(uint32_t mx) {
  const int fe = mx == 0 ? 127 : min(253, 268 - int(mx >> 7));
  const float f = __uint_as_float(mx >= 0x7F80u ? 0x7FC00000u : uint32_t(fe) << 23);
  return make_float2(f, __uint_as_float(uint32_t(254 - fe) << 23));
}

}  // namespace mxfa
