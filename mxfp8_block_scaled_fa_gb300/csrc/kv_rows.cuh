// kv_rows.cuh -- a row of the 4-bit cache (one token of one key head) from bf16, shared by the
// kernels that store: sixteen lanes a row, eight channels a lane.
#pragma once
#include "kv_fp4.cuh"
#include "mx_ptx.cuh"
#include "mxfa_internal.h"

namespace mxfa {

__device__ __forceinline__ uint32_t pack8_e2m1(const float* y) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return r;
}

// Sixteen bytes that nothing reads again soon.
__device__ __forceinline__ uint4 ldg_stream(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// Stores this lane's eight channels of cache row `at`; all lanes of the warp call it, those without a
// row with live = false.
template <int FMT>
__device__ __forceinline__ void kv_store_row(const KvPages& c, bool live, bool is_v, int64_t at, int lane, uint4 x) {
  const uint32_t m2 = __vmaxu2(__vmaxu2(abs2(x.x), abs2(x.y)), __vmaxu2(abs2(x.z), abs2(x.w)));
  uint32_t mx = hmax2(m2);
  mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
  if (FMT == 0) mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
  if (!live) return;
  const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
  float y[8];
  uint32_t sc;
  const bool bad = mx >= 0x7F80u;
  if (FMT == 0) {
    // bf16 exponent field - 2, clamped to the fields of 2^-23 and 2^13
    sc = min(max(int(mx >> 7) - 2, 104), 140);
    const float f = __uint_as_float((254u - sc) << 23);
#pragma unroll
    for (int e = 0; e < 4; e++) {
      y[2 * e] = bf_lo(xs[e]) * f;
      y[2 * e + 1] = bf_hi(xs[e]) * f;
    }
    if (bad) sc = 0xFFu;
  } else {
    const float st = __ldg(is_v ? c.v_scale : c.k_scale);
    sc = cvt_e4m3x2(__fdiv_rn(__uint_as_float(mx << 16), __fmul_rn(6.0f, st)), 0.0f) & 0xFFu;
    const float unit = __fmul_rn(e4m3x2_to_float2(sc).x, st);
#pragma unroll
    for (int e = 0; e < 4; e++) {
      y[2 * e] = unit > 0.0f ? __fdiv_rn(bf_lo(xs[e]), unit) : 0.0f;
      y[2 * e + 1] = unit > 0.0f ? __fdiv_rn(bf_hi(xs[e]), unit) : 0.0f;
    }
    if (bad) sc = 0x7Fu;
  }
  uint8_t* codes = is_v ? c.v : c.k;
  uint8_t* sf = is_v ? c.v_sf : c.k_sf;
  reinterpret_cast<uint32_t*>(codes + at * 64)[lane] = bad ? 0u : pack8_e2m1(y);
  if (FMT == 0) {
    if ((lane & 3) == 0) sf[at * 4 + (lane >> 2)] = uint8_t(sc);
  } else {
    if ((lane & 1) == 0) sf[at * 8 + (lane >> 1)] = uint8_t(sc);
  }
}

}  // namespace mxfa
