// The 4-bit cache: how a page lies in memory and the conversions of its numbers.
//
// A unit is the K or the V of one page and head: codes [d/32][page_size][16] (byte y of chunk c: channels 32 c + 2 y in
// its low and 32 c + 2 y + 1 in its high four bits), behind them the scales [page_size][d/16].  The two units of a page
// and head (K, V) lie side by side, so that a page of a head is one contiguous copy; chunks stand apart so that lanes
// that read neighbouring tokens meet no bank twice.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/msa.h"

namespace msa {

// Bytes of a token in a unit.
template <int D>
constexpr int kv4_unit() {
  return D / 2 + D / 16;
}

msa_status check_kv4_pages(const msa_kv4_pages* p);  // geometry, address, scales
inline float kv4_scale(float s) { return s == 0.f ? 1.f : s; }

// ---------------------------------------------------------------- conversions (all exact or rounded to nearest even)
__device__ __forceinline__ uint32_t e4m3_of(float x) {  // saturates
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
  return r & 0xFFu;
}
// Two e4m3 numbers as fp16
__device__ __forceinline__ uint32_t f16x2_of_e4m3x2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
  return r;
}
__device__ __forceinline__ float e4m3_value(uint32_t one) {
  float f;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, l;\n\t}" : "=f"(f) : "r"(f16x2_of_e4m3x2(one)));
  return f;
}
__device__ __forceinline__ uint32_t e2m1x2_of(float lo, float hi) {  // saturates
  uint32_t r;
  asm("{\n\t.reg .b8 c, z;\n\tcvt.rn.satfinite.e2m1x2.f32 c, %2, %1;\n\tcvt.u32.u8 %0, c;\n\t}" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}
// Eight numbers as codes, the first in the lowest four bits (saturates)
__device__ __forceinline__ uint32_t e2m1x8_of(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}
// Eight codes as fp16 pairs, times `scale` (twice the same fp16): exact, a product has 6 bits
__device__ __forceinline__ void f16_of_codes(uint32_t codes, uint32_t scale, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t.reg .b32 w, x, y, z;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 w, a;\n\tcvt.rn.f16x2.e2m1x2 x, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 y, c;\n\tcvt.rn.f16x2.e2m1x2 z, d;\n\t"
      "mul.rn.f16x2 %0, w, %5;\n\tmul.rn.f16x2 %1, x, %5;\n\t"
      "mul.rn.f16x2 %2, y, %5;\n\tmul.rn.f16x2 %3, z, %5;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(codes), "r"(scale));
}

}  // namespace msa
