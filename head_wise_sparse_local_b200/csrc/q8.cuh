// Device helpers of the paged 8-bit cache.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "q8.h"

namespace rtp {

constexpr float kQ8ScaleMin = 5.42101086242752217e-20f;  // 2^-64, the smallest block scale

// Four e4m3 values (low byte first) as two fp16 pairs, exactly.
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t four, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi) : "r"(four));
}

// Nearest e4m3 values (ties to even) of two floats, lo in the low byte.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// The largest of three numbers; a NaN wins.
__device__ __forceinline__ float max3_nan(float x, float y, float z) {
  float m;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(x), "f"(y), "f"(z));
  return m;
}

// Least power of two s >= 2^-64 with a <= 448 s, for finite a >= 0.  448 is
// 1.75 * 2^8: with a = m 2^e, s is 2^(e-8) where m <= 1.75 and 2^(e-7) above.
__device__ __forceinline__ float q8_scale(float a) {
  const uint32_t u = __float_as_uint(a);
  int e = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = max(e, 127 - 64);
  return __uint_as_float((uint32_t)e << 23);
}

// 1 / s of a power of two 2^-64 <= s <= 2^121, exactly.
__device__ __forceinline__ float q8_inverse(float s) { return __uint_as_float((254u << 23) - __float_as_uint(s)); }

// cos and sin of a rotary angle from its frequency in turns (0.64 fixed
// point).  The product with the position wraps around modulo one turn, so no
// position is too far for the reduction; its upper 32 bits split into the
// nearest quarter turn and a rest within an eighth, whose sine and cosine are
// Taylor sums (to r^9 and r^10: off by less than 2^-26).  Off by 2^-23 at most.
__device__ __forceinline__ void rope_turns(int pos, uint64_t turns, float& c, float& s) {
  const uint32_t lo = (uint32_t)turns, p = (uint32_t)pos;
  const uint32_t f = __umulhi(p, lo) + p * (uint32_t)(turns >> 32) - (pos < 0 ? lo : 0u);
  const uint32_t q = (f + 0x20000000u) >> 30;                                  // quarter turns
  const float r = (float)(int)(f - (q << 30)) * 1.4629180792671596e-09f;      // the rest, 2 pi / 2^32
  const float x = r * r;
  float sn = fmaf(x, 2.7557319e-06f, -1.9841270e-04f);
  sn = fmaf(sn, x, 8.3333333e-03f);
  sn = fmaf(sn, x, -1.6666667e-01f);
  sn = fmaf(sn * x, r, r);
  float cs = fmaf(x, -2.7557319e-07f, 2.4801587e-05f);
  cs = fmaf(cs, x, -1.3888889e-03f);
  cs = fmaf(cs, x, 4.1666667e-02f);
  cs = fmaf(cs, x, -0.5f);
  cs = fmaf(cs, x, 1.f);
  const float u = q & 1u ? sn : cs, v = q & 1u ? cs : sn;
  c = __uint_as_float(__float_as_uint(u) ^ (((q + 1u) & 2u) << 30));  // cos: minus in quarters 1 and 2
  s = __uint_as_float(__float_as_uint(v) ^ ((q & 2u) << 30));       // sin: minus in quarters 2 and 3
}

}  // namespace rtp
