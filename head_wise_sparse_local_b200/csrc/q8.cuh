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

// An element of a table among a kernel's parameters, by an ordinary load: lanes
// that index the constant bank apart are served one after another, and each of
// its lines misses at a kernel's start.
__device__ __forceinline__ uint64_t table_at(const uint64_t* t, int k) {
  uint64_t x;
  asm volatile("ld.u64 %0, [%1];" : "=l"(x) : "l"(t + k));
  return x;
}
__device__ __forceinline__ int table_at(const unsigned char* t, int k) {
  uint32_t x;
  asm volatile("ld.u8 %0, [%1];" : "=r"(x) : "l"(t + k));
  return (int)x;
}

// cos and sin of a rotary angle from its frequency in turns (0.64 fixed
// point): the product with the position wraps around modulo one turn, so no
// position is too far for the reduction, and what is left goes to fp32 once.
__device__ __forceinline__ void rope_turns(int pos, uint64_t turns, float& c, float& s) {
  const long long frac = (long long)((uint64_t)(long long)pos * turns);  // [-1/2, 1/2) turn, times 2^64
  sincospif(__ll2float_rn(frac) * 1.0842021724855044e-19f, &s, &c);     // half turns: 2^-63
}

}  // namespace rtp
