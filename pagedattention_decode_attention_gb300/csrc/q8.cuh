// The 8-bit cache's number format, shared by the kernels that write and read
// it: e4m3 codes with one scale per (block, KV head), K and V apart.
//
// A scale is a power of two.  A floating code keeps its relative precision
// whatever the scale, so rounding the scale up to a power of two costs at most
// one binade of the code's range and nothing of its precision; in return
// dividing by it is exact, and when a block's scale grows the codes it holds
// only move their exponents (they lose what falls under e4m3's smallest
// step, nothing else).
#pragma once

#include <cstdint>

#include <cuda_fp16.h>

namespace pa {
namespace q8 {

constexpr float kCodeMax = 448.f;           // largest finite e4m3 value, 1.75 * 2^8
constexpr int kExpMin = -100, kExpMax = 120;  // exponents a scale may have

// Smallest e in [kExpMin, kExpMax] with peak <= 448 * 2^e, for a finite
// peak >= 0: peak = 1.m * 2^x needs e = x - 8 while 1.m <= 1.75, else one more.
__host__ __device__ __forceinline__ int scale_exponent(uint32_t peak_bits) {
  const int x = int(peak_bits >> 23) - 127;
  const int e = (peak_bits & 0x7FFFFFu) <= 0x600000u ? x - 8 : x - 7;
  return e < kExpMin ? kExpMin : (e > kExpMax ? kExpMax : e);
}

__host__ __device__ __forceinline__ uint32_t pow2_bits(int e) { return uint32_t(e + 127) << 23; }

// Two e4m3 codes (byte 0, byte 1) as two halves (exact).
__device__ __forceinline__ uint32_t decode2(uint16_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(codes));
  return h;
}

__device__ __forceinline__ float2 decode2_float(uint16_t codes) {
  const uint32_t h = decode2(codes);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// lo, hi to two e4m3 codes (byte 0, byte 1), to nearest even; beyond +-448
// saturates, NaN stays NaN.
__device__ __forceinline__ uint16_t encode2(float lo, float hi) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(hi), "f"(lo));
  return c;
}

}  // namespace q8
}  // namespace pa
