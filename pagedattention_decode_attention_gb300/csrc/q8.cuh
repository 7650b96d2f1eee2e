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
#include <type_traits>

#include <cuda_fp16.h>

#include "device_common.cuh"

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

// Eight consecutive elements of a row, as they lie in memory: a 16-bit type's
// stay packed between finding the largest and encoding (half the registers,
// twice the warps).
template <typename T>
struct Row8 {
  static constexpr uint32_t kInf = std::is_same<T, __half>::value ? 0x7C00u : 0x7F80u;
  uint4 v;
  __device__ __forceinline__ void load(const T* src) { v = *reinterpret_cast<const uint4*>(src); }
  // largest magnitude, in the type's bits; not `finite`: infinities and NaN
  // count too (they are above every finite one)
  __device__ __forceinline__ uint32_t top(bool finite) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t x = w[i] & 0x7FFF7FFFu;
      if (finite) {
        if ((x & 0xFFFFu) >= kInf) x &= 0xFFFF0000u;
        if ((x >> 16) >= kInf) x &= 0xFFFFu;
      }
      m = __vmaxu2(m, x);
    }
    return max(m & 0xFFFFu, m >> 16);
  }
  __device__ static __forceinline__ uint32_t float_bits(uint32_t top) {
    if constexpr (std::is_same<T, __half>::value)
      return __float_as_uint(__half2float(__ushort_as_half(uint16_t(top))));
    return top << 16;
  }
  __device__ __forceinline__ uint2 encode(float inv) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = dev::Mma<T>::unpack(w[i]);
      c[i] = encode2(f.x * inv, f.y * inv);
    }
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
  }
};

template <>
struct Row8<float> {
  static constexpr uint32_t kInf = 0x7F800000u;
  uint4 v[2];
  __device__ __forceinline__ void load(const float* src) {
    v[0] = reinterpret_cast<const uint4*>(src)[0];
    v[1] = reinterpret_cast<const uint4*>(src)[1];
  }
  __device__ __forceinline__ uint32_t top(bool finite) const {
    const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t x = w[i] & 0x7FFFFFFFu;
      if (!finite || x < kInf) m = max(m, x);
    }
    return m;
  }
  __device__ static __forceinline__ uint32_t float_bits(uint32_t top) { return top; }
  __device__ __forceinline__ uint2 encode(float inv) const {
    const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c[i] = encode2(__uint_as_float(w[2 * i]) * inv, __uint_as_float(w[2 * i + 1]) * inv);
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
  }
};

// Eight codes times `factor`, as codes again.
__device__ __forceinline__ uint2 rescale8(uint2 c, float factor) {
  uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 a = decode2_float(uint16_t(w[i] & 0xffff)), b = decode2_float(uint16_t(w[i] >> 16));
    w[i] = uint32_t(encode2(a.x * factor, a.y * factor)) |
           uint32_t(encode2(b.x * factor, b.y * factor)) << 16;
  }
  return make_uint2(w[0], w[1]);
}

}  // namespace q8
}  // namespace pa
