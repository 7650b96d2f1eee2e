// Rotary positions: the angles and the rotation, shared by every kernel that
// rotates rows, so that one row rotated by any of them gives the same bits.
//
// A row of head_dim columns at position p is rotated in its first r ("part of
// the head"): pair i of r / 2 by the angle p w_i, times a magnitude m,
//   (a, b) -> m (a cos - b sin, b cos + a sin),
// with pairs (i, i + r / 2), or (2 i, 2 i + 1) where they are interleaved.
//
// A frequency w_i is held as its fraction of a turn, w_i / 2 pi * 2^64 in 64
// bits: the product with the position wraps at a whole turn by itself, so a far
// position's angle is as exact as a near one's (a 32-bit float product at
// position 10^5 is off by 0.004) and no table of cosines is read.
//
// The unit of work is an item: 16 columns of one row that hold 8 pairs (i = 8 j
// .. 8 j + 7 for item j < r / 16), or 16 columns that pass through.
#pragma once

#include <cstdint>
#include <type_traits>

#include "device_common.cuh"
#include "pagedattn.h"
#include "status.h"

namespace pa {
namespace rot {

struct Args {
  const int64_t* freqs;  // [dim / 2], turns * 2^64 per position
  int dim;               // columns rotated, a multiple of 16
  int interleaved;
  float magnitude;
};

// Cosine and sine of the angle position * freq, times m.
//
// The nearest quarter turn comes off in integers; what is left, at most an
// eighth of a turn, goes to 32 bits in three roundings (the integer, 2 pi's
// constant, their product), and the Taylor series of both end below half a step
// there: a^11 / 11! and a^12 / 12! for a <= pi / 4 are 2e-9 a and 2e-10.
__device__ __forceinline__ float2 cos_sin(int position, int64_t freq, float m) {
  const uint64_t turn = uint64_t(int64_t(position)) * uint64_t(freq);
  const uint32_t quarter = uint32_t((turn + (uint64_t(1) << 61)) >> 62);  // 0 .. 3
  const int64_t rest = int64_t(turn - (uint64_t(quarter) << 62));
  const float a = __fmul_rn(__ll2float_rn(rest), 3.406121580e-19f);  // 2 pi / 2^64
  const float z = __fmul_rn(a, a);
  float s = fmaf(z, 1.f / 362880, -1.f / 5040);
  s = fmaf(z, s, 1.f / 120);
  s = fmaf(z, s, -1.f / 6);
  s = fmaf(__fmul_rn(z, a), s, a);
  float c = fmaf(z, -1.f / 3628800, 1.f / 40320);
  c = fmaf(z, c, -1.f / 720);
  c = fmaf(z, c, 1.f / 24);
  c = fmaf(z, c, -0.5f);
  c = fmaf(z, c, 1.f);
  const bool odd = quarter & 1;
  float cq = odd ? s : c, sq = odd ? c : s;
  if (quarter == 1 || quarter == 2) cq = -cq;
  if (quarter >= 2) sq = -sq;
  return make_float2(__fmul_rn(cq, m), __fmul_rn(sq, m));
}

// One pair.  (The products are spelt out: every kernel rounds alike.)
__device__ __forceinline__ void turn_pair(float& a, float& b, float c, float s) {
  const float x = fmaf(a, c, -__fmul_rn(b, s));
  b = fmaf(b, c, __fmul_rn(a, s));
  a = x;
}

// Two products, or two products added to, in one instruction each (sm_100 on).
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mov.b64 w, {%6, %7};\n\tfma.rn.f32x2 z, x, y, w;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

// Two neighbouring pairs of a half layout: turn_pair of each, bit for bit.
__device__ __forceinline__ void turn_two(float* a, float* b, const float* c, const float* s) {
  const float2 x = make_float2(a[0], a[1]), y = make_float2(b[0], b[1]);
  const float2 cc = make_float2(c[0], c[1]), ss = make_float2(s[0], s[1]);
  const float2 u = fma2(x, cc, mul2(y, make_float2(-s[0], -s[1])));
  const float2 v = fma2(y, cc, mul2(x, ss));
  a[0] = u.x;
  a[1] = u.y;
  b[0] = v.x;
  b[1] = v.y;
}

// A warp's angles.  With NJ = D / 16 items a row, lane l keeps the 2 or 1 pairs
// 8 j + q * kPer .. of item j = l % NJ, q = l / NJ (two cosines a lane at
// head_dim 128, each computed once in the warp); gather(j) collects an item's 8.
template <int D>
struct WarpAngles {
  static constexpr int NJ = D / 16;
  static constexpr int kPer = D / 64;
  float2 cs[kPer];

  static __device__ __forceinline__ int pair_of(int lane, int e) {
    return 8 * (lane % NJ) + (lane / NJ) * kPer + e;
  }
  // this lane's frequencies (0 past the rotated columns: an angle of zero)
  static __device__ __forceinline__ void load_freqs(const Args& r, int lane, int64_t (&f)[kPer]) {
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int i = pair_of(lane, e);
      f[e] = i < r.dim / 2 ? r.freqs[i] : 0;
    }
  }
  __device__ __forceinline__ void set(const int64_t (&f)[kPer], int position, float m) {
#pragma unroll
    for (int e = 0; e < kPer; ++e) cs[e] = cos_sin(position, f[e], m);
  }
  // c, s of the pairs of item j (any j of this warp; all lanes take part)
  __device__ __forceinline__ void gather(int j, float (&c)[8], float (&s)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int from = (i / kPer) * NJ + j;
      c[i] = __shfl_sync(0xffffffffu, cs[i % kPer].x, from);
      s[i] = __shfl_sync(0xffffffffu, cs[i % kPer].y, from);
    }
  }
};

// A warp's angles in shared memory, an item's 8 pairs as 4 pieces of 16 bytes
// (two cosines, two sines), items side by side.
template <int D>
struct AngleTable {
  float4 cs[4][D / 16];
  // by all lanes of the warp that holds `a`
  __device__ __forceinline__ void put(const WarpAngles<D>& a, int lane) {
    const int j = lane % (D / 16), q = lane / (D / 16);
    if constexpr (D == 128) {
      cs[q][j] = make_float4(a.cs[0].x, a.cs[1].x, a.cs[0].y, a.cs[1].y);
    } else {
      float* to = reinterpret_cast<float*>(&cs[q >> 1][j]) + (q & 1);
      to[0] = a.cs[0].x;
      to[2] = a.cs[0].y;
    }
  }
  __device__ __forceinline__ void get(int j, float (&c)[8], float (&s)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 x = cs[i][j];
      c[2 * i] = x.x;
      c[2 * i + 1] = x.y;
      s[2 * i] = x.z;
      s[2 * i + 1] = x.w;
    }
  }
};

// Where an item's two 8-column chunks begin (its first and second half).
__device__ __forceinline__ int2 item_columns(const Args& r, int j) {
  if (!r.interleaved && 16 * j < r.dim) return make_int2(8 * j, 8 * j + r.dim / 2);
  return make_int2(16 * j, 16 * j + 8);
}

// An item's 16 values in 32 bits: x[0 .. 7] the first chunk's, x[8 .. 15] the
// second's, rotated in place.
__device__ __forceinline__ void turn_item(bool interleaved, float (&x)[16], const float (&c)[8],
                                          const float (&s)[8]) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn_pair(x[2 * i], x[2 * i + 1], c[i], s[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; i += 2) turn_two(x + i, x + 8 + i, c + i, s + i);
  }
}

// 32 bytes at once (sm_100 on): whole sectors, half the requests.
__device__ __forceinline__ void load32(const void* p, uint4& a, uint4& b) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void store32(void* p, const uint4& a, const uint4& b) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z),
               "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

// Eight elements of a row as they lie in memory.
template <typename T>
struct Chunk {
  static constexpr int kVecs = sizeof(T) == 4 ? 2 : 1;
  uint4 v[kVecs];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) reinterpret_cast<uint4*>(p)[i] = v[i];
  }
  __device__ __forceinline__ void to_float(float* x) const {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(v);
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = dev::Mma<T>::unpack(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
      }
    }
  }
  __device__ __forceinline__ void from_float(const float* x) {
    uint32_t* w = reinterpret_cast<uint32_t*>(v);
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(x[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = dev::Mma<T>::pack(x[2 * i], x[2 * i + 1]);
    }
  }
};

// pa_rotary_kv_append's kernel on checked arguments (positions null:
// context_lens[token] - 1), for the entry points that append as a first launch
// (rotary.cu).
int append_rows(const void* q, const void* k, const void* v, const int32_t* positions,
                const int32_t* context_lens, const Args& rot, void* k_cache, void* v_cache,
                const int64_t* slot_mapping, int num_tokens, int num_q_heads, int num_kv_heads,
                int head_dim, int num_blocks, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                int64_t q_out_stride, int dtype, void* q_out, void* stream, const char* who);

// Host-side checks of a rotation's arguments.
inline int check_args(const int64_t* freqs, int rotary_dim, int interleaved, float magnitude,
                      int head_dim, const char* who, Args* out) {
  if (rotary_dim < 16 || rotary_dim > head_dim || rotary_dim % 16 != 0)
    return fail(PA_ERR_INVALID_ARG, "%s: rotary_dim %d (a multiple of 16, 16 .. head_dim %d)", who,
                rotary_dim, head_dim);
  if (interleaved != 0 && interleaved != 1)
    return fail(PA_ERR_INVALID_ARG, "%s: interleaved must be 0 or 1", who);
  if (!(magnitude - magnitude == 0.f))
    return fail(PA_ERR_INVALID_ARG, "%s: magnitude must be finite", who);
  if (!freqs) return fail(PA_ERR_INVALID_ARG, "%s: NULL pointer", who);
  if (reinterpret_cast<uintptr_t>(freqs) & 7)
    return fail(PA_ERR_INVALID_ARG, "%s: frequencies must be 8-byte aligned", who);
  out->freqs = freqs;
  out->dim = rotary_dim;
  out->interleaved = interleaved;
  out->magnitude = magnitude;
  return PA_OK;
}

// A row stride in elements: whole 16-byte vectors, not negative (0 repeats a
// row).  `own` > 0: rows of that many elements are written and must not meet.
inline int check_stride(int64_t stride, int elem_bytes, int64_t own, const char* name,
                        const char* who) {
  if (stride < 0 || stride >= (int64_t(1) << 40) || (stride * elem_bytes) % 16 != 0)
    return fail(PA_ERR_INVALID_ARG, "%s: %s %lld (whole 16-byte vectors, 0 .. 2^40 elements)", who, name,
                static_cast<long long>(stride));
  if (stride < own)
    return fail(PA_ERR_INVALID_ARG, "%s: %s %lld is less than a row's %lld elements", who, name,
                static_cast<long long>(stride), static_cast<long long>(own));
  return PA_OK;
}

}  // namespace rot
}  // namespace pa
