// The 8-bit paged cache: kv_append_q8 (new tokens quantised into their blocks),
// rotary_kv_append_q8 (the same with queries and keys rotated on the way) and
// block_dequantize (whole blocks read back as 16- or 32-bit values).
//
// Format (q8.cuh): k_cache, v_cache hold e4m3 codes [num_blocks][num_kv_heads]
// [16][head_dim]; k_scale, v_scale one fp32 power of two per (block, KV head).
// A token's value is code * scale.  The tokens of one block share a scale
// because a block is what the pool moves and what attention reads: the scale
// travels with the 16 rows it belongs to and costs 4 bytes per 16 * head_dim.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "device_common.cuh"
#include "pagedattn.h"
#include "q8.cuh"
#include "rotary.cuh"
#include "status.h"
#include "trace.h"

namespace pa {
namespace q8 {
namespace {

constexpr int kBlockSize = 16;
constexpr int kAppendWarps = 8;

struct AppendParams {
  const void* src[2];   // k, v: [num_tokens][num_kv_heads][head_dim]
  uint8_t* cache[2];
  float* scale[2];
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* query_start;
  int num_seqs, num_tokens, num_kv_heads, max_blocks, num_blocks;
  unsigned* status;
};

// One (unit, KV head, K or V), by a warp: it alone reads and writes that
// scale, holds the new rows in registers between finding their largest
// magnitude and encoding them, and rescales the older rows of the block when
// the scale grows.
template <typename T, int D>
__device__ __forceinline__ void append_block(const AppendParams& p, const int4 seq, int unit, int head, int kv,
                                             int lane) {
  constexpr int kLanes = D / 8;             // lanes per row, eight elements each
  constexpr int kRows = 32 / kLanes;        // rows per pass
  constexpr int kPasses = kBlockSize / kRows;
  const int b = seq.x, q0 = seq.y, q1 = seq.z, ctx = seq.w;
  const int begin = ctx - (q1 - q0);        // first new token's position
  const int blk = begin / kBlockSize + (unit - (q0 / kBlockSize + 2 * b));
  const int lo = max(begin - blk * kBlockSize, 0);                 // rows lo .. hi - 1 are new
  const int hi = min(ctx - blk * kBlockSize, kBlockSize);
  const int row0 = lane / kLanes, col = (lane % kLanes) * 8;
  // the new rows (on their way while the table entry is), and the largest
  // finite magnitude among them
  Row8<T> x[kPasses];
  // (row 0 of the block, which lies before the tokens when lo > 0)
  const T* src = static_cast<const T*>(kv ? p.src[1] : p.src[0]) +
                 ((int64_t(q0) + blk * kBlockSize - begin) * p.num_kv_heads + head) * D + col;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int r = i * kRows + row0;
    if (r >= lo && r < hi) x[i].load(src + int64_t(r) * p.num_kv_heads * D);
  }
  const int phys = p.block_tables[size_t(b) * p.max_blocks + blk];
  if (phys < 0 || phys >= p.num_blocks) {
    if (lane == 0) dev::flag_status(p.status, kStatusBounds);
    return;
  }
  const size_t tile = size_t(phys) * p.num_kv_heads + head;
  float* scale_at = (kv ? p.scale[1] : p.scale[0]) + tile;
  const float old = lo > 0 ? *scale_at : 0.f;
  auto largest = [&](bool finite) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int r = i * kRows + row0;
      if (r >= lo && r < hi) m = max(m, x[i].top(finite));
    }
    return __reduce_max_sync(0xffffffffu, m);
  };
  uint32_t top = largest(false);
  if (top >= Row8<T>::kInf) top = largest(true);
  top = Row8<T>::float_bits(top);
  const float want = __uint_as_float(pow2_bits(scale_exponent(top)));
  const float scale = lo > 0 ? fmaxf(old, want) : want;
  const float inv = 1.f / scale;            // exact for a power of two, rounded for a scale of the caller's
  uint8_t* codes = (kv ? p.cache[1] : p.cache[0]) + tile * kBlockSize * D + col;
  if (lo > 0 && scale > old) {
    // older rows of the block: the same values under the larger scale
    const float factor = old / scale;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int r = i * kRows + row0;
      if (r < lo) {
        uint2* at = reinterpret_cast<uint2*>(codes + r * D);
        *at = rescale8(*at, factor);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int r = i * kRows + row0;
    if (r >= lo && r < hi) *reinterpret_cast<uint2*>(codes + r * D) = x[i].encode(inv);
  }
  if (lane == 0 && (lo == 0 || scale > old)) *scale_at = scale;
}

__device__ __forceinline__ bool invalid(const AppendParams& p, int q0, int q1, int ctx) {
  return q0 < 0 || q1 < q0 || q1 > p.num_tokens || q1 - q0 > ctx || ctx > p.max_blocks * kBlockSize;
}

// Whether `unit` is one of sequence b's blocks.
__device__ __forceinline__ bool owns(const AppendParams& p, int unit, int b, int q0, int q1, int ctx) {
  if (q1 == q0 || invalid(p, q0, q1, ctx)) return false;
  const int nth = unit - (q0 / kBlockSize + 2 * b);
  return nth >= 0 && nth <= (ctx - 1) / kBlockSize - (ctx - (q1 - q0)) / kBlockSize;
}

// A unit of several sequences (see append_kernel): each one's in turn, row by
// row from memory (the path that a call in order takes keeps its registers).
template <typename T, int D>
__device__ __forceinline__ void append_in_turn(const AppendParams& p, int unit, int head, int kv, int lane) {
#pragma unroll 1
  for (int b = 0; b < p.num_seqs; ++b) {
    const int q0 = p.query_start[b], q1 = p.query_start[b + 1], ctx = p.context_lens[b];
    if (!owns(p, unit, b, q0, q1, ctx)) continue;
    const int begin = ctx - (q1 - q0);
    const int blk = begin / kBlockSize + (unit - (q0 / kBlockSize + 2 * b));
    const int lo = max(begin - blk * kBlockSize, 0), hi = min(ctx - blk * kBlockSize, kBlockSize);
    const int phys = p.block_tables[size_t(b) * p.max_blocks + blk];
    if (phys < 0 || phys >= p.num_blocks) {
      if (lane == 0) dev::flag_status(p.status, kStatusBounds);
      continue;
    }
    const size_t tile = size_t(phys) * p.num_kv_heads + head;
    float* scale_at = (kv ? p.scale[1] : p.scale[0]) + tile;
    const bool live = lane < D / 8;
    const T* src = static_cast<const T*>(kv ? p.src[1] : p.src[0]) +
                   ((int64_t(q0) + blk * kBlockSize - begin) * p.num_kv_heads + head) * D + 8 * lane;
    uint8_t* codes = (kv ? p.cache[1] : p.cache[0]) + tile * kBlockSize * D + 8 * lane;
    uint32_t top = 0;
#pragma unroll 1
    for (int r = lo; r < hi && live; ++r) {
      Row8<T> x;
      x.load(src + int64_t(r) * p.num_kv_heads * D);
      top = max(top, x.top(true));
    }
    top = Row8<T>::float_bits(__reduce_max_sync(0xffffffffu, top));
    const float want = __uint_as_float(pow2_bits(scale_exponent(top)));
    const float old = lo > 0 ? *scale_at : 0.f;
    const float scale = fmaxf(old, want);
    __syncwarp();
#pragma unroll 1
    for (int r = scale > old ? 0 : lo; r < hi && live; ++r) {
      uint2* at = reinterpret_cast<uint2*>(codes + r * D);
      if (r < lo) {
        *at = rescale8(*at, old / scale);
      } else {
        Row8<T> x;
        x.load(src + int64_t(r) * p.num_kv_heads * D);
        *at = x.encode(1.f / scale);
      }
    }
    if (lane == 0 && (lo == 0 || scale > old)) *scale_at = scale;
  }
}

// A unit is one (sequence, block the call writes to); blockIdx.x numbers them
// with gaps: sequence b's begin at query_start[b] / 16 + 2 b, so the next one's
// begin at least T / 16 + 2 later, and T new tokens touch at most (T + 14) / 16
// + 1 <= T / 16 + 2 blocks: two sequences' units do not meet.  A warp owns one
// (unit, KV head, K or V).  Bound by bytes (2 head_dim elements read and as many
// codes written per token and head): 13.6 K tokens of 8 heads, 84 MB, 14.4 us
// (fp32 rows, 139 MB: 24.4); for a decode step by latency (query_start, then
// table entry and rows together, then the scale).
template <typename T, int D>
__global__ void __launch_bounds__(kAppendWarps * 32, sizeof(T) == 4 ? 2 : 4)
    append_kernel(const AppendParams p) {
  dev::grid_launch_dependents();
  dev::grid_dependency_wait();
  // the unit's sequence.  With query_start in order there is one at most; a
  // sequence that runs backwards (skipped) may be followed by one that begins
  // among the units of an earlier one, and then a unit is each one's in turn.
  __shared__ int4 s_seq;  // it, its first and last query row, its length
  __shared__ int s_hits;
  const int unit = blockIdx.x;
  if (threadIdx.x == 0) s_hits = 0;
  __syncthreads();
  for (int b = threadIdx.x; b < p.num_seqs; b += kAppendWarps * 32) {
    const int q0 = p.query_start[b], q1 = p.query_start[b + 1], ctx = p.context_lens[b];
    if (owns(p, unit, b, q0, q1, ctx)) {
      s_seq = make_int4(b, q0, q1, ctx);
      atomicAdd(&s_hits, 1);
    }
    if (unit == 0 && blockIdx.y == 0 && invalid(p, q0, q1, ctx)) dev::flag_status(p.status, kStatusBounds);
  }
  __syncthreads();
  const int job = blockIdx.y * kAppendWarps + (threadIdx.x >> 5);
  if (job >= 2 * p.num_kv_heads) return;
  const int kv = job & 1, head = job >> 1, lane = threadIdx.x & 31;
  if (s_hits == 1) {
    append_block<T, D>(p, s_seq, unit, head, kv, lane);
  } else if (s_hits > 1) {
    append_in_turn<T, D>(p, unit, head, kv, lane);
  }
}

// ------------------------------------------------- rotated on the way
struct RotaryAppendParams {
  AppendParams a;       // src: k, v
  const void* q;
  void* q_out;
  int64_t stride[3], q_out_stride;  // elements between rows of k, v, q; of q_out
  int num_q_heads;
  const int32_t* positions;         // null: a token's place in its sequence
  rot::Args rot;
};

// The cosines and sines of a unit's rows, an item's 8 pairs as 4 pieces of 16
// bytes (two cosines, two sines), items side by side: the lanes of a row read
// without bank conflicts.
template <int D>
struct UnitAngles {
  float4 cs[kBlockSize][4][D / 16];
  __device__ __forceinline__ void put(int row, int pair, float2 x) {
    float* to = reinterpret_cast<float*>(&cs[row][(pair & 7) >> 1][pair >> 3]) + (pair & 1);
    to[0] = x.x;
    to[2] = x.y;
  }
  __device__ __forceinline__ void get(int row, int j, float (&c)[8], float (&s)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 x = cs[row][i][j];
      c[2 * i] = x.x;
      c[2 * i + 1] = x.y;
      s[2 * i] = x.z;
      s[2 * i + 1] = x.w;
    }
  }
};

// What a warp knows of its unit.
struct Unit {
  int lo, hi;      // rows of the block that are new
  int64_t first;   // the query row that row 0 of the block would be
  int phys;        // -1: not a block
};

// The new rows of one (unit, head of Q, K or V) as they lie in memory: a lane has item lane % NJ of rows lane / NJ, + 32 / NJ, ....
template <typename T, int D>
struct UnitRows {
  static constexpr int NJ = D / 16, kRows = 32 / NJ, kPasses = kBlockSize / kRows;
  rot::Chunk<T> u[kPasses], w[kPasses];
  float old;  // K, V: the block's scale
  int kv, head;
  int2 at;

  __device__ __forceinline__ void load(const RotaryAppendParams& p, const Unit& n, int job, int lane) {
    kv = job < 2 * p.a.num_kv_heads ? job & 1 : 2;  // K, V, Q
    head = kv < 2 ? job >> 1 : job - 2 * p.a.num_kv_heads;
    const int j = lane % NJ, row0 = lane / NJ;
    at = kv != 1 ? rot::item_columns(p.rot, j) : make_int2(16 * j, 16 * j + 8);
    const T* from = static_cast<const T*>(kv == 2 ? p.q : kv ? p.a.src[1] : p.a.src[0]) +
                    (n.first + row0) * p.stride[kv] + head * D;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int r = i * kRows + row0;
      if (r >= n.lo && r < n.hi) {
        u[i].load(from + at.x);
        w[i].load(from + at.y);
      }
      from += kRows * p.stride[kv];
    }
    old = 0.f;
    if (kv < 2 && n.lo > 0 && n.phys >= 0)
      old = (kv ? p.a.scale[1] : p.a.scale[0])[size_t(n.phys) * p.a.num_kv_heads + head];
  }

  // Pass i's values, rotated (V: as they are).
  template <bool INTER>
  __device__ __forceinline__ void values(const RotaryAppendParams& p, const UnitAngles<D>& angles, int lane, int i,
                                         float (&x)[16]) const {
    u[i].to_float(x);
    w[i].to_float(x + 8);
    if (kv != 1 && 16 * (lane % NJ) < p.rot.dim) {
      float c[8], s[8];
      angles.get(i * kRows + lane / NJ, lane % NJ, c, s);
      rot::turn_item(INTER, x, c, s);
    }
  }
};

// The largest finite magnitude.
__device__ __forceinline__ float largest_of(const float (&x)[16]) {
  float m = 0.f;  // (NaN is passed over)
#pragma unroll
  for (int e = 0; e < 16; ++e) m = fmaxf(m, fabsf(x[e]));
  if (m == INFINITY) {
    m = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) m = fabsf(x[e]) < INFINITY ? fmaxf(m, fabsf(x[e])) : m;
  }
  return m;
}

// Rotates and stores what was loaded.  K and V are quantised from 32 bits: a
// rotated key is rounded once, to its code.  (Keys are rotated twice, for the
// block's largest magnitude and for the codes: keeping the 32 or 64 values takes
// a third of the warps, 46.1 us and 42.9 for 9900 tokens of 32 heads of 64.)
template <typename T, int D, bool INTER>
__device__ __forceinline__ void store_unit(const RotaryAppendParams& p, const Unit& n, int lane,
                                           const UnitRows<T, D>& rows, const UnitAngles<D>& angles) {
  using U = UnitRows<T, D>;
  const int kv = rows.kv, row0 = lane / U::NJ;
  const int2 at = rows.at;
  if (kv == 2) {
    T* to = static_cast<T*>(p.q_out) + (n.first + row0) * p.q_out_stride + rows.head * D;
#pragma unroll
    for (int i = 0; i < U::kPasses; ++i) {
      const int r = i * U::kRows + row0;
      if (r >= n.lo && r < n.hi) {
        float x[16];
        rows.template values<INTER>(p, angles, lane, i, x);
        rot::Chunk<T> u, w;
        u.from_float(x);
        w.from_float(x + 8);
        u.store(to + at.x);
        w.store(to + at.y);
      }
      to += U::kRows * p.q_out_stride;
    }
    return;
  }
  if (n.phys < 0) return;
  // the largest finite magnitude (16-bit values by their bits, two at once)
  uint32_t top = 0;
  bool packed = false;
  if constexpr (sizeof(T) == 2) {
    if (kv == 1) {
      uint32_t w = 0;
#pragma unroll
      for (int i = 0; i < U::kPasses; ++i) {
        const int r = i * U::kRows + row0;
        if (r < n.lo || r >= n.hi) continue;
        for (const uint4& v : {rows.u[i].v[0], rows.w[i].v[0]})
          w = __vmaxu2(w, __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                   __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
      }
      top = __reduce_max_sync(0xffffffffu, max(w & 0xFFFFu, w >> 16));
      packed = top < Row8<T>::kInf;
      top = Row8<T>::float_bits(top);
    }
  }
  if (!packed) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < U::kPasses; ++i) {
      const int r = i * U::kRows + row0;
      if (r < n.lo || r >= n.hi) continue;
      float x[16];
      rows.template values<INTER>(p, angles, lane, i, x);
      m = fmaxf(m, largest_of(x));
    }
    top = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
  }
  const float want = __uint_as_float(pow2_bits(scale_exponent(top)));
  const float scale = n.lo > 0 ? fmaxf(rows.old, want) : want;
  const float inv = 1.f / scale;
  const size_t tile = size_t(n.phys) * p.a.num_kv_heads + rows.head;
  uint8_t* codes = (kv ? p.a.cache[1] : p.a.cache[0]) + (tile * kBlockSize + row0) * D;
  if (n.lo > 0 && scale > rows.old) {
    // older rows of the block: the same values under the larger scale
    const float factor = rows.old / scale;
#pragma unroll 1
    for (int r = row0; r < n.lo; r += U::kRows) {
      uint2* a = reinterpret_cast<uint2*>(codes + (r - row0) * D + at.x);
      uint2* b = reinterpret_cast<uint2*>(codes + (r - row0) * D + at.y);
      *a = rescale8(*a, factor);
      *b = rescale8(*b, factor);
    }
  }
#pragma unroll
  for (int i = 0; i < U::kPasses; ++i) {
    const int r = i * U::kRows + row0;
    if (r < n.lo || r >= n.hi) continue;
    float x[16];
    rows.template values<INTER>(p, angles, lane, i, x);
    uint32_t c[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 y = rot::mul2(make_float2(x[2 * e], x[2 * e + 1]), make_float2(inv, inv));
      c[e] = encode2(y.x, y.y);
    }
    *reinterpret_cast<uint2*>(codes + i * U::kRows * D + at.x) = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
    *reinterpret_cast<uint2*>(codes + i * U::kRows * D + at.y) = make_uint2(c[4] | c[5] << 16, c[6] | c[7] << 16);
  }
  if (lane == 0 && (n.lo == 0 || scale > rows.old)) (kv ? p.a.scale[1] : p.a.scale[0])[tile] = scale;
}

// Units as append_kernel's; a warp takes every (8 gridDim.y)-th head of Q, K and V
// of its unit.  Bound by bytes and, nearly, by instructions (1.8 a cycle and SM;
// the angles are shared by a CTA, products go two to an instruction): 10.6 K
// tokens of 32/8 heads, 238 MB, 38.8 us, 0.91 of the copy rate; 10.6 K of 32/32
// heads of 64, 217 MB, 42.8 us, 0.75 (two thirds of its rows are quantised); 6 K
// fp32 rows of 32/8 heads, 259 MB, 42.7 us, 0.90.  Three CTAs an SM (head_dim 128;
// they spill 20 bytes a thread): two 48.5 us, four 53.6 (212 - 264 bytes).
template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kAppendWarps * 32, sizeof(T) == 4 ? 2 : D == 64 ? 4 : 3)
    rotary_append_kernel(const RotaryAppendParams p) {
  constexpr int kThreads = kAppendWarps * 32, kPairs = D / 2;
  dev::grid_launch_dependents();
  dev::grid_dependency_wait();
  __shared__ UnitAngles<D> angles;
  __shared__ int4 s_seq;
  __shared__ int s_hits;
  const int unit = blockIdx.x, lane = threadIdx.x & 31;
  // this thread's pair of every row it computes the angle of
  const int pair = threadIdx.x % kPairs;
  const int64_t freq = pair < p.rot.dim / 2 ? p.rot.freqs[pair] : 0;
  if (threadIdx.x == 0) s_hits = 0;
  __syncthreads();
  for (int b = threadIdx.x; b < p.a.num_seqs; b += kThreads) {
    const int q0 = p.a.query_start[b], q1 = p.a.query_start[b + 1], ctx = p.a.context_lens[b];
    if (owns(p.a, unit, b, q0, q1, ctx)) {
      s_seq = make_int4(b, q0, q1, ctx);
      atomicAdd(&s_hits, 1);
    }
    if (unit == 0 && blockIdx.y == 0 && invalid(p.a, q0, q1, ctx)) dev::flag_status(p.a.status, kStatusBounds);
  }
  __syncthreads();
  const int hits = s_hits;
  const int jobs = 2 * p.a.num_kv_heads + p.num_q_heads, step = gridDim.y * kAppendWarps;
  auto take = [&](const int4 seq) {
    const int begin = seq.w - (seq.z - seq.y);
    const int blk = begin / kBlockSize + (unit - (seq.y / kBlockSize + 2 * seq.x));
    Unit n;
    n.lo = max(begin - blk * kBlockSize, 0);
    n.hi = min(seq.w - blk * kBlockSize, kBlockSize);
    n.first = int64_t(seq.y) + blk * kBlockSize - begin;
    n.phys = p.a.block_tables[size_t(seq.x) * p.a.max_blocks + blk];
    if (n.phys < 0 || n.phys >= p.a.num_blocks) {
      if (threadIdx.x == 0 && blockIdx.y == 0) dev::flag_status(p.a.status, kStatusBounds);
      n.phys = -1;
    }
    int job = blockIdx.y * kAppendWarps + (threadIdx.x >> 5);
    UnitRows<T, D> rows;
    if (job < jobs) rows.load(p, n, job, lane);
    for (int r = n.lo + threadIdx.x / kPairs; r < n.hi; r += kThreads / kPairs) {
      const int position = p.positions ? p.positions[n.first + r] : blk * kBlockSize + r;
      angles.put(r, pair, rot::cos_sin(position, freq, p.rot.magnitude));
    }
    __syncthreads();
    while (job < jobs) {
      store_unit<T, D, INTER>(p, n, lane, rows, angles);
      job += step;
      if (job < jobs) rows.load(p, n, job, lane);
    }
  };
  if (hits == 1) {
    take(s_seq);
  } else if (hits > 1) {
    // a unit of several sequences: each one's in turn
    for (int b = 0; b < p.a.num_seqs; ++b) {
      const int q0 = p.a.query_start[b], q1 = p.a.query_start[b + 1], ctx = p.a.context_lens[b];
      if (!owns(p.a, unit, b, q0, q1, ctx)) continue;
      take(make_int4(b, q0, q1, ctx));
      __syncthreads();
    }
  }
}

// The same where sequences have a token or two on average (a decode step): a unit
// is (token, block the call writes to), unit query_start[b] + i the i-th block of
// sequence b; a CTA takes a unit, a warp 32 / NJ heads of Q, K or V and its rows in
// turn, an item a lane.  A chunk among single tokens pays for those turns: 255
// tokens and a chunk of 256 17.5 us in one call, 9.5 us in two.  A chain of
// latencies: the sequence, its row, table entry and position, the block's scale.
// 128 tokens of 48 heads: 2.6 us, 4.7 by blocks of 16 rows.  (With the registers of
// two CTAs an SM 3.3, though 512 tokens then take 6.6 and not 8.8.)
constexpr int kFewWarps = 16;

template <typename T, int D>
__global__ void __launch_bounds__(kFewWarps * 32) rotary_append_few_kernel(const RotaryAppendParams p) {
  constexpr int NJ = D / 16, kHeads = 32 / NJ;
  dev::grid_launch_dependents();
  __shared__ int4 s_seq;
  __shared__ int s_hits;
  const int unit = blockIdx.x, lane = threadIdx.x & 31, j = lane % NJ;
  if (threadIdx.x == 0) s_hits = 0;
  __syncthreads();
  dev::grid_dependency_wait();
  int64_t freqs[rot::WarpAngles<D>::kPer];
  rot::WarpAngles<D>::load_freqs(p.rot, lane, freqs);
  auto mine = [&](int b, int4& seq) {
    const int q0 = p.a.query_start[b], q1 = p.a.query_start[b + 1], ctx = p.a.context_lens[b];
    seq = make_int4(b, q0, q1, ctx);
    const bool bad = invalid(p.a, q0, q1, ctx);
    if (bad && unit == 0 && blockIdx.y == 0) dev::flag_status(p.a.status, kStatusBounds);
    if (bad || q1 == q0 || unit < q0) return false;
    return unit - q0 <= (ctx - 1) / kBlockSize - (ctx - (q1 - q0)) / kBlockSize;
  };
  for (int b = threadIdx.x; b < p.a.num_seqs; b += blockDim.x) {
    int4 seq;
    if (mine(b, seq)) {
      s_seq = seq;
      atomicAdd(&s_hits, 1);
    }
  }
  __syncthreads();
  // Q, K, V by groups of heads
  const int groups_q = (p.num_q_heads + kHeads - 1) / kHeads, groups_k = (p.a.num_kv_heads + kHeads - 1) / kHeads;
  int group = blockIdx.y * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (group >= groups_q + 2 * groups_k) return;
  const int kv = group < groups_q ? 2 : group < groups_q + groups_k ? 0 : 1;
  group -= kv == 2 ? 0 : kv == 0 ? groups_q : groups_q + groups_k;
  const int head = group * kHeads + lane / NJ;
  const bool live = head < (kv == 2 ? p.num_q_heads : p.a.num_kv_heads);
  const int2 at = kv != 1 ? rot::item_columns(p.rot, j) : make_int2(16 * j, 16 * j + 8);
  const T* src = static_cast<const T*>(kv == 2 ? p.q : kv ? p.a.src[1] : p.a.src[0]) + int64_t(head) * D;
  auto take = [&](const int4 seq) {
    const int begin = seq.w - (seq.z - seq.y);
    const int blk = begin / kBlockSize + unit - seq.y;
    const int lo = max(begin - blk * kBlockSize, 0), hi = min(seq.w - blk * kBlockSize, kBlockSize);
    const int64_t first = int64_t(seq.y) + blk * kBlockSize - begin;
    rot::Chunk<T> u, w;
    float x[16];
    auto load = [&](int r) {
      if (live) {
        u.load(src + (first + r) * p.stride[kv] + at.x);
        w.load(src + (first + r) * p.stride[kv] + at.y);
      }
    };
    auto values = [&](int r) {
      if (kv != 1) {
        const int position = p.positions ? p.positions[first + r] : blk * kBlockSize + r;
        rot::WarpAngles<D> angles;
        float c[8], s[8];
        angles.set(freqs, position, p.rot.magnitude);
        angles.gather(j, c, s);
        u.to_float(x);
        w.to_float(x + 8);
        if (16 * j < p.rot.dim) rot::turn_item(p.rot.interleaved, x, c, s);
      } else {
        u.to_float(x);
        w.to_float(x + 8);
      }
    };
    load(lo);
    int phys = 0;
    float old = 0.f;
    size_t tile = 0;
    if (kv != 2) {
      phys = p.a.block_tables[size_t(seq.x) * p.a.max_blocks + blk];
      if (phys < 0 || phys >= p.a.num_blocks) {
        if (lane == 0) dev::flag_status(p.a.status, kStatusBounds);
        return;
      }
      tile = size_t(phys) * p.a.num_kv_heads + head;
      if (lo > 0 && live) old = (kv ? p.a.scale[1] : p.a.scale[0])[tile];
    }
    float m = 0.f;
    for (int r = lo; r < hi; ++r) {
      if (r > lo) load(r);
      values(r);
      if (kv != 2) {
        m = fmaxf(m, largest_of(x));
      } else if (live) {
        T* to = static_cast<T*>(p.q_out) + (first + r) * p.q_out_stride + int64_t(head) * D;
        u.from_float(x);
        w.from_float(x + 8);
        u.store(to + at.x);
        w.store(to + at.y);
      }
    }
    if (kv == 2) return;
#pragma unroll
    for (int o = NJ / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float want = __uint_as_float(pow2_bits(scale_exponent(__float_as_uint(m))));
    const float scale = lo > 0 ? fmaxf(old, want) : want;
    const float inv = 1.f / scale;
    uint8_t* codes = (kv ? p.a.cache[1] : p.a.cache[0]) + tile * kBlockSize * D;
    const bool grows = live && lo > 0 && scale > old;
    if (grows) {
      const float factor = old / scale;
#pragma unroll 4
      for (int r = 0; r < lo; ++r) {
        uint2* a = reinterpret_cast<uint2*>(codes + r * D + at.x);
        uint2* b = reinterpret_cast<uint2*>(codes + r * D + at.y);
        *a = rescale8(*a, factor);
        *b = rescale8(*b, factor);
      }
    }
    for (int r = lo; r < hi; ++r) {
      if (hi - lo > 1) {
        load(r);
        values(r);
      }
      uint32_t c[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) c[e] = encode2(x[2 * e] * inv, x[2 * e + 1] * inv);
      if (!live) continue;
      *reinterpret_cast<uint2*>(codes + r * D + at.x) = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
      *reinterpret_cast<uint2*>(codes + r * D + at.y) = make_uint2(c[4] | c[5] << 16, c[6] | c[7] << 16);
    }
    if (live && j == 0 && (lo == 0 || grows)) (kv ? p.a.scale[1] : p.a.scale[0])[tile] = scale;
  };
  if (s_hits == 1) {
    take(s_seq);
  } else if (s_hits > 1) {
    // a unit of several sequences: each one's in turn
    for (int b = 0; b < p.a.num_seqs; ++b) {
      int4 seq;
      if (mine(b, seq)) take(seq);
      __syncwarp();
    }
  }
}

// Sixteen values as elements of the output's type: whole 32-byte sectors per
// store where the output is 32-byte aligned.
template <typename T>
__device__ __forceinline__ void store16(T* dst, const float (&x)[16], bool wide) {
  constexpr int kWords = sizeof(T) == 4 ? 16 : 8;
  uint32_t w[kWords];
#pragma unroll
  for (int i = 0; i < kWords; ++i) {
    if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(x[i]);
    else w[i] = dev::Mma<T>::pack(x[2 * i], x[2 * i + 1]);
  }
#pragma unroll
  for (int i = 0; i < kWords; i += 8) {
    uint32_t* at = reinterpret_cast<uint32_t*>(dst) + i;
    if (wide) {
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(w[i]),
                   "r"(w[i + 1]), "r"(w[i + 2]), "r"(w[i + 3]), "r"(w[i + 4]), "r"(w[i + 5]),
                   "r"(w[i + 6]), "r"(w[i + 7])
                   : "memory");
    } else {
      reinterpret_cast<uint4*>(at)[0] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
      reinterpret_cast<uint4*>(at)[1] = make_uint4(w[i + 4], w[i + 5], w[i + 6], w[i + 7]);
    }
  }
}

constexpr int kReadThreads = 256;
constexpr int kReadBatch = 4;  // 16-code chunks a thread has in flight

struct ReadParams {
  const uint8_t* cache[2];
  const float* scale[2];
  void* out[2];
  const int64_t* pairs;
  int num_blocks, num_out_blocks;
  int chunks;       // 16-code chunks of a block: num_kv_heads * head_dim
  int head_shift;   // chunk >> head_shift: its KV head
  int num_kv_heads;
  unsigned* status;
};

// Pair blockIdx.x, K or V blockIdx.y: a block's codes are contiguous, and a
// thread turns chunks of 16 into 16 elements.  Pure data movement: 872 blocks of
// 8 heads, 86 MB read and written, 13.0 us (to fp32, 143 MB: 22.1).
template <typename T>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const ReadParams p) {
  dev::grid_launch_dependents();
  dev::grid_dependency_wait();
  const int64_t src = p.pairs[2 * int64_t(blockIdx.x)], dst = p.pairs[2 * int64_t(blockIdx.x) + 1];
  if (src < 0 || src >= p.num_blocks || dst < 0 || dst >= p.num_out_blocks) {
    if (threadIdx.x == 0) dev::flag_status(p.status, kStatusBounds);
    return;
  }
  const int kv = blockIdx.y;
  const uint4* from = reinterpret_cast<const uint4*>((kv ? p.cache[1] : p.cache[0])) + src * p.chunks;
  const float* scale = (kv ? p.scale[1] : p.scale[0]) + src * p.num_kv_heads;
  T* to = static_cast<T*>((kv ? p.out[1] : p.out[0])) + dst * p.chunks * 16;
  const bool wide = (reinterpret_cast<uintptr_t>(to) & 31) == 0;
  for (int base = blockIdx.z * kReadThreads * kReadBatch; base < p.chunks;
       base += gridDim.z * kReadThreads * kReadBatch) {
    uint4 c[kReadBatch];
    float s[kReadBatch];
#pragma unroll
    for (int u = 0; u < kReadBatch; ++u) {
      const int i = base + u * kReadThreads + threadIdx.x;
      if (i < p.chunks) {
        c[u] = from[i];
        s[u] = scale[i >> p.head_shift];
      }
    }
#pragma unroll
    for (int u = 0; u < kReadBatch; ++u) {
      const int i = base + u * kReadThreads + threadIdx.x;
      if (i >= p.chunks) continue;
      const uint32_t w[4] = {c[u].x, c[u].y, c[u].z, c[u].w};
      float x[16];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 a = decode2_float(uint16_t(w[k] & 0xffff)), b = decode2_float(uint16_t(w[k] >> 16));
        x[4 * k] = a.x * s[u];
        x[4 * k + 1] = a.y * s[u];
        x[4 * k + 2] = b.x * s[u];
        x[4 * k + 3] = b.y * s[u];
      }
      store16<T>(to + int64_t(i) * 16, x, wide);
    }
  }
}

bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; }

int check_shape(int dtype, int head_dim, int num_kv_heads, int num_blocks, const char* who) {
  if (dtype != PA_F32 && dtype != PA_F16 && dtype != PA_BF16)
    return fail(PA_ERR_UNSUPPORTED, "%s: unknown dtype %d", who, dtype);
  if (head_dim != 64 && head_dim != 128)
    return fail(PA_ERR_UNSUPPORTED, "%s: head_dim %d (64 or 128)", who, head_dim);
  if (num_kv_heads <= 0 || num_blocks <= 0)
    return fail(PA_ERR_INVALID_ARG, "%s: num_kv_heads and num_blocks must be positive", who);
  if (num_kv_heads > 1 << 16)
    return fail(PA_ERR_INVALID_ARG, "%s: num_kv_heads %d too large", who, num_kv_heads);
  return PA_OK;
}

cudaLaunchAttribute pdl_attribute() {
  cudaLaunchAttribute a;
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  return a;
}

}  // namespace
}  // namespace q8
}  // namespace pa

using namespace pa;
using namespace pa::q8;

extern "C" {

PA_API int pa_kv_append_q8(const void* k, const void* v, void* k_cache, void* v_cache,
                           float* k_scale, float* v_scale, const int32_t* block_tables,
                           const int32_t* context_lens, const int32_t* query_start, int num_seqs,
                           int num_tokens, int num_kv_heads, int head_dim, int max_blocks_per_seq,
                           int num_blocks, int dtype, void* stream) {
  PA_TRACE("pa_kv_append_q8");
  const char* who = "kv_append_q8";
  int rc = check_shape(dtype, head_dim, num_kv_heads, num_blocks, who);
  if (rc != PA_OK) return rc;
  if (num_seqs < 0 || num_tokens < 0 || max_blocks_per_seq <= 0)
    return fail(PA_ERR_INVALID_ARG, "%s: sizes must be positive", who);
  if (double(max_blocks_per_seq) * kBlockSize >= 2147483647.0 ||
      double(num_tokens) / kBlockSize + 2.0 * num_seqs >= 2147483647.0)
    return fail(PA_ERR_INVALID_ARG, "%s: sizes too large", who);
  if (num_seqs == 0 || num_tokens == 0) return PA_OK;
  if (!k || !v || !k_cache || !v_cache || !k_scale || !v_scale || !block_tables ||
      !context_lens || !query_start)
    return fail(PA_ERR_INVALID_ARG, "%s: NULL pointer", who);
  if (misaligned(k) || misaligned(v) || misaligned(k_cache) || misaligned(v_cache))
    return fail(PA_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", who);
  unsigned* status = device_status_word();
  if (!status) return PA_ERR_CUDA;
  AppendParams p = {};
  p.src[0] = k;
  p.src[1] = v;
  p.cache[0] = static_cast<uint8_t*>(k_cache);
  p.cache[1] = static_cast<uint8_t*>(v_cache);
  p.scale[0] = k_scale;
  p.scale[1] = v_scale;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.query_start = query_start;
  p.num_seqs = num_seqs;
  p.num_tokens = num_tokens;
  p.num_kv_heads = num_kv_heads;
  p.max_blocks = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  p.status = status;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(num_tokens / kBlockSize + 2 * num_seqs),
                     unsigned((2 * num_kv_heads + kAppendWarps - 1) / kAppendWarps));
  cfg.blockDim = dim3(kAppendWarps * 32);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e;
  const bool wide = head_dim == 128;
  if (dtype == PA_F32)
    e = wide ? cudaLaunchKernelEx(&cfg, append_kernel<float, 128>, p)
             : cudaLaunchKernelEx(&cfg, append_kernel<float, 64>, p);
  else if (dtype == PA_F16)
    e = wide ? cudaLaunchKernelEx(&cfg, append_kernel<__half, 128>, p)
             : cudaLaunchKernelEx(&cfg, append_kernel<__half, 64>, p);
  else
    e = wide ? cudaLaunchKernelEx(&cfg, append_kernel<__nv_bfloat16, 128>, p)
             : cudaLaunchKernelEx(&cfg, append_kernel<__nv_bfloat16, 64>, p);
  if (e != cudaSuccess) return fail(PA_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
  return PA_OK;
}

PA_API int pa_rotary_kv_append_q8(const void* q, const void* k, const void* v,
                                  const int32_t* positions, const int64_t* turns, int rotary_dim,
                                  int interleaved, float magnitude, void* k_cache, void* v_cache,
                                  float* k_scale, float* v_scale, const int32_t* block_tables,
                                  const int32_t* context_lens, const int32_t* query_start,
                                  int num_seqs, int num_tokens, int num_q_heads, int num_kv_heads,
                                  int head_dim, int max_blocks_per_seq, int num_blocks,
                                  int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                  int64_t q_out_stride, int dtype, void* q_out, void* stream) {
  PA_TRACE("pa_rotary_kv_append_q8");
  const char* who = "rotary_kv_append_q8";
  int rc = check_shape(dtype, head_dim, num_kv_heads, num_blocks, who);
  if (rc != PA_OK) return rc;
  if (num_seqs < 0 || num_tokens < 0 || max_blocks_per_seq <= 0 || num_q_heads < 0 || num_q_heads > 1 << 16)
    return fail(PA_ERR_INVALID_ARG, "%s: sizes must be positive", who);
  if (double(max_blocks_per_seq) * kBlockSize >= 2147483647.0 ||
      double(num_tokens) / kBlockSize + 2.0 * num_seqs >= 2147483647.0)
    return fail(PA_ERR_INVALID_ARG, "%s: sizes too large", who);
  const int elem = dtype == PA_F32 ? 4 : 2;
  if (rc == PA_OK) rc = rot::check_stride(q_stride, elem, 0, "q_stride", who);
  if (rc == PA_OK) rc = rot::check_stride(k_stride, elem, 0, "k_stride", who);
  if (rc == PA_OK) rc = rot::check_stride(v_stride, elem, 0, "v_stride", who);
  if (rc == PA_OK)
    rc = rot::check_stride(q_out_stride, elem, num_tokens > 1 ? int64_t(num_q_heads) * head_dim : 0,
                           "q_out_stride", who);
  if (rc != PA_OK) return rc;
  if (num_seqs == 0 || num_tokens == 0) return PA_OK;
  RotaryAppendParams p = {};
  rc = rot::check_args(turns, rotary_dim, interleaved, magnitude, head_dim, who, &p.rot);
  if (rc != PA_OK) return rc;
  if (!k || !v || !k_cache || !v_cache || !k_scale || !v_scale || !block_tables ||
      !context_lens || !query_start || (num_q_heads && (!q || !q_out)))
    return fail(PA_ERR_INVALID_ARG, "%s: NULL pointer", who);
  if (misaligned(k) || misaligned(v) || misaligned(k_cache) || misaligned(v_cache) ||
      (num_q_heads && (misaligned(q) || misaligned(q_out))))
    return fail(PA_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", who);
  unsigned* status = device_status_word();
  if (!status) return PA_ERR_CUDA;
  p.a.src[0] = k;
  p.a.src[1] = v;
  p.a.cache[0] = static_cast<uint8_t*>(k_cache);
  p.a.cache[1] = static_cast<uint8_t*>(v_cache);
  p.a.scale[0] = k_scale;
  p.a.scale[1] = v_scale;
  p.a.block_tables = block_tables;
  p.a.context_lens = context_lens;
  p.a.query_start = query_start;
  p.a.num_seqs = num_seqs;
  p.a.num_tokens = num_tokens;
  p.a.num_kv_heads = num_kv_heads;
  p.a.max_blocks = max_blocks_per_seq;
  p.a.num_blocks = num_blocks;
  p.a.status = status;
  p.q = q;
  p.q_out = q_out;
  p.stride[0] = k_stride;
  p.stride[1] = v_stride;
  p.stride[2] = q_stride;
  p.q_out_stride = q_out_stride;
  p.num_q_heads = num_q_heads;
  p.positions = positions;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cudaLaunchConfig_t cfg = {};
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e;
  const bool wide = head_dim == 128;
  if (num_tokens <= 2 * num_seqs) {
    const int per = 32 / (head_dim / 16);
    const int groups = (num_q_heads + per - 1) / per + 2 * ((num_kv_heads + per - 1) / per);
    const int gy = (groups + kFewWarps - 1) / kFewWarps;
    cfg.gridDim = dim3(unsigned(num_tokens), unsigned(gy));
    cfg.blockDim = dim3(unsigned((groups + gy - 1) / gy * 32));
    if (dtype == PA_F32)
      e = wide ? cudaLaunchKernelEx(&cfg, rotary_append_few_kernel<float, 128>, p)
               : cudaLaunchKernelEx(&cfg, rotary_append_few_kernel<float, 64>, p);
    else if (dtype == PA_F16)
      e = wide ? cudaLaunchKernelEx(&cfg, rotary_append_few_kernel<__half, 128>, p)
               : cudaLaunchKernelEx(&cfg, rotary_append_few_kernel<__half, 64>, p);
    else
      e = wide ? cudaLaunchKernelEx(&cfg, rotary_append_few_kernel<__nv_bfloat16, 128>, p)
               : cudaLaunchKernelEx(&cfg, rotary_append_few_kernel<__nv_bfloat16, 64>, p);
  } else {
    // Three heads a warp pay for the CTA's angles and its sequence's search
    // (10.6 K tokens of 48 heads: 43.7 us with six, 39.3 with three, 42.5 with
    // one), as long as there are CTAs for the GPU (1 K: 13.9, 9.8, 6.2).
    const int64_t units = int64_t(num_tokens) / kBlockSize + 2 * num_seqs;
    const int rounds = (2 * num_kv_heads + num_q_heads + kAppendWarps - 1) / kAppendWarps;
    const int64_t fill = (1024 + units - 1) / units;
    int gy = (rounds + 2) / 3;
    if (gy < fill) gy = int(fill < rounds ? fill : rounds);
    cfg.gridDim = dim3(unsigned(units), unsigned(gy));
    cfg.blockDim = dim3(kAppendWarps * 32);
    auto go = [&](auto inter) {
      constexpr bool I = decltype(inter)::value;
      if (dtype == PA_F32)
        return wide ? cudaLaunchKernelEx(&cfg, rotary_append_kernel<float, 128, I>, p)
                    : cudaLaunchKernelEx(&cfg, rotary_append_kernel<float, 64, I>, p);
      if (dtype == PA_F16)
        return wide ? cudaLaunchKernelEx(&cfg, rotary_append_kernel<__half, 128, I>, p)
                    : cudaLaunchKernelEx(&cfg, rotary_append_kernel<__half, 64, I>, p);
      return wide ? cudaLaunchKernelEx(&cfg, rotary_append_kernel<__nv_bfloat16, 128, I>, p)
                  : cudaLaunchKernelEx(&cfg, rotary_append_kernel<__nv_bfloat16, 64, I>, p);
    };
    e = interleaved ? go(std::true_type()) : go(std::false_type());
  }
  if (e != cudaSuccess) return fail(PA_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
  return PA_OK;
}

PA_API int pa_block_dequantize(const void* k_cache, const void* v_cache, const float* k_scale,
                               const float* v_scale, const int64_t* src_dst_pairs, int num_pairs,
                               int num_kv_heads, int head_dim, int num_blocks, int num_out_blocks,
                               int dtype, void* k_out, void* v_out, void* stream) {
  PA_TRACE("pa_block_dequantize");
  const char* who = "block_dequantize";
  int rc = check_shape(dtype, head_dim, num_kv_heads, num_blocks, who);
  if (rc != PA_OK) return rc;
  if (num_pairs < 0 || num_out_blocks <= 0)
    return fail(PA_ERR_INVALID_ARG, "%s: num_pairs < 0 or num_out_blocks <= 0", who);
  if (num_pairs == 0) return PA_OK;
  if (!k_cache || !v_cache || !k_scale || !v_scale || !src_dst_pairs || !k_out || !v_out)
    return fail(PA_ERR_INVALID_ARG, "%s: NULL pointer", who);
  if (misaligned(k_cache) || misaligned(v_cache) || misaligned(k_out) || misaligned(v_out))
    return fail(PA_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", who);
  unsigned* status = device_status_word();
  if (!status) return PA_ERR_CUDA;
  ReadParams p = {};
  p.cache[0] = static_cast<const uint8_t*>(k_cache);
  p.cache[1] = static_cast<const uint8_t*>(v_cache);
  p.scale[0] = k_scale;
  p.scale[1] = v_scale;
  p.out[0] = k_out;
  p.out[1] = v_out;
  p.pairs = src_dst_pairs;
  p.num_blocks = num_blocks;
  p.num_out_blocks = num_out_blocks;
  p.chunks = num_kv_heads * head_dim;
  p.head_shift = head_dim == 128 ? 7 : 6;
  p.num_kv_heads = num_kv_heads;
  p.status = status;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cudaLaunchConfig_t cfg = {};
  const int per_cta = kReadThreads * kReadBatch;
  int z = (p.chunks + per_cta - 1) / per_cta;
  if (z > 64) z = 64;
  cfg.gridDim = dim3(unsigned(num_pairs), 2, unsigned(z));
  cfg.blockDim = dim3(kReadThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = dtype == PA_F32   ? cudaLaunchKernelEx(&cfg, read_kernel<float>, p)
                        : dtype == PA_F16 ? cudaLaunchKernelEx(&cfg, read_kernel<__half>, p)
                                          : cudaLaunchKernelEx(&cfg, read_kernel<__nv_bfloat16>, p);
  if (e != cudaSuccess) return fail(PA_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
  return PA_OK;
}

}  // extern "C"
