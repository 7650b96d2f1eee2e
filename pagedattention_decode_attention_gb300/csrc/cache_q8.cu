// The 8-bit paged cache: kv_append_q8 (new tokens quantised into their blocks)
// and block_dequantize (whole blocks read back as 16- or 32-bit values).
//
// Format (q8.cuh): k_cache, v_cache hold e4m3 codes [num_blocks][num_kv_heads]
// [16][head_dim]; k_scale, v_scale one fp32 power of two per (block, KV head).
// A token's value is code * scale.  The tokens of one block share a scale
// because a block is what the pool moves and what attention reads: the scale
// travels with the 16 rows it belongs to and costs 4 bytes per 16 * head_dim.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "device_common.cuh"
#include "pagedattn.h"
#include "q8.cuh"
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
