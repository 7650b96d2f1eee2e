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

// Eight consecutive elements of a row in 32 bits.
template <typename T>
__device__ __forceinline__ void load8(const T* src, float (&x)[8]);

template <>
__device__ __forceinline__ void load8<float>(const float* src, float (&x)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(src), b = *reinterpret_cast<const float4*>(src + 4);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__half>(const __half* src, float (&x)[8]) {
  const uint4 v = *reinterpret_cast<const uint4*>(src);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = dev::Mma<__half>::unpack(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* src, float (&x)[8]) {
  const uint4 v = *reinterpret_cast<const uint4*>(src);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = dev::Mma<__nv_bfloat16>::unpack(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

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

// A unit is one (sequence, block the call writes to); blockIdx.x numbers them
// with gaps: sequence b's begin at query_start[b] / 16 + 3 b, and T new tokens
// touch at most (T + 30) / 16 blocks, so two sequences' units never meet.  A
// warp owns one (unit, KV head, K or V): it alone reads and writes that
// scale, holds the new rows in registers between finding their largest
// magnitude and encoding them, and rescales the older rows of the block when
// the scale grows.  Bound by bytes (2 head_dim elements read and as many
// codes written per token and head); for a decode step by latency.
template <typename T, int D>
__global__ void __launch_bounds__(kAppendWarps * 32) append_kernel(const AppendParams p) {
  constexpr int kLanes = D / 8;             // lanes per row, eight elements each
  constexpr int kRows = 32 / kLanes;        // rows per pass
  constexpr int kPasses = kBlockSize / kRows;
  dev::grid_launch_dependents();
  dev::grid_dependency_wait();
  // the unit's sequence: the last one whose first unit is not past it
  const int unit = blockIdx.x;
  auto invalid = [&](int q0, int q1, int ctx) {
    return q0 < 0 || q1 < q0 || q1 > p.num_tokens || q1 - q0 > ctx ||
           ctx > p.max_blocks * kBlockSize;
  };
  int mine = 0;
  for (int base = 0; base < p.num_seqs; base += kAppendWarps * 32) {
    const int b = base + threadIdx.x;
    const int q0 = b < p.num_seqs ? p.query_start[b] : 0;
    mine += __syncthreads_count(b < p.num_seqs && q0 / kBlockSize + 3 * b <= unit);
    if (unit == 0 && blockIdx.y == 0 && b < p.num_seqs &&
        invalid(q0, p.query_start[b + 1], p.context_lens[b]))
      dev::flag_status(p.status, kStatusBounds);
  }
  const int b = mine - 1;
  if (b < 0) return;
  const int q0 = p.query_start[b], q1 = p.query_start[b + 1], ctx = p.context_lens[b];
  const int fresh_tokens = q1 - q0;
  if (fresh_tokens == 0 || invalid(q0, q1, ctx)) return;
  const int begin = ctx - fresh_tokens;     // first new token's position
  const int blk = begin / kBlockSize + (unit - (q0 / kBlockSize + 3 * b));
  if (blk > (ctx - 1) / kBlockSize) return;
  const int phys = p.block_tables[size_t(b) * p.max_blocks + blk];
  if (phys < 0 || phys >= p.num_blocks) {
    if (threadIdx.x == 0) dev::flag_status(p.status, kStatusBounds);
    return;
  }
  const int job = blockIdx.y * kAppendWarps + (threadIdx.x >> 5);
  if (job >= 2 * p.num_kv_heads) return;
  const int kv = job & 1, head = job >> 1, lane = threadIdx.x & 31;
  const int lo = max(begin - blk * kBlockSize, 0);                 // rows lo .. hi - 1 are new
  const int hi = min(ctx - blk * kBlockSize, kBlockSize);
  const int row0 = lane / kLanes, col = (lane % kLanes) * 8;
  // the new rows, and the largest finite magnitude among them
  float x[kPasses][8];
  float peak = 0.f;
  // (row 0 of the block, which lies before the tokens when lo > 0)
  const T* src = static_cast<const T*>((kv ? p.src[1] : p.src[0])) +
                 ((int64_t(q0) + blk * kBlockSize - begin) * p.num_kv_heads + head) * D + col;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int r = i * kRows + row0;
    if (r >= lo && r < hi) load8<T>(src + int64_t(r) * p.num_kv_heads * D, x[i]);
  }
  const size_t tile = size_t(phys) * p.num_kv_heads + head;
  const float old = lo > 0 ? (kv ? p.scale[1] : p.scale[0])[tile] : 0.f;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int r = i * kRows + row0;
    if (r >= lo && r < hi) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float a = fabsf(x[i][e]);
        if (a <= 3.402823466e38f) peak = fmaxf(peak, a);
      }
    }
  }
  const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(peak));
  const float want = __uint_as_float(pow2_bits(scale_exponent(top)));
  const float scale = lo > 0 ? fmaxf(old, want) : want;
  const float inv = 1.f / scale;            // exact: a power of two (or the caller's own scale)
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
    if (r >= lo && r < hi) {
      uint2 c;
      c.x = uint32_t(encode2(x[i][0] * inv, x[i][1] * inv)) |
            uint32_t(encode2(x[i][2] * inv, x[i][3] * inv)) << 16;
      c.y = uint32_t(encode2(x[i][4] * inv, x[i][5] * inv)) |
            uint32_t(encode2(x[i][6] * inv, x[i][7] * inv)) << 16;
      *reinterpret_cast<uint2*>(codes + r * D) = c;
    }
  }
  if (lane == 0 && (lo == 0 || scale > old)) (kv ? p.scale[1] : p.scale[0])[tile] = scale;
}

// Sixteen codes times their scale, as sixteen elements.
__device__ __forceinline__ void store16(float* dst, const float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    reinterpret_cast<float4*>(dst)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
}
template <typename T>
__device__ __forceinline__ void store16(T* dst, const float (&x)[16]) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = dev::Mma<T>::pack(x[2 * i], x[2 * i + 1]);
  reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
  reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
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
// thread turns chunks of 16 into 16 elements.  Pure data movement.
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
      store16(to + int64_t(i) * 16, x);
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
      double(num_tokens) / kBlockSize + 3.0 * num_seqs >= 2147483647.0)
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
  cfg.gridDim = dim3(unsigned(num_tokens / kBlockSize + 3 * num_seqs),
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
