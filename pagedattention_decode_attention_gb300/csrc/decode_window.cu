// Decode attention with a sliding window and first tokens that stay visible,
// over 16- and 32-bit caches (pa_paged_attention_decode_window) and over the
// 8-bit cache (pa_paged_attention_decode_q8).
//
// Sequence b has n = context_lens[b] tokens; its one query, the newest token's,
// sees token t when t < n and (t >= n - window or t < num_sinks); window 0
// means all of them.
//   s_t = scale * q . K_t,   out = sum_t softmax(s)_t V_t
// with K_t = k_scale * code for the 8-bit cache.  Blocks none of whose tokens
// are visible are not read, nor are their table entries (a program that has
// freed them may leave any value there).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "device_common.cuh"
#include "pagedattn.h"
#include "q8.cuh"
#include "status.h"
#include "trace.h"

namespace pa {
namespace window {
namespace {

constexpr int kBlockSize = 16;
constexpr int kMaxGroup = 8;

// Workspace: header words, then each sequence's planned length.
constexpr int kHdrSignature = 0;

struct Layout {
  size_t ctx, total;
};

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

Layout workspace_layout(int num_seqs) {
  Layout l;
  l.ctx = 256;
  l.total = align256(l.ctx + size_t(num_seqs) * 4);
  return l;
}

struct Params {
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const float* k_scale;
  const float* v_scale;
  void* out;
  const int32_t* block_tables;
  const int32_t* context_lens;
  int window, num_sinks;
  int num_seqs, num_q_heads, num_kv_heads, group;
  int max_blocks, num_blocks;
  float scale;
  int signature;
  int* header;
  int* ctx;
  unsigned* status;
};

__global__ void plan_kernel(const Params p) {
  dev::grid_launch_dependents();
  dev::grid_dependency_wait();
  for (int b = threadIdx.x; b < p.num_seqs; b += blockDim.x) {
    int n = p.context_lens[b];
    if (n < 0 || n > p.max_blocks * kBlockSize) {
      dev::flag_status(p.status, kStatusBounds);
      n = n < 0 ? 0 : p.max_blocks * kBlockSize;
    }
    p.ctx[b] = n;
  }
  if (threadIdx.x == 0) p.header[kHdrSignature] = p.signature;
}

template <typename T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_float<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_float<uint8_t>(uint8_t x) { return q8::decode2_float(x).x; }

template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// One warp per (sequence, query head), a token at a time, fp32 throughout.
template <typename T, typename C, int D>
__global__ void __launch_bounds__(128) simple_kernel(const Params p) {
  constexpr int E = D / 32;
  dev::grid_launch_dependents();
  dev::grid_dependency_wait();
  const int unit = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (unit >= p.num_seqs * p.num_q_heads) return;
  if (p.header[kHdrSignature] != p.signature) {
    if (unit == 0 && lane == 0) dev::flag_status(p.status, kStatusPlan);
    return;
  }
  const int b = unit / p.num_q_heads, h = unit % p.num_q_heads, g = h / p.group;
  const int n = p.ctx[b];
  const int lo = p.window ? max(n - p.window, 0) : 0;
  const int first = min(p.num_sinks, lo);
  const T* q = static_cast<const T*>(p.q) + size_t(unit) * D + lane * E;
  const C* kc = static_cast<const C*>(p.k_cache);
  const C* vc = static_cast<const C*>(p.v_cache);
  float qr[E], acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    qr[e] = to_float<T>(q[e]);
    acc[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int i = 0; i < first + n - lo; ++i) {
    const int t = i < first ? i : lo + i - first;
    int phys = p.block_tables[size_t(b) * p.max_blocks + t / kBlockSize];
    if (phys < 0 || phys >= p.num_blocks) {
      if (lane == 0) dev::flag_status(p.status, kStatusBounds);
      phys = 0;
    }
    const size_t tile = size_t(phys) * p.num_kv_heads + g;
    const size_t at = (tile * kBlockSize + t % kBlockSize) * D + lane * E;
    const float ks = p.k_scale ? p.k_scale[tile] : 1.f, vs = p.v_scale ? p.v_scale[tile] : 1.f;
    float dot = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) dot = fmaf(qr[e], to_float<C>(kc[at + e]), dot);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
    const float s = dot * ks * p.scale;
    const float mn = fmaxf(m, s);
    const float a = expf(m - mn), w = expf(s - mn);
    l = l * a + w;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * a + w * (to_float<C>(vc[at + e]) * vs);
    m = mn;
  }
  T* out = static_cast<T*>(p.out) + size_t(unit) * D + lane * E;
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) out[e] = from_float<T>(acc[e] * inv);
}

int signature_of(int window, int num_sinks, int num_seqs, int num_q_heads, int num_kv_heads,
                 int head_dim, int max_blocks) {
  uint32_t h = 2166136261u;
  const int v[8] = {window, num_sinks, num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks, 0x51D3};
  for (int x : v) {
    h ^= uint32_t(x);
    h *= 16777619u;
  }
  return int(h | 1u);
}

cudaLaunchAttribute pdl_attribute() {
  cudaLaunchAttribute a;
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  return a;
}

enum class Mode { kPlanAndRun, kPlanOnly, kRunOnly };

struct Call {
  const char* who;
  Mode mode;
  bool q8;
  const void *q, *k_cache, *v_cache;
  const float *k_scale, *v_scale;
  const int32_t *block_tables, *context_lens;
  int window, num_sinks, num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks, num_blocks;
  float scale;
  int dtype;
  void *out, *workspace;
  size_t workspace_bytes;
  void* stream;
};

int check_sizes(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int max_blocks,
                const char* who) {
  if (head_dim != 64 && head_dim != 128)
    return fail(PA_ERR_UNSUPPORTED, "%s: head_dim %d (64 or 128)", who, head_dim);
  if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || max_blocks <= 0)
    return fail(PA_ERR_INVALID_ARG, "%s: sizes must be positive", who);
  if (num_q_heads % num_kv_heads != 0)
    return fail(PA_ERR_INVALID_ARG, "%s: num_q_heads %% num_kv_heads != 0", who);
  if (double(max_blocks) * kBlockSize >= 2147483647.0 ||
      double(num_seqs) * num_kv_heads * max_blocks >= 2147483647.0 ||
      double(num_seqs) * num_q_heads >= 2147483647.0)
    return fail(PA_ERR_INVALID_ARG, "%s: sizes too large for the workspace", who);
  return PA_OK;
}

template <typename T, typename C>
cudaError_t launch_simple(const cudaLaunchConfig_t& cfg, int head_dim, const Params& p) {
  return head_dim == 128 ? cudaLaunchKernelEx(&cfg, simple_kernel<T, C, 128>, p)
                         : cudaLaunchKernelEx(&cfg, simple_kernel<T, C, 64>, p);
}

int entry(const Call& c) {
  const char* who = c.who;
  const bool runs = c.mode != Mode::kPlanOnly;
  if (runs && c.dtype != PA_F32 && c.dtype != PA_F16 && c.dtype != PA_BF16)
    return fail(PA_ERR_UNSUPPORTED, "%s: unknown dtype %d", who, c.dtype);
  if (c.q8 && c.dtype == PA_F32)
    return fail(PA_ERR_UNSUPPORTED, "%s: queries over the 8-bit cache are f16 or bf16", who);
  int rc = check_sizes(c.num_seqs, c.num_q_heads, c.num_kv_heads, c.head_dim, c.max_blocks, who);
  if (rc != PA_OK) return rc;
  if (c.window < 0 || c.num_sinks < 0)
    return fail(PA_ERR_INVALID_ARG, "%s: window and num_sinks must not be negative", who);
  const int group = c.num_q_heads / c.num_kv_heads;
  if (runs && c.dtype != PA_F32 && group > kMaxGroup)
    return fail(PA_ERR_UNSUPPORTED, "%s: %d query heads per KV head (max %d)", who, group, kMaxGroup);
  if (c.num_seqs == 0) return PA_OK;
  if (!c.context_lens) return fail(PA_ERR_INVALID_ARG, "%s: NULL pointer", who);
  if (runs) {
    if (!c.q || !c.k_cache || !c.v_cache || !c.block_tables || !c.out ||
        (c.q8 && (!c.k_scale || !c.v_scale)))
      return fail(PA_ERR_INVALID_ARG, "%s: NULL pointer", who);
    for (const void* ptr : {c.q, c.k_cache, c.v_cache, static_cast<const void*>(c.out)})
      if (reinterpret_cast<uintptr_t>(ptr) & 15)
        return fail(PA_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", who);
    if (c.num_blocks <= 0 || double(c.num_blocks) * c.num_kv_heads * kBlockSize >= 2147483647.0)
      return fail(PA_ERR_INVALID_ARG, "%s: bad num_blocks", who);
  }
  const Layout lay = workspace_layout(c.num_seqs);
  if (!c.workspace || (reinterpret_cast<uintptr_t>(c.workspace) & 255))
    return fail(PA_ERR_INVALID_ARG, "%s: workspace must be non-NULL and 256-byte aligned", who);
  if (c.workspace_bytes < lay.total)
    return fail(PA_ERR_INVALID_ARG, "%s: workspace %zu bytes < %zu needed", who, c.workspace_bytes,
                lay.total);
  unsigned* status = device_status_word();
  if (!status) return PA_ERR_CUDA;
  Params p = {};
  p.q = c.q;
  p.k_cache = c.k_cache;
  p.v_cache = c.v_cache;
  p.k_scale = c.k_scale;
  p.v_scale = c.v_scale;
  p.out = c.out;
  p.block_tables = c.block_tables;
  p.context_lens = c.context_lens;
  p.window = c.window;
  p.num_sinks = c.num_sinks;
  p.num_seqs = c.num_seqs;
  p.num_q_heads = c.num_q_heads;
  p.num_kv_heads = c.num_kv_heads;
  p.group = group;
  p.max_blocks = c.max_blocks;
  p.num_blocks = c.num_blocks;
  p.scale = c.scale;
  p.signature = signature_of(c.window, c.num_sinks, c.num_seqs, c.num_q_heads, c.num_kv_heads,
                             c.head_dim, c.max_blocks);
  uint8_t* ws = static_cast<uint8_t*>(c.workspace);
  p.header = reinterpret_cast<int*>(ws);
  p.ctx = reinterpret_cast<int*>(ws + lay.ctx);
  p.status = status;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cudaLaunchConfig_t cfg = {};
  cfg.stream = static_cast<cudaStream_t>(c.stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (c.mode != Mode::kRunOnly) {
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(256);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, plan_kernel, p);
    if (e != cudaSuccess) return fail(PA_ERR_CUDA, "%s: plan launch failed: %s", who, cudaGetErrorString(e));
  }
  if (!runs) return PA_OK;
  cfg.gridDim = dim3(unsigned((c.num_seqs * c.num_q_heads + 3) / 4));
  cfg.blockDim = dim3(128);
  cudaError_t e;
  if (c.dtype == PA_F32)
    e = launch_simple<float, float>(cfg, c.head_dim, p);
  else if (c.dtype == PA_F16)
    e = c.q8 ? launch_simple<__half, uint8_t>(cfg, c.head_dim, p)
             : launch_simple<__half, __half>(cfg, c.head_dim, p);
  else
    e = c.q8 ? launch_simple<__nv_bfloat16, uint8_t>(cfg, c.head_dim, p)
             : launch_simple<__nv_bfloat16, __nv_bfloat16>(cfg, c.head_dim, p);
  if (e != cudaSuccess) return fail(PA_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
  return PA_OK;
}

}  // namespace
}  // namespace window
}  // namespace pa

using namespace pa;
using pa::window::Mode;

extern "C" {

PA_API int pa_paged_attention_decode_window_workspace_size(int num_seqs, int num_q_heads,
                                                           int num_kv_heads, int head_dim,
                                                           int max_blocks_per_seq, size_t* bytes) {
  const char* who = "paged_attention_decode_window_workspace_size";
  if (!bytes) return fail(PA_ERR_INVALID_ARG, "%s: bytes is NULL", who);
  const int rc = window::check_sizes(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                     max_blocks_per_seq, who);
  if (rc != PA_OK) return rc;
  *bytes = window::workspace_layout(num_seqs).total;
  return PA_OK;
}

PA_API int pa_paged_attention_decode_window_plan(const int32_t* context_lens, int window,
                                                 int num_sinks, int num_seqs, int num_q_heads,
                                                 int num_kv_heads, int head_dim,
                                                 int max_blocks_per_seq, void* workspace,
                                                 size_t workspace_bytes, void* stream) {
  PA_TRACE("pa_paged_attention_decode_window_plan");
  return window::entry({"paged_attention_decode_window_plan", Mode::kPlanOnly, false, nullptr,
                        nullptr, nullptr, nullptr, nullptr, nullptr, context_lens, window,
                        num_sinks, num_seqs, num_q_heads, num_kv_heads, head_dim,
                        max_blocks_per_seq, 0, 0.f, PA_BF16, nullptr, workspace, workspace_bytes,
                        stream});
}

PA_API int pa_paged_attention_decode_window(
    const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
    const int32_t* context_lens, int window, int num_sinks, int num_seqs, int num_q_heads,
    int num_kv_heads, int head_dim, int max_blocks_per_seq, int num_blocks, float scale, int dtype,
    void* out, void* workspace, size_t workspace_bytes, void* stream) {
  PA_TRACE("pa_paged_attention_decode_window");
  return window::entry({"paged_attention_decode_window", Mode::kPlanAndRun, false, q, k_cache,
                        v_cache, nullptr, nullptr, block_tables, context_lens, window, num_sinks,
                        num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq,
                        num_blocks, scale, dtype, out, workspace, workspace_bytes, stream});
}

PA_API int pa_paged_attention_decode_window_run(
    const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
    const int32_t* context_lens, int window, int num_sinks, int num_seqs, int num_q_heads,
    int num_kv_heads, int head_dim, int max_blocks_per_seq, int num_blocks, float scale, int dtype,
    void* out, void* workspace, size_t workspace_bytes, void* stream) {
  PA_TRACE("pa_paged_attention_decode_window_run");
  return window::entry({"paged_attention_decode_window_run", Mode::kRunOnly, false, q, k_cache,
                        v_cache, nullptr, nullptr, block_tables, context_lens, window, num_sinks,
                        num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq,
                        num_blocks, scale, dtype, out, workspace, workspace_bytes, stream});
}

PA_API int pa_paged_attention_decode_q8(
    const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
    const float* v_scale, const int32_t* block_tables, const int32_t* context_lens, int window,
    int num_sinks, int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
    int max_blocks_per_seq, int num_blocks, float scale, int dtype, void* out, void* workspace,
    size_t workspace_bytes, void* stream) {
  PA_TRACE("pa_paged_attention_decode_q8");
  return window::entry({"paged_attention_decode_q8", Mode::kPlanAndRun, true, q, k_cache, v_cache,
                        k_scale, v_scale, block_tables, context_lens, window, num_sinks, num_seqs,
                        num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq, num_blocks, scale,
                        dtype, out, workspace, workspace_bytes, stream});
}

PA_API int pa_paged_attention_decode_q8_run(
    const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
    const float* v_scale, const int32_t* block_tables, const int32_t* context_lens, int window,
    int num_sinks, int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
    int max_blocks_per_seq, int num_blocks, float scale, int dtype, void* out, void* workspace,
    size_t workspace_bytes, void* stream) {
  PA_TRACE("pa_paged_attention_decode_q8_run");
  return window::entry({"paged_attention_decode_q8_run", Mode::kRunOnly, true, q, k_cache, v_cache,
                        k_scale, v_scale, block_tables, context_lens, window, num_sinks, num_seqs,
                        num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq, num_blocks, scale,
                        dtype, out, workspace, workspace_bytes, stream});
}

}  // extern "C"
