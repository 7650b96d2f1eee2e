// Rotary positions (rotary.cuh): query and key rows rotated (pa_rotary), and
// the same on the way into a paged cache, values beside them
// (pa_rotary_kv_append); the frequencies they take (host).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <type_traits>

#include "device_common.cuh"
#include "pagedattn.h"
#include "rotary.cuh"
#include "status.h"
#include "trace.h"

namespace pa {
namespace rot {
namespace {

constexpr int kBlockSize = 16;
constexpr int kThreads = 128;

struct Params {
  const void* src[3];  // q, k, v
  void* dst[3];        // their rows rotated; appending, k's and v's cache
  int64_t src_stride[3], dst_stride[3];
  int heads[3];
  int groups[3];       // warps a token's rows take (see rows_kernel)
  int num_tokens;
  int parts;           // warps that share a token's groups: `share` each, the
  int share, extra;    // first `extra` one more
  bool wide;           // every row begins on a 32-byte boundary
  const int32_t* positions;
  const int32_t* lengths;  // without positions: a token is at lengths[token] - 1
  const int64_t* slots;
  int64_t num_slots;
  Args rot;
  unsigned* status;
};

// An item's two chunks, in whole 32-byte sectors where they lie so (`wide`; for
// 16-bit types the chunks must be neighbours, `joined`).
template <typename T>
__device__ __forceinline__ void load_item(const T* row, int2 at, bool wide, bool joined, Chunk<T>& a, Chunk<T>& b) {
  if constexpr (sizeof(T) == 4) {
    if (wide) {
      load32(row + at.x, a.v[0], a.v[1]);
      load32(row + at.y, b.v[0], b.v[1]);
      return;
    }
  } else if (wide && joined) {
    load32(row + at.x, a.v[0], b.v[0]);
    return;
  }
  a.load(row + at.x);
  b.load(row + at.y);
}
template <typename T>
__device__ __forceinline__ void store_item(T* row, int2 at, bool wide, bool joined, const Chunk<T>& a,
                                           const Chunk<T>& b) {
  if constexpr (sizeof(T) == 4) {
    if (wide) {
      store32(row + at.x, a.v[0], a.v[1]);
      store32(row + at.y, b.v[0], b.v[1]);
      return;
    }
  } else if (wide && joined) {
    store32(row + at.x, a.v[0], b.v[0]);
    return;
  }
  a.store(row + at.x);
  b.store(row + at.y);
}

// A group is 32 / NJ heads of one of a token's q, k and v, one item a lane; a warp
// takes N groups of one token, all its loads before anything else; its angles,
// one or two pairs a lane, are computed while they are on their way.  Bound by
// bytes: 13.2 K tokens rotated (271 MB) 41.3 us, 0.97 of the copy rate; 6.4 K
// appended (157 MB) 24.7 us, 0.94; 3.3 K of 32 bits (107 MB) 16.9 us, 0.94 (19.6
// in 16-byte accesses: half of every 32-byte sector at a time).  128 tokens 2.3
// us: launch and latency.
template <typename T, int D, bool APPEND, int N>
__global__ void __launch_bounds__(kThreads) rows_kernel(const Params p) {
  constexpr int NJ = D / 16, kHeads = 32 / NJ;
  dev::grid_launch_dependents();
  const int lane = threadIdx.x, j = lane % NJ;
  const int64_t token = int64_t(blockIdx.x) * blockDim.z + threadIdx.z;
  const int part = blockIdx.y * blockDim.y + threadIdx.y;
  if (token >= p.num_tokens || part >= p.parts) return;
  const int group0 = N == 1 ? part : part * p.share + min(part, p.extra);
  const int count = N == 1 ? 1 : p.share + (part < p.extra ? 1 : 0);
  int64_t f[WarpAngles<D>::kPer];
  const int2 turned = item_columns(p.rot, j);
  // (what a group is follows from its number, for the whole warp)
  auto locate = [&](int i, int& head) {
    int group = group0 + i, kind = 0;
    while (kind < 2 && group >= p.groups[kind]) group -= p.groups[kind++];
    head = group * kHeads + lane / NJ;
    return kind;
  };
  dev::grid_dependency_wait();
  const int position = p.positions ? p.positions[token] : p.lengths[token] - 1;
  int64_t slot = 0;
  if (APPEND) slot = p.slots[token];
  WarpAngles<D>::load_freqs(p.rot, lane, f);
  Chunk<T> a[N], b[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    int head;
    const int kind = locate(i, head);
    if (i >= count || head >= p.heads[kind]) continue;
    const T* row = static_cast<const T*>(p.src[kind]) + token * p.src_stride[kind] + int64_t(head) * D;
    load_item(row, kind < 2 ? turned : make_int2(16 * j, 16 * j + 8), p.wide, kind == 2 || p.rot.interleaved, a[i],
              b[i]);
  }
  WarpAngles<D> angles;
  angles.set(f, position, p.rot.magnitude);
  float c[8], s[8];
  angles.gather(j, c, s);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    int head;
    const int kind = locate(i, head);
    if (i >= count) break;
    if (kind < 2 && 16 * j < p.rot.dim) {
      float x[16];
      a[i].to_float(x);
      b[i].to_float(x + 8);
      turn_item(p.rot.interleaved, x, c, s);
      a[i].from_float(x);
      b[i].from_float(x + 8);
    }
    T* row = static_cast<T*>(p.dst[kind]);
    if (APPEND && kind > 0) {
      if (slot >= p.num_slots && lane == 0) dev::flag_status(p.status, kStatusBounds);
      if (slot < 0 || slot >= p.num_slots) continue;
      row += ((slot / kBlockSize * p.heads[kind] + head) * kBlockSize + slot % kBlockSize) * D;
    } else {
      row += token * p.dst_stride[kind] + int64_t(head) * D;
    }
    if (head >= p.heads[kind]) continue;
    store_item(row, kind < 2 ? turned : make_int2(16 * j, 16 * j + 8), p.wide, kind == 2 || p.rot.interleaved, a[i],
               b[i]);
  }
}

int elem_bytes(int dtype) { return dtype == PA_F32 ? 4 : 2; }

bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; }

// What both entry points check of their rows.
int check_rows(int num_tokens, int num_q_heads, int num_kv_heads, int head_dim, int dtype,
               const char* who) {
  if (dtype != PA_F32 && dtype != PA_F16 && dtype != PA_BF16)
    return fail(PA_ERR_UNSUPPORTED, "%s: unknown dtype %d", who, dtype);
  if (head_dim != 64 && head_dim != 128)
    return fail(PA_ERR_UNSUPPORTED, "%s: head_dim %d (64 or 128)", who, head_dim);
  if (num_tokens < 0) return fail(PA_ERR_INVALID_ARG, "%s: num_tokens < 0", who);
  if (num_q_heads > 1 << 16 || num_kv_heads > 1 << 16)
    return fail(PA_ERR_INVALID_ARG, "%s: more than 65536 heads", who);
  return PA_OK;
}

template <typename T, int D, bool APPEND>
cudaError_t launch_rows(Params p, int groups, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto go = [&](auto number) {
    constexpr int N = decltype(number)::value;
    p.parts = (groups + N - 1) / N;
    p.share = groups / p.parts;
    p.extra = groups % p.parts;
    const int wide = p.parts < kThreads / 32 ? p.parts : kThreads / 32;
    const int tokens = kThreads / 32 / wide;
    cfg.gridDim = dim3(unsigned((int64_t(p.num_tokens) + tokens - 1) / tokens),
                       unsigned((p.parts + wide - 1) / wide));
    cfg.blockDim = dim3(32, unsigned(wide), unsigned(tokens));
    return cudaLaunchKernelEx(&cfg, rows_kernel<T, D, APPEND, N>, p);
  };
  // A warp's angles cost as much as two groups' rotation, and what a warp has
  // in flight hides its latency: the more groups it takes the better, as long
  // as the warps fill the GPU.  (16-bit rows, one group, three, four: 2.4, 2.5,
  // 2.8 us for 128 tokens of 12 groups; 5.1, 3.9, 5.6 for 1024; 27.5, 23.2, 25.7
  // for 6000; 41.7, 36.6, 35.8 for 7200 of 16.)  A group of 32-bit rows is twice
  // the bytes, and one a warp is enough (17.0 us for 3268 tokens of 8 groups,
  // 17.0 with three, 17.1 with four).
  const int64_t units = int64_t(p.num_tokens) * groups;
  if constexpr (sizeof(T) == 2) {
    if (units > 100000 && (groups + 3) / 4 < (groups + 2) / 3) return go(std::integral_constant<int, 4>());
    if (units > 7000) return go(std::integral_constant<int, 3>());
  }
  return go(std::integral_constant<int, 1>());
}

template <bool APPEND>
int launch(Params& p, int num_tokens, int head_dim, int dtype, void* stream, const char* who) {
  p.status = device_status_word();
  if (!p.status) return PA_ERR_CUDA;
  p.num_tokens = num_tokens;
  uintptr_t ends = 0;
  for (int i = 0; i < 3; ++i) {
    if (!p.heads[i]) continue;
    ends |= reinterpret_cast<uintptr_t>(p.src[i]) | reinterpret_cast<uintptr_t>(p.dst[i]);
    ends |= uintptr_t(p.src_stride[i] * elem_bytes(dtype)) | uintptr_t(p.dst_stride[i] * elem_bytes(dtype));
  }
  p.wide = (ends & 31) == 0;
  const int per = 32 / (head_dim / 16);
  int groups = 0;
  for (int i = 0; i < 3; ++i) groups += p.groups[i] = (p.heads[i] + per - 1) / per;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  const bool wide = head_dim == 128;
  if (dtype == PA_F32)
    e = wide ? launch_rows<float, 128, APPEND>(p, groups, s) : launch_rows<float, 64, APPEND>(p, groups, s);
  else if (dtype == PA_F16)
    e = wide ? launch_rows<__half, 128, APPEND>(p, groups, s) : launch_rows<__half, 64, APPEND>(p, groups, s);
  else
    e = wide ? launch_rows<__nv_bfloat16, 128, APPEND>(p, groups, s)
             : launch_rows<__nv_bfloat16, 64, APPEND>(p, groups, s);
  if (e != cudaSuccess) return fail(PA_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
  return PA_OK;
}

}  // namespace

int append_rows(const void* q, const void* k, const void* v, const int32_t* positions,
                const int32_t* context_lens, const Args& rot, void* k_cache, void* v_cache,
                const int64_t* slot_mapping, int num_tokens, int num_q_heads, int num_kv_heads,
                int head_dim, int num_blocks, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                int64_t q_out_stride, int dtype, void* q_out, void* stream, const char* who) {
  Params p = {};
  const void* src[3] = {q, k, v};
  void* dst[3] = {q_out, k_cache, v_cache};
  const int64_t in[3] = {q_stride, k_stride, v_stride};
  for (int i = 0; i < 3; ++i) {
    p.heads[i] = i ? num_kv_heads : num_q_heads;
    p.src[i] = src[i];
    p.dst[i] = dst[i];
    p.src_stride[i] = in[i];
  }
  p.dst_stride[0] = q_out_stride;
  p.positions = positions;
  p.lengths = context_lens;
  p.slots = slot_mapping;
  p.num_slots = int64_t(num_blocks) * kBlockSize;
  p.rot = rot;
  return launch<true>(p, num_tokens, head_dim, dtype, stream, who);
}

}  // namespace rot
}  // namespace pa

using namespace pa;

extern "C" {

PA_API int pa_rotary_frequencies(int rotary_dim, double base, int scaling, double factor,
                                 int original_context, double low, double high,
                                 double* frequencies) {
  const char* who = "rotary_frequencies";
  const double kTurn = 6.283185307179586476925;
  if (rotary_dim < 16 || rotary_dim > 128 || rotary_dim % 16 != 0)
    return fail(PA_ERR_INVALID_ARG, "%s: rotary_dim %d (a multiple of 16, 16 .. 128)", who, rotary_dim);
  if (!(base > 0.0) || !std::isfinite(base))
    return fail(PA_ERR_INVALID_ARG, "%s: base must be positive", who);
  if (scaling < PA_ROTARY_PLAIN || scaling > PA_ROTARY_BANDS)
    return fail(PA_ERR_INVALID_ARG, "%s: unknown scaling %d", who, scaling);
  if (scaling != PA_ROTARY_PLAIN && (!(factor > 0.0) || !std::isfinite(factor)))
    return fail(PA_ERR_INVALID_ARG, "%s: factor must be positive", who);
  if (scaling == PA_ROTARY_BANDS &&
      (original_context <= 0 || !(low >= 0.0) || !(high > low) || !std::isfinite(high)))
    return fail(PA_ERR_INVALID_ARG, "%s: bands need original_context > 0 and 0 <= low < high", who);
  if (!frequencies) return fail(PA_ERR_INVALID_ARG, "%s: NULL pointer", who);
  if (scaling == PA_ROTARY_BASE) base *= std::pow(factor, rotary_dim / (rotary_dim - 2.0));
  for (int i = 0; i < rotary_dim / 2; ++i) {
    double w = std::pow(base, -2.0 * i / rotary_dim);
    if (scaling == PA_ROTARY_LINEAR) {
      w /= factor;
    } else if (scaling == PA_ROTARY_BANDS) {
      const double turns = original_context * w / kTurn;
      double keep = (turns - low) / (high - low);
      keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
      w *= keep + (1.0 - keep) / factor;
    }
    frequencies[i] = w;
  }
  return PA_OK;
}

PA_API int pa_rotary_turns(const double* frequencies, int num_frequencies, int64_t* turns) {
  const char* who = "rotary_turns";
  const double kTurn = 6.283185307179586476925;
  if (num_frequencies < 0) return fail(PA_ERR_INVALID_ARG, "%s: num_frequencies < 0", who);
  if (num_frequencies > 0 && (!frequencies || !turns))
    return fail(PA_ERR_INVALID_ARG, "%s: NULL pointer", who);
  for (int i = 0; i < num_frequencies; ++i)
    if (!std::isfinite(frequencies[i]))
      return fail(PA_ERR_INVALID_ARG, "%s: frequency %d is not finite", who, i);
  // The quotient in two parts, the second what the first one's rounding leaves
  // over (a turn in two parts too): 2^-102 of it is lost, where one division
  // loses 2^-53, 2^-25 of a turn at position 2^31.
  const double kTurnRest = 2.4492935982947064e-16;       // 2 pi - kTurn
  for (int i = 0; i < num_frequencies; ++i) {
    const double w = frequencies[i];
    double t = w / kTurn;
    double rest = std::fma(-t, kTurnRest, std::fma(-t, kTurn, w)) / kTurn;
    t -= std::rint(t);                                   // whole turns do nothing
    rest -= std::rint(rest);
    t = std::ldexp(t, 64);                               // -2^63 .. 2^63
    const double whole = std::rint(t);
    const double low = std::rint((t - whole) + std::ldexp(rest, 64));
    const uint64_t high = whole >= 9223372036854775808.0 ? uint64_t(1) << 63
                                                         : uint64_t(static_cast<int64_t>(whole));
    const uint64_t more = low >= 9223372036854775808.0 ? uint64_t(1) << 63
                                                       : uint64_t(static_cast<int64_t>(low));
    turns[i] = static_cast<int64_t>(high + more);
  }
  return PA_OK;
}

PA_API int pa_rotary(const void* q, const void* k, const int32_t* positions, const int64_t* turns,
                     int rotary_dim, int interleaved, float magnitude, int num_tokens,
                     int num_q_heads, int num_kv_heads, int head_dim, int64_t q_stride,
                     int64_t k_stride, int64_t q_out_stride, int64_t k_out_stride, int dtype,
                     void* q_out, void* k_out, void* stream) {
  PA_TRACE("pa_rotary");
  const char* who = "rotary";
  int rc = rot::check_rows(num_tokens, num_q_heads, num_kv_heads, head_dim, dtype, who);
  if (rc != PA_OK) return rc;
  if (num_q_heads < 0 || num_kv_heads < 0 || num_q_heads + num_kv_heads == 0)
    return fail(PA_ERR_INVALID_ARG, "%s: no heads", who);
  rot::Params p = {};
  const int elem = rot::elem_bytes(dtype);
  const int64_t qw = int64_t(num_q_heads) * head_dim, kw = int64_t(num_kv_heads) * head_dim;
  if (rc == PA_OK) rc = rot::check_stride(q_stride, elem, 0, "q_stride", who);
  if (rc == PA_OK) rc = rot::check_stride(k_stride, elem, 0, "k_stride", who);
  if (rc == PA_OK) rc = rot::check_stride(q_out_stride, elem, num_tokens > 1 ? qw : 0, "q_out_stride", who);
  if (rc == PA_OK) rc = rot::check_stride(k_out_stride, elem, num_tokens > 1 ? kw : 0, "k_out_stride", who);
  if (rc != PA_OK || num_tokens == 0) return rc;
  rc = rot::check_args(turns, rotary_dim, interleaved, magnitude, head_dim, who, &p.rot);
  if (rc != PA_OK) return rc;
  if (!positions || (num_q_heads && (!q || !q_out)) || (num_kv_heads && (!k || !k_out)))
    return fail(PA_ERR_INVALID_ARG, "%s: NULL pointer", who);
  const void* src[2] = {q, k};
  void* dst[2] = {q_out, k_out};
  const int heads[2] = {num_q_heads, num_kv_heads};
  const int64_t in[2] = {q_stride, k_stride}, out[2] = {q_out_stride, k_out_stride};
  for (int i = 0; i < 2; ++i) {
    if (heads[i] && (rot::misaligned(src[i]) || rot::misaligned(dst[i])))
      return fail(PA_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", who);
    p.src[i] = src[i];
    p.dst[i] = dst[i];
    p.heads[i] = heads[i];
    p.src_stride[i] = in[i];
    p.dst_stride[i] = out[i];
  }
  p.positions = positions;
  return rot::launch<false>(p, num_tokens, head_dim, dtype, stream, who);
}

PA_API int pa_rotary_kv_append(const void* q, const void* k, const void* v,
                               const int32_t* positions, const int64_t* turns, int rotary_dim,
                               int interleaved, float magnitude, void* k_cache, void* v_cache,
                               const int64_t* slot_mapping, int num_tokens, int num_q_heads,
                               int num_kv_heads, int head_dim, int num_blocks, int64_t q_stride,
                               int64_t k_stride, int64_t v_stride, int64_t q_out_stride, int dtype,
                               void* q_out, void* stream) {
  PA_TRACE("pa_rotary_kv_append");
  const char* who = "rotary_kv_append";
  int rc = rot::check_rows(num_tokens, num_q_heads, num_kv_heads, head_dim, dtype, who);
  if (rc != PA_OK) return rc;
  if (num_q_heads < 0 || num_kv_heads <= 0 || num_blocks <= 0)
    return fail(PA_ERR_INVALID_ARG, "%s: num_kv_heads and num_blocks must be positive", who);
  rot::Args args;
  const int elem = rot::elem_bytes(dtype);
  if (rc == PA_OK) rc = rot::check_stride(q_stride, elem, 0, "q_stride", who);
  if (rc == PA_OK) rc = rot::check_stride(k_stride, elem, 0, "k_stride", who);
  if (rc == PA_OK) rc = rot::check_stride(v_stride, elem, 0, "v_stride", who);
  if (rc == PA_OK)
    rc = rot::check_stride(q_out_stride, elem, num_tokens > 1 ? int64_t(num_q_heads) * head_dim : 0,
                           "q_out_stride", who);
  if (rc != PA_OK || num_tokens == 0) return rc;
  rc = rot::check_args(turns, rotary_dim, interleaved, magnitude, head_dim, who, &args);
  if (rc != PA_OK) return rc;
  if (!positions || !slot_mapping || !k || !v || !k_cache || !v_cache ||
      (num_q_heads && (!q || !q_out)))
    return fail(PA_ERR_INVALID_ARG, "%s: NULL pointer", who);
  const void* const tensors[6] = {num_q_heads ? q : nullptr, num_q_heads ? q_out : nullptr, k, v, k_cache,
                                  v_cache};
  for (const void* ptr : tensors)
    if (rot::misaligned(ptr))
      return fail(PA_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", who);
  return rot::append_rows(q, k, v, positions, nullptr, args, k_cache, v_cache, slot_mapping,
                          num_tokens, num_q_heads, num_kv_heads, head_dim, num_blocks, q_stride,
                          k_stride, v_stride, q_out_stride, dtype, q_out, stream, who);
}

}  // extern "C"
