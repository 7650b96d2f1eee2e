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
//
// Bound by the bytes of the visible blocks: 4 G / elem flops per byte at most
// (G query heads per KV head), far under the tensor cores' rate.
//
//  * The visible blocks of a sequence are numbered 0 .. nb - 1 without gaps
//    (first tokens' blocks, then the window's); all (sequence, KV head, block)
//    triples in that order form one line, cut into equal shares, one per CTA
//    of a full grid (one CTA per SM), at least kMinPlaces each, and those into
//    one per warp.  Equal work for every warp whatever the lengths (a
//    (sequence, KV head) takes kSegmentCost places more than it has blocks,
//    for its query rows, first references and output); a long context is
//    spread over the GPU, many short ones share a warp.  The plan kernel
//    writes each warp's starting point.
//  * A warp streams its share through its own shared-memory ring, one tensor
//    copy per K and V tile (16 rows), filled as many blocks ahead as fit; it
//    does not stop at the ends of sequences.
//  * Per block: S^T = K Q^T (16 tokens x 8 heads, m16n8k16), a base-2 softmax
//    against a running reference that moves only when a score exceeds it by
//    more than 8 (so almost every block needs one vote and no shuffle), and
//    O^T += V^T P^T.  The contraction order over head_dim and the order of
//    O's rows are free, so K and V fragments are read in 16-byte chunks:
//    lane (g, t) takes chunks of K's rows g and g + 8, and chunk g of V's rows
//    2t, 2t + 1, 2t + 8, 2t + 9, whose bytes pair up by one permute.
//  * Where a warp's share cuts a sequence, its partial sums meet the other
//    warps' of the CTA in shared memory; where the CTA's share cuts it, the
//    CTA's two open ends go to the workspace and the CTA that arrives last at
//    a sequence merges its pieces in order (the result does not depend on
//    which one that is).
//  * pa_paged_attention_decode_q8_append_run: the warp that takes a sequence's
//    last block quantises the new token into the tile it has in shared memory
//    (and the older rows anew when the scale grows) and stores the same bytes
//    to the cache, so no copy waits for the append.  This stands outside
//    the loop over blocks: 90.7 us on the first batch below, 92.1 inside it.
//  * Before it waits for the kernel in front of it, a launch brings its first
//    blocks into L2 (hints only): 1.3 - 3.4 us less for launches in a row, 0.7 us
//    more for one on an idle GPU.
//
// Measured (GB300, launches in a row, of the copy rate 6.79 TB/s): 128 sequences
// of 128 .. 8192 tokens, 32/8 heads, 8-bit: 87.9 us, 6.23 TB/s of the bytes a
// launch cannot do without (0.92); 64 sequences, window 4096 + 64, bf16: 89.0
// us, 6.54 TB/s (0.96); 64 sequences of 16 .. 2048 tokens, 32/32 heads, 8-bit:
// 38.4 us, 5.42 TB/s (0.80: 2048 short segments); one sequence of 101 tokens:
// 5.8 us; one stream with a window of 1024: 8.8 us.  With the append, two
// launches and one: 94.3 and 90.7 us (first batch), 45.0 and 41.9 (third).  The
// loop itself runs at the copy rate; start (plan words, table entries, first
// copies: 2 us) and end (warps' slack, merges within and between CTAs: 3 - 5 us)
// are what is left.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <mutex>
#include <type_traits>

#include "device_common.cuh"
#include "pagedattn.h"
#include "q8.cuh"
#include "rotary.cuh"
#include "status.h"
#include "tensor_map.h"
#include "trace.h"

namespace pa {
namespace window {
namespace {

constexpr int kBlockSize = 16;
constexpr int kMaxGroup = 8;

// Warps per CTA.  A warp takes a block in about the same time whatever its
// bytes (a chain of latencies: copy, product, softmax, product), so the fewer
// bytes a block has, the more warps it takes to keep HBM busy.  Registers and
// rings of three blocks allow 8 for 16-bit tiles of head_dim 128, 12 for 8-bit
// ones (8: 92.1 us on the 8-bit batch, 90.3 with 12), 16 for 8-bit tiles of 64
// (8: 18.0 us on the long window, 16.7); 16-bit tiles of 64 do best with 12 and
// rings of four (16 with three: 16.2 us on the odd window, 15.3).
__host__ __device__ constexpr int warps_of(bool q8, int head_dim) {
  return head_dim == 64 ? (q8 ? 16 : 12) : (q8 ? 12 : 8);
}
constexpr int kMaxCtas = 256;        // CTAs the workspace has room for
constexpr int kMinPlaces = 32;       // places on the line a CTA takes at least
// what a (sequence, KV head) costs beside its blocks, in blocks (none: 100.6 us
// on the 8-bit batch, 57.6 on the MHA one; 1: 95.5, 44.8; 2: 92.1, 42.9; 3: 92.8,
// 44.1)
constexpr int kSegmentCost = 2;
constexpr int kFillAt = 16;          // where in its 32 blocks a warp reads the next 32's entries
constexpr float kRescale = 8.f;      // log2 by which a score may exceed the reference (Tiles::kLift counts on it)
constexpr int kPlanThreads = 1024;

// Workspace header words: what the plan was made for; places in all, places
// per CTA, whether a sequence has no blocks (its output rows are zero).
constexpr int kHdrSignature = 0, kHdrPlaces = 1, kHdrShare = 2, kHdrEmpty = 3;

// A CTA's two open ends: the one it shares with earlier CTAs (slot 0) and the
// one that goes on in later ones (slot 1): unnormalised output, reference of
// the scores, reference of the weights, sum of the softmax.
template <int D>
struct Piece {
  float o[kMaxGroup][D];
  float m[kMaxGroup], w[kMaxGroup], l[kMaxGroup];
  int id, ends, used;  // sequence * KV heads + head; holds its last block
  int c0, ctas;        // first CTA of the sequence's KV head, and how many share it
  int pad[3];
};

struct Layout {
  size_t seqs, starts, arrivals, pieces, total;
};

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

Layout workspace_layout(int num_seqs, int head_dim) {
  Layout l;
  l.seqs = 256;
  l.starts = align256(l.seqs + size_t(num_seqs) * sizeof(int4));
  l.arrivals = align256(l.starts + size_t(kMaxCtas) * (warps_of(false, head_dim) + warps_of(true, head_dim)) *
                                       2 * sizeof(int4));
  l.pieces = align256(l.arrivals + size_t(kMaxCtas) * 4);
  l.total = align256(l.pieces + size_t(kMaxCtas) * 2 *
                                    (head_dim == 128 ? sizeof(Piece<128>) : sizeof(Piece<64>)));
  return l;
}

struct Params {
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const float* k_scale;
  const float* v_scale;
  // fused append: the new tokens' rows, [num_seqs][num_kv_heads][head_dim], and
  // the cache and scales again, to write
  const void* new_rows[2];
  uint8_t* codes[2];
  float* scales[2];
  // rotation of q's rows and the new K rows (rotary.cuh): positions (null: the
  // newest token's place), elements between rows of q, K and V
  rot::Args rot;
  const int32_t* positions;
  int64_t q_stride, new_stride[2];
  void* out;
  const int32_t* block_tables;
  const int32_t* context_lens;
  int window, num_sinks;
  int num_seqs, num_q_heads, num_kv_heads, group;
  int max_blocks, num_blocks;
  int ncta;
  float scale, scale_log2;
  int signature;
  int* header;
  // per sequence: length, visible blocks, places of a KV head's blocks before
  // the sequence's and of its own on the line
  int4* seqs;
  // per warp: sequence, KV head, block within it, blocks; its seqs entry (for
  // the warp counts of 16-bit and 8-bit caches, one after the other)
  int4* starts;
  int head_dim;
  int* arrivals;     // per CTA: arrivals at the sequence that begins in it and goes on
  void* pieces;      // [kMaxCtas][2] Piece
  unsigned* status;
  unsigned long long timeout_ns;
};

// Which blocks of n tokens are visible: blocks 0 .. first - 1 and first + skip
// .. ceil(n / 16) - 1; tokens under `low` are visible below `sinks` only.
struct Range {
  int low, sinks, first, skip, count;
};

__device__ __forceinline__ Range visible_range(int n, int window, int num_sinks) {
  Range r;
  const int blocks = (n + kBlockSize - 1) / kBlockSize;
  r.low = window > 0 && window < n ? n - window : 0;
  r.sinks = min(num_sinks, r.low);
  const int sink_blocks = (r.sinks + kBlockSize - 1) / kBlockSize, low_block = r.low / kBlockSize;
  r.first = sink_blocks < low_block ? sink_blocks : blocks;
  r.skip = sink_blocks < low_block ? low_block - sink_blocks : 0;
  r.count = blocks - r.skip;
  return r;
}

// One CTA: visible blocks per sequence and their running sum, then each warp's
// starting point by bisection.  Latency-bound (128 sequences 11 us, one 7 us,
// as launched back to back); once per step, not per layer.
//
// Where the batch is so small that every (sequence, KV head) can have CTAs of
// its own (at kMinPlaces a CTA), it gets them: up to kMinPlaces -
// kSegmentCost blocks then meet in one CTA's shared memory, which saves the
// trip through the workspace (one sequence of 101 tokens, 8 KV heads: 5.6 us,
// 9.6 us packed).
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const Params p) {
  __shared__ int s_warp[kPlanThreads / 32];
  __shared__ int s_carry, s_empty, s_ctas;
  dev::grid_launch_dependents();
  dev::grid_dependency_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    s_carry = 0;
    s_empty = 0;
    s_ctas = 0;
  }
  __syncthreads();
  auto length = [&](int b) {
    const int n = p.context_lens[b];
    return n < 0 ? 0 : min(n, p.max_blocks * kBlockSize);
  };
  int ctas = 0;
  for (int b = tid; b < p.num_seqs; b += kPlanThreads) {
    const int n = p.context_lens[b];
    if (n < 0 || n > p.max_blocks * kBlockSize) dev::flag_status(p.status, kStatusBounds);
    const int nb = visible_range(length(b), p.window, p.num_sinks).count;
    if (nb == 0) s_empty = 1;
    else if (ctas <= kMaxCtas) ctas += (nb + kSegmentCost + kMinPlaces - 1) / kMinPlaces;
  }
  if (ctas) atomicAdd(&s_ctas, min(ctas, kMaxCtas + 1));
  __syncthreads();
  const int pad = (long long)s_ctas * p.num_kv_heads <= p.ncta ? kMinPlaces : 1;
  for (int base = 0; base < p.num_seqs; base += kPlanThreads) {
    const int b = base + tid;
    int n = 0, nb = 0;
    if (b < p.num_seqs) {
      n = length(b);
      nb = visible_range(n, p.window, p.num_sinks).count;
    }
    const int places = nb ? (nb + kSegmentCost + pad - 1) / pad * pad : 0;
    int sum = places;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, sum, off);
      if (lane >= off) sum += up;
    }
    if (lane == 31) s_warp[warp] = sum;
    __syncthreads();
    if (warp == 0) {
      int v = s_warp[lane];
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += up;
      }
      s_warp[lane] = v;
    }
    __syncthreads();
    const int before = s_carry + (warp ? s_warp[warp - 1] : 0) + sum - places;
    if (b < p.num_seqs) p.seqs[b] = make_int4(n, nb, before, places);
    __syncthreads();
    if (tid == 0) s_carry += s_warp[kPlanThreads / 32 - 1];
    __syncthreads();
  }
  const int total = s_carry * p.num_kv_heads;
  const int share = max(kMinPlaces, (total + p.ncta - 1) / p.ncta);
  // Place f of the line: the sequence it falls in, and how many of its blocks
  // (KV head by KV head) lie before it.  A KV head's first kSegmentCost places
  // and those behind its last block hold none.
  auto locate = [&](long long f, int4& q, int& block) {
    // the last sequence that begins at or before f (it has tokens: an empty
    // one's successor begins where it does)
    int lo = 0, hi = p.num_seqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((long long)p.seqs[mid].z * p.num_kv_heads <= f) lo = mid;
      else hi = mid - 1;
    }
    q = p.seqs[lo];
    const int r = int(f - (long long)q.z * p.num_kv_heads);
    block = r / q.w * q.y + min(max(r % q.w - kSegmentCost, 0), q.y);
    return lo;
  };
  int4* starts = p.starts;
  for (int q8 = 0; q8 < 2; ++q8) {
    const int warps = warps_of(q8, p.head_dim);
    auto place = [&](int w) {
      return (long long)(w / warps) * share + (long long)(w % warps) * share / warps;
    };
    for (int w = tid; w < p.ncta * warps; w += kPlanThreads) {
      const long long f = place(w), end = place(w + 1);
      int4 at = make_int4(0, 0, 0, 0), q = make_int4(0, 1, 0, 1);
      if (f < total) {
        int block, block2 = 0;
        const int b = locate(f, q, block);
        int4 q2;
        int count = 0, b2 = p.num_seqs;
        if (end < total) b2 = locate(end, q2, block2);
        // blocks up to the next warp's first, sequence by sequence
        if (b2 == b) {
          count = block2 - block;
        } else {
          count = q.y * p.num_kv_heads - block + block2;
          for (int i = b + 1; i < b2; ++i) count += p.seqs[i].y * p.num_kv_heads;
        }
        at = make_int4(b, block / q.y, block % q.y, count);
        // (between two sequences: the next one's first block is the first)
        if (count > 0 && at.y == p.num_kv_heads) {
          int i = b + 1;
          while (p.seqs[i].y == 0) ++i;
          q = p.seqs[i];
          at = make_int4(i, 0, 0, count);
        }
      }
      starts[2 * w] = at;
      starts[2 * w + 1] = q;
    }
    starts += size_t(kMaxCtas) * warps * 2;
  }
  for (int c = tid; c < p.ncta; c += kPlanThreads) p.arrivals[c] = 0;
  if (tid == 0) {
    p.header[kHdrPlaces] = total;
    p.header[kHdrShare] = share;
    p.header[kHdrEmpty] = s_empty;
    p.header[kHdrSignature] = p.signature;
  }
}

// fp32 caches: one warp per (sequence, query head), a token at a time, so K and
// V are read once per query head and a token waits for the one before: 64
// sequences with a window of 4096 + 64, 32/8 heads, 4.6 ms (floor 0.2).  For
// checking against, not for serving.
template <int D>
__global__ void __launch_bounds__(128) f32_kernel(const Params p) {
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
  const int n = p.seqs[b].x;
  const int lo = p.window ? max(n - p.window, 0) : 0;
  const int first = min(p.num_sinks, lo);
  const float* q = static_cast<const float*>(p.q) + size_t(unit) * D + lane * E;
  const float* kc = static_cast<const float*>(p.k_cache);
  const float* vc = static_cast<const float*>(p.v_cache);
  float qr[E], acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    qr[e] = q[e];
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
    float dot = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) dot = fmaf(qr[e], kc[at + e], dot);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
    const float s = dot * p.scale;
    // (scores of -inf before any other: nothing has weight yet)
    const float mn = fmaxf(m, s), ref = mn == -INFINITY ? 0.f : mn;
    const float a = expf(m - ref), w = expf(s - ref);
    l = l * a + w;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * a + w * vc[at + e];
    m = mn;
  }
  float* out = static_cast<float*>(p.out) + size_t(unit) * D + lane * E;
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) out[e] = acc[e] * inv;
}

// ------------------------------------------------------- tensor-core path
// Tiles of the cache: C = the cache's element (uint8_t: e4m3 codes).
// ROT: with room for a warp's query rows, which it rotates there.
template <typename T, bool Q8, int D, bool ROT = false>
struct Tiles {
  using Mm = dev::Mma<typename std::conditional<Q8, __half, T>::type>;
  static constexpr int kElem = Q8 ? 1 : 2;
  // The softmax's weights enter V's product rounded to its 16-bit type: half a
  // step, f16's 2^-11 and bf16's 2^-8 relative, as much as the rounding of an
  // output of that type.  For f16 (and an 8-bit cache's f16 weights) that is
  // accepted: outputs of the f16 window case are 1.7e-4 from 64-bit
  // arithmetic on average, 1.5e-4 with weights in 32 bits.  For bf16 what the
  // rounding leaves over goes through a second product: the windowed batch's
  // output is 0.0017 (one rounding) from 64-bit arithmetic, 0.0023 without, for
  // 89.4 us, 89.2 without (the tensor cores are active 13 % of the time, 9 without).
  static constexpr bool kTwoParts = !Q8 && std::is_same<T, __nv_bfloat16>::value;
  // f16 weights are 2^(x - reference + kLift).  The reference may be the
  // sequence's largest score (a first token that takes most of the softmax),
  // and then everything else lies under it: without the lift f16's full
  // precision ends at 2^-14 of it and its range at 2^-25, so that thousands of
  // small weights lose their bits or all of their share.  A score exceeds the
  // reference by kRescale at most: 2^(7 + 8) stays under f16's 65504.  bf16 has
  // the range of 32 bits.
  static constexpr float kLift = Q8 || std::is_same<T, __half>::value ? 7.f : 0.f;
  static constexpr int kRowBytes = D * kElem;               // of a token's row
  // a copy box is 128 bytes wide: half a row, a row, or two tokens' rows
  static constexpr int kBoxes = kRowBytes / 128 > 1 ? kRowBytes / 128 : 1;
  static constexpr int kTile = kRowBytes * kBlockSize;
  static constexpr int kBoxBytes = kTile / kBoxes;
  static constexpr int kBoxRows = kBoxBytes / 128;
  static constexpr int kStage = 2 * kTile;                  // K tile, V tile
  static constexpr int kWarps = warps_of(Q8, D);
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kStages = (kWarps == 8 ? 24576 : !Q8 ? 16384 : 12288) / kStage - (ROT && D == 64 ? 1 : 0);
  static constexpr int kSteps = D / 16;                     // 16-wide steps of either product
  static constexpr size_t kRing = size_t(kWarps) * kStages * kStage;
  static constexpr size_t kPieces = kRing;                  // Piece[kWarps]
  static constexpr size_t kBars = kPieces + kWarps * sizeof(Piece<D>);
  static constexpr size_t kFlags = kBars + size_t(kWarps) * kStages * 8;  // int[kWarps + 4]
  // rows padded by 16 bytes, so that lanes reading one column of several do not meet in a bank
  static constexpr int kQRow = D + 8;
  static constexpr int kQBytes = ROT ? kMaxGroup * kQRow * 2 + int(sizeof(rot::AngleTable<D>)) : 0;
  static constexpr size_t kRows = (kFlags + (kWarps + 4) * 4 + 15) & ~size_t(15);
  static constexpr size_t kFreqs = kRows + size_t(kWarps) * kQBytes;  // int64[D / 2]
  static constexpr size_t kBytes = ROT ? kFreqs + D / 2 * 8 : kFlags + (kWarps + 4) * 4;
  // merge of a sequence's pieces over CTAs, in the ring's place
  static_assert(kRing >= size_t(kMaxCtas) * kMaxGroup * 12, "merge weights");
  static_assert(size_t(kStages) * kStage >= sizeof(Piece<D>), "a warp's last piece");
  static_assert(kStages >= 3, "two blocks in use, one on its way");
  static_assert(kBytes <= 227 * 1024, "shared memory");
  static_assert(kThreads >= kMaxGroup * D / 4, "a column per thread");
};

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}

// log2 of a positive scale, exact for a power of two.
__device__ __forceinline__ float log2_scale(float x) {
  const uint32_t u = __float_as_uint(x);
  const int e = int(u >> 23) - 127;
  if (e == -127 || e == 128) return log2f(x);  // zero, subnormal; infinity, NaN
  return float(e) + __log2f(__uint_as_float((u & 0x7FFFFFu) | 0x3F800000u));
}

// The tokens of K's rows g, g + 8 as MMA A fragments, eight or four steps.
template <bool Q8, int D>
__device__ __forceinline__ void load_k(uint32_t tile, int g, int t, uint32_t (&f)[D / 16][4]) {
  if constexpr (Q8) {
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
      // head_dim 16 (2t + j) .. + 15 (128), 16 t .. + 15 (64)
      // (64: two tokens to a 128-byte row)
      const uint32_t at = D == 128 ? tile + g * 128 + (((2 * t + j) ^ g) << 4)
                                   : tile + (g >> 1) * 128 + ((((g & 1) * 4 + t) ^ (g >> 1)) << 4);
      const uint4 a = lds128(at), b = lds128(D == 128 ? at + 1024 : (at + 512) ^ 64);
      const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[4 * j + i][0] = q8::decode2(uint16_t(wa[i]));
        f[4 * j + i][1] = q8::decode2(uint16_t(wb[i]));
        f[4 * j + i][2] = q8::decode2(uint16_t(wa[i] >> 16));
        f[4 * j + i][3] = q8::decode2(uint16_t(wb[i] >> 16));
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
      // half j / 2 of the row, its elements 8 (2t + j % 2) .. + 7
      const uint32_t at = tile + (j >> 1) * 2048 + g * 128 + (((2 * t + (j & 1)) ^ g) << 4);
      const uint4 a = lds128(at), b = lds128(at + 1024);
      f[2 * j][0] = a.x;
      f[2 * j][1] = b.x;
      f[2 * j][2] = a.y;
      f[2 * j][3] = b.y;
      f[2 * j + 1][0] = a.z;
      f[2 * j + 1][1] = b.z;
      f[2 * j + 1][2] = a.w;
      f[2 * j + 1][3] = b.w;
    }
  }
}

// V's rows 2t, 2t + 1, 2t + 8, 2t + 9 as A fragments of V^T: fragment m's rows
// g and g + 8 are head_dim dim_of(m) and dim_of(m) + 1.
template <bool Q8, int D>
__device__ __forceinline__ int dim_of(int g, int m) {
  if (Q8 && D == 128) return 16 * g + 2 * m;
  return (m >> 2) * 64 + 8 * g + 2 * (m & 3);
}

template <bool Q8, int D, int W>
__device__ __forceinline__ void pair_rows(const uint32_t (&r)[4][W], uint32_t (&f)[D / 16][4], int m0) {
#pragma unroll
  for (int i = 0; i < W; ++i) {
    if constexpr (Q8) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t sel = h ? 0x7362 : 0x5140;
        const uint32_t a = __byte_perm(r[0][i], r[1][i], sel), b = __byte_perm(r[2][i], r[3][i], sel);
        f[m0 + 2 * i + h][0] = q8::decode2(uint16_t(a));
        f[m0 + 2 * i + h][1] = q8::decode2(uint16_t(a >> 16));
        f[m0 + 2 * i + h][2] = q8::decode2(uint16_t(b));
        f[m0 + 2 * i + h][3] = q8::decode2(uint16_t(b >> 16));
      }
    } else {
      f[m0 + i][0] = __byte_perm(r[0][i], r[1][i], 0x5410);
      f[m0 + i][1] = __byte_perm(r[0][i], r[1][i], 0x7632);
      f[m0 + i][2] = __byte_perm(r[2][i], r[3][i], 0x5410);
      f[m0 + i][3] = __byte_perm(r[2][i], r[3][i], 0x7632);
    }
  }
}

template <int W>
__device__ __forceinline__ void hide_rows(uint32_t keep, uint32_t (&w)[4][W]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < W; ++j)
      if (!(keep >> i & 1)) w[i][j] = 0;
}

// keep: bit i set when V row i of the four is visible (the others read as 0,
// whatever the cache holds there); 15 for all but a few blocks.
template <bool Q8, int D>
__device__ __forceinline__ void load_v(uint32_t tile, int g, int t, uint32_t keep,
                                       uint32_t (&f)[D / 16][4]) {
  const int rows[4] = {2 * t, 2 * t + 1, 2 * t + 8, 2 * t + 9};
  if constexpr (Q8 && D == 64) {
    uint32_t w[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = rows[i];
      const uint2 v = lds64(tile + (r >> 1) * 128 + ((((r & 1) * 4 + (g >> 1)) ^ (r >> 1)) << 4) + (g & 1) * 8);
      w[i][0] = v.x;
      w[i][1] = v.y;
    }
    if (keep != 15) hide_rows(keep, w);
    pair_rows<Q8, D, 2>(w, f, 0);
  } else {
#pragma unroll
    for (int j = 0; j < (Q8 ? 1 : D / 64); ++j) {
      uint32_t w[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = rows[i];
        const uint4 v = lds128(tile + j * 2048 + r * 128 + ((g ^ (r & 7)) << 4));
        w[i][0] = v.x;
        w[i][1] = v.y;
        w[i][2] = v.z;
        w[i][3] = v.w;
      }
      if (keep != 15) hide_rows(keep, w);
      pair_rows<Q8, D, 4>(w, f, 4 * j);
    }
  }
}

// Query row of head g in load_k's order, as loaded (heads past the group are
// zero) ...
template <typename T, bool Q8, int D>
__device__ __forceinline__ void load_q(const T* row, bool live, int t, uint4 (&w)[D / 32]) {
#pragma unroll
  for (int j = 0; j < D / 32; ++j) {
    const int at = Q8 ? (D == 128 ? 32 * t + 8 * j : 16 * t + 8 * j)
                      : (j >> 1) * 64 + (2 * t + (j & 1)) * 8;
    w[j] = make_uint4(0, 0, 0, 0);
    if (live) w[j] = *reinterpret_cast<const uint4*>(row + at);
  }
}

// ... and as B fragments.  For the 8-bit cache a bf16 row is brought to f16 by
// a power of two (returned as its exponent): a row of any size keeps every bit
// down to 2^-38 of its largest element.
template <typename T, bool Q8, int D>
__device__ __forceinline__ int convert_q(const uint4 (&raw)[D / 32], uint32_t (&f)[D / 16][2]) {
  uint32_t w[D / 8];
#pragma unroll
  for (int j = 0; j < D / 32; ++j) {
    w[4 * j] = raw[j].x;
    w[4 * j + 1] = raw[j].y;
    w[4 * j + 2] = raw[j].z;
    w[4 * j + 3] = raw[j].w;
  }
  int e = 0;
  if constexpr (Q8 && std::is_same<T, __nv_bfloat16>::value) {
    // the largest magnitude of the row, as bf16 bits (its four lanes)
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) top = __vmaxu2(top, w[i] & 0x7FFF7FFFu);
    top = max(top & 0xFFFFu, top >> 16);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int x = int(top >> 7);  // biased exponent; 0: nothing, 255: not finite
    e = x == 0 || x == 255 ? 0 : max(x - 127 - 13, -120);
    const float down = __uint_as_float(uint32_t(127 - e) << 23);
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      const float2 v = dev::Mma<__nv_bfloat16>::unpack(w[i]);
      w[i] = dev::Mma<__half>::pack(v.x * down, v.y * down);
    }
  }
#pragma unroll
  for (int i = 0; i < D / 16; ++i) {
    f[i][0] = w[2 * i];
    f[i][1] = w[2 * i + 1];
  }
  return e;
}

// While the kernel before this one finishes (its last CTAs leave most of HBM
// idle): brings the warp's first blocks into L2.  Hints only, made from
// whatever the workspace and tables hold at this moment: every index is
// checked, everything is read again after the dependency wait, and these reads
// go through L2 so that no L1 line of theirs can serve a later one.
template <int TILE>
__device__ __forceinline__ void warm_l2(const Params& p, const int4* mine, int lane, int blocks) {
  const int4 hdr = __ldcg(reinterpret_cast<const int4*>(p.header));
  const int4 at = __ldcg(mine), seq = __ldcg(mine + 1);
  if (hdr.x != p.signature || lane >= blocks || lane >= at.w) return;
  const int b = at.x, h = at.y, v = at.z + lane;
  if (b < 0 || b >= p.num_seqs || h < 0 || h >= p.num_kv_heads || at.z < 0 || v >= seq.y ||
      seq.x <= 0 || seq.x > p.max_blocks * kBlockSize)
    return;
  const Range r = visible_range(seq.x, p.window, p.num_sinks);
  const int block = v < r.first ? v : v + r.skip;
  if (block < 0 || block >= p.max_blocks) return;
  const int phys = __ldcg(p.block_tables + size_t(b) * p.max_blocks + block);
  if (phys < 0 || phys >= p.num_blocks) return;
  const size_t tile = (size_t(phys) * p.num_kv_heads + h) * TILE;
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(static_cast<const uint8_t*>(p.k_cache) + tile),
               "n"(TILE)
               : "memory");
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(static_cast<const uint8_t*>(p.v_cache) + tile),
               "n"(TILE)
               : "memory");
}

// Where 8 bytes of row r of an 8-bit tile, columns 8 c .. 8 c + 7, sit in it.
template <int D>
__device__ __forceinline__ int q8_offset(int r, int c) {
  return D == 128 ? r * 128 + (((c >> 1) ^ (r & 7)) << 4) + (c & 1) * 8
                  : (r >> 1) * 128 + ((((r & 1) * 4 + (c >> 1)) ^ (r >> 1)) << 4) + (c & 1) * 8;
}

// kv_append_q8 of one token, into a tile pair in shared memory (`tiles`: K, then
// V) and the cache: row `off` of block `tile` of K (lanes 0 - 15) and V (16 -
// 31), eight elements a lane.  `old`: this half's scale of the block.  Returns
// its scale afterwards.
template <typename T, int D>
__device__ __forceinline__ float append_row(const Params& p, uint8_t* tiles, size_t tile, int off, float old,
                                            const q8::Row8<T>& x) {
  const int lane = threadIdx.x & 31, kv = lane >> 4, c = lane & 15;
  const bool live = c < D / 8;
  auto largest = [&](bool finite) {
    uint32_t m = live ? x.top(finite) : 0;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
  };
  uint32_t top = largest(false);
  if constexpr (std::is_same<T, float>::value) {
    if (__any_sync(0xffffffffu, top >= q8::Row8<T>::kInf)) {
      const uint32_t fine = largest(true);
      if (top >= q8::Row8<T>::kInf) top = fine;
    }
  } else {
    const uint32_t fine = largest(true);
    if (top >= q8::Row8<T>::kInf) top = fine;
  }
  const float want = __uint_as_float(q8::pow2_bits(q8::scale_exponent(q8::Row8<T>::float_bits(top))));
  const float scale = off > 0 ? fmaxf(old, want) : want;
  const bool grows = off > 0 && scale > old;
  uint8_t* to = tiles + kv * 16 * D;
  uint8_t* cache = (kv ? p.codes[1] : p.codes[0]) + tile * kBlockSize * D + 8 * c;
  if (live && grows) {
    const float factor = old / scale;
    for (int r = 0; r < off; ++r) {
      uint2* at = reinterpret_cast<uint2*>(to + q8_offset<D>(r, c));
      const uint2 y = q8::rescale8(*at, factor);
      *at = y;
      *reinterpret_cast<uint2*>(cache + r * D) = y;
    }
  }
  if (live) {
    const uint2 y = x.encode(1.f / scale);
    *reinterpret_cast<uint2*>(to + q8_offset<D>(off, c)) = y;
    *reinterpret_cast<uint2*>(cache + off * D) = y;
  }
  if (c == 0 && (off == 0 || grows)) (kv ? p.scales[1] : p.scales[0])[tile] = scale;
  return scale;
}

// A query row's 16 rotated values (an item of row lane / NJ; the NJ lanes of a
// row call together) as f16 in the warp's rows, `to` + at.x and at.y, brought to
// f16's range by a power of two of the row's largest (its exponent is
// returned): a row of any size keeps every bit down to 2^-38 of its largest
// element.  f16 queries: x is left with what the rounding left over.
template <int NJ, bool REST>
__device__ __forceinline__ int place_q(float (&x)[16], uint16_t* to, const int2 at, bool live) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(x[i]));
#pragma unroll
  for (int o = NJ / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const int e0 = int(__float_as_uint(top) >> 23);  // biased exponent; 0: nothing, 255: not finite
  const int e = e0 == 0 || e0 == 255 ? 0 : max(e0 - 127 - 13, -120);
  const float down = __uint_as_float(uint32_t(127 - e) << 23);
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 y = rot::mul2(make_float2(x[2 * i], x[2 * i + 1]), make_float2(down, down));
    w[i] = dev::Mma<__half>::pack(y.x, y.y);
    if constexpr (REST) {
      const float2 z = rot::fma2(dev::Mma<__half>::unpack(w[i]), make_float2(-1.f, -1.f), y);
      x[2 * i] = z.x;
      x[2 * i + 1] = z.y;
    }
  }
  if (live) {
    *reinterpret_cast<uint4*>(to + at.x) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(to + at.y) = make_uint4(w[4], w[5], w[6], w[7]);
  }
  return e;
}

// The new K row rotated, 8 columns a lane (lanes 0 - 15; the others hold V's and
// keep it), in 32 bits: a column is y cos + other sin, `other` its pair's other
// column, its sign turned in the pair's first.
template <typename T, int D>
__device__ __forceinline__ q8::Row8<float> rotate_row(const Params& p, const q8::Row8<T>& x,
                                                      const rot::AngleTable<D>& table) {
  const int lane = threadIdx.x & 31, chunk = lane & 15, half = p.rot.dim / 16;
  const bool inter = p.rot.interleaved, second = !inter && chunk >= half;
  const int j = inter ? chunk / 2 : second ? chunk - half : chunk;
  const int from = (lane + (chunk < half ? half : -half)) & 31;
  const uint32_t sign = inter ? 0x00008000u : second ? 0u : 0x80008000u;
  rot::Chunk<T> raw, other;
  raw.v[0] = x.v;
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&x.v);
  uint32_t* o = reinterpret_cast<uint32_t*>(&other.v[0]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t far = __shfl_sync(0xffffffffu, w[i], from);
    o[i] = (inter ? __byte_perm(w[i], 0, 0x1032) : far) ^ sign;
  }
  float y[8], z[8], c[8], s[8];
  raw.to_float(y);
  if (lane < 16 && chunk < 2 * half) {
    other.to_float(z);
    table.get(j, c, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // the angles of columns 2 i, 2 i + 1: their own pairs', or the one they are
      const float2 far = chunk & 1 ? make_float2(c[4 + i], s[4 + i]) : make_float2(c[i], s[i]);
      const float2 cc = inter ? make_float2(far.x, far.x) : make_float2(c[2 * i], c[2 * i + 1]);
      const float2 ss = inter ? make_float2(far.y, far.y) : make_float2(s[2 * i], s[2 * i + 1]);
      const float2 a = rot::fma2(make_float2(y[2 * i], y[2 * i + 1]), cc,
                                 rot::mul2(make_float2(z[2 * i], z[2 * i + 1]), ss));
      y[2 * i] = a.x;
      y[2 * i + 1] = a.y;
    }
  }
  q8::Row8<float> out;
  out.v[0] = make_uint4(__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]), __float_as_uint(y[3]));
  out.v[1] = make_uint4(__float_as_uint(y[4]), __float_as_uint(y[5]), __float_as_uint(y[6]), __float_as_uint(y[7]));
  return out;
}

// ROT (with APPEND): the query rows and the new K row are rotated on the way.  A
// segment's rows are loaded as items (rotary.cuh), rotated in registers, and
// turned into fragments through the warp's shared memory.  They are rounded to
// f16, not to T; where T is f16, what that leaves over (the rest) enters the
// product too (outputs 2.8e-4 from 64-bit arithmetic, 4.1e-4 without): in the
// product's free columns 4 .. 7 and added by a shuffle where a group has at most
// 4 heads (FOLD), else by a second product (64 sequences of 32/32 heads, f16,
// so: 60.9 us folded, 70.5 with the second product).
//
// What it costs (one launch of many): the first batch above 87.1 us, 84.5 with
// its rows rotated already; the third 54.0 and 41.8, 2048 segments and as many
// new tokens, each some 400 instructions more that a warp goes through alone: that
// batch is faster as two launches, rotary first (45.2; bf16 52.1 and 49.2).
template <typename T, bool Q8, int D, bool APPEND, bool ROT, bool FOLD>
__global__ void __launch_bounds__(Tiles<T, Q8, D, ROT>::kThreads, 1)
    attend_kernel(const __grid_constant__ CUtensorMap tmap_k,
                  const __grid_constant__ CUtensorMap tmap_v, const Params p) {
  using S = Tiles<T, Q8, D, ROT>;
  using Mm = typename S::Mm;
  static_assert(!ROT || (Q8 && APPEND), "rotation is built for the 8-bit append");
  constexpr bool kRest = ROT && std::is_same<T, __half>::value;
  constexpr int NJ = D / 16;  // 16-column items of a row's rotation
  constexpr bool fold = kRest && FOLD;
  constexpr int ST = S::kStages, kWarps = S::kWarps, kThreads = S::kThreads;
  constexpr bool kTwoParts = S::kTwoParts;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + size_t(warp) * ST * S::kStage;
  Piece<D>* head_pieces = reinterpret_cast<Piece<D>*>(smem + S::kPieces);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::kBars) + warp * ST;
  if (lane == 0) {
    for (int i = 0; i < ST; ++i) dev::mbar_init(&full[i], 1);
    dev::mbar_fence_init();
    dev::prefetch_tensormap(&tmap_k);
    dev::prefetch_tensormap(&tmap_v);
  }
  __syncwarp();
  dev::grid_launch_dependents();
  const int Hkv = p.num_kv_heads, G = p.group;
  warm_l2<S::kTile>(p, p.starts + 2 * (blockIdx.x * kWarps + warp), lane, 2 * ST);
  dev::grid_dependency_wait();

  // (all of the plan's words at once: one trip to memory)
  const int4 hdr = *reinterpret_cast<const int4*>(p.header);
  const int4* mine = p.starts + 2 * (blockIdx.x * kWarps + warp);
  const int4 start = mine[0], start_seq = mine[1];
  // (a CTA whose wait runs out voids the plan while others may still be
  // starting: a warp that finds none takes no blocks, and its CTA gives up
  // where the warps meet)
  const bool planned = __all_sync(0xffffffffu, hdr.x == p.signature);
  if (!planned && blockIdx.x == 0 && threadIdx.x == 0) dev::flag_status(p.status, kStatusPlan);
  const int total = hdr.y, share = hdr.z;
  if (planned && hdr.w) {
    // rows of sequences without tokens are zero
    for (int b = blockIdx.x; b < p.num_seqs; b += gridDim.x)
      if (p.seqs[b].y == 0) {
        uint4* row = reinterpret_cast<uint4*>(static_cast<T*>(p.out) + size_t(b) * p.num_q_heads * D);
        for (int i = threadIdx.x; i < p.num_q_heads * D / 8; i += kThreads) row[i] = make_uint4(0, 0, 0, 0);
      }
  }
  const int count = planned ? start.w : 0;  // this warp's blocks
  if ((long long)blockIdx.x * share >= total) return;

  const unsigned long long tmo = p.timeout_ns;
  const uint64_t policy = dev::l2_policy_evict_first();

  // ---- copies.  Lane j holds the (block, head) tile of the warp's block
  // 32 c + j; those of the next 32 are read from the tables while the
  // current ones are in use.
  int fb = start.x, fg = start.y, fv = start.z, filled = 0;  // where the next fill begins
  int4 fseq = start_seq;
  Range frange = visible_range(fseq.x, p.window, p.num_sinks);
  int next_phys = 0, next_head = 0;
  auto fill = [&]() {
    int entry = -1;
    const int todo = min(32, count - filled);
    for (int done = 0; done < todo;) {
      const int n = min(todo - done, fseq.y - fv);
      if (lane >= done && lane < done + n) {
        const int v = fv + lane - done;
        entry = p.block_tables[size_t(fb) * p.max_blocks + (v < frange.first ? v : v + frange.skip)];
        next_head = fg;
      }
      done += n;
      fv += n;
      if (fv == fseq.y) {
        fv = 0;
        if (++fg == Hkv && filled + done < count) {
          fg = 0;
          do fseq = p.seqs[++fb];
          while (fseq.y == 0);
          frange = visible_range(fseq.x, p.window, p.num_sinks);
        }
      }
    }
    next_phys = entry;
    filled += todo;
  };
  int tile = 0;
  float next_ks = 0.f, next_vs = 0.f;  // their scales
  auto promote = [&]() {
    int phys = next_phys;
    if (phys < 0 || phys >= p.num_blocks) {
      if (lane < filled - ((filled - 1) & ~31)) dev::flag_status(p.status, kStatusBounds);
      phys = 0;
    }
    tile = phys * Hkv + next_head;
    if constexpr (Q8) {
      next_ks = p.k_scale[tile];
      next_vs = p.v_scale[tile];
    }
  };
  int issued = 0, put = 0;  // blocks copied so far, ring stage of the next
  auto issue = [&]() {
    if ((issued & 31) == 0) promote();
    if ((issued & 31) == kFillAt && filled < count) fill();
    const int at = __shfl_sync(0xffffffffu, tile, issued & 31);
    uint8_t* dst = ring + put * S::kStage;
    uint64_t* bar = &full[put];
    if (lane == 0) {
      dev::mbar_arrive_expect_tx(bar, S::kStage);
#pragma unroll
      for (int x = 0; x < S::kBoxes; ++x) {
        dev::tma_load_2d(dst + x * S::kBoxBytes, &tmap_k, x * (128 / S::kElem), at * S::kBoxRows, bar, policy);
        dev::tma_load_2d(dst + S::kTile + x * S::kBoxBytes, &tmap_v, x * (128 / S::kElem), at * S::kBoxRows, bar,
                         policy);
      }
    }
    ++issued;
    if (++put == ST) put = 0;
  };
  // a segment's query rows are loaded a segment ahead; the first one's before
  // the table entries that the copies wait for
  uint4 raw[D / 32];
  uint16_t* rows = reinterpret_cast<uint16_t*>(smem + S::kRows + size_t(warp) * S::kQBytes);
  rot::AngleTable<D>* table = reinterpret_cast<rot::AngleTable<D>*>(rows + kMaxGroup * S::kQRow);
  int64_t* freqs = reinterpret_cast<int64_t*>(smem + S::kFreqs);
  int turned = -1;            // the sequence whose angles the table holds
  auto fetch_q = [&](int qb, int qh) {
    if constexpr (ROT) {
      const int2 at = rot::item_columns(p.rot, lane % NJ);
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        const int r = i * (32 / NJ) + lane / NJ;
        const T* row = static_cast<const T*>(p.q) + qb * p.q_stride + (qh * G + r) * D;
        raw[2 * i] = raw[2 * i + 1] = make_uint4(0, 0, 0, 0);
        if (r < G) {
          raw[2 * i] = *reinterpret_cast<const uint4*>(row + at.x);
          raw[2 * i + 1] = *reinterpret_cast<const uint4*>(row + at.y);
        }
      }
    } else {
      load_q<T, Q8, D>(static_cast<const T*>(p.q) + (size_t(qb) * p.num_q_heads + qh * G + g) * D, g < G, t, raw);
    }
  };
  int64_t first_freqs[ROT ? D / 64 : 1];
  if (count > 0) {
    fetch_q(start.x, start.y);
    if constexpr (ROT) rot::WarpAngles<D>::load_freqs(p.rot, lane, first_freqs);
    fill();
  }
  for (int i = 0; i < ST && issued < count; ++i) issue();
  if constexpr (ROT) {
    // (every warp of the CTA writes the same, and a lane reads what it wrote:
    // the loop has no registers to spare for them)
    if (count > 0) {
#pragma unroll
      for (int i = 0; i < D / 64; ++i) freqs[rot::WarpAngles<D>::pair_of(lane, i)] = first_freqs[i];
    }
  }

  // ---- the warp's segments: runs of blocks of one (sequence, KV head)
  int b = start.x, h = start.y, v = start.z;
  int4 seq = start_seq;
  int get = 0, parity = 0, done = 0;  // done: blocks taken from the ring
  bool ok = planned;
  float ks = 0.f, lvs = 0.f;  // lane j: K scale and log2 of V's of block 32 c + j
  bool joined = false;        // a stage was written to (fused append)
  Piece<D>* tail = reinterpret_cast<Piece<D>*>(ring);
  if (lane == 0) head_pieces[warp].used = 0;
  bool has_tail = false;
  while (done < count) {
    const Range range = visible_range(seq.x, p.window, p.num_sinks);
    const int run = min(seq.y - v, count - done);
    const bool starts = v == 0, ends = v + run == seq.y;
    uint32_t qf[S::kSteps][2];
    int qexp;
    if constexpr (ROT) {
      __syncwarp();  // (the last segment's rows are read)
      if (turned != b) {
        rot::WarpAngles<D> angles;
        int64_t f[D / 64];
#pragma unroll
        for (int i = 0; i < D / 64; ++i) f[i] = freqs[rot::WarpAngles<D>::pair_of(lane, i)];
        angles.set(f, p.positions ? p.positions[b] : seq.x - 1, p.rot.magnitude);
        table->put(angles, lane);
        turned = b;
        __syncwarp();
      }
      float c[8], sn[8];
      table->get(lane % NJ, c, sn);
      const int2 at = rot::item_columns(p.rot, lane % NJ);
      float x[D / 64][16];
      int e[D / 64] = {};
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        if (i * (32 / NJ) >= G) break;
        rot::Chunk<T> u, w;
        u.v[0] = raw[2 * i];
        w.v[0] = raw[2 * i + 1];
        u.to_float(x[i]);
        w.to_float(x[i] + 8);
        if (16 * (lane % NJ) < p.rot.dim) rot::turn_item(p.rot.interleaved, x[i], c, sn);
        const int r = i * (32 / NJ) + lane / NJ;
        e[i] = place_q<NJ, kRest>(x[i], rows + r * S::kQRow, at, r < G);
        if (fold && r < G) {
          rot::Chunk<__half> a, z;
          a.from_float(x[i]);
          z.from_float(x[i] + 8);
          a.store(reinterpret_cast<__half*>(rows + (r + 4) * S::kQRow + at.x));
          z.store(reinterpret_cast<__half*>(rows + (r + 4) * S::kQRow + at.y));
        }
      }
      __syncwarp();
      const int row = fold && g >= 4 ? g - 4 : g;  // the head of this lane's column
      auto fragments = [&](uint4 (&w)[D / 32]) {
        load_q<__half, Q8, D>(reinterpret_cast<const __half*>(rows + g * S::kQRow), row < G, t, w);
      };
      fragments(raw);
      convert_q<__half, Q8, D>(raw, qf);
      // its exponent: item 0 of the row has it
      qexp = __shfl_sync(0xffffffffu, e[0], (row % (32 / NJ)) * NJ);
      if constexpr (D == 128) {
        const int high = __shfl_sync(0xffffffffu, e[D / 64 - 1], (row % (32 / NJ)) * NJ);
        if (row >= 32 / NJ) qexp = high;
      }
      if constexpr (kRest && !fold) {
        // the rests as fragments, each lane's together
        __syncwarp();
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          if (i * (32 / NJ) >= G) break;
          uint16_t* to = rows + (i * (32 / NJ) + lane / NJ) * S::kQRow;
          rot::Chunk<__half> u, w;
          u.from_float(x[i]);
          w.from_float(x[i] + 8);
          u.store(reinterpret_cast<__half*>(to + at.x));
          w.store(reinterpret_cast<__half*>(to + at.y));
        }
        __syncwarp();
        fragments(raw);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < D / 32; ++i) reinterpret_cast<uint4*>(rows)[i * 32 + lane] = raw[i];
      }
    } else {
      qexp = convert_q<T, Q8, D>(raw, qf);
    }
    // the next segment: the sequence's next head, or the next sequence that
    // has tokens
    int nb = b, nh = h + 1;
    int4 nseq = seq;
    if (run < count - done) {
      if (nh == Hkv) {
        nh = 0;
        do nseq = p.seqs[++nb];
        while (nseq.y == 0);
      }
      fetch_q(nb, nh);
    }
    float f0 = p.scale_log2, f1 = p.scale_log2;
    if constexpr (Q8) {
      f0 *= __uint_as_float(uint32_t(127 + __shfl_sync(0xffffffffu, qexp, 8 * t)) << 23);
      f1 *= __uint_as_float(uint32_t(127 + __shfl_sync(0xffffffffu, qexp, 8 * t + 4)) << 23);
    }
    // the sequence's new token, K by lanes 0 - 15 and V by 16 - 31, its block
    // (-1: not to be stored) and the block's scale, on their way while the
    // segment runs.  A length that is not the planned one stores nothing (the
    // plan cuts what the table cannot hold, and flags it).
    q8::Row8<T> fresh;
    int own = -1;
    float old = 0.f;
    if constexpr (APPEND) {
      if (ends) {
        if ((lane & 15) < D / 8)
          fresh.load(static_cast<const T*>(lane >> 4 ? p.new_rows[1] : p.new_rows[0]) +
                     (ROT ? b * (lane >> 4 ? p.new_stride[1] : p.new_stride[0]) + h * D
                          : int64_t((size_t(b) * Hkv + h) * D)) +
                     8 * (lane & 15));
        const int length = p.context_lens[b];
        const int phys = p.block_tables[size_t(b) * p.max_blocks + (seq.x - 1) / kBlockSize];
        if (length != seq.x) {
          if (length <= p.max_blocks * kBlockSize && lane == 0) dev::flag_status(p.status, kStatusPlan);
        } else if (phys >= 0 && phys < p.num_blocks) {
          own = phys * Hkv + h;
          old = (lane >> 4 ? p.v_scale : p.k_scale)[own];
        }
      }
    }
    float o[S::kSteps][4];
#pragma unroll
    for (int m = 0; m < S::kSteps; ++m) o[m][0] = o[m][1] = o[m][2] = o[m][3] = 0.f;
    // per head (2t, 2t + 1): reference of the scores, of the weights, and
    // this lane's part of the softmax's sum
    float m0 = -INFINITY, m1 = -INFINITY, w0 = -INFINITY, w1 = -INFINITY, l0 = 0.f, l1 = 0.f;

    // N blocks at once: their products interleave, and the wait, the vote and
    // the loop are paid once
    auto take = [&](auto number) -> bool {
      constexpr int N = decltype(number)::value;
      uint32_t kt[N];
      float x[N][4], lv[N];
      uint32_t keep[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (!dev::mbar_wait_bounded(&full[get], parity, tmo, p.status)) ok = false;
        kt[i] = dev::smem_u32(ring + get * S::kStage);
        if (++get == ST) {
          get = 0;
          parity ^= 1;
        }
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return false;
      float bks[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        lv[i] = 0.f;
        bks[i] = 1.f;
        if constexpr (Q8) {
          if ((done & 31) == 0) {
            ks = next_ks;
            lvs = log2_scale(next_vs);
          }
          bks[i] = __shfl_sync(0xffffffffu, ks, done & 31);
          lv[i] = __shfl_sync(0xffffffffu, lvs, done & 31);
        }
        ++done;
      }
      // ---- S^T = K Q^T, each block's in two chains
      float s[N][4], s2[N][4];
#pragma unroll
      for (int i = 0; i < N; ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[i][e] = s2[i][e] = 0.f;
        uint32_t f[S::kSteps][4];
        load_k<Q8, D>(kt[i], g, t, f);
#pragma unroll
        for (int k = 0; k < S::kSteps; k += 2) {
          Mm::run(s[i], f[k][0], f[k][1], f[k][2], f[k][3], qf[k][0], qf[k][1]);
          Mm::run(s2[i], f[k + 1][0], f[k + 1][1], f[k + 1][2], f[k + 1][3], qf[k + 1][0], qf[k + 1][1]);
          if constexpr (kRest && !fold) {
            // (convert_q's order: two steps to 16 bytes)
            const uint4 w = reinterpret_cast<const uint4*>(rows)[k / 2 * 32 + lane];
            Mm::run(s[i], f[k][0], f[k][1], f[k][2], f[k][3], w.x, w.y);
            Mm::run(s2[i], f[k + 1][0], f[k + 1][1], f[k + 1][2], f[k + 1][3], w.z, w.w);
          }
        }
      }
      // ---- base-2 scores of tokens t0 + g (x[0], x[1]) and t0 + g + 8
      // (x[2], x[3]), heads 2t and 2t + 1
      float top0 = -INFINITY, top1 = -INFINITY, high0 = -INFINITY, high1 = -INFINITY;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if constexpr (fold) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[i][e] += s2[i][e];
            s2[i][e] = __shfl_xor_sync(0xffffffffu, s[i][e], 2);
          }
        }
        const float c0 = Q8 ? f0 * bks[i] : f0, c1 = Q8 ? f1 * bks[i] : f1;
        x[i][0] = (s[i][0] + s2[i][0]) * c0;
        x[i][1] = (s[i][1] + s2[i][1]) * c1;
        x[i][2] = (s[i][2] + s2[i][2]) * c0;
        x[i][3] = (s[i][3] + s2[i][3]) * c1;
        keep[i] = 15;
        const int t0 = (v + i < range.first ? v + i : v + i + range.skip) * kBlockSize;
        if (t0 + kBlockSize > seq.x || (t0 < range.low && t0 + kBlockSize > range.sinks)) {
          auto sees = [&](int r) {
            return t0 + r < seq.x && (t0 + r >= range.low || t0 + r < range.sinks);
          };
          if (!sees(g)) x[i][0] = x[i][1] = -INFINITY;
          if (!sees(g + 8)) x[i][2] = x[i][3] = -INFINITY;
          keep[i] = uint32_t(sees(2 * t)) | uint32_t(sees(2 * t + 1)) << 1 |
                    uint32_t(sees(2 * t + 8)) << 2 | uint32_t(sees(2 * t + 9)) << 3;
        }
        const float a0 = fmaxf(x[i][0], x[i][2]), a1 = fmaxf(x[i][1], x[i][3]);
        top0 = fmaxf(top0, a0);
        top1 = fmaxf(top1, a1);
        if constexpr (Q8) {
          high0 = fmaxf(high0, a0 + lv[i]);
          high1 = fmaxf(high1, a1 + lv[i]);
        }
      }
      // ---- references
      bool grow = top0 > m0 + kRescale || top1 > m1 + kRescale;
      if constexpr (Q8) grow = grow || high0 > w0 + kRescale || high1 > w1 + kRescale;
      if (__any_sync(0xffffffffu, grow)) {
        auto all_max = [](float a) {
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
          return a;
        };
        // (a reference of -inf stands for nothing yet: the sums are zero)
        auto raise = [](float& ref, float to) {
          const float old = ref;
          ref = fmaxf(ref, to);
          return old == -INFINITY ? 0.f : dev::fast_exp2(old - ref);
        };
        const float n0 = all_max(top0), n1 = all_max(top1);
        l0 *= raise(m0, n0);
        l1 *= raise(m1, n1);
        const float a0 = raise(w0, Q8 ? all_max(high0) : n0);
        const float a1 = raise(w1, Q8 ? all_max(high1) : n1);
#pragma unroll
        for (int m = 0; m < S::kSteps; ++m) {
          o[m][0] *= a0;
          o[m][1] *= a1;
          o[m][2] *= a0;
          o[m][3] *= a1;
        }
      }
      // (the softmax's sum is lifted like the weights, so the lift divides out)
      const float r0 = m0 == -INFINITY ? 0.f : m0 - S::kLift, r1 = m1 == -INFINITY ? 0.f : m1 - S::kLift;
      uint32_t b0[N], b1[N], e0[N], e1[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float p0 = dev::fast_exp2(x[i][0] - r0), p1 = dev::fast_exp2(x[i][1] - r1);
        float p2 = dev::fast_exp2(x[i][2] - r0), p3 = dev::fast_exp2(x[i][3] - r1);
        l0 += p0 + p2;
        l1 += p1 + p3;
        if constexpr (Q8) {
          // the weights carry the block's value scale: 2^(x + log2 scale),
          // kept near 2^kLift by a reference of their own, so f16 holds them
          // whatever the scales are
          const float d0 = lv[i] - (w0 == -INFINITY ? 0.f : w0 - S::kLift);
          const float d1 = lv[i] - (w1 == -INFINITY ? 0.f : w1 - S::kLift);
          p0 = dev::fast_exp2(x[i][0] + d0);
          p1 = dev::fast_exp2(x[i][1] + d1);
          p2 = dev::fast_exp2(x[i][2] + d0);
          p3 = dev::fast_exp2(x[i][3] + d1);
        }
        // to the tensor cores' 16-bit type, transposed so that the tokens are
        // the contraction
        const uint32_t first = Mm::pack(p0, p1), second = Mm::pack(p2, p3);
        b0[i] = dev::movmatrix_trans(first);
        b1[i] = dev::movmatrix_trans(second);
        if constexpr (kTwoParts) {
          // what the rounding left over, rounded in turn
          const float2 a = Mm::unpack(first), c = Mm::unpack(second);
          e0[i] = dev::movmatrix_trans(Mm::pack(p0 - a.x, p1 - a.y));
          e1[i] = dev::movmatrix_trans(Mm::pack(p2 - c.x, p3 - c.y));
        }
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        uint32_t f[S::kSteps][4];
        load_v<Q8, D>(kt[i] + S::kTile, g, t, keep[i], f);
#pragma unroll
        for (int m = 0; m < S::kSteps; ++m) Mm::run(o[m], f[m][0], f[m][1], f[m][2], f[m][3], b0[i], b1[i]);
        if constexpr (kTwoParts) {
#pragma unroll
          for (int m = 0; m < S::kSteps; ++m) Mm::run(o[m], f[m][0], f[m][1], f[m][2], f[m][3], e0[i], e1[i]);
        }
      }
      v += N;
      // the stages are read: their next blocks
      if constexpr (APPEND) {
        // (writes to them come before the copies)
        if (joined) dev::fence_proxy_async_smem();
        joined = false;
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (issued < count) issue();
      return true;
    };
    // the new token into the sequence's last block, n - 1 blocks ahead of the
    // next to be taken; its scales where take() looks for them
    auto join = [&](int n) {
      const int stage = get + n - 1 < ST ? get + n - 1 : get + n - 1 - ST;
      ok = __all_sync(0xffffffffu, dev::mbar_wait_bounded(&full[stage], parity ^ int(stage < get), tmo, p.status));
      if (!ok) return;
      float now;
      if constexpr (ROT)
        now = append_row<float, D>(p, ring + stage * S::kStage, size_t(own), (seq.x - 1) & 15, old,
                                   rotate_row<T, D>(p, fresh, *table));
      else
        now = append_row<T, D>(p, ring + stage * S::kStage, size_t(own), (seq.x - 1) & 15, old, fresh);
      const float now_k = __shfl_sync(0xffffffffu, now, 0), now_v = __shfl_sync(0xffffffffu, now, 16);
      const int x = done + n - 1;
      if (lane == (x & 31)) {
        if (((done - 1) >> 5) == (x >> 5)) {
          ks = now_k;
          lvs = log2_scale(now_v);
        } else {
          next_ks = now_k;
          next_vs = now_v;
        }
      }
      joined = true;
      __syncwarp();
    };
    int left = run;
    // (with a second product one block at a time: two leave too few registers,
    // 8 heads per KV head in f16 58.4 us and 61.3)
    constexpr bool kPairs = !(kRest && !fold);
    if constexpr (kPairs) {
      for (; left >= 2 && ok; left -= 2) {
        if constexpr (APPEND) {
          if (left == 2 && own >= 0) join(2);
          if (!ok) break;
        }
        take(std::integral_constant<int, 2>());
      }
    }
    for (; left && ok; --left) {
      if constexpr (APPEND) {
        if (left == 1 && own >= 0) join(1);
      }
      if (ok) take(std::integral_constant<int, 1>());
    }
    if (!ok) break;

    // ---- end of the segment: sums over the 8 lanes that share a head
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, off);
      l1 += __shfl_xor_sync(0xffffffffu, l1, off);
    }
    if (starts && ends) {
      const float i0 = l0 != 0.f ? dev::fast_exp2(Q8 ? w0 - m0 : 0.f) / l0 : 0.f;
      const float i1 = l1 != 0.f ? dev::fast_exp2(Q8 ? w1 - m1 : 0.f) / l1 : 0.f;
      T* base = static_cast<T*>(p.out) + (size_t(b) * p.num_q_heads + h * G) * D;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (2 * t + k >= G) continue;
        const float inv = k ? i1 : i0;
        T* row = base + (2 * t + k) * D;
#pragma unroll
        for (int m = 0; m < S::kSteps; m += 4) {
          uint32_t x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = dev::Mma<T>::pack(o[m + e][k] * inv, o[m + e][2 + k] * inv);
          *reinterpret_cast<uint4*>(row + dim_of<Q8, D>(g, m)) = make_uint4(x[0], x[1], x[2], x[3]);
        }
      }
    } else {
      Piece<D>* piece = starts ? tail : &head_pieces[warp];
      if (starts) has_tail = true;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (2 * t + k >= G) continue;
#pragma unroll
        for (int m = 0; m < S::kSteps; ++m)
          *reinterpret_cast<float2*>(&piece->o[2 * t + k][dim_of<Q8, D>(g, m)]) =
              make_float2(o[m][k], o[m][2 + k]);
        if (g == 0) {
          piece->m[2 * t + k] = k ? m1 : m0;
          piece->w[2 * t + k] = k ? w1 : w0;
          piece->l[2 * t + k] = k ? l1 : l0;
        }
      }
      if (lane == 0) {
        piece->id = b * Hkv + h;
        piece->ends = ends;
        piece->used = 1;
        const int f = seq.z * Hkv + h * seq.w + kSegmentCost;  // its first block's place
        piece->c0 = f / share;
        piece->ctas = (f + seq.y - 1) / share - f / share + 1;
      }
    }
    v = 0;
    b = nb;
    h = nh;
    seq = nseq;
  }
  if (!ok) {
    // a wait ran out: let this warp's copies in flight land, then give up
    for (int k = max(0, issued - ST); k < issued; ++k) {
      const int st = k % ST;
      dev::mbar_wait_bounded(&full[st], (k / ST) & 1, tmo, p.status);
    }
  }
  // ---- sequences cut between the CTA's warps: their pieces lie in a run of
  // warps (a last piece, or for one that an earlier CTA began the first
  // warp's, then first pieces), each of which merges a slice of the columns.
  // One cut between CTAs too goes to the workspace.
  int* s_tail = reinterpret_cast<int*>(smem + S::kFlags);
  int *s_open = s_tail + kWarps, *s_merge = s_open + 2;
  if (lane == 0) s_tail[warp] = has_tail;
  if (threadIdx.x < 2) s_open[threadIdx.x] = s_merge[threadIdx.x] = -1;
  if (!__syncthreads_and(ok)) {
    // a wait ran out: the pieces of this CTA are missing, and those of others
    // stay counted (`arrivals`), so no later run may use the plan
    if (threadIdx.x == 0 && planned) atomicExch(&p.header[kHdrSignature], 0);
    return;
  }
  // bit w: warp w has a last piece, a first piece, a first piece that ends its
  // sequence
  const uint32_t tails = __ballot_sync(0xffffffffu, lane < kWarps && s_tail[lane % kWarps]);
  const uint32_t heads = __ballot_sync(0xffffffffu, lane < kWarps && head_pieces[lane % kWarps].used);
  const uint32_t ending =
      __ballot_sync(0xffffffffu, lane < kWarps && head_pieces[lane % kWarps].used && head_pieces[lane % kWarps].ends);
  auto last_piece = [&](int w) { return reinterpret_cast<const Piece<D>*>(smem + size_t(w) * ST * S::kStage); };
  // the run of pieces that begins in warp `from`: it goes on through the first
  // pieces of the warps behind until one ends the sequence or has none
  auto merge = [&](int from, bool from_tail) {
    const Piece<D>* first = from_tail ? last_piece(from) : &head_pieces[from];
    const int id = first->id;
    bool ends = first->ends;
    int last = from;
    if (!ends) {
      const uint32_t more = ~heads >> (from + 1), stop = ending >> (from + 1);  // (bit kWarps of ~heads is set)
      const int without = __ffs(more) - 1, with = stop ? __ffs(stop) - 1 : 32;
      ends = with < without;
      last = from + (ends ? with + 1 : without);
    }
    const bool whole = from_tail && ends;
    Piece<D>* slot = static_cast<Piece<D>*>(p.pieces) + size_t(blockIdx.x) * 2 + (from_tail ? 1 : 0);
    const int n = last - from + 1;
    for (int i = (warp - from) * 32 + lane; i < G * D / 4; i += 32 * n) {
      const int head = i / (D / 4), d = (i % (D / 4)) * 4;
      auto nth = [&](int j) { return j ? &head_pieces[from + j] : first; };
      float m = -INFINITY, w = -INFINITY;
#pragma unroll 4
      for (int j = 0; j < n; ++j) {
        m = fmaxf(m, nth(j)->m[head]);
        w = fmaxf(w, nth(j)->w[head]);
      }
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
      float l = 0.f;
#pragma unroll 4
      for (int j = 0; j < n; ++j) {
        const Piece<D>* x = nth(j);
        const float a = x->w[head] == -INFINITY ? 0.f : dev::fast_exp2(x->w[head] - w);
        const float4 y = *reinterpret_cast<const float4*>(&x->o[head][d]);
        sum.x += a * y.x;
        sum.y += a * y.y;
        sum.z += a * y.z;
        sum.w += a * y.w;
        l += x->m[head] == -INFINITY ? 0.f : dev::fast_exp2(x->m[head] - m) * x->l[head];
      }
      if (whole) {
        const float inv = l != 0.f ? dev::fast_exp2(Q8 ? w - m : 0.f) / l : 0.f;
        T* row = static_cast<T*>(p.out) + (size_t(id / Hkv) * p.num_q_heads + id % Hkv * G + head) * D + d;
        *reinterpret_cast<uint2*>(row) = make_uint2(dev::Mma<T>::pack(sum.x * inv, sum.y * inv),
                                                    dev::Mma<T>::pack(sum.z * inv, sum.w * inv));
      } else {
        *reinterpret_cast<float4*>(&slot->o[head][d]) = sum;
        if (d == 0) {
          slot->m[head] = m;
          slot->w[head] = w;
          slot->l[head] = l;
        }
      }
    }
    if (!whole && warp == from && lane == 0) s_open[from_tail ? 1 : 0] = from;
  };
  if (heads >> warp & 1) {
    // it goes on from the nearest last piece before it, or from an earlier CTA
    const uint32_t before = tails & ((1u << warp) - 1);
    merge(before ? 31 - __clz(before) : 0, before != 0);
  }
  if (has_tail) merge(warp, true);
  __syncthreads();

  // ---- the last CTA to arrive at a sequence cut between CTAs merges it
  // (ends of the CTA that are open, by the warp in which their pieces begin)
  const int open0 = s_open[0], open1 = s_open[1];
  if (open0 < 0 && open1 < 0) return;
  if (lane == 0 && warp < 2) {
    const int from = warp ? open1 : open0;
    if (from >= 0) {
      const Piece<D>* x = warp ? last_piece(from) : &head_pieces[from];
      if (dev::atom_add_acq_rel_gpu(&p.arrivals[x->c0], 1) == x->ctas - 1) {
        p.arrivals[x->c0] = 0;  // ready for the next run
        s_merge[warp] = from;
      }
    }
  }
  __syncthreads();
  const int merge0 = s_merge[0], merge1 = s_merge[1];
  if (merge0 < 0 && merge1 < 0) return;
  const Piece<D>* left = merge0 < 0 ? nullptr : &head_pieces[merge0];
  const Piece<D>* right = merge1 < 0 ? nullptr : last_piece(merge1);
  const int left_id = left ? left->id : -1, left_c0 = left ? left->c0 : 0, left_n = left ? left->ctas : 0;
  const int right_id = right ? right->id : -1, right_c0 = right ? right->c0 : 0, right_n = right ? right->ctas : 0;
  __syncthreads();  // (the weights below overwrite the rings)
  for (int side = 0; side < 2; ++side) {
    const int id = side ? right_id : left_id, c0 = side ? right_c0 : left_c0, n = side ? right_n : left_n;
    if (id < 0) continue;
    // piece k is CTA c0 + k's: its later end for k == 0, its earlier one else
    const Piece<D>* all = static_cast<const Piece<D>*>(p.pieces) + size_t(c0) * 2 + 1;
    auto nth = [&](int k) { return k ? all + 2 * k - 1 : all; };
    float* wsm = reinterpret_cast<float*>(smem);  // [n][8] weights, in the rings' place
    // the columns' first pieces are on their way while the weights are made
    const int head = threadIdx.x / (D / 4), d = (threadIdx.x % (D / 4)) * 4;
    const bool mine = threadIdx.x < G * D / 4;  // kThreads >= 8 D / 4
    constexpr int kAhead = 4;
    float4 ahead[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (mine && k < n) ahead[k] = __ldcg(reinterpret_cast<const float4*>(&nth(k)->o[head][d]));
    if (warp < G) {  // one warp per head
      float m = -INFINITY, w = -INFINITY, l = 0.f;
      float pm = -INFINITY, pw = -INFINITY, pl = 0.f;  // piece `lane`'s
      if (lane < n) {
        pm = __ldcg(&nth(lane)->m[warp]);
        pw = __ldcg(&nth(lane)->w[warp]);
        pl = __ldcg(&nth(lane)->l[warp]);
        m = pm;
        w = pw;
      }
      for (int k = lane + 32; k < n; k += 32) {
        m = fmaxf(m, __ldcg(&nth(k)->m[warp]));
        w = fmaxf(w, __ldcg(&nth(k)->w[warp]));
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, off));
      }
      l = pm == -INFINITY ? 0.f : dev::fast_exp2(pm - m) * pl;
      for (int k = lane + 32; k < n; k += 32) {
        const float x = __ldcg(&nth(k)->m[warp]);
        l += x == -INFINITY ? 0.f : dev::fast_exp2(x - m) * __ldcg(&nth(k)->l[warp]);
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
      const float inv = l != 0.f ? dev::fast_exp2(Q8 ? w - m : 0.f) / l : 0.f;
      if (lane < n) wsm[lane * kMaxGroup + warp] = pw == -INFINITY ? 0.f : dev::fast_exp2(pw - w) * inv;
      for (int k = lane + 32; k < n; k += 32) {
        const float x = __ldcg(&nth(k)->w[warp]);
        wsm[k * kMaxGroup + warp] = x == -INFINITY ? 0.f : dev::fast_exp2(x - w) * inv;
      }
    }
    __syncthreads();
    if (mine) {
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
      auto add = [&](int k, const float4& y) {
        const float a = wsm[k * kMaxGroup + head];
        sum.x += a * y.x;
        sum.y += a * y.y;
        sum.z += a * y.z;
        sum.w += a * y.w;
      };
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (k < n) add(k, ahead[k]);
#pragma unroll 8
      for (int k = kAhead; k < n; ++k) add(k, __ldcg(reinterpret_cast<const float4*>(&nth(k)->o[head][d])));
      T* row = static_cast<T*>(p.out) + (size_t(id / Hkv) * p.num_q_heads + id % Hkv * G + head) * D + d;
      *reinterpret_cast<uint2*>(row) =
          make_uint2(dev::Mma<T>::pack(sum.x, sum.y), dev::Mma<T>::pack(sum.z, sum.w));
    }
    __syncthreads();  // the weights are read
  }
}

constexpr int kMaxDevices = 64;

struct DeviceState {
  std::once_flag once;
  int error = 0;
  int sms = 0;
};
DeviceState g_dev[kMaxDevices];

template <typename T, bool Q8, int D>
cudaError_t configure() {
  const int bytes = int(Tiles<T, Q8, D>::kBytes);
  cudaError_t e = cudaFuncSetAttribute(attend_kernel<T, Q8, D, false, false, false>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if constexpr (Q8) {
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(attend_kernel<T, Q8, D, true, false, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               bytes);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(attend_kernel<T, Q8, D, true, true, false>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, int(Tiles<T, Q8, D, true>::kBytes));
    if (e == cudaSuccess && std::is_same<T, __half>::value)
      e = cudaFuncSetAttribute(attend_kernel<T, Q8, D, true, true, std::is_same<T, __half>::value>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, int(Tiles<T, Q8, D, true>::kBytes));
  }
  return e;
}

int device_setup(int* ncta, const char* who) {
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess || device < 0 || device >= kMaxDevices)
    return fail(PA_ERR_CUDA, "%s: no current CUDA device", who);
  DeviceState& st = g_dev[device];
  std::call_once(st.once, [&] {
    cudaError_t e = cudaDeviceGetAttribute(&st.sms, cudaDevAttrMultiProcessorCount, device);
    if (e == cudaSuccess) e = configure<__half, false, 64>();
    if (e == cudaSuccess) e = configure<__half, false, 128>();
    if (e == cudaSuccess) e = configure<__nv_bfloat16, false, 64>();
    if (e == cudaSuccess) e = configure<__nv_bfloat16, false, 128>();
    if (e == cudaSuccess) e = configure<__half, true, 64>();
    if (e == cudaSuccess) e = configure<__half, true, 128>();
    if (e == cudaSuccess) e = configure<__nv_bfloat16, true, 64>();
    if (e == cudaSuccess) e = configure<__nv_bfloat16, true, 128>();
    st.error = e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
  });
  if (st.error != PA_OK) return fail(st.error, "%s: per-device set-up failed on device %d", who, device);
  *ncta = st.sms < kMaxCtas ? st.sms : kMaxCtas;
  return PA_OK;
}

int signature_of(int window, int num_sinks, int num_seqs, int num_q_heads, int num_kv_heads,
                 int head_dim, int max_blocks, int ncta) {
  uint32_t h = 2166136261u;
  const int v[9] = {window, num_sinks, num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks, ncta, 0x51D3};
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
  bool append = false;
  const void *k_new = nullptr, *v_new = nullptr;
  rot::Args rot = {};  // freqs null: none
  const int32_t* positions = nullptr;
  int64_t q_stride = 0, k_stride = 0, v_stride = 0;
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
      double(num_seqs) * num_kv_heads * (double(max_blocks) + kMinPlaces) >= 2147483647.0 ||
      double(num_seqs) * num_q_heads >= 2147483647.0)
    return fail(PA_ERR_INVALID_ARG, "%s: sizes too large for the workspace", who);
  return PA_OK;
}

template <typename T, bool Q8, int D>
cudaError_t launch_attend(cudaLaunchConfig_t cfg, const CUtensorMap& mk, const CUtensorMap& mv,
                          const Params& p) {
  cfg.gridDim = dim3(unsigned(p.ncta));
  cfg.blockDim = dim3(Tiles<T, Q8, D>::kThreads);
  cfg.dynamicSmemBytes = Tiles<T, Q8, D>::kBytes;
  if constexpr (Q8) {
    if (p.rot.freqs) {
      cfg.dynamicSmemBytes = Tiles<T, Q8, D, true>::kBytes;
      if (std::is_same<T, __half>::value && p.group <= 4)
        return cudaLaunchKernelEx(&cfg, attend_kernel<T, Q8, D, true, true, std::is_same<T, __half>::value>, mk, mv,
                                  p);
      return cudaLaunchKernelEx(&cfg, attend_kernel<T, Q8, D, true, true, false>, mk, mv, p);
    }
    if (p.new_rows[0]) return cudaLaunchKernelEx(&cfg, attend_kernel<T, Q8, D, true, false, false>, mk, mv, p);
  }
  return cudaLaunchKernelEx(&cfg, attend_kernel<T, Q8, D, false, false, false>, mk, mv, p);
}

template <typename T, bool Q8>
cudaError_t launch_attend(const cudaLaunchConfig_t& cfg, int head_dim, const CUtensorMap& mk,
                          const CUtensorMap& mv, const Params& p) {
  return head_dim == 128 ? launch_attend<T, Q8, 128>(cfg, mk, mv, p)
                         : launch_attend<T, Q8, 64>(cfg, mk, mv, p);
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
    if (c.append && (!c.k_new || !c.v_new)) return fail(PA_ERR_INVALID_ARG, "%s: NULL pointer", who);
    for (const void* ptr : {c.q, c.k_cache, c.v_cache, static_cast<const void*>(c.out), c.k_new, c.v_new})
      if (reinterpret_cast<uintptr_t>(ptr) & 15)
        return fail(PA_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", who);
    if (c.num_blocks <= 0 || double(c.num_blocks) * c.num_kv_heads * kBlockSize >= 2147483647.0)
      return fail(PA_ERR_INVALID_ARG, "%s: bad num_blocks", who);
  }
  const Layout lay = workspace_layout(c.num_seqs, c.head_dim);
  if (!c.workspace || (reinterpret_cast<uintptr_t>(c.workspace) & 255))
    return fail(PA_ERR_INVALID_ARG, "%s: workspace must be non-NULL and 256-byte aligned", who);
  if (c.workspace_bytes < lay.total)
    return fail(PA_ERR_INVALID_ARG, "%s: workspace %zu bytes < %zu needed", who, c.workspace_bytes,
                lay.total);
  int ncta = 0;
  rc = device_setup(&ncta, who);
  if (rc != PA_OK) return rc;
  unsigned* status = device_status_word();
  if (!status) return PA_ERR_CUDA;
  Params p = {};
  p.q = c.q;
  p.k_cache = c.k_cache;
  p.v_cache = c.v_cache;
  p.k_scale = c.k_scale;
  p.v_scale = c.v_scale;
  if (c.append) {
    p.new_rows[0] = c.k_new;
    p.new_rows[1] = c.v_new;
    p.codes[0] = static_cast<uint8_t*>(const_cast<void*>(c.k_cache));
    p.codes[1] = static_cast<uint8_t*>(const_cast<void*>(c.v_cache));
    p.scales[0] = const_cast<float*>(c.k_scale);
    p.scales[1] = const_cast<float*>(c.v_scale);
  }
  p.rot = c.rot;
  p.positions = c.positions;
  p.q_stride = c.q_stride;
  p.new_stride[0] = c.k_stride;
  p.new_stride[1] = c.v_stride;
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
  p.head_dim = c.head_dim;
  p.ncta = ncta;
  p.scale = c.scale;
  p.scale_log2 = c.scale * 1.4426950408889634f;
  p.signature = signature_of(c.window, c.num_sinks, c.num_seqs, c.num_q_heads, c.num_kv_heads,
                             c.head_dim, c.max_blocks, ncta);
  uint8_t* ws = static_cast<uint8_t*>(c.workspace);
  p.header = reinterpret_cast<int*>(ws);
  p.seqs = reinterpret_cast<int4*>(ws + lay.seqs);
  // (the plan writes both warp counts' starts, a run reads its own)
  p.starts = reinterpret_cast<int4*>(ws + lay.starts);
  int4* q8_starts = p.starts + size_t(kMaxCtas) * warps_of(false, c.head_dim) * 2;
  p.arrivals = reinterpret_cast<int*>(ws + lay.arrivals);
  p.pieces = ws + lay.pieces;
  p.status = status;
  p.timeout_ns = 1000000000ull;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cudaLaunchConfig_t cfg = {};
  cfg.stream = static_cast<cudaStream_t>(c.stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (c.mode != Mode::kRunOnly) {
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kPlanThreads);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, plan_kernel, p);
    if (e != cudaSuccess) return fail(PA_ERR_CUDA, "%s: plan launch failed: %s", who, cudaGetErrorString(e));
  }
  if (!runs) return PA_OK;
  if (c.q8) p.starts = q8_starts;
  cudaError_t e;
  if (c.dtype == PA_F32) {
    cfg.gridDim = dim3(unsigned((c.num_seqs * c.num_q_heads + 3) / 4));
    cfg.blockDim = dim3(128);
    e = c.head_dim == 128 ? cudaLaunchKernelEx(&cfg, f32_kernel<128>, p)
                          : cudaLaunchKernelEx(&cfg, f32_kernel<64>, p);
  } else {
    alignas(64) CUtensorMap mk, mv;
    auto encode = [&](CUtensorMap* map, const void* cache) {
      return c.q8 ? q8_cache_tensor_map(map, cache, c.num_blocks, c.num_kv_heads, c.head_dim)
                  : cache_tensor_map(map, cache, c.dtype == PA_BF16, c.num_blocks, c.num_kv_heads,
                                     c.head_dim);
    };
    rc = encode(&mk, c.k_cache);
    if (rc == PA_OK) rc = encode(&mv, c.v_cache);
    if (rc != PA_OK) return rc;
    if (c.dtype == PA_F16)
      e = c.q8 ? launch_attend<__half, true>(cfg, c.head_dim, mk, mv, p)
               : launch_attend<__half, false>(cfg, c.head_dim, mk, mv, p);
    else
      e = c.q8 ? launch_attend<__nv_bfloat16, true>(cfg, c.head_dim, mk, mv, p)
               : launch_attend<__nv_bfloat16, false>(cfg, c.head_dim, mk, mv, p);
  }
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
  *bytes = window::workspace_layout(num_seqs, head_dim).total;
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

PA_API int pa_paged_attention_decode_q8_append_run(
    const void* q, const void* k_new, const void* v_new, void* k_cache, void* v_cache,
    float* k_scale, float* v_scale, const int32_t* block_tables, const int32_t* context_lens,
    int window, int num_sinks, int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
    int max_blocks_per_seq, int num_blocks, float scale, int dtype, void* out, void* workspace,
    size_t workspace_bytes, void* stream) {
  PA_TRACE("pa_paged_attention_decode_q8_append_run");
  return window::entry({"paged_attention_decode_q8_append_run", Mode::kRunOnly, true, q, k_cache,
                        v_cache, k_scale, v_scale, block_tables, context_lens, window, num_sinks,
                        num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq,
                        num_blocks, scale, dtype, out, workspace, workspace_bytes, stream, true,
                        k_new, v_new});
}

PA_API int pa_paged_attention_decode_q8_rotary_append_run(
    const void* q, const void* k_new, const void* v_new, const int32_t* positions,
    const int64_t* turns, int rotary_dim, int interleaved, float magnitude, void* k_cache,
    void* v_cache, float* k_scale, float* v_scale, const int32_t* block_tables,
    const int32_t* context_lens, int window, int num_sinks, int num_seqs, int num_q_heads,
    int num_kv_heads, int head_dim, int max_blocks_per_seq, int num_blocks, int64_t q_stride,
    int64_t k_stride, int64_t v_stride, float scale, int dtype, void* out, void* workspace,
    size_t workspace_bytes, void* stream) {
  PA_TRACE("pa_paged_attention_decode_q8_rotary_append_run");
  const char* who = "paged_attention_decode_q8_rotary_append_run";
  window::Call c = {who, Mode::kRunOnly, true, q, k_cache, v_cache, k_scale, v_scale, block_tables,
                    context_lens, window, num_sinks, num_seqs, num_q_heads, num_kv_heads, head_dim,
                    max_blocks_per_seq, num_blocks, scale, dtype, out, workspace, workspace_bytes,
                    stream, true, k_new, v_new};
  int rc = rot::check_stride(q_stride, 2, 0, "q_stride", who);
  if (rc == PA_OK) rc = rot::check_stride(k_stride, 2, 0, "k_stride", who);
  if (rc == PA_OK) rc = rot::check_stride(v_stride, 2, 0, "v_stride", who);
  if (rc == PA_OK && num_seqs > 0)
    rc = rot::check_args(turns, rotary_dim, interleaved, magnitude, head_dim, who, &c.rot);
  if (rc != PA_OK) return rc;
  c.positions = positions;
  c.q_stride = q_stride;
  c.k_stride = k_stride;
  c.v_stride = v_stride;
  return window::entry(c);
}

}  // extern "C"
