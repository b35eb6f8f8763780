// What the kernels of tq_paged_attention share: the split of the work, and the
// join of its parts.
//
// The query heads of a KV head are taken in groups of at most `gh`; a KV head
// with its group is a virtual head, `hv` per sequence.  A unit is 4 blocks of 32
// tokens (fewer at a sequence's end) of one virtual head: what a warp's value
// pass takes at a time.  The units of all sequences and virtual heads, in the
// order (sequence, virtual head, blocks), are one line, cut into equal shares
// (within one unit), one per worker (a warp or a CTA), whatever the sequences'
// lengths; so a long sequence is spread over many workers and a worker may hold
// several short ones.  What a worker has of one (sequence, virtual head) is a
// segment; it leaves the partial (m, l, o) of each of its segments in the
// workspace, m as a power of two's exponent.  Segment (bh, worker c) has slot
// bh + c: from one segment to the next bh or c or both grow, so no two share a
// slot.
#pragma once

#include "tq_device.cuh"
#include "tq_paged.h"

namespace tq {
namespace paged {

constexpr int kUnit = 4;       // blocks
constexpr int kMaxGroup = 16; // query heads per KV head
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct AttnArgs {
  Layout L;
  Table tab;
  const uint32_t* pool;
  int layer;
  const int32_t* lens;
  int B, Hq, G;
  int hv, gh;            // virtual heads per sequence, query heads of one
  float scale2;          // scale log2(e)
  const void* q;
  int dt;
  int64_t q_ld;
  void* out;
  float* lse;
  int workers;           // of the main kernel
  int64_t* prefix;       // [B + 1]: units a head of the sequences before b
  float* qrot;           // [B * Hq][d_pad] (the kernel for any shape)
  float* u;              // [B * Hq][m]
  uint32_t* frag;        // [B * hv] query images (the tensor-core kernel)
  int frag_words;        // of one
  float* part;           // [slots][gh][4 + d_pad]: m, l, -, -, o
  unsigned* err;
};

// Worker c's share of `units` is [share_at(c), share_at(c + 1)): none is empty below min(units, workers).
__device__ __forceinline__ int64_t share_at(const AttnArgs& A, int64_t units, int64_t c) {
  const int64_t w = min64(units, A.workers);
  return c >= w ? units : c * units / w;
}
// The worker whose share unit x is in: the last c with c units / w < x + 1.
__device__ __forceinline__ int worker_of(const AttnArgs& A, int64_t units, int64_t x) {
  return (int)(((x + 1) * min64(units, A.workers) - 1) / units);
}

__device__ __forceinline__ int units_of(const AttnArgs& A, int64_t b) {
  return (int)(((unsigned)clamp_len(A.lens[b], A.L, A.tab.max_pages) + 32u * kUnit - 1u) / (32u * kUnit));
}

struct Segment {
  int b, h, blk, end;  // blocks [blk, end) of (sequence, virtual head)
  int kvh;             // its KV head
  int len;             // tokens of the sequence
};

// The segment from unit `rel` of sequence b on, which has n units a head, for a share of `left` more units.
__device__ __forceinline__ Segment segment_in(const AttnArgs& A, int b, int n, int64_t rel, int64_t left) {
  Segment s;
  s.b = b;
  s.h = (int)(rel / n);
  s.kvh = s.h / (A.hv / A.L.hkv);
  s.len = clamp_len(A.lens[b], A.L, A.tab.max_pages);
  const int first = (int)(rel - (int64_t)s.h * n);
  s.blk = kUnit * first;
  s.end = (int)min64((s.len + 31) / 32, kUnit * (first + min64(n, left)));
  return s;
}

// The segment that unit u0 begins, cut at u1, found in the units' prefix sums; called by a whole warp.
__device__ __forceinline__ Segment segment_at(const AttnArgs& A, int64_t u0, int64_t u1, int lane) {
  const int64_t x = u0 / A.hv;
  int lo = 0, n = A.B;  // the last b with prefix[b] <= x is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const bool le = lane * step < n && A.prefix[lo + lane * step] <= x;
    const int last = __popc(__ballot_sync(0xffffffffu, le)) - 1;
    lo += last * step;
    n = min(step, n - last * step);
  }
  const int64_t p = A.prefix[lo];
  return segment_in(A, lo, (int)(A.prefix[lo + 1] - p), u0 - A.hv * p, u1 - u0);
}

// The segment behind s, for a share that goes on from unit u0 to u1; n1: the units a head of the sequence behind it,
// read beforehand.
__device__ __forceinline__ Segment segment_after(const AttnArgs& A, const Segment& s, int n1, int64_t u0, int64_t u1) {
  int b = s.b, n = (int)(((unsigned)s.len + 32u * kUnit - 1u) / (32u * kUnit));
  int64_t rel = (int64_t)(s.h + 1) * n;
  if (s.h + 1 == A.hv) {
    rel = 0;
    ++b;
    for (n = n1; n == 0;) n = units_of(A, ++b);  // ends: a unit u0 < u1 <= units is some sequence's
  }
  return segment_in(A, b, n, rel, u1 - u0);
}

// Up to this many sequences a warp sums their units itself, and need not wait for the prefix sums.
constexpr int kOwnSums = 1024;

// A worker's first segment and its share [u0, u1) of the units from the lengths alone; B <= kOwnSums, a whole warp.
__device__ __forceinline__ Segment first_segment(const AttnArgs& A, int worker, int64_t& u0, int64_t& u1, int lane) {
  const int per = (A.B + 31) / 32, b0 = lane * per, b1 = min(A.B, b0 + per);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += units_of(A, b);
  long long upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  const int64_t units = __shfl_sync(0xffffffffu, upto, 31) * A.hv;
  u0 = share_at(A, units, worker);
  u1 = share_at(A, units, worker + 1);
  Segment s = {};
  if (u0 >= u1) return s;
  const long long x = u0 / A.hv, before = upto - mine;
  // the last lane whose sequences begin at or before x (it has units: the next lane's begin behind x)
  const int at = __popc(__ballot_sync(0xffffffffu, before <= x)) - 1;
  int b = at * per, n = 0;
  long long p = __shfl_sync(0xffffffffu, before, at);
  for (;; ++b) {
    n = units_of(A, b);
    if (p + n > x) break;
    p += n;
  }
  return segment_in(A, b, n, u0 - A.hv * p, u1 - u0);
}

__host__ __device__ __forceinline__ int part_row(int dp) { return dp + 4; }  // 16-byte rows

__device__ __forceinline__ float* slot_of(const AttnArgs& A, int64_t bh, int worker, int head) {
  return A.part + ((bh + worker) * A.gh + head) * (int64_t)part_row(A.L.dp);
}

__device__ __forceinline__ float load_q(const AttnArgs& A, int64_t i) {
  if (A.dt == TQ_F32) return static_cast<const float*>(A.q)[i];
  if (A.dt == TQ_F16) return __half2float(static_cast<const __half*>(A.q)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(A.q)[i]);
}
__device__ __forceinline__ void store_out(const AttnArgs& A, int64_t i, float v) {
  if (A.dt == TQ_F32) static_cast<float*>(A.out)[i] = v;
  else if (A.dt == TQ_F16) static_cast<__half*>(A.out)[i] = __float2half_rn(v);
  else static_cast<__nv_bfloat16*>(A.out)[i] = __float2bfloat16_rn(v);
}

// Whether the values' sums have to be as exact as fp32's: an output of 16 bits hides what is lost in them.
inline bool fine_sums(int dt) { return dt == TQ_F32; }

// The tensor-core kernel (tq_paged_attn_tc.cuh): what it needs to know of a
// shape, and its launch.  ctas == 0: not a shape of it.
struct TcShape {
  int ctas_per_sm = 0;
  int warps;       // of a CTA
  int nt;          // tiles of four heads of a virtual head
  int steps;       // MMA steps over q' and over u
  int smem;        // bytes of a CTA
};
TcShape tc_shape(int kk, int kv, int m, int dp, int G, bool fine);
cudaError_t tc_launch(const AttnArgs& a, const QParams& kq, const QParams& vq, const TcShape& s, int ctas, cudaStream_t st);

// Codebooks as the tensor-core kernel takes them.
struct TcBooks {
  float kalpha[4];      // odd-subset coefficients of the key codebook
  uint32_t hi[2], lo[2], th[2];  // bytes of the value levels, of 16 bits or (th too) of 24
  float unit;           // value of one step of them
};

}  // namespace paged
}  // namespace tq
