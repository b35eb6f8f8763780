// What the two kernels of tq_paged_attention share: the split of the work, and
// the join of its parts.
//
// The blocks of 32 tokens of all sequences and KV heads, in the order (sequence,
// head, block), are one line of U units, cut into equal shares, one per CTA,
// whatever the sequences' lengths; so a long sequence is spread over many CTAs
// and a CTA may hold several short ones.  What a CTA has of one (sequence, head)
// is a segment; it leaves the partial (m, l, o) of each of its segments in the
// workspace.  Segment (bh, CTA c) has slot bh + c: from one segment to the next
// bh or c or both grow, so no two share a slot.
#pragma once

#include "tq_device.cuh"
#include "tq_paged.h"

namespace tq {
namespace paged {

constexpr int kMinShare = 4;  // blocks: below 128 tokens a CTA's setup outweighs its work
constexpr int kMaxGroup = 16; // query heads per KV head

struct AttnArgs {
  Layout L;
  Table tab;
  const uint32_t* pool;
  int layer;
  const int32_t* lens;
  int B, Hq, G;
  float scale;
  const void* q;
  int dt;
  int64_t q_ld;
  void* out;
  float* lse;
  int ctas;              // of the main kernel
  int64_t* prefix;       // [B + 1]: blocks of the sequences before b
  float* qrot;           // [B * Hq][d_pad]
  float* u;              // [B * Hq][m]
  float* part;           // [slots][G][d_pad + 2]
  unsigned* err;
};

__device__ __forceinline__ int64_t share_of(const AttnArgs& A, int64_t units) {
  const int64_t s = (units + A.ctas - 1) / A.ctas;
  return s < kMinShare ? kMinShare : s;
}

struct Segment {
  int b, h, blk, end;  // blocks [blk, end) of (b, h)
  int len;             // tokens of the sequence
};

// The segment that unit u0 begins, cut at u1.
__device__ __forceinline__ Segment segment_at(const AttnArgs& A, int64_t u0, int64_t u1) {
  const int hkv = A.L.hkv;
  const int64_t x = u0 / hkv;
  int lo = 0, hi = A.B;  // prefix[lo] <= x < prefix[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (A.prefix[mid] <= x) lo = mid;
    else hi = mid;
  }
  const int64_t p = A.prefix[lo];
  const int n = (int)(A.prefix[lo + 1] - p);
  const int64_t rel = u0 - hkv * p;
  Segment s;
  s.b = lo;
  s.h = (int)(rel / n);
  s.blk = (int)(rel - (int64_t)s.h * n);
  s.end = (int)min64(n, s.blk + (u1 - u0));
  s.len = clamp_len(A.lens[lo], A.L, A.tab.max_pages);
  return s;
}

__device__ __forceinline__ float* slot_of(const AttnArgs& A, int64_t bh, int c, int head) {
  return A.part + ((bh + c) * A.G + head) * (int64_t)(A.L.dp + 2);
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

}  // namespace paged
}  // namespace tq
