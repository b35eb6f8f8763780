// tq_paged_attention: one query token per sequence over a paged compressed
// cache (include/tq.h; the estimator and the rotated value average are those of
// tq_decode_attention).  Three launches: the queries' rotation and sketch with
// the split of the work, the attention over the segments, and the join.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "tq_attn_params.h"
#include "tq_paged_attn.cuh"

namespace tq {
namespace paged {
namespace {

inline bool al256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }

// ---------------------------------------------------------------- queries

constexpr float kQMax = 8323072.0f;  // 127 2^16, the largest entry in fixed point: three signed bytes hold it

// P_j of the tensor-core kernel's scores: x / 2^j as an integer.
__device__ __forceinline__ int place_value(float x, int j) {
  return __float2int_rn(x * __int_as_float((127 - j) << 23));
}

// Byte `piece` (0: hi, 1: mid, 2: lo) of v = 2^16 hi + 2^8 mid + lo, |v| <= 127 * 2^16, all three in [-128, 127].
__device__ __forceinline__ uint32_t digit(int v, int piece) {
  const int lo = ((v + 128) & 0xff) - 128;
  const int v1 = (v - lo) >> 8;  // exact
  const int mid = ((v1 + 128) & 0xff) - 128;
  return (uint32_t)((piece == 0 ? (v1 - mid) >> 8 : piece == 1 ? mid : lo) & 0xff);
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A head's numbers in fixed point, by a warp (A32 of them a lane, n in all, 32 a + lane): place values to `p`, and the
// score constants c[0] = 2 w / inv, c[1] = -w k / inv times the sum of what the place values hold (NaN where an entry is
// not finite; the images are then 0).
template <int A32>
__device__ __forceinline__ void fixed_point(const float (&x)[A32], int n, float w, float k, int* p, float* c, int lane) {
  float mx = 1e-30f, bad = 0.f;
#pragma unroll
  for (int a = 0; a < A32; ++a)
    if (32 * a < n) {
      mx = fmaxf(mx, fabsf(x[a]));
      bad = fmaf(x[a], 0.f, bad);
    }
  mx = warp_max(mx);
  bad = warp_sum(bad);
  const float inv = bad == 0.f ? kQMax / mx : 0.f;
  int sum = 0;  // |sum| < d_pad (kQMax + 2^2) < 2^31
#pragma unroll
  for (int a = 0; a < A32; ++a)
    if (32 * a < n) {
      const int v = place_value(x[a] * inv, lane & 3);  // coordinate j is bit j mod 4 of its half byte
      p[32 * a + lane] = v;
      sum += v << (lane & 3);
    }
  sum = __reduce_add_sync(0xffffffffu, sum);
  if (lane == 0) {
    const float u = w * (mx / kQMax);
    c[0] = 2.f * u;
    c[1] = bad == 0.f ? -u * k * (float)sum : bad;
  }
}

// Block (b, h): q' = H D q / sqrt(d_pad) and u = S q' of the query heads of KV
// head h, and, for h = 0, the units of the sequences before b.  With NT tiles
// of heads the images that the tensor-core kernel takes (its B operands, thread
// by thread, and four constants per head), with NT = 0 q' and u.
//
// A call of few sequences waits for this kernel's latency, so everything is
// spread over the block: a warp per head rotates and takes the fixed point, u's
// products (d_pad m G of them, S 32 KB in fp16 at d_pad = m = 128) go to the
// tensor cores, a warp per 16 rows of S with all its loads in flight, and a
// warp per (step, tile) writes images.  q' is scaled by a power of two and split
// into two halves of 11 bits (S is exact in fp16): u is off by 2^-23 of q' s
// largest entry times |S row|, and by fp32 sums.
template <int A32, int NT>
__global__ void __launch_bounds__(512) queries_kernel(const AttnArgs A, const QParams kq, float alpha_sum) {
  constexpr int dp = 32 * A32, LD = dp + 8, HN = 4 * NT, NQ = NT + 1;
  __shared__ __align__(16) __half qh[2 * kMaxGroup][LD];       // columns 2 h, 2 h + 1: the halves of head h
  __shared__ int pq[NT ? kMaxGroup : 1][NT ? dp : 1];          // place values of q'
  __shared__ float unit[kMaxGroup];
  __shared__ long long s_sum[16];
  // u, and then its place values, in the halves' place (m <= d_pad there)
  float (*us)[dp] = reinterpret_cast<float (*)[dp]>(&qh[0][0]);
  static_assert(sizeof(float) * kMaxGroup * dp <= sizeof(qh), "u fits");
  let_next_start();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, tig = lane & 3;
  const int b = blockIdx.x / A.L.hkv, h = blockIdx.x % A.L.hkv;
  const int m = kq.m, steps = A32 + m / 32, groups = A.hv / A.L.hkv;
  const int n_tiles = (A.G + 3) / 4;
  const int64_t row0 = (int64_t)b * A.Hq + (int64_t)h * A.G;
  uint32_t* const f0 = A.frag + ((int64_t)b * A.hv + (int64_t)h * groups) * A.frag_words;
  auto constants = [&](int head) {  // of a head: four floats
    const int grp = head / A.gh;
    return reinterpret_cast<float*>(f0 + (int64_t)grp * A.frag_words + steps * NQ * 64) + 4 * (head - grp * A.gh);
  };
  if (warp < 4 * n_tiles) {  // at most 16
    float v[A32] = {};
    if (warp < A.G) {
      const int64_t at = b * A.q_ld + (int64_t)(h * A.G + warp) * kq.d;
#pragma unroll
      for (int a = 0; a < A32; ++a) {
        const int j = 32 * a + lane;
        v[a] = j < kq.d ? load_q(A, at + j) : 0.f;
      }
      apply_signs<A32>(v, kq.dmask, lane);
      warp_fwht<A32>(v, lane);
    }
    float mx = 0.f;
#pragma unroll
    for (int a = 0; a < A32; ++a) {
      v[a] *= kq.inv_sqrt_dpad;
      mx = fmaxf(mx, fabsf(v[a]));
      if (NT == 0 && warp < A.G) A.qrot[(row0 + warp) * dp + 32 * a + lane] = v[a];
    }
    mx = warp_max(mx);
    // 2^e above mx, within what has a reciprocal
    const int e = min(max((__float_as_int(mx) >> 23) + 1, 27), 253);
    const float up = __int_as_float(e << 23), down = __int_as_float((254 - e) << 23);
    if (lane == 0) unit[warp] = up;
#pragma unroll
    for (int a = 0; a < A32; ++a) {
      const float x = v[a] * down;
      const __half hi = __float2half_rn(x);
      qh[2 * warp][32 * a + lane] = hi;
      qh[2 * warp + 1][32 * a + lane] = __float2half_rn(x - __half2float(hi));
    }
    if constexpr (NT > 0)
      if (warp < A.G) fixed_point<A32>(v, dp, A.scale2, alpha_sum, pq[warp], constants(warp), lane);
  }
  if (h == 0) {
    long long sum = 0;
    for (int i = tid; i < b; i += 512) sum += units_of(A, i);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) s_sum[warp] = sum;
  }
  __syncthreads();
  if (h == 0 && tid == 0) {
    long long sum = 0;
    for (int i = 0; i < 16; ++i) sum += s_sum[i];
    A.prefix[b] = sum;
    if (b == A.B - 1) A.prefix[A.B] = sum + units_of(A, b);
  }
  // u: rows 16 r .. of S; a thread's 16 bytes of a row are the K slots of two products, the same in both operands
  float acc[kMaxGroup / 4][4];
  for (int r = warp; r < (m + 15) / 16; r += 16) {
    uint4 s0[A32], s1[A32];
    const int i0 = 16 * r + g, i1 = i0 + 8;  // m is a multiple of 32
#pragma unroll
    for (int a = 0; a < A32; ++a) {
      s0[a] = *reinterpret_cast<const uint4*>(kq.S16 + (int64_t)i0 * dp + 32 * a + 8 * tig);
      s1[a] = *reinterpret_cast<const uint4*>(kq.S16 + (int64_t)i1 * dp + 32 * a + 8 * tig);
    }
#pragma unroll
    for (int t = 0; t < kMaxGroup / 4; ++t) {
      if (t >= n_tiles) break;
      float (&d)[4] = acc[t];
      d[0] = d[1] = d[2] = d[3] = 0.f;
#pragma unroll
      for (int a = 0; a < A32; ++a) {
        const uint4 q = *reinterpret_cast<const uint4*>(&qh[8 * t + g][32 * a + 8 * tig]);
        mma_f16(d, s0[a].x, s1[a].x, s0[a].y, s1[a].y, q.x, q.y);
        mma_f16(d, s0[a].z, s1[a].z, s0[a].w, s1[a].w, q.z, q.w);
      }
      if (NT == 0 && 4 * t + tig < A.G) {
        A.u[(row0 + 4 * t + tig) * m + i0] = (d[0] + d[1]) * unit[4 * t + tig];
        A.u[(row0 + 4 * t + tig) * m + i1] = (d[2] + d[3]) * unit[4 * t + tig];
      }
    }
  }
  if constexpr (NT > 0) {
    __syncthreads();  // the halves have been read; m <= 256: a warp has had 16 rows at most
    if (warp < m / 16) {
#pragma unroll
      for (int t = 0; t < kMaxGroup / 4; ++t)
        if (t < n_tiles) {
          us[4 * t + tig][16 * warp + g] = (acc[t][0] + acc[t][1]) * unit[4 * t + tig];
          us[4 * t + tig][16 * warp + g + 8] = (acc[t][2] + acc[t][3]) * unit[4 * t + tig];
        }
    }
    __syncthreads();
    if (warp < A.G) {
      float v[A32];
#pragma unroll
      for (int a = 0; a < A32; ++a) v[a] = 32 * a < m ? us[warp][32 * a + lane] : 0.f;
      fixed_point<A32>(v, m, A.scale2 * kq.kappa, 1.f, reinterpret_cast<int*>(us[warp]), constants(warp) + 2, lane);
    }
    // places of a last group that no head has
    for (int e = A.G + tid; e < groups * A.gh; e += 512)
      *reinterpret_cast<float4*>(constants(e)) = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int e = A.gh + tid; e < HN; e += 512)  // and of a group of fewer than HN
      for (int grp = 0; grp < groups; ++grp)
        *reinterpret_cast<float4*>(f0 + (int64_t)grp * A.frag_words + steps * NQ * 64 + 4 * e) = make_float4(0.f, 0.f, 0.f, 0.f);
    __syncthreads();
    // images: a warp per (group, step, tile)
    for (int e = warp; e < groups * steps * NQ; e += 16) {
      const int t = e % NQ, at = e / NQ, grp = at / steps, step = at - grp * steps;
      const int slot = t < NT ? 4 * t + (g >> 1) : (g >> 1) + 4 * (g & 1), piece = t < NT ? g & 1 : 2;
      const int head = grp * A.gh + slot;
      uint32_t w[2] = {0, 0};
      if (slot < A.gh && head < A.G) {
        const bool which = step >= A32;
        const int n = which ? m : dp, st = which ? step - A32 : step;
        // bits of the thread's word, of both half bytes; in two-word planes two threads share one, a half byte each
        const int j0 = n == 64 ? 32 * (tig & 1) + 4 * (tig >> 1) + 2 * st : 32 * (tig + (st & ~3)) + (st & 3);
        const int* p = (which ? reinterpret_cast<const int*>(us[head]) : pq[head]) + j0;
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int i = 0; i < 4; ++i) w[r] |= digit(p[8 * i + (n == 64 ? r : 4 * r)], piece) << (8 * i);
      }
      reinterpret_cast<uint2*>(f0 + (int64_t)grp * A.frag_words)[(at - grp * steps) * NQ * 32 + t * 32 + lane] =
          make_uint2(w[0], w[1]);
    }
  }
}

// ---------------------------------------------------------------- attention, any shape

// Index of token t's code for a coordinate from its value words.
__device__ __forceinline__ int value_index(const uint32_t (&w)[4], int kv, int t) {
  const int s = t & 3, i = t >> 2;
  if (kv == 1) return (w[0] >> t) & 1;
  if (kv == 4) {
    const uint32_t x = s == 0 ? w[0] : s == 1 ? w[1] : s == 2 ? w[2] : w[3];
    const int nib = (x >> (4 * i)) & 15;
    return nib >= 8 ? 15 - nib : 8 + nib;
  }
  int idx = ((s < 2 ? w[0] : w[1]) >> (4 * i + 2 * (s & 1))) & 3;
  if (kv == 3) idx |= ((w[2] >> ((t + 2) & 31)) & 1) << 2;
  return idx;
}

// 128 threads: a warp's lanes are the tokens of a block for the scores of its
// heads, a thread's coordinates tid + 128 c for the values.
template <int NC>
__global__ void __launch_bounds__(128) attention_any_kernel(const AttnArgs A, const QParams kq, const QParams vq) {
  extern __shared__ float dyn[];
  __shared__ float kc[kMaxLevels], vc[kMaxLevels];
  __shared__ float p_s[32][kMaxGroup];
  __shared__ float corr_s[kMaxGroup], m_s[kMaxGroup], l_s[kMaxGroup];
  const Layout& L = A.L;
  const int G = A.G, dp = L.dp, m = kq.m;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float* qs = dyn;           // [G][dp]
  float* us = dyn + G * dp;  // [G][m]
  if (tid < kMaxLevels) {
    kc[tid] = kq.centroids[tid];
    vc[tid] = vq.centroids[tid];
  }
  wait_for_previous();
  let_next_start();
  const int64_t units = A.prefix[A.B] * L.hkv;
  int64_t u0 = share_at(A, units, blockIdx.x);
  const int64_t u1 = share_at(A, units, blockIdx.x + 1);
  while (u0 < u1) {
    const Segment sg = segment_at(A, u0, u1, lane);
    u0 += (sg.end - sg.blk + kUnit - 1) / kUnit;
    const int64_t row0 = (int64_t)sg.b * A.Hq + (int64_t)sg.h * G;
    __syncthreads();
    for (int e = tid; e < G * dp; e += 128) qs[e] = A.qrot[row0 * dp + e];
    for (int e = tid; e < G * m; e += 128) us[e] = A.u[row0 * m + e];
    if (tid < G) {
      m_s[tid] = -INFINITY;
      l_s[tid] = 0.f;
    }
    __syncthreads();
    float o[kMaxGroup][NC];
#pragma unroll
    for (int g = 0; g < kMaxGroup; ++g)
#pragma unroll
      for (int c = 0; c < NC; ++c) o[g][c] = 0.f;
    for (int blk = sg.blk; blk < sg.end; ++blk) {
      const int64_t at = record_at(L, A.tab, sg.b, blk, A.layer, sg.kvh);
      if (at < 0) continue;
      const uint32_t* rec = A.pool + at;
      const int nt = min(32, sg.len - 32 * blk);  // tokens of the block
      const bool valid = lane < nt;
      float am[4], aq[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) am[i] = aq[i] = 0.f;
      float kn = 0.f, kr = 0.f, vn = 0.f;
      if (valid) {
        for (int w = 0; w < dp / 32; ++w) {
          uint32_t pw[4];
#pragma unroll
          for (int p = 0; p < 4; ++p) pw[p] = p < kq.k ? rec[key_word_at(L, lane, p * (dp / 32) + w)] : 0u;
          for (int i = 0; i < 32; ++i) {
            int idx = 0;
#pragma unroll
            for (int p = 0; p < 4; ++p) idx |= (int)((pw[p] >> i) & 1u) << p;
            const float c = kc[idx];
#pragma unroll
            for (int hh = 0; hh < 4; ++hh)
              if (warp + 4 * hh < G) am[hh] = fmaf(qs[(warp + 4 * hh) * dp + 32 * w + i], c, am[hh]);
          }
        }
        for (int w = 0; w < L.sw; ++w) {
          const uint32_t x = rec[key_word_at(L, lane, L.kw + w)];
          for (int i = 0; i < 32; ++i) {
            const float sg1 = ((x >> i) & 1u) ? 1.f : -1.f;
#pragma unroll
            for (int hh = 0; hh < 4; ++hh)
              if (warp + 4 * hh < G) aq[hh] = fmaf(us[(warp + 4 * hh) * m + 32 * w + i], sg1, aq[hh]);
          }
        }
        kn = __uint_as_float(rec[L.o_kn + lane]);
        kr = kq.kappa * get_rnorm(reinterpret_cast<const float*>(rec + L.o_kr), lane, L.r16);
        vn = __uint_as_float(rec[L.o_vn + lane]);
      }
#pragma unroll
      for (int hh = 0; hh < 4; ++hh) {
        const int g = warp + 4 * hh;
        if (g < G) {
          const float x = valid ? A.scale2 * (kn * (am[hh] + kr * aq[hh])) : -INFINITY;
          const float old = m_s[g], top = fmaxf(old, warp_max(x));
          const float base = top == -INFINITY ? 0.f : top;  // scores of -inf have no weight, the first ones neither
          const float p = valid ? exp2f(x - base) : 0.f;
          const float corr = exp2f(old - base);
          const float sum = warp_sum(p);
          p_s[lane][g] = p * vn;
          if (lane == 0) {
            corr_s[g] = corr;
            m_s[g] = top;
            l_s[g] = l_s[g] * corr + sum;
          }
        }
      }
      __syncthreads();
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int j = tid + 128 * c;
        if (j >= dp) continue;
        uint32_t pw[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) pw[p] = p < L.kv ? rec[L.o_v + p * dp + j] : 0u;
#pragma unroll
        for (int g = 0; g < kMaxGroup; ++g)
          if (g < G) o[g][c] *= corr_s[g];
        for (int t = 0; t < nt; ++t) {
          const float v = vc[value_index(pw, L.kv, t)];
#pragma unroll
          for (int g = 0; g < kMaxGroup; ++g)
            if (g < G) o[g][c] = fmaf(p_s[t][g], v, o[g][c]);
        }
      }
      __syncthreads();
    }
    const int64_t bh = (int64_t)sg.b * L.hkv + sg.h;
#pragma unroll
    for (int g = 0; g < kMaxGroup; ++g) {
      if (g < G) {
        float* pp = slot_of(A, bh, blockIdx.x, g);
#pragma unroll
        for (int c = 0; c < NC; ++c)
          if (tid + 128 * c < dp) pp[4 + tid + 128 * c] = o[g][c];
        if (tid == 0) {
          pp[0] = m_s[g];
          pp[1] = l_s[g];
        }
      }
    }
  }
}

// ---------------------------------------------------------------- join

constexpr int kJoinWarps = 8;

// Block (b, query head): the parts' maximum, then warp w sums parts w, w + 8,
// ... and warp 0 adds the warps' sums, rotates back and stores.
template <int A32>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const AttnArgs A, const QParams vq) {
  constexpr int dp = 32 * A32;
  __shared__ float sm[kJoinWarps], sl[kJoinWarps], sv[kJoinWarps][dp];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / A.Hq, hq = blockIdx.x % A.Hq;
  const int kh = hq / A.G, gq = hq % A.G;
  const int h = kh * (A.hv / A.L.hkv) + gq / A.gh, g = gq % A.gh;  // virtual head, place in it
  wait_for_previous();
  const int64_t p0 = A.prefix[b];
  const int64_t n = A.prefix[b + 1] - p0;
  const int64_t units = A.prefix[A.B] * A.hv;
  const int64_t s0 = A.hv * p0 + h * n, bh = (int64_t)b * A.hv + h;
  // parts c0 .. c1; none of an empty sequence
  const int c0 = n ? worker_of(A, units, s0) : 0, c1 = n ? worker_of(A, units, s0 + n - 1) : -1;
  float top = -INFINITY;
  for (int c = c0 + tid; c <= c1; c += 32 * kJoinWarps) top = fmaxf(top, slot_of(A, bh, c, g)[0]);
  top = warp_max(top);
  if (lane == 0) sm[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, sm[w]);
  float l = 0.f, v[A32];
#pragma unroll
  for (int a = 0; a < A32; ++a) v[a] = 0.f;
#pragma unroll 4
  for (int c = c0 + warp; c <= c1; c += kJoinWarps) {
    const float* pp = slot_of(A, bh, c, g);
    const float pl = pp[1];
    // holes only: nothing in it (a NaN sum is not zero: it goes on)
    const float e = pl == 0.f ? 0.f : exp2f(pp[0] - top);
    l = fmaf(e, pl, l);
#pragma unroll
    for (int a = 0; a < A32; ++a) v[a] = pl == 0.f ? v[a] : fmaf(e, pp[4 + 32 * a + lane], v[a]);
  }
  if (lane == 0) sl[warp] = l;
#pragma unroll
  for (int a = 0; a < A32; ++a) sv[warp][32 * a + lane] = v[a];
  __syncthreads();
  if (warp != 0) return;
  l = 0.f;
#pragma unroll
  for (int a = 0; a < A32; ++a) v[a] = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    l += sl[w];
#pragma unroll
    for (int a = 0; a < A32; ++a) v[a] += sv[w][32 * a + lane];
  }
  // no token: zeros; (a NaN sum is not zero and stays one)
  const float inv = l == 0.f ? 0.f : vq.inv_sqrt_dpad / l;
  warp_fwht<A32>(v, lane);
  apply_signs<A32>(v, vq.dmask, lane);
#pragma unroll
  for (int a = 0; a < A32; ++a) {
    const int j = 32 * a + lane;
    if (j < vq.d) store_out(A, ((int64_t)b * A.Hq + hq) * vq.d + j, v[a] * inv);
  }
  if (lane == 0 && A.lse) A.lse[(int64_t)b * A.Hq + hq] = l == 0.f ? -INFINITY : kLn2 * (top + log2f(l));
}

// What attention_any_kernel may take of shared memory for the queries of a group (q' and u); its own arrays fit beside it.
constexpr size_t kAnyQueries = 200 * 1024;

// How a call is run: the tensor-core kernel where it has the shape, else the one for any.
struct Plan {
  TcShape tc;
  int hv, gh, ctas, workers;
  int frag_words;
  size_t prefix, qrot, u, frag, part;  // workspace bytes
  size_t all() const { return prefix + qrot + u + frag + part; }
};

size_t round256(size_t b) { return (b + 255) & ~(size_t)255; }

Plan plan_of(const tq_paged* pg, int B, int Hq, bool fine) {
  const Layout& L = pg->lay;
  const int G = Hq / L.hkv;
  Plan p = {};
  p.tc = tc_shape(pg->kq.k, L.kv, pg->kq.m, L.dp, G, fine);
  const size_t heads = (size_t)B * Hq;
  if (p.tc.ctas_per_sm) {
    const int hn = 4 * p.tc.nt, groups = (G + hn - 1) / hn;
    p.gh = groups == 1 ? G : hn;
    p.hv = L.hkv * groups;
    p.ctas = sm_count() * p.tc.ctas_per_sm;
    p.workers = p.ctas * p.tc.warps;
    p.frag_words = p.tc.steps * (p.tc.nt + 1) * 64 + hn * 4;
    p.frag = round256((size_t)B * p.hv * p.frag_words * 4);
  } else {
    p.gh = G;
    p.hv = L.hkv;
    p.ctas = p.workers = sm_count() * 4;
    p.qrot = round256(heads * L.dp * 4);
    p.u = round256(heads * pg->kq.m * 4);
  }
  p.prefix = round256(((size_t)B + 1) * 8);
  p.part = round256(((size_t)B * p.hv + p.workers) * p.gh * part_row(L.dp) * 4);
  return p;
}

template <int A32>
cudaError_t run(const AttnArgs& a, const tq_paged* pg, const Plan& p, cudaStream_t st) {
  const dim3 pairs((unsigned)(a.B * a.L.hkv));
  cudaError_t e;
  if (p.tc.ctas_per_sm) {
    float alpha[8], alpha_sum;
    attn::odd_feature_coefs(pg->kq.centroids, pg->kq.k, alpha, &alpha_sum);
    if (p.tc.nt == 1) queries_kernel<A32, 1><<<pairs, 512, 0, st>>>(a, pg->kq, alpha_sum);
    else if constexpr (A32 < 8) queries_kernel<A32, 2><<<pairs, 512, 0, st>>>(a, pg->kq, alpha_sum);
    e = tc_launch(a, pg->kq, pg->vq, p.tc, p.ctas, st);
  } else {
    queries_kernel<A32, 0><<<pairs, 512, 0, st>>>(a, pg->kq, 0.f);
    constexpr int NC = A32 > 4 ? 2 : 1;
    const size_t smem = (size_t)a.G * (a.L.dp + pg->kq.m) * sizeof(float);
    // function attributes are per device: set on every call (a cheap host call), always to the same value, since
    // calls of other threads and shapes share it
    e = cudaFuncSetAttribute(attention_any_kernel<NC>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kAnyQueries);
    if (e == cudaSuccess) e = launch_after(attention_any_kernel<NC>, dim3(a.workers), 128, smem, st, a, pg->kq, pg->vq);
  }
  if (e != cudaSuccess) return e;
  e = launch_after(join_kernel<A32>, dim3((unsigned)(a.B * a.Hq)), 32 * kJoinWarps, 0, st, a, pg->vq);
  const cudaError_t last = cudaGetLastError();
  return e != cudaSuccess ? e : last;
}

// What does not fit the kernels' shared memory: the queries of a group.
bool too_wide(const tq_paged* pg, int G) { return (size_t)G * (pg->lay.dp + pg->kq.m) * sizeof(float) > kAnyQueries; }

}  // namespace
}  // namespace paged
}  // namespace tq

extern "C" tq_status tq_paged_attention_workspace_size(const tq_paged* pg, int B, int Hq, size_t* bytes) {
  using namespace tq::paged;
  if (!pg || !bytes || B < 0 || B > (1 << 20) || Hq < pg->lay.hkv || Hq % pg->lay.hkv) return TQ_ERR_INVALID_ARG;
  if (Hq / pg->lay.hkv > kMaxGroup || too_wide(pg, Hq / pg->lay.hkv)) return TQ_ERR_UNSUPPORTED;
  // for queries of every type
  *bytes = B == 0 ? 0 : std::max(plan_of(pg, B, Hq, false).all(), plan_of(pg, B, Hq, true).all());
  return TQ_OK;
}

extern "C" tq_status tq_paged_attention(const tq_paged* pg, const void* q, tq_dtype dt, int64_t q_ld, int B, int Hq,
                                        const uint32_t* pool, int64_t n_pages, int layer, const int32_t* lens,
                                        const int32_t* tables, int64_t table_ld, int max_pages, float scale, void* out,
                                        float* lse, void* ws, size_t ws_bytes, void* stream) {
  using namespace tq::paged;
  size_t need = 0;
  const tq_status s = tq_paged_attention_workspace_size(pg, B, Hq, &need);
  if (s != TQ_OK) return s;
  const Layout& L = pg->lay;
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess || device != pg->device) return TQ_ERR_INVALID_ARG;
  if ((dt != TQ_F32 && dt != TQ_F16 && dt != TQ_BF16) || layer < 0 || layer >= L.layers) return TQ_ERR_INVALID_ARG;
  if (B == 0) return TQ_OK;
  if (bad_pool(L, pool, n_pages) || bad_table(L, tables, table_ld, max_pages)) return TQ_ERR_INVALID_ARG;
  const uintptr_t esz = dt == TQ_F32 ? 4 : 2;
  if (!q || !out || !lens || mis4(lens) || mis4(lse) || reinterpret_cast<uintptr_t>(q) % esz ||
      reinterpret_cast<uintptr_t>(out) % esz || (B > 1 && q_ld < (int64_t)Hq * pg->kq.d))
    return TQ_ERR_INVALID_ARG;
  if ((int64_t)B * Hq > 0x7fffffffll) return TQ_ERR_UNSUPPORTED;
  if (!ws || ws_bytes < need || !al256(ws)) return TQ_ERR_WORKSPACE;
  const Plan z = plan_of(pg, B, Hq, fine_sums(dt));
  char* w = static_cast<char*>(ws);
  AttnArgs a = {};
  a.L = L;
  a.tab = {tables, table_ld, max_pages, n_pages};
  a.pool = pool;
  a.layer = layer;
  a.lens = lens;
  a.B = B;
  a.Hq = Hq;
  a.G = Hq / L.hkv;
  a.hv = z.hv;
  a.gh = z.gh;
  a.scale2 = (float)((double)scale * 1.4426950408889634);
  a.q = q;
  a.dt = dt;
  a.q_ld = q_ld;
  a.out = out;
  a.lse = lse;
  a.workers = z.workers;
  a.prefix = reinterpret_cast<int64_t*>(w);
  a.qrot = reinterpret_cast<float*>(w + z.prefix);
  a.u = reinterpret_cast<float*>(w + z.prefix + z.qrot);
  a.frag = reinterpret_cast<uint32_t*>(w + z.prefix + z.qrot + z.u);
  a.frag_words = z.frag_words;
  a.part = reinterpret_cast<float*>(w + z.prefix + z.qrot + z.u + z.frag);
  a.err = tq::error_word();
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (L.dp / 32) {
    case 1: e = run<1>(a, pg, z, st); break;
    case 2: e = run<2>(a, pg, z, st); break;
    case 4: e = run<4>(a, pg, z, st); break;
    default: e = run<8>(a, pg, z, st); break;
  }
  return e == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}
