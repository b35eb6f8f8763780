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

// Largest entry in fixed point: the difference of two neighbouring place values,
// at most 3/2 of it and a rounding, fits three signed bytes (127 2^16 and less).
constexpr float kQMax = 5548000.0f;

// P_j of the tensor-core kernel's scores: x / 2^j as an integer.
__device__ __forceinline__ int place_value(float x, int j) { return __float2int_rn(x * (1.f / (float)(1 << j))); }

// Byte `piece` (0: hi, 1: mid, 2: lo) of v = 2^16 hi + 2^8 mid + lo, |v| <= 127 * 2^16, all three in [-128, 127].
__device__ __forceinline__ uint32_t digit(int v, int piece) {
  const int lo = ((v + 128) & 0xff) - 128;
  const int v1 = (v - lo) >> 8;  // exact
  const int mid = ((v1 + 128) & 0xff) - 128;
  return (uint32_t)((piece == 0 ? (v1 - mid) >> 8 : piece == 1 ? mid : lo) & 0xff);
}

// Block (b, h): q' = H D q / sqrt(d_pad) and u = S q' of the query heads of KV
// head h, and, for h = 0, the blocks of the sequences before b.  With NT tiles
// of heads the images that the tensor-core kernel takes (its B operands, thread
// by thread, and four constants per head), with NT = 0 q' and u.
//
// u takes d_pad m G products from S (64 KB at d_pad = m = 128, in L2 after the
// first block): a thread has one row and a part of the coordinates, so that
// its loads of S are in flight together.
template <int A32, int NT>
__global__ void __launch_bounds__(512) queries_kernel(const AttnArgs A, const QParams kq, float alpha_sum) {
  constexpr int dp = 32 * A32;
  __shared__ float qs[kMaxGroup][dp];
  __shared__ float us[NT ? kMaxGroup : 1][NT ? dp : 1];  // m <= d_pad there
  __shared__ float ps[4][512];
  __shared__ float inv_s[2][kMaxGroup];
  __shared__ long long s_sum[16];
  let_next_start();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / A.L.hkv, h = blockIdx.x % A.L.hkv;
  const int m = kq.m;
  if (h == 0) {
    long long sum = 0;
    for (int i = tid; i < b; i += 512) sum += blocks_of(A, i);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) s_sum[warp] = sum;
  }
  const int64_t row0 = (int64_t)b * A.Hq + (int64_t)h * A.G;
  for (int g = warp; g < A.G; g += 16) {
    const int64_t at = b * A.q_ld + (int64_t)(h * A.G + g) * kq.d;
    float v[A32];
#pragma unroll
    for (int a = 0; a < A32; ++a) {
      const int j = 32 * a + lane;
      v[a] = j < kq.d ? load_q(A, at + j) : 0.f;
    }
    apply_signs<A32>(v, kq.dmask, lane);
    warp_fwht<A32>(v, lane);
#pragma unroll
    for (int a = 0; a < A32; ++a) {
      v[a] *= kq.inv_sqrt_dpad;
      qs[g][32 * a + lane] = v[a];
      if (NT == 0) A.qrot[(row0 + g) * dp + 32 * a + lane] = v[a];
    }
  }
  __syncthreads();
  if (h == 0 && tid == 0) {
    long long sum = 0;
    for (int i = 0; i < 16; ++i) sum += s_sum[i];
    A.prefix[b] = sum;
    if (b == A.B - 1) A.prefix[A.B] = sum + blocks_of(A, b);
  }
  const int parts = m < 512 ? 512 / m : 1, len = (dp + parts - 1) / parts;  // of the coordinates
  for (int g0 = 0; g0 < A.G; g0 += 4) {
    for (int e = tid; e < m * parts; e += 512) {
      const int i = e % m, j0 = e / m * len, j1 = min(dp, j0 + len);
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 32
      for (int j = j0; j < j1; ++j) {
        const float s = kq.St[(int64_t)j * m + i];
#pragma unroll
        for (int g = 0; g < 4; ++g) acc[g] = fmaf(s, qs[min(g0 + g, A.G - 1)][j], acc[g]);
      }
      if (parts > 1) {
#pragma unroll
        for (int g = 0; g < 4; ++g) ps[g][e] = acc[g];
      } else {
#pragma unroll
        for (int g = 0; g < 4; ++g)
          if (g0 + g < A.G) A.u[(row0 + g0 + g) * m + i] = acc[g];
      }
    }
    __syncthreads();
    if (parts > 1) {
      for (int e = tid; e < 4 * m; e += 512) {
        const int g = e / m, i = e - g * m;
        float s = 0.f;
        for (int p = 0; p < parts; ++p) s += ps[g][p * m + i];
        if (g0 + g < A.G) {
          if (NT == 0) A.u[(row0 + g0 + g) * m + i] = s;
          else us[g0 + g][i] = s;
        }
      }
    }
    __syncthreads();
  }
  if constexpr (NT > 0) {
    constexpr int HN = 4 * NT, NQ = NT + 1;
    const int steps = A32 + m / 32, groups = A.hv / A.L.hkv;
    uint32_t* f0 = A.frag + ((int64_t)b * A.hv + (int64_t)h * groups) * A.frag_words;
    // a warp per (q' or u, head): the fixed point's unit, and the sum of what it holds
    for (int e = warp; e < 2 * groups * HN; e += 16) {
      const int which = e / (groups * HN), hh = e - which * groups * HN;
      const int grp = hh / HN, slot = hh - grp * HN, head = grp * A.gh + slot;
      const bool there = slot < A.gh && head < A.G;
      const float* x = which ? us[there ? head : 0] : qs[there ? head : 0];
      const int n = which ? m : dp;
      const int in_byte = n == 64 ? 3 : 7;  // coordinate j is bit j & in_byte of its byte (or half byte)
      float mx = 1e-30f, bad = 0.f;
      for (int j = lane; j < n; j += 32) {
        mx = fmaxf(mx, fabsf(x[j]));
        bad = fmaf(x[j], 0.f, bad);  // NaN once an entry is not finite
      }
      mx = warp_max(mx);
      bad = warp_sum(bad);
      const float inv = bad == 0.f ? kQMax / mx : 0.f;
      int sum = 0;  // |sum| < d_pad (kQMax + 2^6) < 2^31
      for (int j = lane; j < n; j += 32) sum += place_value(x[j] * inv, j & in_byte) << (j & in_byte);
      sum = __reduce_add_sync(0xffffffffu, sum);
      if (lane == 0) {
        if (there) inv_s[which][head] = inv;
        const float w = A.scale2 * (which ? kq.kappa : 1.f) * (mx / kQMax);
        float* c = reinterpret_cast<float*>(f0 + (int64_t)grp * A.frag_words + steps * NQ * 64) + 4 * slot + 2 * which;
        c[0] = there ? 2.f * w : 0.f;
        c[1] = !there ? 0.f : bad == 0.f ? -w * (which ? 1.f : alpha_sum) * (float)sum : bad;
      }
    }
    __syncthreads();
    for (int e = tid; e < groups * steps * NQ * 64; e += 512) {
      const int r = e & 1, ln = (e >> 1) & 31, t = (e >> 6) % NQ, at = (e >> 6) / NQ;
      const int grp = at / steps, step = at - grp * steps;
      const int g = ln >> 2, tig = ln & 3;
      const int slot = t < NT ? 4 * t + (g >> 1) : (g >> 1) + 4 * (g & 1), piece = t < NT ? g & 1 : 2;
      const int head = grp * A.gh + slot;
      uint32_t w = 0;
      if (slot < A.gh && head < A.G) {
        const bool which = step >= A32;
        const int n = which ? m : dp, st = which ? step - A32 : step;
        // the product of k low bits of the bytes of the thread's word; in two-word planes two threads share one
        const int k = n == 64 ? 2 * st + 1 + r : (st & 3) + 1 + 4 * r, top = n == 64 ? 4 : 8;
        const int j0 = n == 64 ? 32 * (tig & 1) + 4 * (tig >> 1) : 32 * (tig + (st & ~3));
        const float* x = which ? us[head] : qs[head];
        const float inv = inv_s[which][head];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float* xi = x + j0 + 8 * i;
          const int p = place_value(xi[k - 1] * inv, k - 1);
          w |= digit(k < top ? p - place_value(xi[k] * inv, k) : p, piece) << (8 * i);
        }
      }
      f0[(int64_t)grp * A.frag_words + (step * NQ + t) * 64 + 2 * ln + r] = w;
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
  const int64_t units = A.prefix[A.B] * L.hkv, share = share_of(A, units);
  int64_t u0 = blockIdx.x * share;
  const int64_t u1 = min64(units, u0 + share);
  while (u0 < u1) {
    const Segment sg = segment_at(A, u0, u1, lane);
    u0 += sg.end - sg.blk;
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
          const float p = valid ? exp2f(x - top) : 0.f;
          const float corr = exp2f(old - top);
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
  const int64_t share = share_of(A, A.prefix[A.B] * A.hv);
  const int64_t s0 = A.hv * p0 + h * n, bh = (int64_t)b * A.hv + h;
  // parts c0 .. c1; none of an empty sequence
  const int c0 = (int)(s0 / share), c1 = n ? (int)((s0 + n - 1) / share) : c0 - 1;
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

// How a call is run: the tensor-core kernel where it has the shape, else the one for any.
struct Plan {
  TcShape tc;
  int hv, gh, ctas, workers;
  int frag_words;
  size_t prefix, qrot, u, frag, part;  // workspace bytes
  size_t all() const { return prefix + qrot + u + frag + part; }
};

size_t round256(size_t b) { return (b + 255) & ~(size_t)255; }

Plan plan_of(const tq_paged* pg, int B, int Hq) {
  const Layout& L = pg->lay;
  const int G = Hq / L.hkv;
  Plan p = {};
  p.tc = tc_shape(pg->kq.k, L.kv, pg->kq.m, L.dp, G);
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
    // function attributes are per device: set on every call (a cheap host call)
    e = cudaFuncSetAttribute(attention_any_kernel<NC>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess) e = launch_after(attention_any_kernel<NC>, dim3(a.workers), 128, smem, st, a, pg->kq, pg->vq);
  }
  if (e != cudaSuccess) return e;
  e = launch_after(join_kernel<A32>, dim3((unsigned)(a.B * a.Hq)), 32 * kJoinWarps, 0, st, a, pg->vq);
  const cudaError_t last = cudaGetLastError();
  return e != cudaSuccess ? e : last;
}

// What does not fit the kernels' shared memory: the queries of a group.
bool too_wide(const tq_paged* pg, int G) { return (size_t)G * (pg->lay.dp + pg->kq.m) * sizeof(float) > 200 * 1024; }

}  // namespace
}  // namespace paged
}  // namespace tq

extern "C" tq_status tq_paged_attention_workspace_size(const tq_paged* pg, int B, int Hq, size_t* bytes) {
  using namespace tq::paged;
  if (!pg || !bytes || B < 0 || B > (1 << 20) || Hq < pg->lay.hkv || Hq % pg->lay.hkv) return TQ_ERR_INVALID_ARG;
  if (Hq / pg->lay.hkv > kMaxGroup || too_wide(pg, Hq / pg->lay.hkv)) return TQ_ERR_UNSUPPORTED;
  *bytes = B == 0 ? 0 : plan_of(pg, B, Hq).all();
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
  if ((dt != TQ_F32 && dt != TQ_F16 && dt != TQ_BF16) || layer < 0 || layer >= L.layers) return TQ_ERR_INVALID_ARG;
  if (B == 0) return TQ_OK;
  if (bad_pool(L, pool, n_pages) || bad_table(L, tables, table_ld, max_pages)) return TQ_ERR_INVALID_ARG;
  const uintptr_t esz = dt == TQ_F32 ? 4 : 2;
  if (!q || !out || !lens || mis4(lens) || mis4(lse) || reinterpret_cast<uintptr_t>(q) % esz ||
      reinterpret_cast<uintptr_t>(out) % esz || (B > 1 && q_ld < (int64_t)Hq * pg->kq.d))
    return TQ_ERR_INVALID_ARG;
  if ((int64_t)B * Hq > 0x7fffffffll) return TQ_ERR_UNSUPPORTED;
  if (!ws || ws_bytes < need || !al256(ws)) return TQ_ERR_WORKSPACE;
  const Plan z = plan_of(pg, B, Hq);
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
