// tq_qk_norm_rope: RMS norm per head and rotary positions of queries and keys
// in one pass (include/tq.h).
//
// Per row (token, head):  y = x rsqrt(mean(x^2) + eps) w, then each pair (a, b)
// of the first `rot` coordinates becomes (a cos - b sin, b cos + a sin) with
// the angle pos f_i.  An angle is needed as a fraction of a turn, so f_i is
// kept as F_i = f_i / (2 pi) 2^64 and the fraction is the product pos F_i
// modulo 2^64: one integer multiplication, exact but for F_i's own rounding
// (pos 2^-65 of a turn).
//
// The work is memory: each element is read and written once.  A group of lanes
// owns a row, each lane holding matching vectors of both halves of the pairs,
// so the rotation needs no exchange and the norm one group reduction.  The
// sines and cosines of a token serve all of a group's heads.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>

#include "tq_device.cuh"
#include "tq_internal.h"

struct tq_rope {
  int rot, interleaved;
  float mscale;
  uint64_t turn[128];  // F_i
};

namespace tq {
namespace rope {

struct Side {  // q or k
  const void* x;
  void* y;
  const void* w;
  int64_t xt, xh, yt, yh;
  int heads;
};

struct Args {
  Side s[2];
  const int64_t* pos;
  int64_t items;  // (token, block of heads)
  int d, rot, blocks, hpg;  // blocks of hpg heads per token
  int lanes;      // of a group: a power of two
  float eps, mscale, inv_d;
  uint64_t turn[128];
};

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T e[V];
};

template <typename T, int V>
__device__ __forceinline__ void load(const T* p, float (&v)[V]) {
  const Vec<T, V> r = *reinterpret_cast<const Vec<T, V>*>(p);
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = to_f32(r.e[i]);
}
template <typename T, int V>
__device__ __forceinline__ void store(T* p, const float (&v)[V]) {
  Vec<T, V> r;
#pragma unroll
  for (int i = 0; i < V; ++i) r.e[i] = from_f32<T>(v[i]);
  *reinterpret_cast<Vec<T, V>*>(p) = r;
}

// A chunk is what one lane handles at a time, two vectors at `a` and `b` of the
// row: V pairs, or, behind the rotated part, 2 V coordinates that pass (the
// last of them perhaps V: b = -1).
template <int V, bool PAIRS>
__device__ __forceinline__ void chunk_at(int c, int np, const Args& A, int& a, int& b) {
  if (c < np) {
    a = PAIRS ? 2 * V * c : V * c;
    b = PAIRS ? a + V : a + A.rot / 2;
  } else {
    a = A.rot + 2 * V * (c - np);
    b = a + V < A.d ? a + V : -1;
  }
}

// cos and sin (times mscale) of the V pairs of chunk c.
template <int V>
__device__ __forceinline__ void turns(const Args& A, int c, uint64_t pos, float (&co)[V], float (&si)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    // the top 32 bits of the fraction as a signed number of half turns
    const int hi = (int)(uint32_t)((pos * A.turn[V * c + i]) >> 32);
    sincospif((float)hi * 0x1p-31f, &si[i], &co[i]);
    co[i] *= A.mscale;
    si[i] *= A.mscale;
  }
}

template <int V, bool PAIRS>
__device__ __forceinline__ void rotate(float (&x)[V], float (&z)[V], const float (&co)[V], const float (&si)[V]) {
  if constexpr (!PAIRS) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float a = x[i], b = z[i];
      x[i] = a * co[i] - b * si[i];
      z[i] = b * co[i] + a * si[i];
    }
  } else {
    float t[2 * V];
#pragma unroll
    for (int i = 0; i < V; ++i) t[i] = x[i], t[V + i] = z[i];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float a = t[2 * i], b = t[2 * i + 1];
      t[2 * i] = a * co[i] - b * si[i];
      t[2 * i + 1] = b * co[i] + a * si[i];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = t[i], z[i] = t[V + i];
  }
}

// Rows of one side: V pairs (or coordinates that pass) a lane, U heads' loads in flight.
template <typename T, int V, bool PAIRS, int U>
__device__ __forceinline__ void norm_rope_rows(const Args& A, const Side& s, int64_t tok, int h0, int h1, int lane,
                                               unsigned mask, bool there, bool turn, int a, int b, const float (&co)[V],
                                               const float (&si)[V]) {
  const T* x = static_cast<const T*>(s.x) + tok * s.xt + a;
  T* y = static_cast<T*>(s.y) + tok * s.yt + a;
  const int ab = b - a;
  float g0[V], g1[V];
  if (s.w && there) {
    load<T, V>(static_cast<const T*>(s.w) + a, g0);
    if (b >= 0) load<T, V>(static_cast<const T*>(s.w) + b, g1);
  }
  for (int h = h0; h < h1; h += U) {
    Vec<T, V> r0[U], r1[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (there && h + u < h1) {
        r0[u] = *reinterpret_cast<const Vec<T, V>*>(x + (h + u) * s.xh);
        if (b >= 0) r1[u] = *reinterpret_cast<const Vec<T, V>*>(x + (h + u) * s.xh + ab);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (h + u >= h1) break;
      float p[V], q[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        p[i] = there ? to_f32(r0[u].e[i]) : 0.f;
        q[i] = there && b >= 0 ? to_f32(r1[u].e[i]) : 0.f;
      }
      if (s.w) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) sum = fmaf(p[i], p[i], fmaf(q[i], q[i], sum));
        for (int o = A.lanes >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(mask, sum, o);
        const float inv = rsqrtf(sum * A.inv_d + A.eps);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          p[i] *= inv * g0[i];
          q[i] *= inv * g1[i];
        }
      }
      if (!there) continue;
      if (b >= 0) {
        if (turn) rotate<V, PAIRS>(p, q, co, si);
        store<T, V>(y + (h + u) * s.yh + ab, q);
      }
      store<T, V>(y + (h + u) * s.yh, p);
    }
  }
}

// A group of lanes takes hpg heads of a token, a chunk of the row per lane: the
// row is read once, and the sines serve all of the heads.
template <typename T, int V, bool PAIRS>
__global__ void __launch_bounds__(256) norm_rope_kernel(const __grid_constant__ Args A) {
  const int lane = threadIdx.x & (A.lanes - 1);
  const unsigned mask = (A.lanes == 32 ? 0xffffffffu : ((1u << A.lanes) - 1u)) << ((threadIdx.x & 31) & ~(A.lanes - 1));
  const int64_t item = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / A.lanes;
  if (item >= A.items) return;
  const int64_t tok = item / A.blocks;
  const int h0 = (int)(item - tok * A.blocks) * A.hpg, hq = A.s[0].heads;
  const int h1 = min(h0 + A.hpg, hq + A.s[1].heads);
  const int np = A.rot / 2 / V, nc = np + (A.d - A.rot + 2 * V - 1) / (2 * V);
  const bool there = lane < nc, turn = lane < np;
  int a = 0, b = -1;
  if (there) chunk_at<V, PAIRS>(lane, np, A, a, b);
  float co[V] = {}, si[V] = {};
  if (turn) turns<V>(A, lane, (uint64_t)A.pos[tok], co, si);
  constexpr int U = V > 1 ? 4 : 2;
  if (h0 < hq) norm_rope_rows<T, V, PAIRS, U>(A, A.s[0], tok, h0, min(h1, hq), lane, mask, there, turn, a, b, co, si);
  if (h1 > hq) norm_rope_rows<T, V, PAIRS, U>(A, A.s[1], tok, max(h0, hq) - hq, h1 - hq, lane, mask, there, turn, a, b, co, si);
}

// Rows of more than 32 chunks (long heads, or no alignment for vectors): a warp per (token, head), chunk by chunk.
template <typename T, int V, bool PAIRS>
__global__ void __launch_bounds__(256) norm_rope_wide_kernel(const __grid_constant__ Args A) {
  const int lane = threadIdx.x & 31;
  const int64_t item = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  if (item >= A.items) return;
  const int64_t tok = item / A.blocks;
  const int h = (int)(item - tok * A.blocks);
  const bool isk = h >= A.s[0].heads;
  const Side& s = A.s[isk ? 1 : 0];
  const int hh = isk ? h - A.s[0].heads : h;
  const int np = A.rot / 2 / V, nc = np + (A.d - A.rot + 2 * V - 1) / (2 * V);
  const uint64_t pos = A.rot ? (uint64_t)A.pos[tok] : 0;
  const T* x = static_cast<const T*>(s.x) + tok * s.xt + hh * s.xh;
  T* y = static_cast<T*>(s.y) + tok * s.yt + hh * s.yh;
  const T* w = static_cast<const T*>(s.w);
  float inv = 1.f;
  if (w) {
    float sum = 0.f;
    for (int c = lane; c < nc; c += 32) {
      int a, b;
      chunk_at<V, PAIRS>(c, np, A, a, b);
      float u[V];
      load<T, V>(x + a, u);
#pragma unroll
      for (int i = 0; i < V; ++i) sum = fmaf(u[i], u[i], sum);
      if (b >= 0) {
        load<T, V>(x + b, u);
#pragma unroll
        for (int i = 0; i < V; ++i) sum = fmaf(u[i], u[i], sum);
      }
    }
    inv = rsqrtf(warp_sum(sum) * A.inv_d + A.eps);
  }
  for (int c = lane; c < nc; c += 32) {
    int a, b;
    chunk_at<V, PAIRS>(c, np, A, a, b);
    float u[V], v[V], g[V];
    load<T, V>(x + a, u);
    if (w) {
      load<T, V>(w + a, g);
#pragma unroll
      for (int i = 0; i < V; ++i) u[i] = u[i] * inv * g[i];
    }
    if (b >= 0) {
      load<T, V>(x + b, v);
      if (w) {
        load<T, V>(w + b, g);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = v[i] * inv * g[i];
      }
      if (c < np) {
        float co[V], si[V];
        turns<V>(A, c, pos, co, si);
        rotate<V, PAIRS>(u, v, co, si);
      }
      store<T, V>(y + b, v);
    }
    store<T, V>(y + a, u);
  }
}

template <typename T, int V>
int launch(const Args& a, bool pairs, bool wide, cudaStream_t st) {
  const int64_t blocks = ceil_div(a.items * a.lanes, 256);
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  const unsigned n = (unsigned)blocks;
  if (wide && pairs) norm_rope_wide_kernel<T, V, true><<<n, 256, 0, st>>>(a);
  else if (wide) norm_rope_wide_kernel<T, V, false><<<n, 256, 0, st>>>(a);
  else if (pairs) norm_rope_kernel<T, V, true><<<n, 256, 0, st>>>(a);
  else norm_rope_kernel<T, V, false><<<n, 256, 0, st>>>(a);
  return cudaGetLastError();
}

// Whether vectors of v elements fit every row: their starts and the pieces
// that a lane takes.
bool fits(const Args& a, bool pairs, int esz, int v) {
  const uintptr_t unit = (uintptr_t)v * esz;
  for (const Side& s : a.s) {
    if (!s.heads) continue;
    if (reinterpret_cast<uintptr_t>(s.x) % unit || reinterpret_cast<uintptr_t>(s.y) % unit ||
        reinterpret_cast<uintptr_t>(s.w) % unit)
      return false;
    for (int64_t st : {s.xt, s.xh, s.yt, s.yh})
      if (st % v) return false;
  }
  return a.d % v == 0 && (a.rot / 2) % v == 0 && (!pairs || a.rot % (2 * v) == 0);
}

}  // namespace rope
}  // namespace tq

extern "C" tq_status tq_rope_create(int rot, int interleaved, double base, tq_rope_scaling scaling, double factor,
                                    double orig_len, double low, double high, tq_rope** out) {
  if (!out) return TQ_ERR_INVALID_ARG;
  *out = nullptr;
  if (rot < 2 || rot > 256 || rot % 2 || !(base > 1.0) || !std::isfinite(base)) return TQ_ERR_INVALID_ARG;
  if (scaling < TQ_ROPE_PLAIN || scaling > TQ_ROPE_YARN) return TQ_ERR_INVALID_ARG;
  if (scaling != TQ_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor))) return TQ_ERR_INVALID_ARG;
  if (scaling >= TQ_ROPE_BANDS &&
      (!(orig_len > 0.0) || !(low > 0.0) || !(high > low) || !std::isfinite(orig_len) || !std::isfinite(high)))
    return TQ_ERR_INVALID_ARG;
  tq_rope* r = new (std::nothrow) tq_rope();
  if (!r) return TQ_ERR_INTERNAL;
  r->rot = rot;
  r->interleaved = interleaved != 0;
  r->mscale = scaling == TQ_ROPE_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
  const double two_pi = 2.0 * M_PI;
  // the pair number at which a pair makes `turns` turns over orig_len
  auto pair_of = [&](double turns) { return rot * std::log(orig_len / (turns * two_pi)) / (2.0 * std::log(base)); };
  for (int i = 0; i < rot / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot), keep = 1.0;  // keep: the share of f that is not slowed down
    if (scaling == TQ_ROPE_LINEAR) keep = 0.0;
    if (scaling == TQ_ROPE_BANDS) keep = std::fmin(1.0, std::fmax(0.0, (orig_len * f / two_pi - low) / (high - low)));
    if (scaling == TQ_ROPE_YARN) {
      const double first = std::fmax(std::floor(pair_of(high)), 0.0);
      const double last = std::fmin(std::ceil(pair_of(low)), rot - 1.0);
      keep = 1.0 - std::fmin(1.0, std::fmax(0.0, (i - first) / std::fmax(last - first, 1e-3)));
    }
    if (scaling != TQ_ROPE_PLAIN) f = f * keep + f / factor * (1.0 - keep);
    r->turn[i] = (uint64_t)((long double)f / (2.0L * M_PIl) * 0x1p64L + 0.5L);
  }
  *out = r;
  return TQ_OK;
}

extern "C" tq_status tq_rope_destroy(tq_rope* r) {
  delete r;
  return TQ_OK;
}

extern "C" tq_status tq_qk_norm_rope(const tq_rope* rope, tq_dtype dt, int64_t n_tok, int d, int Hq, const void* q,
                                     int64_t q_tok, int64_t q_head, int Hkv, const void* k, int64_t k_tok,
                                     int64_t k_head, const int64_t* pos, const void* wq, const void* wk, float eps,
                                     void* q_out, int64_t qo_tok, int64_t qo_head, void* k_out, int64_t ko_tok,
                                     int64_t ko_head, void* stream) {
  using namespace tq::rope;
  if (dt != TQ_F32 && dt != TQ_F16 && dt != TQ_BF16) return TQ_ERR_INVALID_ARG;
  if (n_tok < 0 || d < 1 || d > 4096 || Hq < 0 || Hkv < 0 || Hq > 65536 || Hkv > 65536) return TQ_ERR_INVALID_ARG;
  if (rope && d < rope->rot) return TQ_ERR_INVALID_ARG;
  if (!(eps >= 0.0f)) return TQ_ERR_INVALID_ARG;
  if (n_tok == 0 || Hq + Hkv == 0) return TQ_OK;
  const int esz = dt == TQ_F32 ? 4 : 2;
  if (rope && (!pos || reinterpret_cast<uintptr_t>(pos) % 8)) return TQ_ERR_INVALID_ARG;
  Args a = {};
  a.s[0] = {q, q_out, wq, q_tok, q_head, qo_tok, qo_head, Hq};
  a.s[1] = {k, k_out, wk, k_tok, k_head, ko_tok, ko_head, Hkv};
  for (const Side& s : a.s) {
    if (!s.heads) continue;
    if (!s.x || !s.y || reinterpret_cast<uintptr_t>(s.x) % esz || reinterpret_cast<uintptr_t>(s.y) % esz ||
        reinterpret_cast<uintptr_t>(s.w) % esz)
      return TQ_ERR_INVALID_ARG;
    if (s.xt < 0 || s.xh < 0 || (n_tok > 1 && s.yt < d) || (s.heads > 1 && s.yh < d)) return TQ_ERR_INVALID_ARG;
  }
  a.pos = pos;
  a.d = d;
  a.rot = rope ? rope->rot : 0;
  a.eps = eps;
  a.mscale = rope ? rope->mscale : 1.0f;
  if (rope)
    for (int i = 0; i < rope->rot / 2; ++i) a.turn[i] = rope->turn[i];
  const bool pairs = rope && rope->interleaved;
  int v = dt == TQ_F32 ? 4 : 8;
  while (v > 1 && !fits(a, pairs, esz, v)) v = v == 8 ? 4 : 1;
  a.inv_d = 1.0f / (float)d;
  const int chunks = a.rot / 2 / v + (d - a.rot + 2 * v - 1) / (2 * v);
  const bool wide = chunks > 32;
  a.lanes = 1;
  while (a.lanes < 32 && a.lanes < chunks) a.lanes *= 2;
  // as many heads a group as leave two groups for every place on the GPU (2048 threads per SM): the sines cost as
  // much as two to three heads' memory time, and a call of few rows is over sooner with a head each
  const int64_t heads = Hq + Hkv, places = (int64_t)tq::sm_count() * 2048 / a.lanes;
  a.hpg = wide ? 1 : (int)std::min<int64_t>(16, std::max<int64_t>(1, n_tok * heads / (2 * places)));
  a.blocks = (int)tq::ceil_div(heads, a.hpg);
  a.hpg = (int)tq::ceil_div(heads, a.blocks);  // even shares
  a.items = n_tok * a.blocks;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int e;
  if (dt == TQ_F32) e = v == 4 ? launch<float, 4>(a, pairs, wide, st) : launch<float, 1>(a, pairs, wide, st);
  else if (dt == TQ_F16)
    e = v == 8 ? launch<__half, 8>(a, pairs, wide, st) : v == 4 ? launch<__half, 4>(a, pairs, wide, st) : launch<__half, 1>(a, pairs, wide, st);
  else
    e = v == 8 ? launch<__nv_bfloat16, 8>(a, pairs, wide, st)
               : v == 4 ? launch<__nv_bfloat16, 4>(a, pairs, wide, st) : launch<__nv_bfloat16, 1>(a, pairs, wide, st);
  return e == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}
