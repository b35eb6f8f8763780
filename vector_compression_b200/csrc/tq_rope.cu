// tq_qk_norm_rope: RMS norm per head and rotary positions of queries and keys
// in one pass (include/tq.h).
//
// Per row (token, head):  y = x rsqrt(mean(x^2) + eps) w, then each pair (a, b)
// of the first `rot` coordinates becomes (a cos - b sin, b cos + a sin) with
// the angle pos f_i.  An angle is needed as a fraction of a turn, so f_i is
// kept as F_i = f_i / (2 pi) 2^64 and the fraction is the product pos F_i
// modulo 2^64: one integer multiplication, exact but for what F_i is off by.
// That is below 2 (its rounding, and f_i made in extended precision, of 2^-63),
// so the fraction is off by pos 2^-63 of a turn; f_i made in double would make
// that pos 2^-57.
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
#include <type_traits>

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
  int64_t items, n_tok;  // (block of heads, token)
  int d, rot, blocks, hpg;  // blocks of hpg heads per token
  int lanes;      // of a group: a power of two
  float eps, mscale, inv_d;
  uint64_t turn[128];
};

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T e[V];
};

__device__ __forceinline__ void unpack2(const float* p, float& a, float& b) { a = p[0], b = p[1]; }
__device__ __forceinline__ void unpack2(const __half* p, float& a, float& b) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(p));
  a = f.x, b = f.y;
}
__device__ __forceinline__ void unpack2(const __nv_bfloat16* p, float& a, float& b) {
  const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
  a = __uint_as_float(w << 16), b = __uint_as_float(w & 0xffff0000u);
}
template <typename T, int V>
__device__ __forceinline__ void unpack(const Vec<T, V>& r, float (&v)[V]) {
  if constexpr (V == 1) v[0] = to_f32(r.e[0]);
  else
#pragma unroll
    for (int i = 0; i < V; i += 2) unpack2(r.e + i, v[i], v[i + 1]);
}
__device__ __forceinline__ void pack2(float* d, float a, float b) { d[0] = a, d[1] = b; }
__device__ __forceinline__ void pack2(__half* d, float a, float b) { *reinterpret_cast<__half2*>(d) = __floats2half2_rn(a, b); }
__device__ __forceinline__ void pack2(__nv_bfloat16* d, float a, float b) {
  *reinterpret_cast<__nv_bfloat162*>(d) = __floats2bfloat162_rn(a, b);
}
__device__ __forceinline__ void pack1(float* d, float a) { *d = a; }
__device__ __forceinline__ void pack1(__half* d, float a) { *d = __float2half_rn(a); }
__device__ __forceinline__ void pack1(__nv_bfloat16* d, float a) { *d = __float2bfloat16_rn(a); }

template <typename T, int V>
__device__ __forceinline__ void load(const T* p, float (&v)[V]) {
  unpack(*reinterpret_cast<const Vec<T, V>*>(p), v);
}
template <typename T, int V>
__device__ __forceinline__ void store(T* p, const float (&v)[V]) {
  Vec<T, V> r;
  if constexpr (V == 1) pack1(r.e, v[0]);
  else
#pragma unroll
    for (int i = 0; i < V; i += 2) pack2(r.e + i, v[i], v[i + 1]);
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

// cos and sin (times mscale) of the V pairs of chunk c.  For 16-bit results the
// hardware's sine of an angle within half a turn is enough: it is off by 2^-21,
// the result's rounding by 2^-12 or 2^-9.
template <typename T, int V>
__device__ __forceinline__ void turns(const Args& A, int c, uint64_t pos, float (&co)[V], float (&si)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    // the top 32 bits of the fraction as a signed number of half turns
    const float x = (float)(int)(uint32_t)((pos * A.turn[V * c + i]) >> 32);
    if constexpr (sizeof(T) == 2) {
      const float y = x * (0x1p-31f * 3.14159265358979f);
      si[i] = __sinf(y);
      co[i] = __cosf(y);
    } else {
      sincospif(x * 0x1p-31f, &si[i], &co[i]);
    }
    co[i] *= A.mscale;
    si[i] *= A.mscale;
  }
}

// Position of pair i of a chunk in its two vectors.
template <int V, bool PAIRS>
__device__ __forceinline__ void pair_at(float (&x)[V], float (&z)[V], int i, float*& a, float*& b) {
  if (PAIRS) {  // coordinates 2 i and 2 i + 1 of the 2 V
    a = 2 * i < V ? &x[2 * i % V] : &z[2 * i % V];
    b = 2 * i + 1 < V ? &x[(2 * i + 1) % V] : &z[(2 * i + 1) % V];
  } else {
    a = &x[i];
    b = &z[i];
  }
}
// The factors of a chunk's pairs, (a, b) -> (a f0 - b f1, b f2 + a f3): the weights' (g0, g1) times the turn's.
template <int V>
struct Factors {
  float f0[V], f1[V], f2[V], f3[V];
};
template <int V, bool PAIRS>
__device__ __forceinline__ void rotate(float (&x)[V], float (&z)[V], const Factors<V>& f) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float *pa, *pb;
    pair_at<V, PAIRS>(x, z, i, pa, pb);
    const float a = *pa, b = *pb;
    *pa = a * f.f0[i] - b * f.f1[i];
    *pb = b * f.f2[i] + a * f.f3[i];
  }
}

// `n` rows of one side from x and y on, V pairs (or coordinates that pass) a lane, U rows' loads in flight.
// FULL: every lane has a whole chunk.
template <typename T, int V, bool PAIRS, bool NORM, bool FULL, int U>
__device__ __forceinline__ void norm_rope_rows(const Args& A, const T* x, int64_t xh, T* y, int64_t yh, int n, int ab,
                                               unsigned mask, bool there, bool both, bool turn, const Factors<V>& f) {
  auto rows = [&](auto count) {
    constexpr int C = decltype(count)::value;
    Vec<T, V> r0[C], r1[C];
#pragma unroll
    for (int u = 0; u < C; ++u) {
      if (!FULL) r0[u] = {}, r1[u] = {};
      if (FULL || there) r0[u] = *reinterpret_cast<const Vec<T, V>*>(x);
      if (FULL || both) r1[u] = *reinterpret_cast<const Vec<T, V>*>(x + ab);
      x += xh;
    }
    float p[C][V], q[C][V];
#pragma unroll
    for (int u = 0; u < C; ++u) {
      unpack(r0[u], p[u]);
      unpack(r1[u], q[u]);
    }
    if (NORM) {
      float inv[C];
#pragma unroll
      for (int u = 0; u < C; ++u) {
        inv[u] = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) inv[u] = fmaf(p[u][i], p[u][i], fmaf(q[u][i], q[u][i], inv[u]));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        if (o < A.lanes)
#pragma unroll
          for (int u = 0; u < C; ++u) inv[u] += __shfl_xor_sync(mask, inv[u], o);
#pragma unroll
      for (int u = 0; u < C; ++u) {
        inv[u] = rsqrtf(inv[u] * A.inv_d + A.eps);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          p[u][i] *= inv[u];
          q[u][i] *= inv[u];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < C; ++u) {
      if (turn) {
        rotate<V, PAIRS>(p[u], q[u], f);
      } else if (NORM) {  // f0 and f2: the weights of the two vectors
#pragma unroll
        for (int i = 0; i < V; ++i) {
          p[u][i] *= f.f0[i];
          q[u][i] *= f.f2[i];
        }
      }
      if (FULL || there) store<T, V>(y, p[u]);
      if (FULL || both) store<T, V>(y + ab, q[u]);
      y += yh;
    }
  };
  for (; n >= U; n -= U) rows(std::integral_constant<int, U>{});
  if (U > 2 && n >= 2) {
    rows(std::integral_constant<int, 2>{});
    n -= 2;
  }
  for (; n > 0; --n) rows(std::integral_constant<int, 1>{});
}

// A group of lanes takes hpg heads of a token, a chunk of the row per lane: the
// row is read once, and the sines serve all of the heads.
template <typename T, int V, bool PAIRS, bool FULL>
__global__ void __launch_bounds__(256, V == 8 ? 2 : 3) norm_rope_kernel(const __grid_constant__ Args A) {
  const int lane = threadIdx.x & (A.lanes - 1);
  const unsigned mask = (A.lanes == 32 ? 0xffffffffu : ((1u << A.lanes) - 1u)) << ((threadIdx.x & 31) & ~(A.lanes - 1));
  const int64_t item = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / A.lanes;
  if (item >= A.items) return;
  // tokens run fastest: the groups of a warp have the same heads, and take the same turns
  const int64_t blk = A.items <= 0x7fffffff ? (uint32_t)item / (uint32_t)A.n_tok : item / A.n_tok, tok = item - blk * A.n_tok;
  const int h0 = (int)blk * A.hpg, hq = A.s[0].heads;
  const int h1 = min(h0 + A.hpg, hq + A.s[1].heads);
  const int np = A.rot / 2 / V, nc = np + (A.d - A.rot + 2 * V - 1) / (2 * V);
  const bool there = lane < nc, turn = lane < np;
  int a = 0, b = -1;
  if (there) chunk_at<V, PAIRS>(lane, np, A, a, b);
  const bool both = b >= 0;
  // a group with heads of both sides: fp32's sines are made once; the 16-bit ones are short, and eight pairs of them
  // held over both sides spill
  constexpr bool kOnce = sizeof(T) == 4;
  const uint64_t pos = turn ? (uint64_t)A.pos[tok] : 0;
  float co1[V] = {}, si1[V] = {};
  if (kOnce && turn) turns<T, V>(A, lane, pos, co1, si1);
  // rows in flight against registers: four of eight-element vectors at two blocks per SM (16384 x 40 x 128 fp16: 63 us,
  // with norms 70) or two of the smaller ones at three; two at three blocks are 63 and 75 there, four spill
  constexpr int U = V == 8 ? 4 : 2;
#pragma unroll 1
  for (int side = 0; side < 2; ++side) {
    const Side& s = A.s[side];
    const int first = side ? max(h0, hq) - hq : h0, n = (side ? h1 - hq : min(h1, hq)) - first;
    if (n <= 0) continue;
    const T* x = static_cast<const T*>(s.x) + tok * s.xt + first * s.xh + a;
    T* y = static_cast<T*>(s.y) + tok * s.yt + first * s.yh + a;
    Factors<V> f;
    float co[V] = {}, si[V] = {};
    if constexpr (kOnce) {
#pragma unroll
      for (int i = 0; i < V; ++i) co[i] = co1[i], si[i] = si1[i];
    } else if (turn) {
      turns<T, V>(A, lane, pos, co, si);
    }
    if (s.w) {
      float g0[V] = {}, g1[V] = {};
      if (there) load<T, V>(static_cast<const T*>(s.w) + a, g0);
      if (both) load<T, V>(static_cast<const T*>(s.w) + b, g1);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        f.f0[i] = g0[i];
        f.f2[i] = g1[i];
        if (turn) {
          float *pa, *pb;
          pair_at<V, PAIRS>(g0, g1, i, pa, pb);
          f.f0[i] = *pa * co[i];
          f.f1[i] = *pb * si[i];
          f.f2[i] = *pb * co[i];
          f.f3[i] = *pa * si[i];
        }
      }
      norm_rope_rows<T, V, PAIRS, true, FULL, U>(A, x, s.xh, y, s.yh, n, b - a, mask, there, both, turn, f);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) f.f0[i] = f.f2[i] = co[i], f.f1[i] = f.f3[i] = si[i];
      norm_rope_rows<T, V, PAIRS, false, FULL, U>(A, x, s.xh, y, s.yh, n, b - a, mask, there, both, turn, f);
    }
  }
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
        turns<T, V>(A, c, pos, co, si);
        Factors<V> f;
#pragma unroll
        for (int i = 0; i < V; ++i) f.f0[i] = f.f2[i] = co[i], f.f1[i] = f.f3[i] = si[i];
        rotate<V, PAIRS>(u, v, f);
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
  const bool full = a.lanes * 2 * V == a.d;  // the chunks are 2 V coordinates each
  if (wide && pairs) norm_rope_wide_kernel<T, V, true><<<n, 256, 0, st>>>(a);
  else if (wide) norm_rope_wide_kernel<T, V, false><<<n, 256, 0, st>>>(a);
  else if (pairs && full) norm_rope_kernel<T, V, true, true><<<n, 256, 0, st>>>(a);
  else if (pairs) norm_rope_kernel<T, V, true, false><<<n, 256, 0, st>>>(a);
  else if (full) norm_rope_kernel<T, V, false, true><<<n, 256, 0, st>>>(a);
  else norm_rope_kernel<T, V, false, false><<<n, 256, 0, st>>>(a);
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

// Whether two of a side's output rows (t yt + h yh, d elements each) share an element.
bool rows_overlap(const Side& s, int64_t n_tok, int d) {
  if ((n_tok > 1 && s.yt < d) || (s.heads > 1 && s.yh < d)) return true;
  if (n_tok == 1 || s.heads == 1) return false;
  // heads within a token, or tokens within a head (a quotient, since a product could pass 64 bits)
  if (s.yh <= (s.yt - d) / (s.heads - 1) || s.yt <= (s.yh - d) / (n_tok - 1)) return false;
  // heads of one token between those of others: row (t, h + j) against (t + i, h), the two i around j yh / yt
  for (int64_t j = 1; j < s.heads; ++j) {
    const __int128 at = (__int128)j * s.yh;
    const __int128 i = at / s.yt;
    const int64_t past = (int64_t)(at - i * s.yt);
    if ((i < n_tok && past < d) || (i + 1 < n_tok && s.yt - past < d)) return true;
  }
  return false;
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
  using real = long double;
  for (int i = 0; i < rot / 2; ++i) {
    real f = std::pow((real)base, (real)(-2 * i) / rot), keep = 1;  // keep: the share of f that is not slowed down
    if (scaling == TQ_ROPE_LINEAR) keep = 0;
    if (scaling == TQ_ROPE_BANDS)
      keep = std::fmin((real)1, std::fmax((real)0, (orig_len * f / (2 * M_PIl) - low) / ((real)high - low)));
    if (scaling == TQ_ROPE_YARN) {
      const double first = std::fmax(std::floor(pair_of(high)), 0.0);
      const double last = std::fmin(std::ceil(pair_of(low)), rot - 1.0);
      keep = 1 - std::fmin((real)1, std::fmax((real)0, (i - (real)first) / std::fmax(last - first, 1e-3)));
    }
    if (scaling != TQ_ROPE_PLAIN) f = f * keep + f / factor * (1 - keep);
    r->turn[i] = (uint64_t)(f / (2 * M_PIl) * 0x1p64L + 0.5L);
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
    if (s.xt < 0 || s.xh < 0 || rows_overlap(s, n_tok, d)) return TQ_ERR_INVALID_ARG;
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
  // as many heads a group as leave a group for every place on the GPU (512 threads per SM): the heads share a token's
  // sines, and a call of few rows is over sooner with a head each (500 x 18 x 192 fp32: 6.0 us, with two or three
  // groups a place 9.1; 1000 x 40 x 128 fp16: 6.4, 7.9 and 12.2)
  const int64_t heads = Hq + Hkv, places = (int64_t)tq::sm_count() * 512 / a.lanes;
  a.hpg = wide ? 1 : (int)std::min<int64_t>(16, std::max<int64_t>(1, n_tok * heads / places));
  a.blocks = (int)tq::ceil_div(heads, a.hpg);
  a.hpg = (int)tq::ceil_div(heads, a.blocks);  // even shares
  a.items = n_tok * a.blocks;
  a.n_tok = n_tok;
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
