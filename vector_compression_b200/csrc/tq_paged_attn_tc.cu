// The shapes of the tensor-core attention over pages, and the choice among its
// instantiations (tq_paged_attn_tc_*.cu).
#include <cmath>

#include "tq_attn_params.h"
#include "tq_paged_attn_tc.cuh"

namespace tq {
namespace paged {

namespace tc {
#define TQ_TC_KEYS(DP, MQ)                                                                                        \
  template <> cudaError_t launch_keys<1, DP, MQ>(const AttnArgs&, const TcBooks&, int, int, int, cudaStream_t); \
  template <> cudaError_t launch_keys<2, DP, MQ>(const AttnArgs&, const TcBooks&, int, int, int, cudaStream_t); \
  template <> cudaError_t launch_keys<3, DP, MQ>(const AttnArgs&, const TcBooks&, int, int, int, cudaStream_t);
TQ_TC_KEYS(64, 64)
TQ_TC_KEYS(128, 64)
TQ_TC_KEYS(128, 128)
TQ_TC_KEYS(256, 256)
#undef TQ_TC_KEYS

template <int KK, int KV, int NT, int DP, int MQ, bool FINE>
void fill(TcShape& s) {
  using S = Shape<KK, KV, NT, DP, MQ, FINE>;
  s.ctas_per_sm = S::CTAS;
  s.warps = S::WARPS;
  s.nt = NT;
  s.steps = S::STEPS;
  s.smem = S::SMEM;
}
template <int KK, int KV, int DP, int MQ, bool FINE>
void shape_nt(TcShape& s, int G) {
  // eight heads at a time where there are more than four: one pass over the cache serves them all.  At d_pad 256
  // their images and sums do not fit a warp's registers beside each other: groups of four, the cache read again
  if constexpr (DP < 256) {
    if (G > 4) return fill<KK, KV, 2, DP, MQ, FINE>(s);
  }
  fill<KK, KV, 1, DP, MQ, FINE>(s);
}
template <int KK, int DP, int MQ, bool FINE>
void shape_kv(TcShape& s, int kv, int G) {
  switch (kv) {
    case 1: return shape_nt<KK, 1, DP, MQ, FINE>(s, G);
    case 2: return shape_nt<KK, 2, DP, MQ, FINE>(s, G);
    case 3: return shape_nt<KK, 3, DP, MQ, FINE>(s, G);
    case 4: return shape_nt<KK, 4, DP, MQ, FINE>(s, G);
  }
}
template <int DP, int MQ, bool FINE>
void shape_kk(TcShape& s, int kk, int kv, int G) {
  switch (kk) {
    case 1: return shape_kv<1, DP, MQ, FINE>(s, kv, G);
    case 2: return shape_kv<2, DP, MQ, FINE>(s, kv, G);
    case 3: return shape_kv<3, DP, MQ, FINE>(s, kv, G);
  }
}
template <int DP, int MQ>
void shape_form(TcShape& s, int kk, int kv, int G, bool fine) {
  fine ? shape_kk<DP, MQ, true>(s, kk, kv, G) : shape_kk<DP, MQ, false>(s, kk, kv, G);
}
template <int DP, int MQ>
cudaError_t launch_shape(const AttnArgs& a, const TcBooks& k, int kk, int kv, int nt, int ctas, cudaStream_t st) {
  switch (kk) {
    case 1: return launch_keys<1, DP, MQ>(a, k, kv, nt, ctas, st);
    case 2: return launch_keys<2, DP, MQ>(a, k, kv, nt, ctas, st);
    default: return launch_keys<3, DP, MQ>(a, k, kv, nt, ctas, st);
  }
}
}  // namespace tc

TcShape tc_shape(int kk, int kv, int m, int dp, int G, bool fine) {
  TcShape s;
  if (dp == 64 && m == 64) tc::shape_form<64, 64>(s, kk, kv, G, fine);
  if (dp == 128 && m == 64) tc::shape_form<128, 64>(s, kk, kv, G, fine);
  if (dp == 128 && m == 128) tc::shape_form<128, 128>(s, kk, kv, G, fine);
  if (dp == 256 && m == 256) tc::shape_form<256, 256>(s, kk, kv, G, fine);
  return s;
}

cudaError_t tc_launch(const AttnArgs& a, const QParams& kq, const QParams& vq, const TcShape& s, int ctas, cudaStream_t st) {
  TcBooks k = {};
  float alpha[8], sum;
  attn::odd_feature_coefs(kq.centroids, kq.k, alpha, &sum);
  for (int f = 0; f < 4; ++f) k.kalpha[f] = f < 1 << (kq.k - 1) ? alpha[f] : 0.f;
  // value levels in 16 or 24 bits; of four-bit codes the upper half, as (v + 1/2) units, so that the lower half is the
  // complement
  const int n = 1 << vq.k, first = vq.k == 4 ? 8 : 0;
  const float top = vq.centroids[n - 1];
  const bool fine = fine_sums(a.dt);
  const double half = vq.k == 4 ? 0.5 : 0.0, steps = (fine ? 8388607.0 : 32767.0) + half;
  k.unit = (float)(top / steps);
  for (int i = first; i < n; ++i) {
    const int v = (int)std::lrint(vq.centroids[i] / (double)top * steps - half);
    const int at = i - first;
    const int to = 8 * (at % 4), up = fine ? 8 : 0;
    k.hi[at / 4] |= (uint32_t)((v >> (8 + up)) & 0xff) << to;
    k.lo[at / 4] |= (uint32_t)((v >> up) & 0xff) << to;
    if (fine) k.th[at / 4] |= (uint32_t)(v & 0xff) << to;
  }
  if (a.L.dp == 64) return tc::launch_shape<64, 64>(a, k, kq.k, vq.k, s.nt, ctas, st);
  if (a.L.dp == 128 && kq.m == 64) return tc::launch_shape<128, 64>(a, k, kq.k, vq.k, s.nt, ctas, st);
  if (a.L.dp == 128) return tc::launch_shape<128, 128>(a, k, kq.k, vq.k, s.nt, ctas, st);
  return tc::launch_shape<256, 256>(a, k, kq.k, vq.k, s.nt, ctas, st);
}

}  // namespace paged
}  // namespace tq
