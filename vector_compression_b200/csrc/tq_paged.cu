// The paged compressed cache: its description, the append of encoded tokens,
// and the page operations fork and compaction (include/tq.h).  All of them move
// bits and nothing else; memory traffic and launch latency are what they cost.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <new>

#include "tq_device.cuh"
#include "tq_paged.h"

namespace tq {
namespace paged {
namespace {

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool al256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }

// ---------------------------------------------------------------- append

struct AppendArgs {
  Layout L;
  Table tab;
  uint32_t* pool;
  int layer;
  const uint32_t *kcodes, *ksigns, *vcodes;
  const float *knorms, *krnorms, *vnorms;
  int64_t n_tok;
  int B;
  const int32_t *cu, *start;
  int per;    // tokens that a warp looks through for the first ones of runs
  int parts;  // of a run
};

// Transposes 32 x 32 bit matrices held one row per lane: afterwards bit t of
// lane j's word is bit j of lane t's.  The lanes with bit s swap their low parts
// with the partners' high parts: for s = 16 and 8 whole bytes, a permute each,
// then a rotation and a selection.
struct Transpose {
  uint32_t sel16, sel8, keep[3];
  int rot[3];
  __device__ __forceinline__ explicit Transpose(int lane) {
    sel16 = lane & 16 ? 0x3276u : 0x5410u;
    sel8 = lane & 8 ? 0x3715u : 0x6240u;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const int s = 4 >> i;
      const uint32_t m = s == 4 ? 0x0f0f0f0fu : s == 2 ? 0x33333333u : 0x55555555u;
      keep[i] = lane & s ? ~m : m;
      rot[i] = lane & s ? 32 - s : s;
    }
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t w) const {
    w = __byte_perm(w, __shfl_xor_sync(0xffffffffu, w, 16), sel16);
    w = __byte_perm(w, __shfl_xor_sync(0xffffffffu, w, 8), sel8);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const uint32_t o = __shfl_xor_sync(0xffffffffu, w, 4 >> i);
      w = (w & keep[i]) | (__funnelshift_l(o, o, rot[i]) & ~keep[i]);
    }
    return w;
  }
};

// The sequence that token i belongs to, its first and last+1 new token (packed
// numbers) and its start; false when i belongs to none.  Called by a whole warp.
__device__ __forceinline__ bool find_sequence(const AppendArgs& A, int i, int lane, int& b, int& t0, int& t1, int& start) {
  int lo = 0, n = A.B;  // the last b with cu[b] <= i is in [lo, lo + n)
  while (n > 32) {
    const int step = (n + 31) / 32;
    const uint32_t le = __ballot_sync(0xffffffffu, lane * step < n && A.cu[lo + lane * step] <= i);
    const int last = le ? 31 - __clz((int)le) : 0;
    lo += last * step;
    n = min(step, n - last * step);
  }
  // of at most 32 each lane holds one: what is asked of the found one is there already
  const int c0 = lane < n ? A.cu[lo + lane] : 0, c1 = lane < n ? A.cu[lo + lane + 1] : 0;
  const int st = lane < n ? A.start[lo + lane] : 0;
  const uint32_t le = __ballot_sync(0xffffffffu, lane < n && c0 <= i);
  const int last = le ? 31 - __clz((int)le) : 0;
  b = lo + last;
  t0 = __shfl_sync(0xffffffffu, c0, last);
  t1 = min(__shfl_sync(0xffffffffu, c1, last), (int)A.n_tok);
  start = __shfl_sync(0xffffffffu, st, last);
  return t0 <= i && i < t1;
}

// Bits of the plane words p (bit t: token t) that go to value word q.
template <int KV>
__device__ __forceinline__ uint32_t place(const uint32_t (&p)[KV], int q) {
  if (KV == 1) return p[0];
  constexpr uint32_t m = 0x11111111u;
  if (KV == 4) {
    // sign and magnitude: bit 3 below zero, bits 0..2 the distance from the middle
    const uint32_t n = ~p[3 % KV];
    return (((p[0] ^ n) >> q) & m) | ((((p[1 % KV] ^ n) >> q) & m) << 1) | ((((p[2 % KV] ^ n) >> q) & m) << 2) |
           (((n >> q) & m) << 3);
  }
  if (q == 2) return __funnelshift_l(p[2 % KV], p[2 % KV], 2);
  if (q == 0) return (p[0] & m) | ((p[1 % KV] & m) << 1) | ((p[0] & 2 * m) << 1) | ((p[1 % KV] & 2 * m) << 2);
  return ((p[0] >> 2) & m) | ((p[1 % KV] >> 1) & 2 * m) | ((p[0] >> 1) & 4 * m) | (p[1 % KV] & 8 * m);
}

// Where a run goes: the record of its block, given the page as read from the table; null in a hole.
__device__ __forceinline__ uint32_t* record_of(const AppendArgs& A, int32_t page, int blk, int h) {
  const int64_t at = record_in(A.L, A.tab, page, blk, A.layer, h);
  return at < 0 ? nullptr : A.pool + at;
}

template <int G>
struct Granule {
  using type = uint32_t;
};
template <>
struct Granule<2> {
  using type = uint2;
};
template <>
struct Granule<4> {
  using type = uint4;
};

// The key words of this lane's token, in granules of G words that lie in one of the two rows each.
template <int G>
__device__ __forceinline__ void write_keys(const AppendArgs& A, int32_t page, int blk, int h, int64_t row, int lane) {
  using V = typename Granule<G>::type;
  const Layout& L = A.L;
  const uint32_t *c = A.kcodes + row * L.kw, *s = A.ksigns + row * L.sw;
  uint32_t* rec = nullptr;
  for (int p0 = 0; p0 < L.nk; p0 += 4 * G) {
    V v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int p = p0 + i * G;
      if (p < L.nk) v[i] = *reinterpret_cast<const V*>(p < L.kw ? c + p : s + (p - L.kw));
    }
    if (!rec && !(rec = record_of(A, page, blk, h))) return;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (p0 + i * G < L.nk) *reinterpret_cast<V*>(rec + (p0 + i * G) * 32 + lane * G) = v[i];
  }
}

constexpr int kPartWords = 2;  // value words per plane (32 coordinates each) of a part

// The new tokens that one 32-token block of one head gets (a run): tok .. tok +
// len - 1 at places off ...; a lane is a token for the keys and a coordinate of
// 32 for the values.  Part 0 is the keys and norms, part 1 + i some of the
// coordinates' value words: warps of their own, a run's latency is theirs.  What
// is written is read before the page's number is looked at, so that the two
// latencies are one.
template <int KV>
__device__ __forceinline__ void write_run(const AppendArgs& A, int32_t page, int blk, int h, int tok, int off,
                                          int len, int part, int lane) {
  const Layout& L = A.L;
  const bool mine = lane >= off && lane < off + len;
  const int64_t row0 = (int64_t)tok * L.hkv + h, row = row0 + (lane - off) * L.hkv;
  if (part == 0) {
    if (!mine) return;
    const float kn = A.knorms[row], vn = A.vnorms[row];
    const uint32_t kr = L.r16 ? reinterpret_cast<const uint16_t*>(A.krnorms)[row] : __float_as_uint(A.krnorms[row]);
    if (L.gr == 4 && L.kw % 4 == 0) write_keys<4>(A, page, blk, h, row, lane);
    else if (L.gr == 2 && L.kw % 2 == 0) write_keys<2>(A, page, blk, h, row, lane);
    uint32_t* rec = record_of(A, page, blk, h);
    if (!rec) return;
    if (L.kw % L.gr != 0 || L.gr == 1) {  // a granule with words of both rows
      const uint32_t *c = A.kcodes + row * L.kw, *s = A.ksigns + row * L.sw;
      for (int w = 0; w < L.nk; ++w) rec[key_word_at(L, lane, w)] = w < L.kw ? c[w] : s[w - L.kw];
    }
    rec[L.o_kn + lane] = __float_as_uint(kn);
    rec[L.o_vn + lane] = __float_as_uint(vn);
    if (L.r16) reinterpret_cast<uint16_t*>(rec + L.o_kr)[lane] = (uint16_t)kr;
    else rec[L.o_kr + lane] = kr;
    return;
  }
  const uint32_t own = (len == 32 ? 0xffffffffu : ((1u << len) - 1u)) << off;  // the run's tokens
  const int wpp = L.dp / 32, jw0 = (part - 1) * kPartWords;
  // plane words of the part's coordinates: of a lane's token, or of a coordinate's few tokens
  uint32_t p[kPartWords][KV];
#pragma unroll
  for (int j = 0; j < kPartWords; ++j)
#pragma unroll
    for (int q = 0; q < KV; ++q) p[j][q] = 0;
  if (len <= 4) {  // below that many tokens picking their bits is shorter than the transposition of 32
    for (int i = 0; i < len; ++i) {
      const uint32_t* v = A.vcodes + (row0 + (int64_t)i * L.hkv) * (KV * wpp);
#pragma unroll
      for (int j = 0; j < kPartWords; ++j)
#pragma unroll
        for (int q = 0; q < KV; ++q)
          if (jw0 + j < wpp) p[j][q] |= ((v[q * wpp + jw0 + j] >> lane) & 1u) << (off + i);
    }
  } else if (mine) {
    const uint32_t* v = A.vcodes + row * (KV * wpp);
#pragma unroll
    for (int j = 0; j < kPartWords; ++j)
#pragma unroll
      for (int q = 0; q < KV; ++q)
        if (jw0 + j < wpp) p[j][q] = v[q * wpp + jw0 + j];
  }
  uint32_t* rec = record_of(A, page, blk, h);
  if (!rec) return;
  const Transpose transpose(lane);
  // the bits of the run's fields: the same placement of codes of ones (of four-bit codes a field's bits lie in one word)
  uint32_t ones[KV];
#pragma unroll
  for (int q = 0; q < KV; ++q) ones[q] = own;
#pragma unroll
  for (int j = 0; j < kPartWords; ++j) {
    if (jw0 + j >= wpp) break;
    uint32_t* w = rec + L.o_v + 32 * (jw0 + j) + lane;
    if (len > 4) {
#pragma unroll
      for (int q = 0; q < KV; ++q) p[j][q] = transpose(p[j][q]);
    }
#pragma unroll
    for (int q = 0; q < KV; ++q) {
      uint32_t v = place<KV>(p[j], q);
      if (len < 32) {
        const uint32_t msk = KV == 4 ? ((own >> q) & 0x11111111u) * 15u : place<KV>(ones, q);
        v = (w[q * L.dp] & ~msk) | (v & msk);
      }
      w[q * L.dp] = v;
    }
  }
}

// Block (4 tiles of tokens, head and part), a warp per tile.
template <int KV>
__global__ void __launch_bounds__(128, 6) append_kernel(const AppendArgs A) {
  const Layout& L = A.L;
  const int lane = threadIdx.x & 31;
  const int h = blockIdx.y / A.parts, part = blockIdx.y - h * A.parts;
  const int64_t first = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 5)) * A.per;
  if (first >= A.n_tok) return;
  const int end = (int)min64(A.n_tok, first + A.per);
  int b = 0, t0 = 0, t1 = 0, start = 0;
  for (int tok = (int)first; tok < end;) {
    if (!A.cu) {
      b = t0 = tok;
      t1 = tok + 1;
      start = A.start[b];
    } else if (tok >= t1 && !find_sequence(A, tok, lane, b, t0, t1, start)) {
      t1 = ++tok;
      continue;
    }
    const int64_t pos = (int64_t)start + tok - t0;
    const int off = (int)pos & 31;
    const int len = min(32 - off, t1 - tok);
    // a sequence's first new token begins a run, and so does every block's first
    if ((tok == t0 || off == 0) && pos >= 0 && pos < (int64_t)A.tab.max_pages * L.page) {
      const int blk = (int)(pos >> 5);
      write_run<KV>(A, page_entry(L, A.tab, b, blk), blk, h, tok, off, len, part, lane);
    }
    tok += len;
  }
}

// ---------------------------------------------------------------- copying

// Copies n 16-byte words by the calling warp, four in flight per lane.
__device__ __forceinline__ void warp_copy(uint4* dst, const uint4* src, int64_t n, int lane) {
  int64_t i = lane;
  for (; i + 96 < n; i += 128) {
    const uint4 a = src[i], b = src[i + 32], c = src[i + 64], d = src[i + 96];
    dst[i] = a;
    dst[i + 32] = b;
    dst[i + 64] = c;
    dst[i + 96] = d;
  }
  for (; i < n; i += 32) dst[i] = src[i];
}

struct ForkArgs {
  Layout L;
  uint32_t* pool;
  int64_t n_pages;
  int32_t* tables;
  int64_t ld;
  int max_pages;
  int32_t* lens;
  int B;
  const int32_t *parents, *children, *fresh;
  int n;
};

// Item (i, segment): a warp copies the used blocks of the tail page of fork i
// for one layer and head; segment 0's warp also writes the child's table row
// and length.
__global__ void __launch_bounds__(256) fork_kernel(const ForkArgs A) {
  const Layout& L = A.L;
  const int lane = threadIdx.x & 31;
  const int64_t segs = (int64_t)L.layers * L.hkv;
  const int64_t warps = ((int64_t)gridDim.x * blockDim.x) >> 5;
  for (int64_t item = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5; item < A.n * segs; item += warps) {
    const int i = (int)(item / segs);
    const int64_t seg = item - i * segs;
    const int par = A.parents[i], ch = A.children[i];
    if (par < 0 || par >= A.B || ch < 0 || ch >= A.B) continue;
    const int len = clamp_len(A.lens[par], L, A.max_pages);
    const int full = len / L.page, rest = len - full * L.page;
    const int32_t* from = A.tables + par * A.ld;
    const int fresh = A.fresh[i];
    // a hole stays one: there is nothing to copy into a fresh page
    const int32_t src = rest ? from[full] : -1;
    const bool ok = src >= 0 && src < A.n_pages && fresh >= 0 && fresh < A.n_pages;
    if (seg == 0) {
      int32_t* to = A.tables + ch * A.ld;
      for (int p = lane; p < A.max_pages; p += 32)
        to[p] = p < full ? from[p] : (p == full && ok) ? fresh : -1;
      if (lane == 0) A.lens[ch] = len;
    }
    if (!ok) continue;
    const int64_t at = seg * L.nb * L.words;
    warp_copy(reinterpret_cast<uint4*>(A.pool + fresh * L.page_words + at),
              reinterpret_cast<const uint4*>(A.pool + src * L.page_words + at),
              (int64_t)((rest + 31) / 32) * (L.words / 4), lane);
  }
}

// ---------------------------------------------------------------- compaction

struct CompactArgs {
  Layout L;
  uint32_t* pool;
  int64_t n_pages;
  const int32_t* tables;
  int32_t* tables_out;
  int64_t ld;
  int max_pages;
  const int32_t* lens;
  int B;
  int32_t* n_used;
  // workspace
  uint32_t* used;   // a bit per page
  int32_t* rank;    // per page: number among the pages to move, -1 for the others
  int32_t* from;    // pages to move, ascending
  int32_t* to;      // unused pages below n_used, ascending
  int32_t* moves;   // how many
};

// The page that entry p of row b names, -1 where the row does not need one.
__device__ __forceinline__ int32_t live_entry(const CompactArgs& A, int64_t b, int p) {
  const int len = clamp_len(A.lens[b], A.L, A.max_pages);
  if ((int64_t)p * A.L.page >= len) return -1;
  const int32_t id = A.tables[b * A.ld + p];
  return id < 0 || id >= A.n_pages ? -1 : id;
}

__global__ void __launch_bounds__(256) mark_kernel(const CompactArgs A) {
  let_next_start();
  const int64_t n = (int64_t)A.B * A.max_pages;
  for (int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; e < n; e += (int64_t)gridDim.x * blockDim.x) {
    const int64_t b = e / A.max_pages;
    const int32_t id = live_entry(A, b, (int)(e - b * A.max_pages));
    if (id >= 0) atomicOr(&A.used[id >> 5], 1u << (id & 31));  // bits: the order does not matter
  }
}

// Each block owns 256 words of the bit map; it counts the words before its own
// and all words itself (the map is small), so the blocks need not wait for one
// another.
__global__ void __launch_bounds__(256) plan_kernel(const CompactArgs A) {
  __shared__ int s_sum[8][2];
  __shared__ int s_scan[8];
  wait_for_previous();
  let_next_start();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int words = (int)((A.n_pages + 31) / 32);
  const int w0 = blockIdx.x * 256;
  int before = 0, total = 0;
  for (int w = tid; w < words; w += 256) {
    const int c = __popc(A.used[w]);
    total += c;
    before += w < w0 ? c : 0;
  }
  before = __reduce_add_sync(0xffffffffu, before);
  total = __reduce_add_sync(0xffffffffu, total);
  if (lane == 0) s_sum[warp][0] = before, s_sum[warp][1] = total;
  const int w = w0 + tid;
  const uint32_t bits = w < words ? A.used[w] : 0u;
  int scan = __popc(bits);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += x;
  }
  if (lane == 31) s_scan[warp] = scan;
  __syncthreads();
  before = total = 0;
#pragma unroll
  for (int v = 0; v < 8; ++v) {
    before += s_sum[v][0] + (v < warp ? s_scan[v] : 0);
    total += s_sum[v][1];
  }
  before += scan - __popc(bits);  // used pages before this thread's word
  // used pages below n_used, and so how many have to move
  __shared__ int s_below[8];
  int below = 0;
  for (int v = tid; v <= total / 32 && v < words; v += 256) {
    const uint32_t x = A.used[v];
    below += __popc(v < total / 32 ? x : x & ((1u << (total & 31)) - 1u));
  }
  below = __reduce_add_sync(0xffffffffu, below);
  if (lane == 0) s_below[warp] = below;
  __syncthreads();
  below = 0;
#pragma unroll
  for (int v = 0; v < 8; ++v) below += s_below[v];
  if (blockIdx.x == 0 && tid == 0) {
    *A.n_used = total;
    *A.moves = total - below;
  }
  if (w >= words) return;
  for (int i = 0; i < 32 && (int64_t)32 * w + i < A.n_pages; ++i) {
    const int id = 32 * w + i;
    const int ahead = before + __popc(bits & ((1u << i) - 1u));
    const bool used = (bits >> i) & 1u;
    int r = -1;
    if (used && id >= total) {
      r = ahead - below;
      A.from[r] = id;
    } else if (!used && id < total) {
      A.to[id - ahead] = id;
    }
    A.rank[id] = r;
  }
}

// mark and plan in one CTA, the bit map and its prefix sums in shared memory.
__global__ void __launch_bounds__(1024) plan_small_kernel(const CompactArgs A) {
  extern __shared__ uint32_t map[];  // [words] bits, then [words] used pages before a word
  __shared__ int s_warp[32];
  let_next_start();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n_pages = (int)A.n_pages, words = (n_pages + 31) / 32;
  int* pre = reinterpret_cast<int*>(map + words);
  for (int w = tid; w < words; w += 1024) map[w] = 0;
  __syncthreads();
  const int n = A.B * A.max_pages;
  for (int e = tid; e < n; e += 1024) {
    const int b = e / A.max_pages;
    const int32_t id = live_entry(A, b, e - b * A.max_pages);
    if (id >= 0) atomicOr(&map[id >> 5], 1u << (id & 31));  // bits: the order does not matter
  }
  __syncthreads();
  const int per = (words + 1023) / 1024, w0 = min(tid * per, words), w1 = min(w0 + per, words);
  int own = 0;
  for (int w = w0; w < w1; ++w) own += __popc(map[w]);
  int upto = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  if (lane == 31) s_warp[warp] = upto;
  __syncthreads();
  const int sums = s_warp[lane];
  const int total = __reduce_add_sync(0xffffffffu, sums);
  int before = __reduce_add_sync(0xffffffffu, lane < warp ? sums : 0) + upto - own;
  for (int w = w0; w < w1; ++w) {
    pre[w] = before;
    before += __popc(map[w]);
  }
  __syncthreads();
  // used pages below n_used, and so how many have to move
  const int below = total >= n_pages ? total : pre[total >> 5] + __popc(map[total >> 5] & ((1u << (total & 31)) - 1u));
  if (tid == 0) {
    *A.n_used = total;
    *A.moves = total - below;
  }
  for (int id = tid; id < n_pages; id += 1024) {
    const uint32_t bits = map[id >> 5];
    const int ahead = pre[id >> 5] + __popc(bits & ((1u << (id & 31)) - 1u));
    const bool used = (bits >> (id & 31)) & 1u;
    int r = -1;
    if (used && id >= total) {
      r = ahead - below;
      A.from[r] = id;
    } else if (!used && id < total) {
      A.to[id - ahead] = id;
    }
    A.rank[id] = r;
  }
}

// Moves the pages, in pieces of `piece` 16-byte words (a warp each), and
// rewrites the tables.  Sources lie at and above n_used, destinations below it
// on unused pages: no piece is read after another has written it.
__global__ void __launch_bounds__(256) move_kernel(const CompactArgs A, int piece) {
  const int lane = threadIdx.x & 31;
  wait_for_previous();
  const int64_t tid = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, threads = (int64_t)gridDim.x * blockDim.x;
  const int64_t n = (int64_t)A.B * A.max_pages;
  for (int64_t e = tid; e < n; e += threads) {
    const int64_t b = e / A.max_pages;
    const int p = (int)(e - b * A.max_pages);
    int32_t id = live_entry(A, b, p);
    if (id >= 0 && A.rank[id] >= 0) id = A.to[A.rank[id]];
    A.tables_out[b * A.ld + p] = id;
  }
  const int64_t quads = A.L.page_words / 4, pieces = (quads + piece - 1) / piece;
  const int64_t items = *A.moves * pieces;
  for (int64_t it = tid >> 5; it < items; it += threads >> 5) {
    const int64_t m = it / pieces, at = (it - m * pieces) * piece;
    warp_copy(reinterpret_cast<uint4*>(A.pool + A.to[m] * A.L.page_words) + at,
              reinterpret_cast<const uint4*>(A.pool + A.from[m] * A.L.page_words) + at, min64(piece, quads - at), lane);
  }
}

// One CTA plans up to this many table entries and 32-page words of the map.
constexpr int64_t kSmallEntries = 32768, kSmallWords = 4096;

size_t round256(size_t b) { return (b + 255) & ~(size_t)255; }

}  // namespace
}  // namespace paged
}  // namespace tq

extern "C" tq_status tq_paged_create(const tq_params* kp, const tq_params* vp, int layers, int Hkv, int page,
                                     tq_paged** out) {
  if (!out) return TQ_ERR_INVALID_ARG;
  *out = nullptr;
  if (layers < 1 || layers > 4096 || Hkv < 1 || Hkv > 1024 || page < 32 || page > 65536 || page % 32)
    return TQ_ERR_INVALID_ARG;
  if (!kp || !vp || kp->mode != TQ_MODE_PROD || (vp->mode != TQ_MODE_MSE && vp->mode != TQ_MODE_MSE_UNBIASED))
    return TQ_ERR_INVALID_ARG;
  if (kp->q.d != vp->q.d || kp->q.rot != vp->q.rot) return TQ_ERR_INVALID_ARG;
  if (kp->q.rot != TQ_ROT_HADAMARD) return TQ_ERR_UNSUPPORTED;
  tq_paged* pg = new (std::nothrow) tq_paged();
  if (!pg) return TQ_ERR_INTERNAL;
  pg->kq = kp->q;
  pg->vq = vp->q;
  pg->device = kp->device;
  tq::paged::Layout& L = pg->lay;
  L.kw = kp->q.code_words;
  L.sw = kp->q.sign_words;
  L.nk = L.kw + L.sw;
  L.gr = L.nk % 4 == 0 ? 4 : L.nk % 2 == 0 ? 2 : 1;
  L.kv = vp->q.k;
  L.dp = vp->q.d_pad;
  L.r16 = kp->q.rnorm_f16;
  L.o_kn = 32 * L.nk;
  L.o_kr = L.o_kn + 32;
  L.o_v = L.o_kr + (L.r16 ? 16 : 32);
  L.o_vn = L.o_v + L.kv * L.dp;
  L.words = L.o_vn + 32;
  L.nb = page / 32;
  L.nb_shift = -1;
  for (int i = 0; i < 16; ++i)
    if (L.nb == 1 << i) L.nb_shift = i;
  L.layers = layers;
  L.hkv = Hkv;
  L.page = page;
  L.page_words = (int64_t)layers * Hkv * L.nb * L.words;
  *out = pg;
  return TQ_OK;
}

extern "C" tq_status tq_paged_destroy(tq_paged* pg) {
  delete pg;
  return TQ_OK;
}

extern "C" tq_status tq_paged_info(const tq_paged* pg, int* block_words, int64_t* page_words) {
  if (!pg) return TQ_ERR_INVALID_ARG;
  if (block_words) *block_words = pg->lay.words;
  if (page_words) *page_words = pg->lay.page_words;
  return TQ_OK;
}

extern "C" tq_status tq_paged_append(const tq_paged* pg, uint32_t* pool, int64_t n_pages, int layer,
                                     const uint32_t* kcodes, const uint32_t* ksigns, const float* knorms,
                                     const float* krnorms, const uint32_t* vcodes, const float* vnorms, int64_t n_tok,
                                     int B, const int32_t* cu, const int32_t* start, const int32_t* tables,
                                     int64_t table_ld, int max_pages, void* stream) {
  using namespace tq::paged;
  if (!pg) return TQ_ERR_INVALID_ARG;
  const Layout& L = pg->lay;
  if (n_tok < 0 || n_tok > 0x7fffffffll || B < 0 || layer < 0 || layer >= L.layers || (!cu && n_tok != B))
    return TQ_ERR_INVALID_ARG;
  if (n_tok == 0 || B == 0) return TQ_OK;
  if (bad_pool(L, pool, n_pages) || bad_table(L, tables, table_ld, max_pages)) return TQ_ERR_INVALID_ARG;
  if (!kcodes || !ksigns || !knorms || !krnorms || !vcodes || !vnorms || !start || mis4(start) || mis4(cu))
    return TQ_ERR_INVALID_ARG;
  // key words are read in granules where those lie in one row each, the others one by one: any row can be the first
  const uintptr_t unit = L.kw % L.gr == 0 ? 4 * L.gr : 4;
  if (!aligned(kcodes, unit) || !aligned(ksigns, unit) || !aligned(vcodes, 4) || !aligned(knorms, 4) ||
      !aligned(vnorms, 4) || !aligned(krnorms, L.r16 ? 2 : 4))
    return TQ_ERR_INVALID_ARG;
  // A step's tokens are a run each, and wait for no other: a warp each.  Of prompts a warp looks through 32, in which
  // one block begins; of shorter sequences through 8, of which several can begin a run.
  const int per = !cu ? 1 : n_tok / B >= 64 ? 32 : 8;
  const int parts = 1 + (L.dp / 32 + kPartWords - 1) / kPartWords;
  AppendArgs a = {L, {tables, table_ld, max_pages, n_pages}, pool, layer, kcodes, ksigns, vcodes, knorms, krnorms,
                  vnorms, n_tok, B, cu, start, per, parts};
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const dim3 grid((unsigned)tq::ceil_div(tq::ceil_div(n_tok, per), 4), L.hkv * parts);
  switch (L.kv) {
    case 1: append_kernel<1><<<grid, 128, 0, st>>>(a); break;
    case 2: append_kernel<2><<<grid, 128, 0, st>>>(a); break;
    case 3: append_kernel<3><<<grid, 128, 0, st>>>(a); break;
    default: append_kernel<4><<<grid, 128, 0, st>>>(a); break;
  }
  return cudaGetLastError() == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

extern "C" tq_status tq_paged_fork(const tq_paged* pg, uint32_t* pool, int64_t n_pages, int32_t* tables,
                                   int64_t table_ld, int max_pages, int32_t* lens, int B, const int32_t* parents,
                                   const int32_t* children, const int32_t* fresh, int n, void* stream) {
  using namespace tq::paged;
  if (!pg || n < 0 || B < 0) return TQ_ERR_INVALID_ARG;
  const Layout& L = pg->lay;
  if (n == 0) return TQ_OK;
  if (bad_pool(L, pool, n_pages) || bad_table(L, tables, table_ld, max_pages)) return TQ_ERR_INVALID_ARG;
  if (!lens || !parents || !children || !fresh || mis4(lens) || mis4(parents) || mis4(children) || mis4(fresh))
    return TQ_ERR_INVALID_ARG;
  ForkArgs a = {L, pool, n_pages, tables, table_ld, max_pages, lens, B, parents, children, fresh, n};
  const int64_t items = (int64_t)n * L.layers * L.hkv;
  const int64_t blocks = std::min<int64_t>(tq::ceil_div(items, 8), (int64_t)tq::sm_count() * 8);
  fork_kernel<<<(unsigned)blocks, 256, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

extern "C" tq_status tq_paged_compact_workspace_size(int64_t n_pages, size_t* bytes) {
  if (!bytes || n_pages < 1 || n_pages > 0x7fffffffll) return TQ_ERR_INVALID_ARG;
  using tq::paged::round256;
  *bytes = 256 + round256((size_t)(n_pages + 31) / 32 * 4) + 3 * round256((size_t)n_pages * 4);
  return TQ_OK;
}

extern "C" tq_status tq_paged_compact(const tq_paged* pg, uint32_t* pool, int64_t n_pages, const int32_t* tables,
                                      int32_t* tables_out, int64_t table_ld, int max_pages, const int32_t* lens,
                                      int B, int32_t* n_used, void* ws, size_t ws_bytes, void* stream) {
  using namespace tq::paged;
  if (!pg || B < 0) return TQ_ERR_INVALID_ARG;
  const Layout& L = pg->lay;
  if (bad_pool(L, pool, n_pages) || !n_used || mis4(n_used)) return TQ_ERR_INVALID_ARG;
  if (B > 0 && (bad_table(L, tables, table_ld, max_pages) || bad_table(L, tables_out, table_ld, max_pages) || !lens ||
                mis4(lens)))
    return TQ_ERR_INVALID_ARG;
  size_t need = 0;
  tq_paged_compact_workspace_size(n_pages, &need);
  if (!ws || ws_bytes < need || !al256(ws)) return TQ_ERR_WORKSPACE;
  char* w = static_cast<char*>(ws);
  const size_t map = round256((size_t)(n_pages + 31) / 32 * 4), list = round256((size_t)n_pages * 4);
  CompactArgs a = {L, pool, n_pages, tables, tables_out, table_ld, max_pages, lens, B, n_used,
                   reinterpret_cast<uint32_t*>(w + 256), reinterpret_cast<int32_t*>(w + 256 + map),
                   reinterpret_cast<int32_t*>(w + 256 + map + list), reinterpret_cast<int32_t*>(w + 256 + map + 2 * list),
                   reinterpret_cast<int32_t*>(w)};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int64_t entries = (int64_t)B * max_pages, words = (n_pages + 31) / 32;
  const int sms = tq::sm_count();
  cudaError_t e = cudaSuccess;
  if (entries <= kSmallEntries && words <= kSmallWords) {
    plan_small_kernel<<<1, 1024, (size_t)words * 8, st>>>(a);
  } else {
    e = cudaMemsetAsync(a.used, 0, (size_t)words * 4, st);
    if (e == cudaSuccess && entries > 0)
      mark_kernel<<<(unsigned)std::min<int64_t>(tq::ceil_div(entries, 256), (int64_t)sms * 8), 256, 0, st>>>(a);
    if (e == cudaSuccess) {
      const dim3 plan((unsigned)tq::ceil_div(words, 256));
      if (entries > 0) e = launch_after(plan_kernel, plan, 256, 0, st, a);
      else plan_kernel<<<plan, 256, 0, st>>>(a);  // behind the memset
    }
  }
  if (e == cudaSuccess) e = launch_after(move_kernel, dim3((unsigned)(sms * 8)), 256, 0, st, a, 512);
  if (e != cudaSuccess) return TQ_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}
