// Attention over a paged compressed cache on the 8-bit integer tensor cores,
// for d_pad 64, 128 and 256 (tq_paged_attn.cuh: the split of the work).
//
// A warp is a worker: it takes its share of 32-token block records four at a
// time (a unit, here a group), keys and values each staged by bulk copies; the
// next group's keys load while this one's values are summed, its values while
// the next keys are scored.  No warp waits for another.
//
// Scores.  With the codebook an odd function of its index bits, C[idx] = sum_S
// alpha_S (2 b_S - 1) over the odd subsets S of the bits (b_S their XOR), the
// contractions are against 0/1 bits: <q', b_S> per subset and <u, sigma>.  An
// MMA's A rows are tokens, its K four bytes of the word that each of four
// threads holds: (word or word >> 4) & (0x01010101 << j) are four of its bits
// with value 2^j, nine instructions for a word's 32.  The B operand carries
// q' / 2^j in fixed point, three signed bytes: hi and mid of heads 4 nt ..
// 4 nt + 3 are tile nt (columns 2 h, 2 h + 1), lo of all of them one more tile
// (columns 2 h, 2 h + 1: heads h and 4 + h), so that thread column tig holds all
// of head tig (and 4 + tig).  The queries' images are made once per call
// (queries_kernel).  Seven masks of whole bytes (differences of q' / 2^j, j =
// 0 .. 7) were 2% faster and 16 times coarser.
//
// Values.  The value words of a coordinate (tq_paged_create) turn into 3-bit
// selectors of eight tokens with two to four bit operations, and byte permutes
// of a table turn the selectors into the levels' bytes: 16-bit levels, signed
// hi and unsigned lo byte, four tokens a permute.  Rows are coordinates, K the
// tokens 4 i + s of the group's four blocks (thread column tig: block tig), B
// the weights p ||v|| as two bytes (columns 2 h, 2 h + 1) relative to the
// group's largest.  Products and sums are exact integers; the roundings are
// those of q', u (2^-24 to 2^-21 of the largest entry by the bit's place), the
// levels and the weights (2^-16 of the largest), and fp32 outside.
//
// 16-bit levels and weights put an output 2e-5 to 6e-5 off (of its 2-norm), a
// tenth of the rounding to fp16 that follows, and a hundred times what fp32
// holds.  So fp32 outputs take the FINE form: levels of 24 bits and weights of
// 23 (what a float's significand gives without further instructions), three
// bytes each, of whose nine products the one below 2^-30 is left out: 2e-7 to
// 5e-7, as fp32 sums.  The third byte of the weights is a tile of its own, laid
// out as that of the queries.  A call of the case below takes 97 us so instead of
// 85, one of 48 sequences of 0 to 6000 tokens with 2 x 8 heads 41 instead of 38.
//
// What bounds it (8 sequences of 31 thousand tokens, 8 KV heads of 4 query
// heads, d = m = 128, 3 bits: 79 us, 2.7 TB/s, of 33 us that the bytes take): the
// ALU (52% busy: masks, permutes) and the tensor pipe (39%), which overlap only
// in part; with 4, 8 and 12 warps an SM it takes 104, 80 and 78 us.
#pragma once

#include "tq_paged_attn.cuh"
#include "tq_wait.cuh"

namespace tq {
namespace paged {
namespace tc {

template <int KK, int KV, int NT, int DP, int MQ, bool FINE>
struct Shape {
  static constexpr int WPP = DP / 32, SW = MQ / 32, NK = KK * WPP + SW;
  static constexpr int GR = NK % 4 == 0 ? 4 : 2;
  static constexpr int FK = 1 << (KK - 1);  // odd subsets
  static constexpr int NQ = NT + 1;         // tiles of the scores
  static constexpr int STEPS = WPP + SW;
  static constexpr int KB = 32 * NK + 64;        // staged words of a block's keys
  static constexpr int VB = KV * DP + 32 + 8;    // and values: 8 mod 32, so that four blocks are on different banks
  static constexpr int WC = 36;                  // words of a column of weights (32 and a gap)
  // the group's scores (a thread's own four of each block), and then its weights
  static constexpr int WT = NT + FINE;           // tiles of the weights
  static constexpr int XW = 4 * 32 * 4 * NT > 8 * WT * WC ? 4 * 32 * 4 * NT : 8 * WT * WC;
  // the running sums: in shared memory the loop over coordinates need not be unrolled (a fourth of the code, which a
  // short call fetches for one use) and 16 registers a tile are free; at d_pad 256 two warps of an SM's eight would not fit
  static constexpr bool O_SMEM = DP < 256;
  static constexpr int OW = O_SMEM ? DP / 32 * 32 * 4 * NT : 0;
  static constexpr int WARP_BYTES = 4 * (4 * KB + 4 * VB + XW + OW) + 16;
  static constexpr int WARPS = 2;
  static constexpr int SMEM = WARPS * WARP_BYTES;
  // resident CTAs: the shared memory's limit, and the registers'.  Two tiles of heads at five CTAs (168 registers, ten
  // warps on four schedulers) took 81 us where four take 69 (8 sequences of 31 thousand tokens, 4 KV heads of 8)
  static constexpr int BY_SMEM = 233472 / (SMEM + 1024);
  static constexpr int BY_REGS = DP == 64 ? 8 : DP == 128 ? (NT == 1 ? 6 : 4) : 4;
  static constexpr int CTAS = BY_SMEM < BY_REGS ? BY_SMEM : BY_REGS;
  static_assert(NK % 2 == 0 && CTAS >= 1, "shape");
};

__device__ __forceinline__ uint32_t smem_at(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ void mma_us(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint2 b) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b.x), "r"(b.y));
}
__device__ __forceinline__ void mma_su(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint2 b) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.u8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b.x), "r"(b.y));
}
__device__ __forceinline__ void mma_uu(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint2 b) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.u8.u8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b.x), "r"(b.y));
}

__device__ __forceinline__ float pow2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Place of word base + wt of token 0 in the staged key words, wt in [0, 4); a token is GR words further.
template <int GR>
__device__ __forceinline__ int word_place(int base, int wt) {
  if (GR == 4) return base / 4 * 128 + base % 4 + wt;
  return (base / 2 + wt / 2) * 64 + wt % 2;
}

// Selectors (nibbles) of the eight tokens 4 i + s from a coordinate's value words.
template <int KV>
__device__ __forceinline__ uint32_t selectors(const uint32_t (&w)[KV], int s) {
  if (KV == 1) return (w[0] >> s) & 0x11111111u;
  if (KV == 4) return w[s % KV];
  const uint32_t a = w[(s >> 1) % KV] >> (2 * (s & 1));
  if (KV == 2) return a & 0x33333333u;
  const uint32_t b = s < 2 ? w[KV - 1] >> s : __funnelshift_r(w[KV - 1], w[KV - 1], s);
  return (a & 0x33333333u) | (b & 0x44444444u);
}

// A byte of four tokens' levels; x: their selectors in the low 16 bits (KV = 4:
// without the signs), flip: 0xff where the level is below zero.
template <int KV>
__device__ __forceinline__ uint32_t levels(const uint32_t (&book)[2], uint32_t x, uint32_t flip) {
  const uint32_t v = __byte_perm(book[0], KV >= 3 ? book[1] : 0u, x);
  return KV == 4 ? v ^ flip : v;
}

template <int KK, int KV, int NT, int DP, int MQ, bool FINE>
__global__ void __launch_bounds__(64, Shape<KK, KV, NT, DP, MQ, FINE>::CTAS)
    attention_tc_kernel(const __grid_constant__ AttnArgs A, const __grid_constant__ TcBooks K) {
  using S = Shape<KK, KV, NT, DP, MQ, FINE>;
  constexpr int WPP = S::WPP, SW = S::SW, NQ = S::NQ, FK = S::FK, STEPS = S::STEPS, WT = S::WT;
  constexpr float kWeight = FINE ? 8388607.f : 65535.f;  // the largest weight of a group
  constexpr float kNone = FINE ? 1e-31f : 1e-33f;  // weights up to this count as 0: kWeight divided by more is finite
  extern __shared__ __align__(128) unsigned char smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, tig = lane & 3;
  uint32_t* kb = reinterpret_cast<uint32_t*>(smem + warp * S::WARP_BYTES);
  uint32_t* vb = kb + 4 * S::KB;
  uint32_t* wb = vb + 4 * S::VB;
  float4* xs = reinterpret_cast<float4*>(wb) + lane;             // [4 blocks][NT][lanes]
  float4* os = reinterpret_cast<float4*>(wb + S::XW) + lane;     // [DP / 32][NT][lanes]
  const uint32_t bar_k = smem_at(wb + S::XW + S::OW), bar_v = bar_k + 8;
  if (lane == 0) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bar_k));
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bar_v));
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncwarp();
  let_next_start();

  // the first records are on their way before the queries are ready
  const int worker = blockIdx.x * S::WARPS + warp;
  const bool own_sums = A.B <= kOwnSums;
  int64_t u, u_end;
  Segment sg;
  if (own_sums) {
    sg = first_segment(A, worker, u, u_end, lane);
  } else {
    wait_for_previous();
    const int64_t units = A.prefix[A.B] * A.hv;
    u = share_at(A, units, worker);
    u_end = share_at(A, units, worker + 1);
    if (u < u_end) sg = segment_at(A, u, u_end, lane);
  }
  const int64_t u_first = u;
  if (u >= u_end) {
    if (own_sums) wait_for_previous();  // the join's launch counts on this one being behind the queries
    return;
  }

  const uint32_t key_bytes = A.L.o_v * 4u, val_bytes = (A.L.words - A.L.o_v) * 4u;
  // lane i < 4 knows of block i of the group at sg.blk: its record (-1: none) and its tokens
  int64_t at = -1;
  int nt = 0;
  // the table is read long before its entry is looked at
  auto entry = [&](const Segment& s) -> int32_t {
    return lane < kUnit && s.blk + lane < s.end ? page_entry(A.L, A.tab, s.b, s.blk + lane) : -1;
  };
  auto describe = [&](const Segment& s, int32_t page, int64_t& a, int& n) {
    const int blk = s.blk + lane;
    a = record_in(A.L, A.tab, page, blk, A.layer, s.kvh);
    n = a >= 0 ? min(32, s.len - 32 * blk) : 0;
  };
  auto stage = [&](int64_t a, bool keys) {
    const uint32_t there = __ballot_sync(0xffffffffu, a >= 0);
    const uint32_t bytes = keys ? key_bytes : val_bytes, bar = keys ? bar_k : bar_v;
    if (lane == 0) expect(bar, __popc(there) * bytes);
    __syncwarp();
    if (a >= 0)
      bulk_copy(smem_at(keys ? kb + lane * S::KB : vb + lane * S::VB), A.pool + a + (keys ? 0 : A.L.o_v), bytes, bar);
  };
  describe(sg, entry(sg), at, nt);
  stage(at, true);
  stage(at, false);

  // the segment's query images and score constants
  uint2 bq[STEPS][NQ];
  float kc[NT][FK + 1];  // per odd subset, and the constant
  float2 uc[NT];         // of the signs
  auto queries = [&](const Segment& s) {
    const uint32_t* f = A.frag + ((int64_t)s.b * A.hv + s.h) * A.frag_words;
#pragma unroll
    for (int i = 0; i < STEPS; ++i)
#pragma unroll
      for (int t = 0; t < NQ; ++t) bq[i][t] = reinterpret_cast<const uint2*>(f)[(i * NQ + t) * 32 + lane];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const float4 c = reinterpret_cast<const float4*>(f + STEPS * NQ * 64)[4 * t + tig];
#pragma unroll
      for (int i = 0; i < FK; ++i) kc[t][i] = c.x * K.kalpha[i];
      kc[t][FK] = c.y;
      uc[t] = make_float2(c.z, c.w);
    }
  };
  if (own_sums) wait_for_previous();
  queries(sg);

  // thread (g, tig): the tokens 16 h + 4 (r ^ h) + s, r = 0..3, of a block (rows g and g + 8 of two m-tiles;
  // eight neighbouring tokens modulo 8 per row set, so that their words are on different banks)
  const int th = g >> 2, ts = g & 3;
  const uint32_t pack_sel = th ? 0x1504u : 0x5140u;  // bytes 0, 0, 1, 1 of two tokens, in the order of i
  const uint32_t pack_top = th ? 0x0026u : 0x0062u;  // byte 2 of them
  const int wt = WPP == 2 ? tig & 1 : tig, ws = MQ == 64 ? tig & 1 : tig;  // this thread's word of a plane, of the signs
  const int ksh = WPP == 2 ? 4 * (tig >> 1) : 0, ssh = MQ == 64 ? 4 * (tig >> 1) : 0;

  float m_run[NT], l_run[NT], w_run[NT];
  float4 o[S::O_SMEM ? 1 : DP / 32][NT];  // head 4 nt + tig, coordinates 32 c + 4 g ..
  auto o_get = [&](int c, int n) -> float4 {
    if constexpr (S::O_SMEM) return os[(c * NT + n) * 32];
    else return o[c][n];
  };
  auto o_put = [&](int c, int n, float4 v) {
    if constexpr (S::O_SMEM) os[(c * NT + n) * 32] = v;
    else o[c][n] = v;
  };
  auto start_sums = [&]() {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m_run[n] = -INFINITY;
      l_run[n] = w_run[n] = 0.f;
#pragma unroll
      for (int c = 0; c < DP / 32; ++c) o_put(c, n, make_float4(0.f, 0.f, 0.f, 0.f));
    }
  };
  start_sums();

  int units_behind = units_of(A, min(sg.b + 1, A.B - 1));  // a head of the next sequence, read a segment ahead
  bool ok = true;
  uint32_t phase = 0, k_phase = 0;  // of this group, and of the keys staged last
  for (;; phase ^= 1u) {
    // what comes after this group
    Segment nx = sg;
    ++u;
    nx.blk += kUnit;
    const bool last = nx.blk >= sg.end, done = u >= u_end;
    if (last && !done) nx = segment_after(A, sg, units_behind, u, u_end);
    const int32_t page = done ? -1 : entry(nx);

    // ---------------- scores, as powers of two
    if (!(ok = __all_sync(0xffffffffu, bounded_wait<true>(bar_k, phase, A.err)))) break;
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
      const int ni = __shfl_sync(0xffffffffu, nt, i);
      float x[NT][4];
      if (ni == 0) {
#pragma unroll
        for (int n = 0; n < NT; ++n) xs[(i * NT + n) * 32] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        continue;
      }
      const uint32_t* kw = kb + i * S::KB;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const int t1 = 16 * th + 4 * ((2 * m) ^ th) + ts, t2 = 16 * th + 4 * ((2 * m + 1) ^ th) + ts;
        int acc[FK + 1][NQ][4];
#pragma unroll
        for (int f = 0; f <= FK; ++f)
#pragma unroll
          for (int t = 0; t < NQ; ++t) acc[f][t][0] = acc[f][t][1] = acc[f][t][2] = acc[f][t][3] = 0;
        // the products of a step go to FK + 1 times NQ sums, so that none waits for the one before
        constexpr int W4 = (WPP + 3) / 4;
#pragma unroll
        for (int hf = 0; hf < W4; ++hf) {
          uint32_t w1[FK + 1], w2[FK + 1], h1[FK + 1], h2[FK + 1];
#pragma unroll
          for (int p = 0; p < KK; ++p) {
            const int base = word_place<S::GR>(p * WPP, wt) + hf * 128;  // hf > 0 only with granules of four
            w1[p] = kw[base + t1 * S::GR] >> ksh;
            w2[p] = kw[base + t2 * S::GR] >> ksh;
          }
          if (FK > KK) {
            w1[FK - 1] = w1[0] ^ w1[1 % KK] ^ w1[KK - 1];
            w2[FK - 1] = w2[0] ^ w2[1 % KK] ^ w2[KK - 1];
          }
          {
            const int base = word_place<S::GR>(KK * WPP, ws) + hf * 128;
            w1[FK] = kw[base + t1 * S::GR] >> ssh;
            w2[FK] = kw[base + t2 * S::GR] >> ssh;
          }
#pragma unroll
          for (int f = 0; f <= FK; ++f) {
            h1[f] = w1[f] >> 4;
            h2[f] = w2[f] >> 4;
          }
#pragma unroll
          for (int st = 0; st < 4; ++st) {
#pragma unroll
            for (int f = 0; f <= FK; ++f) {
              if (4 * hf + st >= (f < FK ? WPP : SW)) continue;
              // bit st of both half bytes, or, where two threads share a word and have one half byte each, two of it
              const bool half = f < FK ? WPP == 2 : SW == 2;
              const uint32_t ka = 0x01010101u << (half ? 2 * st % 4 : st), kc2 = half ? 2 * ka : ka;
              const int step = 4 * hf + st + (f < FK ? 0 : WPP);
#pragma unroll
              for (int t = 0; t < NQ; ++t)
                mma_us(acc[f][t], w1[f] & ka, w2[f] & ka, (half ? w1[f] : h1[f]) & kc2, (half ? w2[f] : h2[f]) & kc2,
                       bq[step][t]);
            }
          }
        }
        const float n1 = __uint_as_float(kw[32 * S::NK + t1]), n2 = __uint_as_float(kw[32 * S::NK + t2]);
        const float* rp = reinterpret_cast<const float*>(kw + 32 * S::NK + 32);
        const float r1 = get_rnorm(rp, t1, A.L.r16), r2 = get_rnorm(rp, t2, A.L.r16);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          // 2^16 hi + 2^8 mid + lo: hi and mid in columns 2 h and 2 h + 1 of tile n, lo in column n of the last.
          // The whole, a sum of bits times entries, is below 2^31, so that the parts may wrap around.
          auto whole = [&](const int (&d)[NQ][4], int row) {
            return (float)(int)(256u * (256u * (uint32_t)d[n][2 * row] + (uint32_t)d[n][2 * row + 1]) +
                                (uint32_t)d[NT][2 * row + n]);
          };
          float a1 = kc[n][FK], a2 = kc[n][FK];
#pragma unroll
          for (int f = 0; f < FK; ++f) {
            a1 = fmaf(kc[n][f], whole(acc[f], 0), a1);
            a2 = fmaf(kc[n][f], whole(acc[f], 1), a2);
          }
          const float y1 = n1 * fmaf(r1, fmaf(uc[n].x, whole(acc[FK], 0), uc[n].y), a1);
          const float y2 = n2 * fmaf(r2, fmaf(uc[n].x, whole(acc[FK], 1), uc[n].y), a2);
          x[n][2 * m] = y1;
          x[n][2 * m + 1] = y2;
        }
      }
      if (ni < 32) {  // slots without a token hold anything
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (16 * th + 4 * (r ^ th) + ts >= ni)
#pragma unroll
            for (int n = 0; n < NT; ++n) x[n][r] = -INFINITY;
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) xs[(i * NT + n) * 32] = make_float4(x[n][0], x[n][1], x[n][2], x[n][3]);
    }
    __syncwarp();  // the keys have been read
    int64_t nat = -1;
    int nnt = 0;
    if (!done) {
      describe(nx, page, nat, nnt);
      stage(nat, true);
      k_phase ^= 1u;
    }

    // ---------------- weights
    if (!(ok = __all_sync(0xffffffffu, bounded_wait<true>(bar_v, phase, A.err)))) break;
    float x[NT][4][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 v = xs[(i * NT + n) * 32];
        x[n][i][0] = v.x;
        x[n][i][1] = v.y;
        x[n][i][2] = v.z;
        x[n][i][3] = v.w;
      }
    __syncwarp();  // the scores' place is the weights' from here on
    float back[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float mx = -INFINITY;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        mx = fmaxf(mx, fmaxf(fmaxf(x[n][i][0], x[n][i][1]), fmaxf(x[n][i][2], x[n][i][3])));
#pragma unroll
      for (int k = 4; k < 32; k *= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
      const float top = fmaxf(m_run[n], mx), base = top == -INFINITY ? 0.f : top;
      const float corr = pow2(m_run[n] - base);
      m_run[n] = top;
      float l = 0.f, wsum = 0.f, big = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float* vn = reinterpret_cast<const float*>(vb + i * S::VB + KV * DP);
        const int ni = __shfl_sync(0xffffffffu, nt, i);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float p = pow2(x[n][i][r] - base);
          // the norm of a slot without a token can be anything; a token's that is NaN stays one
          const int t = 16 * th + 4 * (r ^ th) + ts;
          const float w = t < ni ? max_nan(p * vn[t], 0.f) : 0.f;
          l += p;
          big = max_nan(big, w);
          if (KV == 4) wsum += w;
          x[n][i][r] = w;
        }
      }
      if (__any_sync(0xffffffffu, corr != 1.f)) {  // seldom after a sequence's first groups
        l_run[n] *= corr;
        if (KV == 4) w_run[n] *= corr;
#pragma unroll
        for (int c = 0; c < DP / 32; ++c) {
          const float4 t = o_get(c, n);
          o_put(c, n, make_float4(t.x * corr, t.y * corr, t.z * corr, t.w * corr));
        }
      }
      l_run[n] += l;
      if (KV == 4) w_run[n] += wsum;
#pragma unroll
      for (int k = 4; k < 32; k *= 2) big = max_nan(big, __shfl_xor_sync(0xffffffffu, big, k));
      // a weight that is not finite makes all of its head's sums NaN (infinity times 0), whatever its integer is
      const float inv = big <= kNone ? 0.f : kWeight / big;
      back[n] = big <= kNone ? 0.f : fmaf(big, 0.f, big * ((FINE ? 0x1p24f : 0x1p8f) / kWeight) * K.unit);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // the integer part in the low 16 or 23 bits (2^23 itself: 2^7 in byte 2)
        uint32_t b[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) b[r] = __float_as_uint(fmaf(x[n][i][r], inv, 8388608.f));
        const uint32_t lh0 = __byte_perm(b[0], b[1], pack_sel), lh1 = __byte_perm(b[2], b[3], pack_sel);
        uint32_t* col = wb + (8 * n + 2 * tig) * S::WC + 8 * i + 2 * ts + th;
        const uint32_t b1 = __byte_perm(lh0, lh1, 0x7632), b0 = __byte_perm(lh0, lh1, 0x5410);
        if constexpr (FINE) {
          col[0] = __byte_perm(__byte_perm(b[0], b[1], pack_top), __byte_perm(b[2], b[3], pack_top), 0x5410);
          col[S::WC] = b1;
          col[(8 * (NT - n) + n) * S::WC] = b0;  // column 2 tig + n of the last tile
        } else {
          col[0] = b1;
          col[S::WC] = b0;
        }
      }
    }
    __syncwarp();

    // ---------------- values
    uint2 bw[WT][4];
#pragma unroll
    for (int n = 0; n < WT; ++n) {
      const uint4* col = reinterpret_cast<const uint4*>(wb + (8 * n + g) * S::WC + 8 * tig);
      const uint4 a = col[0], b = col[1];
      bw[n][0] = make_uint2(a.x, a.y);
      bw[n][1] = make_uint2(a.z, a.w);
      bw[n][2] = make_uint2(b.x, b.y);
      bw[n][3] = make_uint2(b.z, b.w);
    }
    const uint32_t* vw = vb + tig * S::VB + 4 * g;
#pragma unroll S::O_SMEM ? 1 : DP / 32
    for (int c = 0; c < DP / 32; ++c) {
      uint32_t w[4][KV];
#pragma unroll
      for (int q = 0; q < KV; ++q) {
        const uint4 v = *reinterpret_cast<const uint4*>(vw + q * DP + 32 * c);
        w[0][q] = v.x;
        w[1][q] = v.y;
        w[2][q] = v.z;
        w[3][q] = v.w;
      }
      // rows g and g + 8 of m-tile mt: coordinates 2 mt and 2 mt + 1 of the four; the levels' bytes
      int ah[2][WT][4], al[2][WT][4], at[2][NT][4];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int n = 0; n < WT; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            ah[mt][n][k] = al[mt][n][k] = 0;
            if (n < NT) at[mt][n][k] = 0;
          }
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          uint32_t h[2][2], l[2][2], t[2][2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint32_t y = selectors<KV>(w[2 * mt + r], s);
            const uint32_t neg = KV == 4 ? (y >> 3) & 0x11111111u : 0u;
            const uint32_t z = KV == 4 ? y & 0x77777777u : y;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const uint32_t flip = KV == 4 ? __byte_perm(0x0000ff00u, 0u, neg >> (16 * half)) : 0u;
              h[r][half] = levels<KV>(K.hi, z >> (16 * half), flip);
              l[r][half] = levels<KV>(K.lo, z >> (16 * half), flip);
              if (FINE) t[r][half] = levels<KV>(K.th, z >> (16 * half), flip);
            }
          }
#pragma unroll
          for (int n = 0; n < WT; ++n) {
            mma_su(ah[mt][n], h[0][0], h[1][0], h[0][1], h[1][1], bw[n][s]);
            mma_uu(al[mt][n], l[0][0], l[1][0], l[0][1], l[1][1], bw[n][s]);
            if (FINE && n < NT) mma_uu(at[mt][n], t[0][0], t[1][0], t[0][1], t[1][1], bw[n][s]);
          }
        }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        auto sum = [&](int mt, int r) {
          const int hh = ah[mt][n][2 * r], hl = ah[mt][n][2 * r + 1], lh = al[mt][n][2 * r], ll = al[mt][n][2 * r + 1];
          // in units of 2^8: what the shift drops is below a unit, of 2^30 where the weights are large
          if (!FINE) return (float)(256 * hh + hl + lh + (ll >> 8));
          // in units of 2^24, of 2^29 where the weights are large; the two bytes below are of 2^16 and 2^8, and what the
          // shift drops is below 2^16
          const int below = ah[mt][NT][2 * r + n] + ll + at[mt][n][2 * r] + ((al[mt][NT][2 * r + n] + at[mt][n][2 * r + 1]) >> 8);
          return fmaf((float)below, 0x1p-8f, (float)(256 * hh + hl + lh));
        };
        float4 t = o_get(c, n);
        t.x = fmaf(back[n], sum(0, 0), t.x);
        t.y = fmaf(back[n], sum(0, 1), t.y);
        t.z = fmaf(back[n], sum(1, 0), t.z);
        t.w = fmaf(back[n], sum(1, 1), t.w);
        o_put(c, n, t);
      }
    }
    __syncwarp();  // values and weights have been read
    if (!done) stage(nat, false);

    // ---------------- the segment's part
    if (last) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float l = l_run[n], ws = w_run[n];
#pragma unroll
        for (int k = 4; k < 32; k *= 2) {
          l += __shfl_xor_sync(0xffffffffu, l, k);
          if (KV == 4) ws += __shfl_xor_sync(0xffffffffu, ws, k);
        }
        if (4 * n + tig < A.gh) {
          float* pp = slot_of(A, (int64_t)sg.b * A.hv + sg.h, worker, 4 * n + tig);
          if (g == 0) *reinterpret_cast<float2*>(pp) = make_float2(m_run[n], l);
          // four-bit levels stand half a step low (their negatives are complements)
          const float up = KV == 4 ? 0.5f * K.unit * ws : 0.f;
#pragma unroll
          for (int c = 0; c < DP / 32; ++c) {
            const float4 t = o_get(c, n);
            *reinterpret_cast<float4*>(pp + 4 + 32 * c + 4 * g) = make_float4(t.x + up, t.y + up, t.z + up, t.w + up);
          }
        }
      }
      start_sums();
      if (!done) {
        queries(nx);
        units_behind = units_of(A, min(nx.b + 1, A.B - 1));
      }
    }
    if (done) break;
    sg = nx;
    at = nat;
    nt = nnt;
  }
  if (!ok) {
    // a wait ran out (the error word is set): leave empty parts, so that nothing
    // downstream reads an old workspace, once the copies in flight have landed
    bounded_wait<true>(bar_k, k_phase, nullptr);
    bounded_wait<true>(bar_v, phase, nullptr);
    for (u = u_first; u < u_end;) {
      sg = segment_at(A, u, u_end, lane);
      u += (sg.end - sg.blk + kUnit - 1) / kUnit;
      if (lane < A.gh)
        *reinterpret_cast<float2*>(slot_of(A, (int64_t)sg.b * A.hv + sg.h, worker, lane)) = make_float2(-INFINITY, 0.f);
    }
  }
}

// One (d_pad, m, key bits) per source file.
template <int KK, int KV, int NT, int DP, int MQ, bool FINE>
cudaError_t launch_form(const AttnArgs& a, const TcBooks& k, int ctas, cudaStream_t st) {
  using S = Shape<KK, KV, NT, DP, MQ, FINE>;
  auto kern = attention_tc_kernel<KK, KV, NT, DP, MQ, FINE>;
  // function attributes are per device: set on every call (a cheap host call)
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
  if (e != cudaSuccess) return e;
  return launch_after(kern, dim3(ctas), 32 * S::WARPS, S::SMEM, st, a, k);
}

template <int KK, int KV, int NT, int DP, int MQ>
cudaError_t launch_one(const AttnArgs& a, const TcBooks& k, int ctas, cudaStream_t st) {
  return fine_sums(a.dt) ? launch_form<KK, KV, NT, DP, MQ, true>(a, k, ctas, st)
                         : launch_form<KK, KV, NT, DP, MQ, false>(a, k, ctas, st);
}

template <int KK, int DP, int MQ>
cudaError_t launch_values(const AttnArgs& a, const TcBooks& k, int kv, int nt, int ctas, cudaStream_t st) {
  if constexpr (DP == 256) {
    if (nt != 1) return cudaErrorInvalidValue;
    switch (kv) {
      case 1: return launch_one<KK, 1, 1, DP, MQ>(a, k, ctas, st);
      case 2: return launch_one<KK, 2, 1, DP, MQ>(a, k, ctas, st);
      case 3: return launch_one<KK, 3, 1, DP, MQ>(a, k, ctas, st);
      default: return launch_one<KK, 4, 1, DP, MQ>(a, k, ctas, st);
    }
  } else {
    switch (kv * 2 + nt - 1) {
      case 2: return launch_one<KK, 1, 1, DP, MQ>(a, k, ctas, st);
      case 3: return launch_one<KK, 1, 2, DP, MQ>(a, k, ctas, st);
      case 4: return launch_one<KK, 2, 1, DP, MQ>(a, k, ctas, st);
      case 5: return launch_one<KK, 2, 2, DP, MQ>(a, k, ctas, st);
      case 6: return launch_one<KK, 3, 1, DP, MQ>(a, k, ctas, st);
      case 7: return launch_one<KK, 3, 2, DP, MQ>(a, k, ctas, st);
      case 8: return launch_one<KK, 4, 1, DP, MQ>(a, k, ctas, st);
      default: return launch_one<KK, 4, 2, DP, MQ>(a, k, ctas, st);
    }
  }
}

// Defined by the source file of its (d_pad, m, key bits).
template <int KK, int DP, int MQ>
cudaError_t launch_keys(const AttnArgs& a, const TcBooks& k, int kv, int nt, int ctas, cudaStream_t st);

}  // namespace tc
}  // namespace paged
}  // namespace tq
