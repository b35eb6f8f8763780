// The paged compressed KV cache: its description and the places of a block
// record's parts (include/tq.h, tq_paged_create).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "tq_internal.h"

namespace tq {
namespace paged {

// Everything the kernels need to find a token: offsets in 32-bit words.
struct Layout {
  int kw, sw, nk;      // code words, sign words, key words of a token
  int gr;              // words of a granule
  int kv, dp;          // value bits, rotated dimension
  int r16;             // residual norms are fp16
  int o_kn, o_kr, o_v, o_vn;
  int words;           // of a record
  int nb;              // records of a page per layer and head
  int nb_shift;        // its logarithm, -1 where it is no power of two
  int layers, hkv, page;
  int64_t page_words;
};

// One page table argument.
struct Table {
  const int32_t* rows;
  int64_t ld;
  int max_pages;
  int64_t n_pages;
};

#ifdef __CUDACC__
// The page of block `blk` (32 tokens) of a sequence, as its table row says.
__device__ __forceinline__ int page_of(const Layout& L, int blk) { return L.nb_shift >= 0 ? blk >> L.nb_shift : blk / L.nb; }
__device__ __forceinline__ int32_t page_entry(const Layout& L, const Table& t, int64_t b, int blk) {
  return t.rows[b * t.ld + page_of(L, blk)];
}
// First word of the record of block `blk` in layer `layer`, head h, given its
// page; -1 in a hole.  64-bit: a pool can be larger than 2^31 words.
__device__ __forceinline__ int64_t record_in(const Layout& L, const Table& t, int32_t page, int blk, int layer, int h) {
  if (page < 0 || page >= t.n_pages) return -1;
  return page * L.page_words + ((int64_t)(layer * L.hkv + h) * L.nb + (blk - page_of(L, blk) * L.nb)) * L.words;
}
__device__ __forceinline__ int64_t record_at(const Layout& L, const Table& t, int64_t b, int blk, int layer, int h) {
  return record_in(L, t, page_entry(L, t, b, blk), blk, layer, h);
}
__device__ __forceinline__ int key_word_at(const Layout& L, int t, int w) {
  return (w / L.gr) * (32 * L.gr) + t * L.gr + w % L.gr;
}
__device__ __forceinline__ int clamp_len(int len, const Layout& L, int max_pages) {
  const int top = max_pages * L.page;
  return len < 0 ? 0 : len > top ? top : len;
}
// Launches that depend on the one before them may be set up early: a kernel
// waits here before it reads what that one wrote ...
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// ... and says here that its successor may be set up.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... Ps, typename... As>
cudaError_t launch_after(void (*kern)(Ps...), dim3 grid, int threads, size_t smem, cudaStream_t st, As... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}
#endif

// Checks shared by the entry points (no handle's contents but the layout).
inline bool bad_pool(const Layout& L, const void* pool, int64_t n_pages) {
  return !pool || (reinterpret_cast<uintptr_t>(pool) & 15u) || n_pages < 1 || n_pages > 0x7fffffffll ||
         L.page_words < 1;
}
inline bool bad_table(const Layout& L, const void* rows, int64_t ld, int max_pages) {
  return !rows || (reinterpret_cast<uintptr_t>(rows) & 3u) || max_pages < 1 || ld < max_pages ||
         (int64_t)max_pages * L.page > 0x7fffffffll;
}
inline bool mis4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

}  // namespace paged
}  // namespace tq

struct tq_paged {
  tq::QParams kq, vq;
  int device;  // of kq's sketch
  tq::paged::Layout lay;
};
