// Tensor-core attention over pages: d_pad 128, m 64, 1-bit key codes.
#include "tq_paged_attn_tc.cuh"

namespace tq {
namespace paged {
namespace tc {

template <>
cudaError_t launch_keys<1, 128, 64>(const AttnArgs& a, const TcBooks& k, int kv, int nt, int ctas, cudaStream_t st) {
  return launch_values<1, 128, 64>(a, k, kv, nt, ctas, st);
}

}  // namespace tc
}  // namespace paged
}  // namespace tq
