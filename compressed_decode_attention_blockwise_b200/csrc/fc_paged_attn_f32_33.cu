// Paged decode attention over f32 pages; limbs of the query: 3, of P: 3.
#include "fc_paged_attn.cuh"

namespace fc {
int launch_paged_attention_f32_33(const PagedArgs& a, int64_t D, cudaStream_t s) {
  return launch_paged_sizes<float, 3, 3>(a, D, s);
}
}  // namespace fc
