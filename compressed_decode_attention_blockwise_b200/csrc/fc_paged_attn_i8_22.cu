// Paged decode attention over i8 pages; limbs of the query: 2, of P: 2.
#include "fc_paged_attn.cuh"

namespace fc {
int launch_paged_attention_i8_22(const PagedArgs& a, int64_t D, cudaStream_t s) {
  return launch_paged_sizes<int8_t, 2, 2>(a, D, s);
}
}  // namespace fc
