// Paged decode attention over bf16 pages; limbs of the query: 1, of P: 2.
#include "fc_paged_attn.cuh"

namespace fc {
int launch_paged_attention_bf16_12(const PagedArgs& a, int64_t D, cudaStream_t s) {
  return launch_paged_sizes<__nv_bfloat16, 1, 2>(a, D, s);
}
}  // namespace fc
