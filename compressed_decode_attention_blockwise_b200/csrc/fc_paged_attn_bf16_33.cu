// Paged decode attention over bf16 pages; limbs of the query: 3, of P: 3.
#include "fc_paged_attn.cuh"

namespace fc {
int launch_paged_attention_bf16_33(const PagedArgs& a, int64_t D, cudaStream_t s) {
  return launch_paged_sizes<__nv_bfloat16, 3, 3>(a, D, s);
}
}  // namespace fc
