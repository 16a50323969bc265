// Paged decode attention over i8 pages (one translation unit per page type).
#include "fc_paged_attn.cuh"

namespace fc {
int launch_paged_attention_i8(const PagedArgs& a, int64_t D, cudaStream_t s) {
  return launch_paged_dtype<int8_t>(a, D, s);
}
}  // namespace fc
