// Paged decode attention over f32 pages (one translation unit per page type).
#include "fc_paged_attn.cuh"

namespace fc {
int launch_paged_attention_f32(const PagedArgs& a, int64_t D, cudaStream_t s) {
  return launch_paged_dtype<float>(a, D, s);
}
}  // namespace fc
