// Paged decode attention over bf16 pages (one translation unit per page type).
#include "fc_paged_attn.cuh"

namespace fc {
int launch_paged_attention_bf16(const PagedArgs& a, int64_t D, cudaStream_t s) {
  return launch_paged_dtype<__nv_bfloat16>(a, D, s);
}
}  // namespace fc
