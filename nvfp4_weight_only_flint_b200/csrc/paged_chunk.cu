#include "paged_attn.cuh"
namespace flint {
size_t paged_chunk_workspace(int, int, int, int, int) { return 0; }
int paged_chunk_launch(const PagedAttnParams&, int, size_t, cudaStream_t) {
  return flint_fail_external(FLINT_ERR_UNSUPPORTED_SHAPE, "max_q_len * n_q_heads / n_kv_heads must be at most 16");
}
}  // namespace flint
