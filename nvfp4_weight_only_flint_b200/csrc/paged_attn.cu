// paged_attn.cu -- the C entry of attention over the paged cache: argument
// checks and the choice between the decode and the chunk kernel.
#include "paged_attn.cuh"

using namespace flint;

extern "C" size_t flint_paged_attention_workspace_bytes(int32_t T, int32_t B, int32_t n_q_heads, int32_t n_kv_heads,
                                                        int32_t max_q_len) {
  if (T < 1 || B < 1 || n_kv_heads < 1 || n_q_heads < 1 || n_q_heads % n_kv_heads != 0 || max_q_len < 1) return 0;
  const int group = n_q_heads / n_kv_heads;
  if (group > kDecodeRows || B > 32768 || n_q_heads > 1024 || T > (1 << 24)) return 0;
  if (max_q_len > T) max_q_len = T;
  // never less than a smaller call takes: one workspace serves the decode steps beside the prompt pieces
  const size_t decode = paged_decode_workspace(B, n_kv_heads);
  if (static_cast<long long>(max_q_len) * group <= kDecodeRows) return decode;
  const size_t chunk = paged_chunk_workspace(n_q_heads, n_kv_heads, max_q_len);
  return chunk > decode ? chunk : decode;
}

extern "C" int flint_paged_attention(const uint16_t* q, int32_t T, const int32_t* q_start, const int32_t* kv_len,
                                     int32_t B, const int32_t* block_table, int32_t max_pages, int32_t page_size,
                                     int64_t n_pages, const void* k_cache, const void* v_cache, int32_t cache_dtype,
                                     const float* k_scale, const float* v_scale, int32_t n_q_heads,
                                     int32_t n_kv_heads, int32_t head_dim, int32_t max_q_len, int32_t window,
                                     float scale, uint16_t* out, void* workspace, size_t workspace_bytes,
                                     int32_t* status, void* stream) {
  if (head_dim != kPagedHeadDim) return flint_fail_external(FLINT_ERR_UNSUPPORTED_SHAPE, "head_dim must be 128");
  if (n_q_heads < 1 || n_kv_heads < 1 || max_q_len < 0 || window < 0 || !(scale > 0.f) || !(scale < INFINITY))
    return flint_fail_external(FLINT_ERR_INVALID_ARG, "flint_paged_attention: bad sizes");
  if (n_q_heads % n_kv_heads != 0 || n_q_heads / n_kv_heads > kDecodeRows)
    return flint_fail_external(FLINT_ERR_UNSUPPORTED_SHAPE, "n_q_heads / n_kv_heads must be an integer <= 16");
  if (B > 32768 || n_q_heads > 1024 || T > (1 << 24))
    return flint_fail_external(FLINT_ERR_UNSUPPORTED_SHAPE,
                               "at most 32768 sequences, 1024 query heads and 2^24 new tokens");
  PagedAttnParams p{};
  const int rc = paged_batch(&p.b, T, q_start, kv_len, B, block_table, max_pages, page_size,
                             n_pages, cache_dtype, k_cache, v_cache, k_scale, v_scale, status);
  if (rc != FLINT_OK) return rc;
  if (T == 0 || B == 0) return FLINT_OK;
  if (!q || !out) return flint_fail_external(FLINT_ERR_INVALID_ARG, "flint_paged_attention: NULL pointer");
  if (!paged_aligned16(q) || !paged_aligned16(out) || !paged_aligned16(workspace))
    return flint_fail_external(FLINT_ERR_MISALIGNED, "flint_paged_attention: misaligned pointer");
  if (max_q_len < 1 || n_pages < 1)
    return flint_fail_external(FLINT_ERR_INVALID_ARG, "flint_paged_attention: max_q_len and n_pages must be at least 1");
  p.q = q;
  p.k = k_cache;
  p.v = v_cache;
  p.k_scale = cache_dtype == FLINT_KV_E4M3 ? k_scale : nullptr;
  p.v_scale = cache_dtype == FLINT_KV_E4M3 ? v_scale : nullptr;
  p.out = out;
  p.status = status;
  p.ws = static_cast<char*>(workspace);
  p.Hq = n_q_heads;
  p.Hkv = n_kv_heads;
  p.group = n_q_heads / n_kv_heads;
  // a window no shorter than the longest sequence is none: positions minus the window stay within int
  p.window = window < kPagedMaxPos ? window : 0;
  p.max_q = max_q_len < T ? max_q_len : T;  // as for the workspace size
  p.scale = scale;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return static_cast<long long>(p.max_q) * p.group <= kDecodeRows
             ? paged_decode_launch(p, cache_dtype, workspace_bytes, st)
             : paged_chunk_launch(p, cache_dtype, workspace_bytes, st);
}
