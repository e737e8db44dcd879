// paged.cuh -- the paged KV cache as its writers and readers see it, and the
// batch of sequences with new tokens that both are called with.
//
// Cache: K and V pools [n_pages][page_size][Hkv][128], bf16 or E4M3 with an
// fp32 scale per kv head. Position p of sequence s lives in page
// block_table[s][p / page_size] at row p % page_size. The page size is a power
// of two >= 16, so a 16-key block never crosses a page and divisions are shifts.
//
// Batch: sequence s owns the token rows q_start[s] .. q_start[s+1] - 1; they
// are its last n = q_start[s+1] - q_start[s] positions, kv_len[s] - n ..
// kv_len[s] - 1. All of it is device data, so a captured graph replays with
// other lengths; nothing read from it is trusted as an index.
#pragma once

#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "common.cuh"
#include "flint_moe.h"

namespace flint {

constexpr int kPagedHeadDim = 128;
constexpr int kPagedMinPage = 16;
constexpr int kPagedMaxPage = 1024;
constexpr int kPagedMaxPos = 1 << 30;  // positions per sequence: key arithmetic stays in int

struct PagedBatch {
  const int32_t* q_start;      // [B + 1]
  const int32_t* kv_len;       // [B]
  const int32_t* block_table;  // [B][max_pages]
  int B, T, max_pages, page_shift;
  int max_pos;                 // positions a block-table row can hold (<= kPagedMaxPos)
  long long n_pages;
};

struct PagedSeq {
  int row0, n, kv;  // first token row, new tokens, cached positions (new ones included)
};

// A sequence's rows and length, or n = 0 for one without new tokens or outside
// the call's rows; a kv_len that cannot hold the new tokens or does not fit the
// block table gives kv = 0 (its tokens see nothing). *bad reports either.
__device__ __forceinline__ PagedSeq paged_seq(const PagedBatch& b, int s, bool* bad) {
  PagedSeq r;
  const int q0 = __ldg(b.q_start + s), q1 = __ldg(b.q_start + s + 1);
  r.row0 = q0;
  r.n = q1 - q0;
  r.kv = __ldg(b.kv_len + s);
  *bad = false;
  if (q0 < 0 || q1 > b.T || q1 < q0) {
    r.n = r.kv = 0;
    *bad = true;
  } else if (r.n > 0 && (r.kv < r.n || r.kv > b.max_pos)) {
    r.kv = 0;
    *bad = true;
  }
  return r;
}

inline bool paged_aligned16(const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15u) == 0; }

// Host side: checks the batch's arguments and fills `b`; FLINT_OK, or the
// recorded error.
inline int paged_batch(PagedBatch* b, int32_t T, const int32_t* q_start, const int32_t* kv_len, int32_t B,
                       const int32_t* block_table, int32_t max_pages, int32_t page_size, int64_t n_pages,
                       int32_t cache_dtype, const void* k_cache, const void* v_cache, const float* k_scale,
                       const float* v_scale, const int32_t* status) {
  if (page_size < kPagedMinPage || page_size > kPagedMaxPage || (page_size & (page_size - 1)) != 0)
    return flint_fail_external(FLINT_ERR_UNSUPPORTED_SHAPE, "page_size must be a power of two in 16..1024");
  if (cache_dtype != FLINT_KV_BF16 && cache_dtype != FLINT_KV_E4M3)
    return flint_fail_external(FLINT_ERR_INVALID_ARG, "cache_dtype is not a flint_kv_dtype");
  if (T < 0 || B < 0 || max_pages < 0 || n_pages < 0)
    return flint_fail_external(FLINT_ERR_INVALID_ARG, "negative size");
  if (n_pages > INT64_C(0x7fffffff) / page_size)
    return flint_fail_external(FLINT_ERR_UNSUPPORTED_SHAPE, "at most 2^31 - 1 cache rows");
  if (T == 0 || B == 0) return FLINT_OK;
  if (!q_start || !kv_len || (max_pages > 0 && !block_table) || (n_pages > 0 && (!k_cache || !v_cache)))
    return flint_fail_external(FLINT_ERR_INVALID_ARG, "NULL pointer");
  if (cache_dtype == FLINT_KV_E4M3 && (!k_scale || !v_scale))
    return flint_fail_external(FLINT_ERR_INVALID_ARG, "an E4M3 cache needs k_scale and v_scale");
  if (!paged_aligned16(k_cache) || !paged_aligned16(v_cache) ||
      ((reinterpret_cast<uintptr_t>(q_start) | reinterpret_cast<uintptr_t>(kv_len) |
        reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(k_scale) |
        reinterpret_cast<uintptr_t>(v_scale) | reinterpret_cast<uintptr_t>(status)) & 3u))
    return flint_fail_external(FLINT_ERR_MISALIGNED, "misaligned pointer");
  b->q_start = q_start;
  b->kv_len = kv_len;
  b->block_table = block_table;
  b->B = B;
  b->T = T;
  b->max_pages = max_pages;
  int sh = 0;
  while ((1 << sh) < page_size) ++sh;
  b->page_shift = sh;
  const long long mp = static_cast<long long>(max_pages) << sh;
  b->max_pos = static_cast<int>(mp < kPagedMaxPos ? mp : kPagedMaxPos);
  b->n_pages = n_pages;
  return FLINT_OK;
}

// Two fp32 -> two E4M3 codes (a in the low byte), round to nearest even,
// saturating at +-448.
__device__ __forceinline__ uint32_t pack_e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
// Two E4M3 codes (low 16 bits of w) -> f16x2, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
  uint32_t h;
  const uint16_t b = static_cast<uint16_t>(w);
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(b));
  return h;
}

}  // namespace flint
