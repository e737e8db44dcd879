// paged_attn.cuh -- what the two attention kernels over the paged cache (few
// new tokens per sequence: paged_decode.cu; many: paged_chunk.cu) share: the
// call's parameters and the register-fragment wrappers.
#pragma once

#include "paged.cuh"

namespace flint {

struct PagedAttnParams {
  PagedBatch b;
  const uint16_t* q;     // [T][Hq][128] bf16
  const void* k;         // pools
  const void* v;
  const float* k_scale;  // [Hkv], null for a bf16 cache
  const float* v_scale;
  uint16_t* out;         // [T][Hq][128] bf16
  int32_t* status;
  char* ws;
  int Hq, Hkv, group, window, max_q;
  float scale;
};

// Query token i of a sequence with n new tokens and kv positions sits at
// position kv - n + i and attends keys (position - window, position] (window
// <= 0: all up to its own). The keys some token of the sequence attends:
// [paged_first_key, kv), the start rounded down to a 16-key block.
__device__ __forceinline__ int paged_first_key(int kv, int n, int window) {
  return window > 0 ? max(0, kv - n - window + 1) & ~(kPagedMinPage - 1) : 0;
}

// 2^x, flushing results below the smallest normal to zero
__device__ __forceinline__ float exp2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLog2e = 1.4426950408889634f;

int paged_decode_launch(const PagedAttnParams& p, int cache_dtype, size_t ws_bytes, cudaStream_t st);
size_t paged_decode_workspace(int B, int n_kv_heads);
int paged_chunk_launch(const PagedAttnParams& p, int cache_dtype, size_t ws_bytes, cudaStream_t st);
size_t paged_chunk_workspace(int n_q_heads, int n_kv_heads, int max_q);

// New tokens times query heads per kv head that one 16-row register tile
// holds: such calls take the decode kernel, others the chunk kernel with its
// 128-row tiles. Two tokens of a group of 8 (16 rows), decode / chunk kernel, us:
// 1 x 4,098 keys 13.5 / 23.9, 64 x 4,098 107 / 126, 8 x 32,002 102 / 118, in E4M3
// 13.0 / 27.1, 74.8 / 142, 72.1 / 130.
constexpr int kDecodeRows = 16;

}  // namespace flint
