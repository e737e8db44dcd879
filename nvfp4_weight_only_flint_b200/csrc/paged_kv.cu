// paged_kv.cu -- the attention prologue of a layer on a paged KV cache: Q/K RMS
// normalisation, rotary embedding and the append of the batch's new keys and
// values to their pages ("[Model] Add Flint (RecursiveSI/flint)", section "What
// happened": one fused kernel in the per-layer decode chain). The arithmetic is
// that of k_qk_norm_rope_kv (attn.cu); the cache rows come from the block table
// and the positions from the sequences' lengths instead of per-token arrays.
//
//   y = x / sqrt(mean(x^2) + eps) * w   (skipped without weights)
//   (y_i, y_{i+64}) turned by the angle row of the token's position
//   q_out = bf16(y); K row = bf16(y) or E4M3(y / k_scale); V row likewise from x
//
// One half-warp takes kHeads consecutive heads of one token: lane l holds
// elements 8l .. 8l+7 of each (a 16-byte load; all heads' loads are issued
// before the first is used), so the cos/sin row, the page lookup and the
// search for the token's sequence are done once for kHeads heads.
// HBM-bound: (Hq + 2 Hkv) 256 bytes read and Hq 256 + 2 Hkv 128 e written per
// token (e = 2 or 1 bytes), the cos/sin row (512 bytes) once per position.
#include "paged.cuh"

namespace flint {
namespace {

constexpr int kHeads = 4;
constexpr int kThreads = 128;
constexpr int kUnitsPerCta = kThreads / 16;

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

struct AppendParams {
  PagedBatch b;
  const uint16_t* qkv;
  const uint16_t* q_w;  // null: no normalisation
  const uint16_t* k_w;
  const float* cos_sin;
  const float* k_scale;
  const float* v_scale;
  uint16_t* q_out;
  void* k_cache;
  void* v_cache;
  int32_t* status;
  int Hq, Hkv, max_pos, rope, units;  // units: half-warps per token
  float eps;
};

template <bool kE4M3>
__global__ void __launch_bounds__(kThreads) k_paged_append(AppendParams p) {
  const int lane = threadIdx.x & 15;
  const unsigned hmask = 0xFFFFu << (threadIdx.x & 16);
  const unsigned unit = blockIdx.x * kUnitsPerCta + (threadIdx.x >> 4);
  const int t = static_cast<int>(unit / static_cast<unsigned>(p.units));
  if (t >= p.b.T) return;
  const int h0 = static_cast<int>(unit - static_cast<unsigned>(t) * p.units) * kHeads;
  const int H = p.Hq + 2 * p.Hkv;
  const int nh = min(kHeads, H - h0);
  uint4 raw[kHeads];
  const uint4* src = reinterpret_cast<const uint4*>(p.qkv + (static_cast<size_t>(t) * H + h0) * kPagedHeadDim) + lane;
#pragma unroll
  for (int i = 0; i < kHeads; ++i)
    if (i < nh) raw[i] = __ldcs(src + i * 16);
  uint4 wq = make_uint4(0, 0, 0, 0), wk = wq;
  if (p.q_w != nullptr) {
    wq = __ldg(reinterpret_cast<const uint4*>(p.q_w) + lane);
    wk = __ldg(reinterpret_cast<const uint4*>(p.k_w) + lane);
  }
  // the token's sequence: the last s in [0, B) with q_start[s] <= t, by a
  // search of 16 probes a step (the half-warp's lanes)
  int lo = -1, hi = p.b.B + 1;  // q_start[lo] <= t < q_start[hi] in sorted data
  while (hi - lo > 1) {
    const int step = (hi - lo + 16) / 17;
    const int probe = lo + (lane + 1) * step;
    const bool le = probe < hi && __ldg(p.b.q_start + probe) <= t;
    const int c = __popc(__ballot_sync(hmask, le) & hmask);
    lo += c * step;
    hi = min(lo + step, hi);
  }
  if (lo < 0 || lo >= p.b.B) return;  // a row of no sequence: left as it is
  bool bad;
  const PagedSeq sq = paged_seq(p.b, lo, &bad);
  const int pos = sq.kv - sq.n + (t - sq.row0);
  // a sequence whose length cannot hold its tokens: no position, no page
  const bool placed = sq.kv > 0 && t - sq.row0 < sq.n;
  long long slot = -1;
  if (placed) {
    const int page = __ldg(p.b.block_table + static_cast<size_t>(lo) * p.b.max_pages + (pos >> p.b.page_shift));
    if (page >= 0 && page < p.b.n_pages)
      slot = (static_cast<long long>(page) << p.b.page_shift) + (pos & ((1 << p.b.page_shift) - 1));
  }
  const bool turn = p.rope && placed && pos < p.max_pos;
  if (lane == 0 && p.status != nullptr && (slot < 0 || (p.rope && !turn))) atomicOr(p.status, FLINT_DEVCHECK_INDEX);
  // angles of pairs (c, c + 64): lanes 0..7 hold the first halves, 8..15 the second
  float cc[8], sn[8];
  if (turn) {
    const float* row = p.cos_sin + static_cast<size_t>(pos) * kPagedHeadDim + 8 * (lane & 7);
    const float4 c0 = __ldg(reinterpret_cast<const float4*>(row)), c1 = __ldg(reinterpret_cast<const float4*>(row + 4));
    const float4 s0 = __ldg(reinterpret_cast<const float4*>(row + 64)), s1 = __ldg(reinterpret_cast<const float4*>(row + 68));
    cc[0] = c0.x; cc[1] = c0.y; cc[2] = c0.z; cc[3] = c0.w;
    cc[4] = c1.x; cc[5] = c1.y; cc[6] = c1.z; cc[7] = c1.w;
    sn[0] = s0.x; sn[1] = s0.y; sn[2] = s0.z; sn[3] = s0.w;
    sn[4] = s1.x; sn[5] = s1.y; sn[6] = s1.z; sn[7] = s1.w;
    // second halves turn with + partner sin, first halves with - partner sin
    if (lane < 8) {
#pragma unroll
      for (int j = 0; j < 8; ++j) sn[j] = -sn[j];
    }
  }
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    if (i >= nh) break;
    const int h = h0 + i;
    const uint32_t rw[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
    float y[8];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      y[2 * q] = bf_lo(rw[q]);
      y[2 * q + 1] = bf_hi(rw[q]);
    }
    const bool is_v = h >= p.Hq + p.Hkv;
    if (!is_v) {
      if (p.q_w != nullptr) {
        const uint4 w4 = h < p.Hq ? wq : wk;
        const uint32_t ww[4] = {w4.x, w4.y, w4.z, w4.w};
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(y[j], y[j], ss);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(hmask, ss, o);
        const float r = 1.f / sqrtf(ss / static_cast<float>(kPagedHeadDim) + p.eps);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          y[2 * q] = y[2 * q] * r * bf_lo(ww[q]);
          y[2 * q + 1] = y[2 * q + 1] * r * bf_hi(ww[q]);
        }
      }
      if (turn) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float partner = __shfl_xor_sync(hmask, y[j], 8);
          y[j] = fmaf(y[j], cc[j], partner * sn[j]);
        }
      }
    }
    if (h < p.Hq) {
      uint4* dst = reinterpret_cast<uint4*>(p.q_out + (static_cast<size_t>(t) * p.Hq + h) * kPagedHeadDim);
      dst[lane] = make_uint4(pack_bf(y[0], y[1]), pack_bf(y[2], y[3]), pack_bf(y[4], y[5]), pack_bf(y[6], y[7]));
      continue;
    }
    if (slot < 0) continue;
    const int g = is_v ? h - p.Hq - p.Hkv : h - p.Hq;
    const size_t at = (static_cast<size_t>(slot) * p.Hkv + g) * kPagedHeadDim;
    void* pool = is_v ? p.v_cache : p.k_cache;
    if constexpr (kE4M3) {
      // one rounding, from fp32: the quotient is not rounded to bf16 first
      const float sc = __ldg((is_v ? p.v_scale : p.k_scale) + g);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = y[j] / sc;
      const uint2 o = make_uint2(pack_e4m3x2(y[0], y[1]) | (pack_e4m3x2(y[2], y[3]) << 16),
                                 pack_e4m3x2(y[4], y[5]) | (pack_e4m3x2(y[6], y[7]) << 16));
      reinterpret_cast<uint2*>(static_cast<uint8_t*>(pool) + at)[lane] = o;
    } else {
      // values are copied bit for bit
      reinterpret_cast<uint4*>(static_cast<uint16_t*>(pool) + at)[lane] =
          is_v ? raw[i] : make_uint4(pack_bf(y[0], y[1]), pack_bf(y[2], y[3]), pack_bf(y[4], y[5]), pack_bf(y[6], y[7]));
    }
  }
}

}  // namespace
}  // namespace flint

using namespace flint;

extern "C" int flint_qk_norm_rope_paged_kv(const uint16_t* qkv, int32_t T, int32_t n_q_heads, int32_t n_kv_heads,
                                           int32_t head_dim, const uint16_t* q_norm_w, const uint16_t* k_norm_w,
                                           const float* cos_sin, int32_t max_pos, int32_t rope, float eps,
                                           const int32_t* q_start, const int32_t* kv_len, int32_t B,
                                           const int32_t* block_table, int32_t max_pages, int32_t page_size,
                                           int64_t n_pages, int32_t cache_dtype, const float* k_scale,
                                           const float* v_scale, uint16_t* q_out, void* k_cache, void* v_cache,
                                           int32_t* status, void* stream) {
  if (head_dim != kPagedHeadDim) return flint_fail_external(FLINT_ERR_UNSUPPORTED_SHAPE, "head_dim must be 128");
  if (n_q_heads < 1 || n_kv_heads < 1 || !(eps >= 0.f))
    return flint_fail_external(FLINT_ERR_INVALID_ARG, "flint_qk_norm_rope_paged_kv: bad sizes");
  if (n_q_heads > 65535 || n_kv_heads > 65535)
    return flint_fail_external(FLINT_ERR_UNSUPPORTED_SHAPE, "at most 65535 heads");
  AppendParams p{};
  const int rc = paged_batch(&p.b, "flint_qk_norm_rope_paged_kv", T, q_start, kv_len, B, block_table, max_pages,
                             page_size, n_pages, cache_dtype, k_cache, v_cache, k_scale, v_scale);
  if (rc != FLINT_OK) return rc;
  if (T == 0 || B == 0) return FLINT_OK;
  if (!qkv || !q_out || (q_norm_w == nullptr) != (k_norm_w == nullptr) || (rope && (!cos_sin || max_pos < 1)))
    return flint_fail_external(FLINT_ERR_INVALID_ARG, "flint_qk_norm_rope_paged_kv: NULL pointer");
  if (!paged_aligned16(qkv) || !paged_aligned16(q_out) || !paged_aligned16(q_norm_w) || !paged_aligned16(k_norm_w) ||
      (rope && !paged_aligned16(cos_sin)))
    return flint_fail_external(FLINT_ERR_MISALIGNED, "flint_qk_norm_rope_paged_kv: misaligned pointer");
  p.qkv = qkv;
  p.q_w = q_norm_w;
  p.k_w = k_norm_w;
  p.cos_sin = cos_sin;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.q_out = q_out;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.status = status;
  p.Hq = n_q_heads;
  p.Hkv = n_kv_heads;
  p.max_pos = max_pos;
  p.rope = rope ? 1 : 0;
  p.eps = eps;
  p.units = (n_q_heads + 2 * n_kv_heads + kHeads - 1) / kHeads;
  // units are counted in 32 bits
  const long long blocks = (static_cast<long long>(T) * p.units + kUnitsPerCta - 1) / kUnitsPerCta;
  if (blocks > 0x7fffffffLL / kUnitsPerCta) return flint_fail_external(FLINT_ERR_UNSUPPORTED_SHAPE, "too many tokens");
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cache_dtype == FLINT_KV_E4M3)
    k_paged_append<true><<<static_cast<unsigned>(blocks), kThreads, 0, st>>>(p);
  else
    k_paged_append<false><<<static_cast<unsigned>(blocks), kThreads, 0, st>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return flint_fail_external(FLINT_ERR_CUDA, cudaGetErrorString(e));
  return FLINT_OK;
}
