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
// One half-warp takes kHeads consecutive heads of one token; lane l holds
// elements 4l .. 4l + 3 and their rotation partners 64 + 4l .. 64 + 4l + 3 of
// each (two 8-byte loads, a half-warp reading two 128-byte runs; all heads'
// loads are issued before the first is used), so no element changes lanes, and
// the angles, the page lookup and the search for the token's sequence are done
// once for kHeads heads. Partners in other lanes, four heads a half-warp and
// IEEE root and quotients took 41 us for 7,803 tokens against 34.6, bound by
// instruction issue; what is left is the latency of the lookups in front of the
// angles (4.65 TB/s; 3, 5 or 8 heads a half-warp 36, 35 and 38 us). Calls of few
// tokens take two heads a half-warp (the launch below).
// HBM-bound: (Hq + 2 Hkv) 256 bytes read and Hq 256 + 2 Hkv 128 e written per
// token (e = 2 or 1 bytes), the cos/sin row (512 bytes) once per position.
#include "paged.cuh"

namespace flint {
namespace {

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

template <bool kE4M3, int kHeads>
__global__ void __launch_bounds__(kThreads) k_paged_append(AppendParams p) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 15;
  const unsigned hmask = 0xFFFFu << (threadIdx.x & 16);
  const unsigned unit = blockIdx.x * kUnitsPerCta + (threadIdx.x >> 4);
  const int t = static_cast<int>(unit / static_cast<unsigned>(p.units));
  if (t >= p.b.T) return;
  const int h0 = static_cast<int>(unit - static_cast<unsigned>(t) * p.units) * kHeads;
  const int H = p.Hq + 2 * p.Hkv;
  const int nh = min(kHeads, H - h0);
  uint2 raw[kHeads][2];
  const uint2* src = reinterpret_cast<const uint2*>(p.qkv + (static_cast<size_t>(t) * H + h0) * kPagedHeadDim) + lane;
#pragma unroll
  for (int i = 0; i < kHeads; ++i)
    if (i < nh) {
      raw[i][0] = __ldcs(src + i * 32);
      raw[i][1] = __ldcs(src + i * 32 + 16);
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
  // a sequence whose length cannot hold its tokens: no position, no page. In a q_start that is not sorted the search
  // may end at a sequence that begins behind t.
  const bool placed = sq.kv > 0 && t >= sq.row0 && t - sq.row0 < sq.n;
  long long slot = -1;
  if (placed) {
    const int page = __ldg(p.b.block_table + static_cast<size_t>(lo) * p.b.max_pages + (pos >> p.b.page_shift));
    if (page >= 0 && page < p.b.n_pages)
      slot = (static_cast<long long>(page) << p.b.page_shift) + (pos & ((1 << p.b.page_shift) - 1));
  }
  const bool turn = p.rope && placed && pos < p.max_pos;
  if (lane == 0 && p.status != nullptr && (slot < 0 || (p.rope && !turn))) atomicOr(p.status, FLINT_DEVCHECK_INDEX);
  // angles of this lane's four pairs (c, c + 64)
  float cc[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
  if (turn) {
    const float4* row = reinterpret_cast<const float4*>(p.cos_sin + static_cast<size_t>(pos) * kPagedHeadDim) + lane;
    const float4 c = __ldg(row), s = __ldg(row + 16);
    cc[0] = c.x; cc[1] = c.y; cc[2] = c.z; cc[3] = c.w;
    sn[0] = s.x; sn[1] = s.y; sn[2] = s.z; sn[3] = s.w;
  }
  // weights of the query heads, then of the key heads, by this lane's elements
  float w[8];
  int w_of = -1;  // 0: w holds the queries' weights, 1: the keys'
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    if (i >= nh) break;
    const int h = h0 + i;
    const bool is_v = h >= p.Hq + p.Hkv;
    float y[8] = {bf_lo(raw[i][0].x), bf_hi(raw[i][0].x), bf_lo(raw[i][0].y), bf_hi(raw[i][0].y),
                  bf_lo(raw[i][1].x), bf_hi(raw[i][1].x), bf_lo(raw[i][1].y), bf_hi(raw[i][1].y)};
    if (!is_v) {
      if (p.q_w != nullptr) {
        if (w_of != (h >= p.Hq)) {
          w_of = h >= p.Hq;
          const uint2* wp = reinterpret_cast<const uint2*>(w_of ? p.k_w : p.q_w) + lane;
          const uint2 w0 = __ldg(wp), w1 = __ldg(wp + 16);
          w[0] = bf_lo(w0.x); w[1] = bf_hi(w0.x); w[2] = bf_lo(w0.y); w[3] = bf_hi(w0.y);
          w[4] = bf_lo(w1.x); w[5] = bf_hi(w1.x); w[6] = bf_lo(w1.y); w[7] = bf_hi(w1.y);
        }
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(y[j], y[j], ss);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(hmask, ss, o);
        // rsqrtf: within 2 ulp of the root's reciprocal
        const float r = rsqrtf(fmaf(ss, 1.f / kPagedHeadDim, p.eps));
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] *= r * w[j];
      }
      if (turn) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float a = y[j], b = y[4 + j];
          y[j] = fmaf(a, cc[j], -b * sn[j]);
          y[4 + j] = fmaf(b, cc[j], a * sn[j]);
        }
      }
    }
    if (h < p.Hq) {
      uint2* dst = reinterpret_cast<uint2*>(p.q_out + (static_cast<size_t>(t) * p.Hq + h) * kPagedHeadDim) + lane;
      dst[0] = make_uint2(pack_bf(y[0], y[1]), pack_bf(y[2], y[3]));
      dst[16] = make_uint2(pack_bf(y[4], y[5]), pack_bf(y[6], y[7]));
      continue;
    }
    if (slot < 0) continue;
    const int g = is_v ? h - p.Hq - p.Hkv : h - p.Hq;
    const size_t at = (static_cast<size_t>(slot) * p.Hkv + g) * kPagedHeadDim;
    void* pool = is_v ? p.v_cache : p.k_cache;
    if constexpr (kE4M3) {
      // one rounding, from the fp32 quotient y / scale, which is not rounded to bf16 first. bf16 values often lie halfway
      // between two codes, where a product with the reciprocal, off by an ulp, picks the wrong one: the reciprocal is
      // taken in two floats (Brisebarre and Muller, "Correctly rounded multiplication by arbitrary precision
      // constants"), so the error in front of the fma's rounding is 2^-47. (A division an element: 1,504 tokens 10.9 us.)
      const float scale = __ldg((is_v ? p.v_scale : p.k_scale) + g);
      const float inv = 1.f / scale;
      const float inv_lo = scale >= 0x1p-24f ? fmaf(-scale, inv, 1.f) * inv : 0.f;  // 0: y inv_lo could overflow
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = fmaf(y[j], inv, y[j] * inv_lo);
      uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(pool) + at) + lane;
      dst[0] = pack_e4m3x2(y[0], y[1]) | (pack_e4m3x2(y[2], y[3]) << 16);
      dst[16] = pack_e4m3x2(y[4], y[5]) | (pack_e4m3x2(y[6], y[7]) << 16);
    } else {
      // values are copied bit for bit
      uint2* dst = reinterpret_cast<uint2*>(static_cast<uint16_t*>(pool) + at) + lane;
      dst[0] = is_v ? raw[i][0] : make_uint2(pack_bf(y[0], y[1]), pack_bf(y[2], y[3]));
      dst[16] = is_v ? raw[i][1] : make_uint2(pack_bf(y[4], y[5]), pack_bf(y[6], y[7]));
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
  const int rc = paged_batch(&p.b, T, q_start, kv_len, B, block_table, max_pages,
                             page_size, n_pages, cache_dtype, k_cache, v_cache, k_scale, v_scale, status);
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
  // heads a half-warp, 2 / 4, us: bf16 128 tokens 3.1 / 3.6, 512 4.1 / 5.2, 640 5.8 / 5.3, 2,048 12.4 / 12.4; E4M3
  // 128 3.4 / 4.1, 384 4.0 / 4.8, 512 5.8 / 5.4, 2,048 13.7 / 12.9
  const int heads = T <= 512 ? 2 : 4;
  p.units = (n_q_heads + 2 * n_kv_heads + heads - 1) / heads;
  // units are counted in 32 bits
  const long long blocks = (static_cast<long long>(T) * p.units + kUnitsPerCta - 1) / kUnitsPerCta;
  if (blocks > 0x7fffffffLL / kUnitsPerCta) return flint_fail_external(FLINT_ERR_UNSUPPORTED_SHAPE, "too many tokens");
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool e4m3 = cache_dtype == FLINT_KV_E4M3;
  auto kern = heads == 2 ? (e4m3 ? k_paged_append<true, 2> : k_paged_append<false, 2>)
                         : (e4m3 ? k_paged_append<true, 4> : k_paged_append<false, 4>);
  const cudaError_t e = launch_pdl(kern, static_cast<unsigned>(blocks), kThreads, 0, st, p);
  if (e != cudaSuccess) return flint_fail_external(FLINT_ERR_CUDA, cudaGetErrorString(e));
  return FLINT_OK;
}
