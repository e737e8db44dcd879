// sample.cu -- the next token of each row of logits, from given uniform numbers,
// with temperature, top-k, top-p and min-p ("Recursive Flint: 40B Local Coding
// Model, Benchmarks", architecture table, row "Vocabulary": the output head's
// 150,144 logits are what a decode step ends with).
//
// With w_i = exp((x_i - max x) / temperature) and the order "larger logit
// first, then lower index":
//   top-k   the first k tokens;
//   top-p   of those, each token whose predecessors hold less than top_p of
//           their mass;
//   min-p   of those, each token with w_i >= min_p (the largest w is 1);
//   token   the first index i, in vocabulary order, whose running sum of kept
//           w exceeds u times the kept total.
//
// No sort of the row: top-k and top-p both keep a prefix of the order, which is
// looked for in a histogram of 1,024 bins, linear in the logit (1/32 nat a bin).
//   top-k (k <= 512): the k-th largest of the threads' own maxima (known from
//     the load) bounds the k-th token from below, so the histogram is of one
//     value per thread. The tokens above the bound, little more than k, are
//     gathered in one CTA, ordered, cut by every filter and drawn from.
//   top-p: the histogram holds each bin's tokens and mass; the bins up to the
//     one the share ends in are gathered if they hold at most 1,024 tokens.
//   Otherwise that bin alone is gathered, its tokens ordered to find the one the
//     prefix ends with, and the draw passes over the whole row once more. (A bin
//     of more than 1,024 tokens, equal ones mostly, is first cut by the bit
//     patterns in order, 10 bits a level.)
//
// One thread-block cluster per row: each CTA keeps its share of the row in
// shared memory (one pass over HBM: 4 bytes a logit, the floor), the CTAs'
// histograms meet through distributed shared memory, and every CTA draws the
// same conclusion from them.
//
// Masses are sums of integers w 2^s (s = 44 for 150,144 tokens), 64 bits wide:
// the same in any order, so a run's result does not depend on the order of the
// shared-memory atomics; a token below 2^-46 of the largest is never drawn, far
// below what a 24-bit u can reach. Each w is right to 2^-27 of itself: a flat
// row of 150,144 tokens has its running sums within 1e-6 of one token's width
// (plain fp32 weights: 3e-5, a wrong token in one row of 15,000). Whole rows are
// bound by the instructions per token, so z = (x - max x) log2(e) / T is formed
// in one fp64 fma whose low word is z in fixed point, 26 bits behind the point,
// and the rest is integer and fp32: about 28 instructions. The same with fp64
// throughout, or with the argument in two floats, took 46 and 62.
#include <cooperative_groups.h>

#include <cfloat>
#include <cmath>
#include <utility>

#include "common.cuh"

namespace cg = cooperative_groups;

namespace flint {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 1024;
constexpr float kBinsPerNat = 32.f;
constexpr int kCand = 2 * kThreads;      // tokens the gathered form takes
constexpr int kCountSort = 256;          // up to here ranks are counted, above the tokens are sorted
constexpr int kTabCopies = 16;           // of the 2^(j / 64) table: one per bank pair
constexpr int kMaxSlice = 46 * 1024;     // keys of a CTA's share held in shared memory
constexpr uint32_t kNegInfKey = 0x007FFFFFu;  // key of -inf; NaN counts as -inf
constexpr int kClusterMax = 8;

typedef unsigned long long u64;

// 2^(j / 64) 2^28 as a float and rounded to an integer
struct ExpEntry {
  float f;
  int32_t i;
};

struct SampleParams {
  ExpEntry exp2_tab[64];
  const void* logits;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* u;
  int32_t* tokens;
  float* logprobs;
  int32_t* status;
  long long stride;
  int V, slice, up;
  double far;  // s + 2
};

// Order-preserving integer of a clean float (no NaN, no -0) and back.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

// The value as the row holds it: NaN as -inf, -0 as +0.
__device__ __forceinline__ float clean(float x) { return fmaxf(x, -INFINITY) + 0.f; }

struct Hist {
  uint32_t n[kBins], lo[kBins], hi[kBins];
};

__device__ __forceinline__ u64 warp_incl(u64 v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  return v;
}

// 64-bit mass into a bin as two 32-bit shared atomics; the carry goes with the
// low half's old value, so the sum is exact.
__device__ __forceinline__ void add_mass(Hist& h, int b, u64 m) {
  const uint32_t lo = static_cast<uint32_t>(m), hi = static_cast<uint32_t>(m >> 32);
  const uint32_t old = atomicAdd(&h.lo[b], lo);
  const uint32_t up = hi + (old + lo < old ? 1u : 0u);
  if (up) atomicAdd(&h.hi[b], up);
}

// x >> n, 0 from n = 32 on (as the instruction has it)
__device__ __forceinline__ uint32_t shift_right(uint32_t x, int n) {
  uint32_t r;
  asm("shr.u32 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(n));
  return r;
}

// Weights of a row, 2^z with z = (x - max x) log2(e) / T. One fma gives 63 + z
// in units of 2^-26 in the low word of a double (exact but for the last bit):
// with 63 + z = 64 bits e.jjjjjjffff..., 2^(j / 64) comes from the table, 2^f - 1
// (f < 1/64) from its Taylor series (degree 4: 1.2e-12; below 2^-6, so good to
// 2^-29 in fp32), 2^e from a shift. What a shift of more
// than 32 drops is half a unit of 2^-s on average, which the last bit stands for
// (units of 2^-(s + 1)); equal large weights stay multiples of 2^17, so their
// sums and shares of them are exact.
// Tokens below `far` (2^-(s + 2) of the largest; masked ones) have no mass.
struct Scale {
  double c, k;  // 2^26 log2(e) / T;  1.5 2^52 + 63 2^26 - c x_max
  float far;
  int up;       // how far 2^32 times the 28-bit weight goes right, for exponent bits e = 0
  __device__ __forceinline__ u64 mass(float x, const ExpEntry (*tab)[kTabCopies]) const {
    constexpr float kL = 0.693147180559945309417f / 64;  // ln 2 / 64, for f in units of 1/64
    const uint32_t z = static_cast<uint32_t>(__double2loint(__fma_rn(static_cast<double>(x), c, k)));
    const float f = __uint_as_float(((z << 3) & 0x7FFFF8u) | 0x3F800000u) - 1.f;
    float q = fmaf(kL * kL * kL * kL / 24, f, kL * kL * kL / 6);
    q = fmaf(q, f, kL * kL / 2);
    q = fmaf(q, f, kL) * f;
    const ExpEntry t = tab[(z >> 20) & 63][threadIdx.x & (kTabCopies - 1)];
    // adding 2^23 rounds 2^28 2^(j/64) (2^f - 1) < 2^23 to an integer in the low bits
    const uint32_t w =
        static_cast<uint32_t>(t.i + static_cast<int>(__float_as_uint(fmaf(q, t.f, 8388608.f)) - 0x4B000000u));
    const int sh = up - static_cast<int>(z >> 26);  // 3 or more
    const uint32_t lo = shift_right(__funnelshift_rc(0u, w, sh), max(sh - 32, 0)), hi = shift_right(w, sh);
    const u64 m = (static_cast<u64>(hi) << 32) | lo | (sh > 32 ? 1u : 0u);
    return x >= far ? m : 0;
  }
};

// A row's state, in shared memory: what the passes below share.
struct Row {
  Scale sc;
  float bin_inv, T, u, top_p;  // bins per logit; the row's parameters
  float x_max;
  u64 m_max;           // the largest token's mass
  float cut;           // the kept prefix ends at this logit (-inf: it is the whole row) ...
  uint32_t cut_ties;   // ... with this many of the tokens equal to it
  uint32_t cut_count;  // how many are equal to it
  float least;         // min-p: the lowest logit it keeps, or -inf
  int n, base, top_k;  // tokens of this CTA, the first one's index
};

// Where a histogram's running value reaches what is wanted.
struct Found {
  int bin;         // kBins: nowhere
  uint32_t upto;   // tokens up to and with the bin
  uint32_t in;     // tokens in it
  u64 above;       // running value in front of it
  u64 want;
};

static_assert(kBins == kCand && kBins == 2 * kThreads, "scratch of find and finish_many; find's two bins a thread");

struct Shared {
  Hist h;
  u64 cand[kCand];     // gathered tokens: key, then ~index
  u64 mass_of[kCand];
  ExpEntry exp2_tab[64][kTabCopies];
  Row row;
  Found found;
  u64 seg_val[kClusterMax];  // of each CTA's part of the bins: value, tokens
  uint32_t seg_n[kClusterMax];
  u64 key;             // largest key of this CTA, then ~place
  u64 mass;            // final pass: this CTA's kept mass above the cut, ties at it
  uint32_t ties;
  // block-local scratch
  u64 wsum[kWarps];
  uint32_t wcnt[kWarps];
  uint32_t cand_n[2];  // one per try
  uint32_t local_n, push_at;
};

// What every row runs is inlined in the order it runs in, and the rarer forms
// (narrowing, sorting) are functions of their own: a row's kernel runs most of
// its instructions once, so fetching them counts. All of it as functions: one
// row with top-k and top-p 13.2 us against 12.2.
__device__ __forceinline__ u64 mass_of(const Shared& sh, float x) { return sh.row.sc.mass(x, sh.exp2_tab); }

// First-level bin: (x_max - x) / (T / 32), the last one for everything below 32 nats.
__device__ __forceinline__ int bin_of(float x, float x_max, float bin_inv) {
  if (x == x_max) return 0;
  const float d = (x_max - x) * bin_inv;
  return d < static_cast<float>(kBins - 1) ? static_cast<int>(d) : kBins - 1;
}
// Bounds of the logits that can lie in bin b, with room for rounding.
__device__ __forceinline__ float bin_top(const Row& r, int b) {
  if (b == 0) return r.x_max;
  const float d = __fmul_rd(static_cast<float>(b), r.T * (1.f / kBinsPerNat * (1.f - 0x1p-18f)));
  return fminf(r.x_max, clean(__fsub_ru(r.x_max, d)));
}
__device__ __forceinline__ float bin_bottom(const Row& r, int b) {
  if (b >= kBins - 1) return -INFINITY;
  const float d = __fmul_ru(static_cast<float>(b + 1), r.T * (1.f / kBinsPerNat * (1.f + 0x1p-18f)));
  return fminf(r.x_max, clean(__fsub_rd(r.x_max, d)));
}

// A row's share: in shared memory, or read again from global memory.
template <typename TL, bool kResident>
struct Share {
  const float* held;
  const TL* src;
  bool inf_row;
  bool vec;  // src is 16-byte aligned
  __device__ __forceinline__ float global(int i) const {
    if constexpr (sizeof(TL) == 4) return clean(__ldg(reinterpret_cast<const float*>(src) + i));
    else return clean(bf16_bits_to_f32(__ldg(reinterpret_cast<const uint16_t*>(src) + i)));
  }
  // a row whose maximum is +inf: the infinite tokens count as zeros, all others as masked
  __device__ __forceinline__ float fix(float x) const { return !inf_row ? x : x == INFINITY ? 0.f : -INFINITY; }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (kResident) return held[i];
    return fix(global(i));
  }
  // four tokens at i, a multiple of 4; NaN past the end
  __device__ __forceinline__ void get4(int i, int end, float (&x)[4]) const {
    if (kResident && i + 4 <= end) {
      const float4 v = *reinterpret_cast<const float4*>(held + i);
      x[0] = v.x;
      x[1] = v.y;
      x[2] = v.z;
      x[3] = v.w;
      return;
    }
    if (!kResident && vec && i + 4 <= end) {
      if constexpr (sizeof(TL) == 4) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(reinterpret_cast<const float*>(src) + i));
        x[0] = v.x;
        x[1] = v.y;
        x[2] = v.z;
        x[3] = v.w;
      } else {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(src) + i));
        x[0] = __uint_as_float(v.x << 16);
        x[1] = __uint_as_float(v.x & 0xFFFF0000u);
        x[2] = __uint_as_float(v.y << 16);
        x[3] = __uint_as_float(v.y & 0xFFFF0000u);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) x[q] = fix(clean(x[q]));
      return;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) x[q] = i + q < end ? get(i + q) : __int_as_float(0x7FC00000);
  }
};

__device__ __forceinline__ bool any_in(const float (&x)[4], float lo, float hi) {
  return (x[0] >= lo && x[0] <= hi) || (x[1] >= lo && x[1] <= hi) || (x[2] >= lo && x[2] <= hi) ||
         (x[3] >= lo && x[3] <= hi);
}

__device__ __forceinline__ u64 warp_sum64(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Histogram of the tokens with keys in [klo, khi]: level 1 (b1 < 0) by bin_of,
// later levels (only tokens of first-level bin b1) by the key's distance from khi.
template <bool kByMass, typename S>
__device__ __forceinline__ void hist_pass(Shared& sh, const S s, uint32_t klo, uint32_t khi, int shift, int b1) {
  const int n = sh.row.n;
  Hist& h = sh.h;
  const Scale sc = sh.row.sc;
  const float x_max = sh.row.x_max, bin_inv = sh.row.bin_inv;
  const float xlo = value_of(klo), xhi = value_of(khi);
  uint32_t far_n = 0;
  u64 far_m = 0;
#pragma unroll 1
  for (int i = 4 * threadIdx.x; i < n; i += 4 * kThreads) {
    float x[4];
    s.get4(i, n, x);
    if (b1 >= 0 && !any_in(x, xlo, xhi)) continue;  // most of a later level's tokens
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (!(x[q] >= xlo && x[q] <= xhi)) continue;
      int b = bin_of(x[q], x_max, bin_inv);
      if (b1 >= 0) {
        if (b != b1) continue;
        b = static_cast<int>((khi - key_of(x[q])) >> shift);
      }
      u64 m = 0;
      if constexpr (kByMass) m = sc.mass(x[q], sh.exp2_tab);
      if (b1 < 0 && b == kBins - 1) {  // the bulk of a cold row: summed in registers
        ++far_n;
        far_m += m;
      } else {
        atomicAdd(&h.n[b], 1u);
        if constexpr (kByMass) add_mass(h, b, m);
      }
    }
  }
  if (b1 < 0) {
    far_n = __reduce_add_sync(0xffffffffu, far_n);
    if constexpr (kByMass) far_m = warp_sum64(far_m);
    if ((threadIdx.x & 31) == 0 && far_n != 0) {
      atomicAdd(&h.n[kBins - 1], far_n);
      if constexpr (kByMass) add_mass(h, kBins - 1, far_m);
    }
  }
}

// The bin of the merged histogram (all CTAs' h) in which the running value (the
// mass, or the count), `above` in front of the first bin, reaches `want`; every
// CTA gets the same answer. want_p >= 0: want is that share of the total mass,
// known here. Each CTA merges its part of the bins and scans it; the parts'
// totals go to all, and the part that holds the bin tells it to all. (Every CTA
// merging all bins took 5 us a call, three words from each of 8 CTAs a bin.)
// The histogram is cleared.
template <bool kByMass>
__device__ __forceinline__ Found find(Shared& sh, u64 above, u64 want, float want_p) {
  cg::cluster_group cl = cg::this_cluster();
  const int C = static_cast<int>(cl.num_blocks()), rank = static_cast<int>(cl.block_rank());
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int part = kBins / C, part0 = rank * part;  // C a power of two
  uint32_t* cnt_of = reinterpret_cast<uint32_t*>(sh.cand);
  if (tid == 0) sh.found.bin = kBins;
  cl.sync();
#pragma unroll
  for (int r = 0; r < kBins / kThreads; ++r) {  // this part's bins from each CTA
    const int e = tid + r * kThreads, c = e / part, b = part0 + (e & (part - 1));
    const Hist* h = cl.map_shared_rank(&sh.h, c);
    cnt_of[e] = h->n[b];
    if constexpr (kByMass) sh.mass_of[e] = (static_cast<u64>(h->hi[b]) << 32) + h->lo[b];
  }
  __syncthreads();
  // two neighbouring bins a thread (threads past the part: none)
  uint32_t n0 = 0, n1 = 0;
  u64 v0 = 0, v1 = 0;
  if (2 * tid < part) {
#pragma unroll 1
    for (int e = 2 * tid; e < kBins; e += part) {
      n0 += cnt_of[e];
      n1 += cnt_of[e + 1];
      if constexpr (kByMass) {
        v0 += sh.mass_of[e];
        v1 += sh.mass_of[e + 1];
      }
    }
  }
  if constexpr (!kByMass) {
    v0 = n0;
    v1 = n1;
  }
  u64 inc = warp_incl(v0 + v1, lane);
  uint32_t n_inc = static_cast<uint32_t>(warp_incl(n0 + n1, lane));
  if (lane == 31) {
    sh.wsum[warp] = inc;
    sh.wcnt[warp] = n_inc;
  }
  __syncthreads();
  {
    const u64 w = lane < kWarps ? sh.wsum[lane] : 0;
    const uint32_t wn = lane < kWarps ? sh.wcnt[lane] : 0;
    const u64 wi = warp_incl(w, lane);
    const uint32_t wni = static_cast<uint32_t>(warp_incl(wn, lane));
    inc += __shfl_sync(0xffffffffu, wi - w, warp);
    n_inc += __shfl_sync(0xffffffffu, wni - wn, warp);
    const u64 all = __shfl_sync(0xffffffffu, wi, 31);
    const uint32_t all_n = __shfl_sync(0xffffffffu, wni, 31);
    if (warp == 0 && lane < C) {
      Shared* to = cl.map_shared_rank(&sh, lane);
      to->seg_val[rank] = all;
      to->seg_n[rank] = all_n;
    }
  }
  cl.sync();
  u64 total = 0, before = above;
  uint32_t n_before = 0;
#pragma unroll 1
  for (int c = 0; c < C; ++c) {
    if (c < rank) {
      before += sh.seg_val[c];
      n_before += sh.seg_n[c];
    }
    total += sh.seg_val[c];
  }
  if (kByMass && want_p >= 0.f) {
    // ties at the floor beyond those that top-k keeps hold no mass
    if (sh.row.cut != -INFINITY) total -= static_cast<u64>(sh.row.cut_count - sh.row.cut_ties) * mass_of(sh, sh.row.cut);
    want = static_cast<u64>(ceil(static_cast<double>(want_p) * static_cast<double>(total)));
    want = want < 1 ? 1 : want > total ? total : want;  // the total may round up as a double
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const u64 end = before + inc - (q == 0 ? v1 : 0), start = end - (q == 0 ? v0 : v1);
    if (start < want && end >= want) {
      const Found f{part0 + 2 * tid + q, n_before + n_inc - (q == 0 ? n1 : 0), q == 0 ? n0 : n1, start, want};
#pragma unroll 1
      for (int c = 0; c < C; ++c) cl.map_shared_rank(&sh, c)->found = f;
    }
  }
  for (int i = tid; i < kBins; i += kThreads) sh.h.n[i] = sh.h.lo[i] = sh.h.hi[i] = 0;
  cl.sync();
  return sh.found;
}

// Gathers the tokens of logits in [from, to] and of first-level bins b0 to b1 in
// the first CTA: each CTA collects its own, asks for room once, and pushes them
// (those past kCand not). Their number is in the first CTA's cand_n[slot].
template <typename S>
__device__ __forceinline__ void gather(Shared& sh, const S s, float from, float to, int b0, int b1, int slot) {
  cg::cluster_group cl = cg::this_cluster();
  Shared* lead = cl.map_shared_rank(&sh, 0);
  const int n = sh.row.n, base = sh.row.base;
  const float x_max = sh.row.x_max, bin_inv = sh.row.bin_inv;
#pragma unroll 2
  for (int i = 4 * threadIdx.x; i < n; i += 4 * kThreads) {
    float x[4];
    s.get4(i, n, x);
    if (!any_in(x, from, to)) continue;
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
      const float y = q == 0 ? x[0] : q == 1 ? x[1] : q == 2 ? x[2] : x[3];
      if (!(y >= from && y <= to)) continue;
      const int b = bin_of(y, x_max, bin_inv);
      if (b < b0 || b > b1) continue;
      const uint32_t at = atomicAdd(&sh.local_n, 1u);
      if (at < kCand)
        sh.mass_of[at] = (static_cast<u64>(key_of(y)) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(base + i + q));
    }
  }
  __syncthreads();
  const uint32_t mine = sh.local_n;
  if (threadIdx.x == 0) sh.push_at = mine != 0 ? atomicAdd(&lead->cand_n[slot], mine) : 0;
  __syncthreads();
  const uint32_t at = sh.push_at;
  for (uint32_t i = threadIdx.x; i < mine && at + i < kCand; i += kThreads) lead->cand[at + i] = sh.mass_of[i];
  if (threadIdx.x == 0) sh.local_n = 0;
  cl.sync();
}

// Sum of one value per thread.
__device__ __forceinline__ u64 block_sum(Shared& sh, u64 v) {
  v = warp_sum64(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh.wsum[threadIdx.x >> 5] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  return warp_sum64(lane < kWarps ? sh.wsum[lane] : 0);
}

__device__ __forceinline__ u64 share_of(float p, u64 total) {
  const u64 w = static_cast<u64>(ceil(static_cast<double>(fmaxf(p, 0.f)) * static_cast<double>(total)));
  return w < 1 ? 1 : w;
}

// Writes the row's token if the running mass reaches the target within [before, before + m). Its log-probability comes
// from its logit, logit(), and the largest token's share: m itself may be a few units only. (ln(m / total): 8 unfiltered
// rows 13.9 us against 14.2, 128 mixed ones 120.4 against 121.9; registers are spilled for the logit.)
template <typename F>
__device__ __forceinline__ void draw(const Shared& sh, const SampleParams& p, int row, F logit, int id, u64 m, u64 before,
                                     u64 total) {
  const Row& r = sh.row;
  const u64 target = static_cast<u64>(static_cast<double>(r.u) * static_cast<double>(total));
  if (!(before <= target && target < before + m)) return;
  p.tokens[row] = id;
  if (p.logprobs == nullptr) return;
  const double below =
      (static_cast<double>(logit()) - static_cast<double>(r.x_max)) * (r.sc.c * (0.69314718055994530942 * 0x1p-26));
  p.logprobs[row] =
      static_cast<float>(below + log(static_cast<double>(r.m_max) / static_cast<double>(total)));
}

// Sorts the first n2 (a power of two <= kCand) words of v descending; whole block.
__device__ __noinline__ void sort_desc(u64* v, int n2) {
  const int t = threadIdx.x;
  for (int k = 2; k <= n2; k <<= 1) {
    for (int j = k >> 1; j > 0; j >>= 1) {
      if (t < (n2 >> 1)) {
        const int i = ((t & ~(j - 1)) << 1) | (t & (j - 1));
        const u64 a = v[i], b = v[i + j];
        if ((a < b) == ((i & k) == 0)) {
          v[i] = b;
          v[i + j] = a;
        }
      }
      // pairs at most 32 apart stay within a warp's 64 words
      if (j > 32) __syncthreads();
      else __syncwarp();
    }
    __syncthreads();
  }
}

// Draws from up to kCountSort gathered tokens, which contain the kept prefix:
// `parts` threads per token count the tokens (and their mass) in front of it,
// first in the order of the logits, then of the vocabulary. want: the mass at
// which top-p ends the prefix, 0 if that is still to be taken of the first top_k.
__device__ __forceinline__ void finish_few(Shared& sh, const SampleParams& p, int row, int n_cand, u64 want) {
  const int tid = threadIdx.x;
  const int n_k = sh.row.top_k > 0 ? min(n_cand, sh.row.top_k) : n_cand;
  int n2 = 32;
  while (n2 < n_cand) n2 <<= 1;
  const int parts = kThreads / n2;  // 2 .. 16
  const int i = tid / parts, sub = tid & (parts - 1);
  const bool live = i < n_cand;
  const u64 ci = live ? sh.cand[i] : 0;
  u64 m = sub == 0 && live ? mass_of(sh, value_of(static_cast<uint32_t>(ci >> 32))) : 0;
  if (sub == 0 && live) sh.mass_of[i] = m;
  __syncthreads();
  int rank = 0;
  u64 before = 0;
#pragma unroll 4
  for (int j = sub; j < n_cand; j += parts) {
    const u64 mj = sh.mass_of[j];
    const bool front = sh.cand[j] > ci;
    rank += front ? 1 : 0;
    before += front ? mj : 0;
  }
#pragma unroll 1
  for (int o = parts >> 1; o > 0; o >>= 1) {
    rank += __shfl_xor_sync(0xffffffffu, rank, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  if (rank >= n_k) m = 0;
  if (sh.row.top_p < 1.f) {
    if (want == 0) want = share_of(sh.row.top_p, block_sum(sh, m));
    if (before >= want) m = 0;
  }
  if (value_of(static_cast<uint32_t>(ci >> 32)) < sh.row.least) m = 0;
  const u64 total = block_sum(sh, m);  // its barriers also end the reads of mass_of
  if (sub == 0 && live) sh.mass_of[i] = m;
  __syncthreads();
  before = 0;
#pragma unroll 4
  for (int j = sub; j < n_cand; j += parts) {
    const u64 mj = sh.mass_of[j];
    before += static_cast<uint32_t>(sh.cand[j]) > static_cast<uint32_t>(ci) ? mj : 0;
  }
#pragma unroll 1
  for (int o = parts >> 1; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
  if (sub == 0)
    draw(sh, p, row, [&] { return value_of(static_cast<uint32_t>(ci >> 32)); },
         static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(ci)), m, before, total);
}

// The same from up to kCand gathered tokens, sorted; two tokens per thread.
__device__ __noinline__ void finish_many(Shared& sh, const SampleParams& p, int row, int n_cand, u64 want) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n_k = sh.row.top_k > 0 ? min(n_cand, sh.row.top_k) : n_cand;
  int n2 = kCountSort;
  while (n2 < n_cand) n2 <<= 1;
  for (int i = n_cand + tid; i < n2; i += kThreads) sh.cand[i] = 0;
  __syncthreads();
  sort_desc(sh.cand, n2);
  u64 c[2], m[2], before = 0, total = 0;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int i = 2 * tid + q;
    c[q] = i < n_k ? sh.cand[i] : 0;
    m[q] = i < n_k ? mass_of(sh, value_of(static_cast<uint32_t>(c[q] >> 32))) : 0;
  }
#pragma unroll 1
  for (int round = 0; round < 2; ++round) {
    // running mass in the order of the logits, then of the vocabulary
    const u64 inc = warp_incl(m[0] + m[1], lane);
    __syncthreads();
    if (lane == 31) sh.wsum[warp] = inc;
    __syncthreads();
    before = inc - m[0] - m[1];
    total = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += sh.wsum[w];
      total += sh.wsum[w];
    }
    if (round == 1) break;
    if (sh.row.top_p < 1.f) {
      const u64 end = want != 0 ? want : share_of(sh.row.top_p, total);
      if (before + m[0] >= end) m[1] = 0;
      if (before >= end) m[0] = 0;
    }
    // what holds mass, by index (largest ~index first)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int i = 2 * tid + q;
      if (value_of(static_cast<uint32_t>(c[q] >> 32)) < sh.row.least) m[q] = 0;
      if (i < n2) {
        sh.cand[i] = m[q] > 0 ? (c[q] << 32) | static_cast<uint32_t>(i) : 0;
        sh.mass_of[i] = m[q];
        sh.h.n[i] = static_cast<uint32_t>(c[q] >> 32);  // the histogram is done with
      }
    }
    __syncthreads();
    sort_desc(sh.cand, n2);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int i = 2 * tid + q;
      c[q] = i < n2 ? sh.cand[i] : 0;
      m[q] = c[q] != 0 ? sh.mass_of[static_cast<uint32_t>(c[q])] : 0;
    }
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    if (m[q] != 0)
      draw(sh, p, row, [&] { return value_of(sh.h.n[static_cast<uint32_t>(c[q])]); },
           static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(c[q] >> 32)), m[q], before, total);
    before += m[q];
  }
}

__device__ __forceinline__ void finish(Shared& sh, const SampleParams& p, int row, uint32_t n_cand, u64 want) {
  if (n_cand <= kCountSort) finish_few(sh, p, row, static_cast<int>(n_cand), want);
  else finish_many(sh, p, row, static_cast<int>(n_cand), want);
}

// Narrows to the logit at which the running count or mass reaches `want`, over
// the prefix kept so far; want_p: want is that share of its mass. True if the
// row was finished from a gather.
template <bool kByMass, typename S>
__device__ __noinline__ bool narrow(Shared& sh, const SampleParams& p, const S s, int row, u64 want, float want_p) {
  cg::cluster_group cl = cg::this_cluster();
  const int rank = static_cast<int>(cl.block_rank()), tid = threadIdx.x;
  const float floor_x = sh.row.cut;
  uint32_t klo = key_of(floor_x), khi = key_of(sh.row.x_max);
  int shift = 0, b1 = -1;
  u64 above = 0;
#pragma unroll 1
  for (int step = 0; step < 6; ++step) {  // at most five levels: 1 + ceil(32 / 10)
    __syncthreads();
    hist_pass<kByMass>(sh, s, klo, khi, shift, b1);
    const Found f = find<kByMass>(sh, above, want, step == 0 ? want_p : -1.f);
    if (f.bin >= kBins) return false;
    above = f.above;
    want = f.want;
    if (step == 0) {
      b1 = f.bin;
      const float bottom = fmaxf(floor_x, bin_bottom(sh.row, b1));
      if (f.upto <= kCand) {
        gather(sh, s, bottom, INFINITY, 0, b1, 1);
        if (rank == 0) finish(sh, p, row, f.upto, kByMass ? want : 0);
        return true;
      }
      klo = key_of(bottom);
      khi = max(klo, key_of(bin_top(sh.row, b1)));
    } else {
      khi -= static_cast<uint32_t>(f.bin) << shift;
      klo = shift > 0 ? max(klo, khi - ((1u << shift) - 1u)) : khi;
    }
    if (f.in <= kCand || (klo == khi && step > 0)) {
      float x = value_of(khi);
      uint32_t keep = 0, equal = f.in;
      if (f.in <= kCand) {
        // the tokens of the bin, in order: the prefix ends with the one at which the value is reached
        gather(sh, s, value_of(klo), value_of(khi), b1, b1, 1);
        if (rank == 0) {
          int n2 = 2;
          while (n2 < static_cast<int>(f.in)) n2 <<= 1;
          for (int i = f.in + tid; i < n2; i += kThreads) sh.cand[i] = 0;
          __syncthreads();
          sort_desc(sh.cand, n2);
          u64 v[2];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int i = 2 * tid + q;
            v[q] = i >= static_cast<int>(f.in) ? 0
                   : kByMass                   ? mass_of(sh, value_of(static_cast<uint32_t>(sh.cand[i] >> 32)))
                                               : 1;
          }
          const int lane = tid & 31, warp = tid >> 5;
          u64 inc = warp_incl(v[0] + v[1], lane);
          __syncthreads();
          if (lane == 31) sh.wsum[warp] = inc;
          __syncthreads();
          for (int w = 0; w < warp; ++w) inc += sh.wsum[w];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const u64 end = above + inc - (q == 0 ? v[1] : 0);
            if (end - v[q] < want && end >= want) {
              const int i = 2 * tid + q;
              const uint32_t k = static_cast<uint32_t>(sh.cand[i] >> 32);
              int lo = i, hi = i;  // the run of equal logits
              while (lo > 0 && static_cast<uint32_t>(sh.cand[lo - 1] >> 32) == k) --lo;
              while (hi + 1 < static_cast<int>(f.in) && static_cast<uint32_t>(sh.cand[hi + 1] >> 32) == k) ++hi;
              sh.found = Found{static_cast<int>(k), static_cast<uint32_t>(hi - lo + 1), static_cast<uint32_t>(i - lo + 1),
                               0, 0};
            }
          }
          __syncthreads();
        }
        cl.sync();
        const Found* from = &cl.map_shared_rank(&sh, 0)->found;
        x = value_of(static_cast<uint32_t>(from->bin));
        equal = from->upto;
        keep = from->in;
      } else if (kByMass) {  // equal tokens only
        const u64 w = mass_of(sh, x);
        keep = w > 0 ? static_cast<uint32_t>(min(static_cast<u64>(f.in), (want - above + w - 1) / w)) : f.in;
      } else {
        keep = static_cast<uint32_t>(want - above);
      }
      if (x == floor_x) keep = min(keep, sh.row.cut_ties);
      if (rank == 0 && tid == 0) sh.cand_n[1] = 0;
      cl.sync();  // read by all
      if (tid == 0) {
        sh.row.cut = x;
        sh.row.cut_ties = keep;
        sh.row.cut_count = equal;
      }
      __syncthreads();
      return false;
    }
    shift = max(0, 32 - __clz(khi - klo) - 10);
  }
  return false;
}

// Four tokens at i (a multiple of 4) as far as `end`: their mass if above the cut
// and not below `least`; how many are equal to the cut.
template <typename S>
__device__ __forceinline__ uint32_t weigh4(const Shared& sh, const S& s, const Scale& sc, float cut, float least, int i,
                                           int end, float (&x)[4], u64 (&m)[4]) {
  s.get4(i, end, x);
  uint32_t t = 0;
  if (cut != -INFINITY) {
#pragma unroll
    for (int q = 0; q < 4; ++q) t += x[q] == cut ? 1u : 0u;
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) m[q] = 0;
  const float most = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
  if (most > cut && most >= least) {  // not so in most of a filtered row
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      m[q] = sc.mass(x[q], sh.exp2_tab);
      if (!(x[q] > cut && x[q] >= least)) m[q] = 0;
    }
  }
  return t;
}

// The draw over the whole row: each warp weighs a run of consecutive tokens.
template <typename S>
__device__ __forceinline__ void draw_all(Shared& sh, const SampleParams& p, const S s, int row) {
  cg::cluster_group cl = cg::this_cluster();
  const int C = static_cast<int>(cl.num_blocks()), rank = static_cast<int>(cl.block_rank());
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = sh.row.n;
  const uint32_t cut_ties = sh.row.cut_ties;
  const float cut = sh.row.cut, least = sh.row.least;
  const Scale sc = sh.row.sc;
  const u64 m_cut = cut >= least ? mass_of(sh, cut) : 0;  // 0 for -inf
  const int span = ((n + kWarps - 1) / kWarps + 127) & ~127;
  u64 mass = 0;
  uint32_t ties = 0;
  // round 0: the runs' masses; round 1: the run that holds the target, by its whole CTA
  int i0 = warp * span + 4 * lane, end = min(n, (warp + 1) * span), stride = 128;
  u64 at = 0, total = 0, target = 0;
  uint32_t seen = 0;
#pragma unroll 1
  for (int round = 0;; ++round) {
#pragma unroll 1
    for (int i = i0; round == 1 ? i - 4 * tid < end : i < end; i += stride) {
      float x4[4];
      u64 m[4];
      const uint32_t mine = weigh4(sh, s, sc, cut, least, i, end, x4, m);
      if (round == 0) {
        ties += mine;
        mass += (m[0] + m[1]) + (m[2] + m[3]);
        continue;
      }
      const uint32_t tie_i = static_cast<uint32_t>(warp_incl(mine, lane));
      __syncthreads();
      if (lane == 31) sh.wcnt[warp] = tie_i;
      __syncthreads();
      const uint32_t tw = lane < kWarps ? sh.wcnt[lane] : 0;
      const uint32_t tw_i = static_cast<uint32_t>(warp_incl(tw, lane));
      uint32_t tie = seen + __shfl_sync(0xffffffffu, tw_i - tw, warp) + tie_i - mine;
      u64 sum = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (x4[q] == cut && tie++ < cut_ties) m[q] = m_cut;
        sum += m[q];
      }
      const u64 inc = warp_incl(sum, lane);
      if (lane == 31) sh.wsum[warp] = inc;
      __syncthreads();
      const u64 mw = lane < kWarps ? sh.wsum[lane] : 0;
      const u64 mw_i = warp_incl(mw, lane);
      u64 x = at + __shfl_sync(0xffffffffu, mw_i - mw, warp) + inc - sum;
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        const u64 mq = q == 0 ? m[0] : q == 1 ? m[1] : q == 2 ? m[2] : m[3];
        if (mq != 0) draw(sh, p, row, [&] { return s.get(i + q); }, sh.row.base + i + q, mq, x, total);
        x += mq;
      }
      seen += __shfl_sync(0xffffffffu, tw_i, 31);
      at += __shfl_sync(0xffffffffu, mw_i, 31);
      if (at > target) return;
    }
    if (round == 1) return;
    mass = warp_sum64(mass);
    ties = __reduce_add_sync(0xffffffffu, ties);
    __syncthreads();
    if (lane == 0) {
      sh.wsum[warp] = mass;
      sh.wcnt[warp] = ties;
    }
    __syncthreads();
    // every warp: lane w holds warp w's; running sums over the CTA's warps
    const u64 w_mass = lane < kWarps ? sh.wsum[lane] : 0;
    const uint32_t w_ties = lane < kWarps ? sh.wcnt[lane] : 0;
    const u64 w_mass_i = warp_incl(w_mass, lane);
    const uint32_t w_ties_i = static_cast<uint32_t>(warp_incl(w_ties, lane));
    if (tid == 31) {
      sh.mass = w_mass_i;
      sh.ties = w_ties_i;
    }
    cl.sync();
    // lane c: CTA c's kept mass (its ties as far as the cut takes them), and running sums
    const u64 c_mass = lane < C ? *cl.map_shared_rank(&sh.mass, lane) : 0;
    const uint32_t c_ties = lane < C ? *cl.map_shared_rank(&sh.ties, lane) : 0;
    cl.sync();  // the last read of another CTA's shared memory
    const uint32_t c_ties_i = static_cast<uint32_t>(warp_incl(c_ties, lane));
    const u64 c_kept = c_mass + static_cast<u64>(min(c_ties_i, cut_ties) - min(c_ties_i - c_ties, cut_ties)) * m_cut;
    const u64 c_kept_i = warp_incl(c_kept, lane);
    total = __shfl_sync(0xffffffffu, c_kept_i, 31);
    const u64 before = __shfl_sync(0xffffffffu, c_kept_i - c_kept, rank);
    const uint32_t ties_before = __shfl_sync(0xffffffffu, c_ties_i - c_ties, rank);
    target = static_cast<u64>(static_cast<double>(sh.row.u) * static_cast<double>(total));
    // lane w: the interval of the running mass that warp w's run covers; exactly
    // one run of the cluster holds the target
    const uint32_t lo_t = min(cut_ties, ties_before + w_ties_i - w_ties), hi_t = min(cut_ties, ties_before + w_ties_i);
    const u64 lo_m = before + (w_mass_i - w_mass) + static_cast<u64>(lo_t - min(cut_ties, ties_before)) * m_cut;
    const u64 hi_m = lo_m + w_mass + static_cast<u64>(hi_t - lo_t) * m_cut;
    const unsigned hit = __ballot_sync(0xffffffffu, lane < kWarps && lo_m <= target && target < hi_m);
    if (hit == 0) return;
    const int owner = __ffs(hit) - 1;
    at = __shfl_sync(0xffffffffu, lo_m, owner);
    seen = __shfl_sync(0xffffffffu, ties_before + w_ties_i - w_ties, owner);
    i0 = owner * span + 4 * tid;
    end = min(n, (owner + 1) * span);
    stride = 4 * kThreads;
  }
}

template <typename TL, bool kResident>
__global__ void __launch_bounds__(kThreads, 2) k_sample(const __grid_constant__ SampleParams p) {
  extern __shared__ __align__(16) float s_held[];
  __shared__ Shared sh;
  cg::cluster_group cl = cg::this_cluster();
  const int C = static_cast<int>(cl.num_blocks()), rank = static_cast<int>(cl.block_rank());
  const int row = blockIdx.x / C;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int base = rank * p.slice;
  const int n = max(0, min(p.slice, p.V - base));
  Share<TL, kResident> s{s_held, static_cast<const TL*>(p.logits) + static_cast<size_t>(row) * p.stride + base, false, false};
  s.vec = (reinterpret_cast<uintptr_t>(s.src) & 15u) == 0;
  const float T = p.temperature != nullptr ? __ldg(p.temperature + row) : 1.f;
  const float u = __ldg(p.u + row);
  const int top_k = p.top_k != nullptr ? __ldg(p.top_k + row) : 0;
  const float top_p = p.top_p != nullptr ? __ldg(p.top_p + row) : 1.f;
  const float min_p = p.min_p != nullptr ? __ldg(p.min_p + row) : 0.f;

  // ---- the row's share into shared memory; the largest (key, lowest index).
  // 16-byte loads where the row allows them, kBatch in flight per thread.
  constexpr int kVec = 16 / sizeof(TL), kBatch = 5;
  float own_max = -INFINITY;
  int own_at = 0;  // the first four tokens (or one) that hold it: a thread's indices only grow
  const int n_vec = s.vec ? n / kVec : 0;
#pragma unroll 1
  for (int i0 = tid; i0 < n_vec; i0 += kThreads * kBatch) {
    uint4 v[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
      if (i0 + b * kThreads < n_vec) v[b] = __ldg(reinterpret_cast<const uint4*>(s.src) + i0 + b * kThreads);
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int i = i0 + b * kThreads;
      if (i >= n_vec) break;
      const uint32_t x[4] = {v[b].x, v[b].y, v[b].z, v[b].w};
      float f[kVec];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if constexpr (sizeof(TL) == 4) {
          f[q] = clean(__uint_as_float(x[q]));
        } else {
          f[2 * q] = clean(__uint_as_float(x[q] << 16));
          f[2 * q + 1] = clean(__uint_as_float(x[q] & 0xFFFF0000u));
        }
      }
#pragma unroll
      for (int q = 0; q < kVec; q += 4) {
        const float most = fmaxf(fmaxf(f[q], f[q + 1]), fmaxf(f[q + 2], f[q + 3]));
        own_at = most > own_max ? i * kVec + q : own_at;
        own_max = fmaxf(own_max, most);
      }
      if constexpr (kResident) {
#pragma unroll
        for (int q = 0; q < kVec; q += 4)
          reinterpret_cast<float4*>(s_held)[(i * kVec + q) / 4] = make_float4(f[q], f[q + 1], f[q + 2], f[q + 3]);
      }
    }
  }
#pragma unroll 4
  for (int i = n_vec * kVec + tid; i < n; i += kThreads) {
    const float x = s.global(i);
    if constexpr (kResident) s_held[i] = x;
    own_at = x > own_max ? i : own_at;
    own_max = fmaxf(own_max, x);
  }
  // largest key of a warp and, of equals, the lowest place
  auto warp_best = [&](uint32_t k, uint32_t not_at) -> u64 {
    const uint32_t m = __reduce_max_sync(0xffffffffu, k);
    const uint32_t at = __reduce_max_sync(0xffffffffu, k == m ? not_at : 0u);
    return (static_cast<u64>(m) << 32) | at;
  };
  u64 best = warp_best(key_of(own_max), 0xFFFFFFFFu - static_cast<uint32_t>(base + own_at));
  if (lane == 0) sh.wsum[warp] = best;
  for (int i = tid; i < kBins; i += kThreads) sh.h.n[i] = sh.h.lo[i] = sh.h.hi[i] = 0;
  for (int i = tid; i < 64 * kTabCopies; i += kThreads)
    sh.exp2_tab[i / kTabCopies][i % kTabCopies] = p.exp2_tab[i / kTabCopies];
  if (tid == 64) sh.cand_n[0] = sh.cand_n[1] = sh.local_n = 0;
  __syncthreads();
  if (warp == 0) {
    best = lane < kWarps ? sh.wsum[lane] : 0;
    best = warp_best(static_cast<uint32_t>(best >> 32), static_cast<uint32_t>(best));
    if (lane == 0) sh.key = best;
  }
  cl.sync();
  // every warp: lane c reads CTA c's, all at once
  best = lane < C ? *cl.map_shared_rank(&sh.key, lane) : 0;
  best = warp_best(static_cast<uint32_t>(best >> 32), static_cast<uint32_t>(best));
  const uint32_t max_key = static_cast<uint32_t>(best >> 32);

  const bool bad_arg = !(T >= 0.f) || !(u >= 0.f && u < 1.f);
  if (bad_arg || max_key == kNegInfKey || T == 0.f) {  // the whole cluster agrees
    const bool none = bad_arg || max_key == kNegInfKey;
    int at = static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(best));
    if (!none && at >= base && at < base + n && tid == 0) {
      // the first of the four (one where the row is not aligned)
      while ((kResident ? s_held[at - base] : s.global(at - base)) != value_of(max_key)) ++at;
      p.tokens[row] = at;
      if (p.logprobs != nullptr) p.logprobs[row] = 0.f;
    }
    if (none && rank == 0 && tid == 0) {
      if (p.status != nullptr) atomicOr(p.status, bad_arg ? FLINT_DEVCHECK_INDEX : FLINT_DEVCHECK_NONFINITE);
      p.tokens[row] = -1;
      if (p.logprobs != nullptr) p.logprobs[row] = -INFINITY;
    }
    cl.sync();  // no CTA leaves while another reads its shared memory
    return;
  }
  // A row whose maximum is +inf: the infinite tokens share the mass (Share::get).
  float x_max = value_of(max_key);
  if (x_max == INFINITY) {
    s.inf_row = true;
    x_max = 0.f;
    if constexpr (kResident)
      for (int i = tid; i < n; i += kThreads) s_held[i] = s_held[i] == INFINITY ? 0.f : -INFINITY;
    own_max = own_max == INFINITY ? 0.f : -INFINITY;
  }
  if (tid == 0) {
    Row& r = sh.row;
    const double ln_unit = static_cast<double>(T) * 0.69314718055994530942;  // logits per factor of two
    const double c = fmin(0x1p26 / ln_unit, 1e38);
    r.sc.c = c;
    r.sc.k = 6755399441055744.0 + 63.0 * 0x1p26 - c * static_cast<double>(x_max);
    r.sc.far = fminf(x_max, __double2float_ru(static_cast<double>(x_max) - p.far * ln_unit));
    if (!(r.sc.far > -INFINITY)) r.sc.far = -FLT_MAX;  // an infinite T: every token that is not masked
    r.sc.up = p.up;
    r.x_max = x_max;
    r.m_max = mass_of(sh, x_max);
    r.bin_inv = kBinsPerNat / T;
    r.T = T;
    r.u = u;
    r.top_p = top_p;
    r.cut = -INFINITY;
    r.cut_ties = r.cut_count = 0;
    // min-p: w >= min_p is x >= x_max + T ln(min_p), up to the next float
    r.least = -INFINITY;
    if (min_p > 0.f && T < INFINITY)
      r.least = fminf(x_max, __double2float_ru(static_cast<double>(x_max) +
                                               static_cast<double>(T) * log(fmin(static_cast<double>(min_p), 1.0))));
    r.n = n;
    r.base = base;
    r.top_k = top_k;
  }
  __syncthreads();

  if (top_k > 0 && top_k < p.V) {
    if (top_k <= kCand / 2) {
      // as many threads' maxima as top_k lie in the bins up to f.bin: so do the first top_k tokens
      // (a thread without a token counts as masked: in the last bin, which bounds nothing)
      atomicAdd(&sh.h.n[bin_of(own_max, sh.row.x_max, sh.row.bin_inv)], 1u);
      const Found f = find<false>(sh, 0, static_cast<u64>(top_k), -1.f);
      if (f.bin < kBins - 1) {
        gather(sh, s, bin_bottom(sh.row, f.bin), INFINITY, 0, kBins, 0);
        const uint32_t got = *cl.map_shared_rank(&sh.cand_n[0], 0);
        auto read = cl.barrier_arrive();  // the first CTA stays until the others have read it
        if (got <= kCand && rank == 0) finish(sh, p, row, got, 0);
        cl.barrier_wait(std::move(read));
        if (got <= kCand) return;
      }
    }
    if (narrow<false>(sh, p, s, row, static_cast<u64>(top_k), -1.f)) return;
  }
  if (top_p < 1.f && narrow<true>(sh, p, s, row, 0, fmaxf(top_p, 0.f))) return;
  draw_all(sh, p, s, row);
}

struct ExpTable {
  ExpEntry v[64];
  ExpTable() {
    for (int j = 0; j < 64; ++j) {
      const double x = std::ldexp(std::exp2(j / 64.0), 28);
      v[j] = ExpEntry{static_cast<float>(x), static_cast<int32_t>(std::lrint(x))};
    }
  }
};

template <typename TL>
cudaError_t launch(SampleParams& p, int rows, cudaStream_t st) {
  // 4,096 tokens or more a CTA, up to 8 CTAs a row. (16 CTAs: one row with
  // top-k and top-p 13.7 us against 13.1; the histograms' all-to-all exchange
  // grows faster than the passes shrink.)
  // Rows longer than eight CTAs' shared memory are read again from L2 by each
  // pass. (Doing so for many short rows, 4 CTAs each and twice as many rows at
  // once, made 128 rows of top-k 58 us against 66, but 128 mixed ones 159
  // against 127: their longest rows decide.)
  int cluster = 1;
  while (cluster < kClusterMax && p.V > cluster * 4096) cluster *= 2;
  p.slice = ((p.V + cluster - 1) / cluster + 7) & ~7;  // whole 16-byte vectors of either type
  const bool resident = p.slice <= kMaxSlice;
  auto kern = resident ? k_sample<TL, true> : k_sample<TL, false>;
  const cudaError_t e = flint_ensure_smem(reinterpret_cast<const void*>(kern));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(rows) * cluster);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = resident ? static_cast<size_t>(p.slice) * 4 : 0;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cluster;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace
}  // namespace flint

using namespace flint;

extern "C" int flint_sample(const void* logits, int32_t rows, int32_t vocab, int64_t row_stride, int32_t logits_dtype,
                            const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                            const float* u, int32_t* tokens, float* logprobs, int32_t* status, void* stream) {
  if (logits_dtype != FLINT_LOGITS_F32 && logits_dtype != FLINT_LOGITS_BF16)
    return flint_fail_external(FLINT_ERR_INVALID_ARG, "logits_dtype is not a flint_logits_dtype");
  if (rows < 0 || vocab < 1 || row_stride < vocab)
    return flint_fail_external(FLINT_ERR_INVALID_ARG, "flint_sample: bad sizes");
  if (vocab > (1 << 24) || rows > (1 << 24))
    return flint_fail_external(FLINT_ERR_UNSUPPORTED_SHAPE, "at most 2^24 rows and tokens");
  if (rows == 0) return FLINT_OK;
  if (!logits || !u || !tokens) return flint_fail_external(FLINT_ERR_INVALID_ARG, "flint_sample: NULL pointer");
  const uintptr_t es = logits_dtype == FLINT_LOGITS_F32 ? 3u : 1u;
  if ((reinterpret_cast<uintptr_t>(logits) & es) ||
      ((reinterpret_cast<uintptr_t>(temperature) | reinterpret_cast<uintptr_t>(top_k) |
        reinterpret_cast<uintptr_t>(top_p) | reinterpret_cast<uintptr_t>(min_p) | reinterpret_cast<uintptr_t>(u) |
        reinterpret_cast<uintptr_t>(tokens) | reinterpret_cast<uintptr_t>(logprobs) |
        reinterpret_cast<uintptr_t>(status)) & 3u))
    return flint_fail_external(FLINT_ERR_MISALIGNED, "flint_sample: misaligned pointer");
  SampleParams p{};
  p.logits = logits;
  p.temperature = temperature;
  p.top_k = top_k;
  p.top_p = top_p;
  p.min_p = min_p;
  p.u = u;
  p.tokens = tokens;
  p.logprobs = logprobs;
  p.status = status;
  p.stride = row_stride;
  p.V = vocab;
  int lg = 0;
  while ((1 << lg) < vocab) ++lg;
  const int mass_bits = 62 - lg < 56 ? 62 - lg : 56;  // the row's mass, in units of 2^-(s + 1), stays below 2^63
  static const ExpTable table;
  for (int j = 0; j < 64; ++j) p.exp2_tab[j] = table.v[j];
  p.up = 63 + 32 - (mass_bits + 1 - 28);
  p.far = mass_bits + 2;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      logits_dtype == FLINT_LOGITS_F32 ? launch<float>(p, rows, st) : launch<uint16_t>(p, rows, st);
  if (e != cudaSuccess) return flint_fail_external(FLINT_ERR_CUDA, cudaGetErrorString(e));
  return FLINT_OK;
}
