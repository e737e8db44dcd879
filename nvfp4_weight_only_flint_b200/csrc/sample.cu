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
// No sort of the row: top-k and top-p both keep a prefix of the order. A
// histogram of 256 bins, linear in the logit (1/8 nat a bin), finds the bin the
// prefix ends in. If the bins up to it hold at most 1,024 tokens (k = 50,
// top-p = 0.9 and the like), those alone are gathered in one CTA, sorted,
// cut and drawn from. Otherwise the end is narrowed to one logit value by
// further histograms over the bit patterns in order, 8 bits a level, and the
// draw passes over the whole row once more.
//
// One thread-block cluster per row: each CTA keeps its share of the row in
// shared memory as order-preserving integer keys (one pass over HBM: 4 bytes a
// logit, the floor), the CTAs' histograms meet through distributed shared
// memory, and every CTA draws the same conclusion from them.
//
// Masses are sums of rint(w 2^s) in 64-bit integers (s = 44 for 150,144
// tokens): exact and the same in any order, so a run's result does not depend
// on the order of the shared-memory atomics; a token below 2^-45 of the
// largest is never drawn, far below what a 24-bit u can reach. w is computed in
// double (2^(j/64) from a table times a degree-5 Taylor polynomial of the rest,
// off by 2.2e-15: 12 fp64 operations): 150,144 fp32 weights would put the sums
// of a flat row 1e-8 off and its draw wrong about once in 10^4.
#include <cooperative_groups.h>

#include "common.cuh"

namespace cg = cooperative_groups;

namespace flint {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 256;
constexpr int kCand = 2 * kThreads;      // tokens the gathered form sorts
constexpr int kMaxCluster = 8;
constexpr int kMaxSlice = 48 * 1024;     // keys of a CTA's share held in shared memory
constexpr uint32_t kNegInfKey = 0x007FFFFFu;  // key of -inf; NaN counts as -inf
constexpr uint32_t kZeroKey = 0x80000000u;

typedef unsigned long long u64;

struct SampleParams {
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
  int V, slice, mass_bits;
};

// Order-preserving integer of a float (-0 and +0 alike) and back.
__device__ __forceinline__ uint32_t key_of(float x) {
  if (x != x) return kNegInfKey;
  const uint32_t b = __float_as_uint(x + 0.f);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

struct Hist {
  uint32_t n[kBins], lo[kBins], hi[kBins];
};

struct Shared {
  Hist h[2];
  u64 cand[kCand];     // gathered tokens: key, then ~index
  u64 mass_of[kCand];
  double exp2_tab[64];  // 2^(j / 64 + s)
  u64 key;             // best (key, index) of this CTA
  u64 mass;            // final pass: this CTA's kept mass above the cut, ties at it
  uint32_t ties;
  // block-local scratch
  u64 wsum[kWarps];
  uint32_t wcnt[kWarps];
  u64 pick_above, want;
  uint32_t pick_bin, pick_n, cand_n;
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

// Weights of a row in log2 units: z = (x - max x) log2(e) / T.
struct Scale {
  double c;      // log2(e) / T
  float x_max;
  __device__ __forceinline__ double z(uint32_t k) const {
    return (static_cast<double>(value_of(k)) - static_cast<double>(x_max)) * c;
  }
};

// rint(2^(z + s)) for z <= 0; 0 below 2^-46 (and for the NaN of a masked token
// at infinite temperature). z = n / 64 + r with r in [0, 1/64): 2^(n / 64) from
// the table and the exponent field, 2^r by its Taylor series.
__device__ __forceinline__ u64 mass_at(double z, const double* tab) {
  if (!(z >= -46.0)) return 0;
  constexpr double kL = 0.693147180559945309417;  // ln 2
  constexpr double kMagic = 6755399441055744.0;   // 1.5 * 2^52: the sum's low word is the integer
  const double m = __fma_rd(z, 64.0, kMagic);
  const int n = __double2loint(m);
  const double r = __fma_rn(m - kMagic, -1.0 / 64, z);
  double p = kL * kL * kL * kL * kL / 120;
  p = __fma_rn(p, r, kL * kL * kL * kL / 24);
  p = __fma_rn(p, r, kL * kL * kL / 6);
  p = __fma_rn(p, r, kL * kL / 2);
  p = __fma_rn(p, r, kL);
  p = __fma_rn(p, r, 1.0);
  const double v = tab[n & 63] * p;
  const double w = __hiloint2double(__double2hiint(v) + ((n >> 6) << 20), __double2loint(v));
  // w <= 2^44: adding 2^52 rounds it to an integer in the low bits
  return static_cast<u64>(__double_as_longlong(w + 4503599627370496.0)) & 0xFFFFFFFFFFFFFull;
}

// Sorts the first n2 (a power of two <= kCand) words of v descending; whole block.
__device__ __forceinline__ void sort_desc(u64* v, int n2) {
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

template <typename TL, bool kResident>
__global__ void __launch_bounds__(kThreads, 2) k_sample(SampleParams p) {
  extern __shared__ __align__(16) uint32_t s_keys[];
  __shared__ Shared sh;
  cg::cluster_group cl = cg::this_cluster();
  const int C = static_cast<int>(cl.num_blocks()), rank = static_cast<int>(cl.block_rank());
  const int row = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int base = rank * p.slice;
  const int n = max(0, min(p.slice, p.V - base));
  const TL* src = static_cast<const TL*>(p.logits) + static_cast<size_t>(row) * p.stride + base;
  const float T = p.temperature != nullptr ? __ldg(p.temperature + row) : 1.f;
  const float u = __ldg(p.u + row);
  const int top_k = p.top_k != nullptr ? __ldg(p.top_k + row) : 0;
  const float top_p = p.top_p != nullptr ? __ldg(p.top_p + row) : 1.f;
  const float min_p = p.min_p != nullptr ? __ldg(p.min_p + row) : 0.f;

  // ---- the row's share into shared memory; the largest (key, lowest index).
  // 16-byte loads where the row allows them, kBatch in flight per thread.
  constexpr int kVec = 16 / sizeof(TL), kBatch = 5;
  u64 best = 0;
  auto see = [&](uint32_t k, int i) {
    const u64 c = (static_cast<u64>(k) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(base + i));
    best = c > best ? c : best;
  };
  auto one = [&](int i) {
    if constexpr (sizeof(TL) == 4) return key_of(__ldg(reinterpret_cast<const float*>(src) + i));
    else return key_of(bf16_bits_to_f32(__ldg(reinterpret_cast<const uint16_t*>(src) + i)));
  };
  const int n_vec = (reinterpret_cast<uintptr_t>(src) & 15u) == 0 ? n / kVec : 0;
  for (int i0 = tid; i0 < n_vec; i0 += kThreads * kBatch) {
    uint4 v[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
      if (i0 + b * kThreads < n_vec) v[b] = __ldg(reinterpret_cast<const uint4*>(src) + i0 + b * kThreads);
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int i = i0 + b * kThreads;
      if (i >= n_vec) break;
      const uint32_t x[4] = {v[b].x, v[b].y, v[b].z, v[b].w};
      uint32_t k[kVec];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if constexpr (sizeof(TL) == 4) {
          k[q] = key_of(__uint_as_float(x[q]));
        } else {
          k[2 * q] = key_of(__uint_as_float(x[q] << 16));
          k[2 * q + 1] = key_of(__uint_as_float(x[q] & 0xFFFF0000u));
        }
      }
#pragma unroll
      for (int q = 0; q < kVec; ++q) see(k[q], i * kVec + q);
      if constexpr (kResident) {
#pragma unroll
        for (int q = 0; q < kVec; q += 4)
          reinterpret_cast<uint4*>(s_keys)[(i * kVec + q) / 4] = make_uint4(k[q], k[q + 1], k[q + 2], k[q + 3]);
      }
    }
  }
  for (int i0 = n_vec * kVec + tid; i0 < n; i0 += kThreads * 8) {
    uint32_t k[8];
#pragma unroll
    for (int b = 0; b < 8; ++b)
      if (i0 + b * kThreads < n) k[b] = one(i0 + b * kThreads);
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      const int i = i0 + b * kThreads;
      if (i >= n) break;
      if constexpr (kResident) s_keys[i] = k[b];
      see(k[b], i);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const u64 x = __shfl_xor_sync(0xffffffffu, best, o);
    best = x > best ? x : best;
  }
  if (lane == 0) sh.wsum[warp] = best;
  for (int i = tid; i < kBins; i += kThreads) sh.h[0].n[i] = sh.h[0].lo[i] = sh.h[0].hi[i] = 0;
  if (tid < 64) sh.exp2_tab[tid] = ldexp(exp2(static_cast<double>(tid) / 64), p.mass_bits);
  if (tid == 64) sh.cand_n = 0;
  __syncthreads();
  if (warp == 0) {
    best = lane < kWarps ? sh.wsum[lane] : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const u64 x = __shfl_xor_sync(0xffffffffu, best, o);
      best = x > best ? x : best;
    }
    if (lane == 0) sh.key = best;
  }
  cl.sync();
  best = 0;
  for (int c = 0; c < C; ++c) {
    const u64 x = *cl.map_shared_rank(&sh.key, c);
    best = x > best ? x : best;
  }
  uint32_t max_key = static_cast<uint32_t>(best >> 32);
  const int arg_max = static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(best));

  const bool bad_arg = !(T >= 0.f) || !(u >= 0.f && u < 1.f);
  if (bad_arg || max_key == kNegInfKey || T == 0.f) {  // the whole cluster agrees
    if (rank == 0 && tid == 0) {
      const bool none = bad_arg || max_key == kNegInfKey;
      if (none && p.status != nullptr) atomicOr(p.status, bad_arg ? FLINT_DEVCHECK_INDEX : FLINT_DEVCHECK_NONFINITE);
      p.tokens[row] = none ? -1 : arg_max;
      if (p.logprobs != nullptr) p.logprobs[row] = none ? -INFINITY : 0.f;
    }
    cl.sync();  // no CTA leaves while another reads its shared memory
    return;
  }

  // A row whose maximum is +inf: the infinite tokens share the mass. They count
  // as zeros, all others as masked.
  const bool inf_row = value_of(max_key) == INFINITY;
  const uint32_t inf_key = max_key;
  if (inf_row) max_key = kZeroKey;
  auto fix = [&](uint32_t k) { return !inf_row ? k : k == inf_key ? kZeroKey : kNegInfKey; };
  auto get = [&](int i) -> uint32_t {
    if constexpr (kResident) return fix(s_keys[i]);
    else return fix(one(i));
  };
  // f(key, index in the share) over the share, in no particular order
  auto each = [&](auto&& f) {
    if constexpr (kResident) {
      for (int i = tid; i < (n >> 2); i += kThreads) {
        const uint4 k = reinterpret_cast<const uint4*>(s_keys)[i];
        f(fix(k.x), 4 * i);
        f(fix(k.y), 4 * i + 1);
        f(fix(k.z), 4 * i + 2);
        f(fix(k.w), 4 * i + 3);
      }
      for (int i = (n & ~3) + tid; i < n; i += kThreads) f(fix(s_keys[i]), i);
    } else {
      for (int i = tid; i < n; i += kThreads) f(fix(one(i)), i);
    }
  };
  const Scale sc{1.4426950408889634074 / static_cast<double>(T), value_of(max_key)};
  const double z_min = min_p > 0.f ? log2(fmin(static_cast<double>(min_p), 1.0)) : -INFINITY;

  const float bin_inv = 8.f / T;
  auto bin1 = [&](uint32_t k) -> int {
    if (k == max_key) return 0;
    const float d = (sc.x_max - value_of(k)) * bin_inv;
    return d < static_cast<float>(kBins - 1) ? static_cast<int>(d) : kBins - 1;
  };

  uint32_t cut_key = 0;       // the prefix ends at this key (0: it is the whole row) ...
  uint32_t cut_ties = 0;      // ... with this many of the keys equal to it
  uint32_t cut_count = 0;     // how many are equal to it
  int level = 0;              // histogram buffer in use

  // The gathered form: the n_cand tokens of keys >= floor_key in bins up to
  // `bin` contain the prefix. want_mass: the mass at which top-p ends it, 0 if
  // that is still to be taken of the first top_k tokens.
  auto gathered = [&](uint32_t floor_key, int bin, int n_cand, u64 want_mass) {
    Shared* lead = cl.map_shared_rank(&sh, 0);
    each([&](uint32_t k, int i) {
      if (k < floor_key || bin1(k) > bin) return;
      lead->cand[atomicAdd(&lead->cand_n, 1u)] =
          (static_cast<u64>(k) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(base + i));
    });
    cl.sync();
    if (rank != 0) return;
    int n2 = 2;
    while (n2 < n_cand) n2 <<= 1;
    for (int i = n_cand + tid; i < n2; i += kThreads) sh.cand[i] = 0;
    __syncthreads();
    sort_desc(sh.cand, n2);
    const int n_k = top_k > 0 ? min(n_cand, top_k) : n_cand;
    // running mass of the sorted tokens, two per thread
    auto scan2 = [&](u64 m0, u64 m1, u64& before0, u64& total) {
      const u64 inc = warp_incl(m0 + m1, lane);
      __syncthreads();
      if (lane == 31) sh.wsum[warp] = inc;
      __syncthreads();
      u64 b = 0, all = 0;
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) b += sh.wsum[w];
        all += sh.wsum[w];
      }
      before0 = b + inc - m0 - m1;
      total = all;
    };
    u64 c[2], m[2];
    double z[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int i = 2 * tid + q;
      c[q] = i < n_k ? sh.cand[i] : 0;
      z[q] = i < n_k ? sc.z(static_cast<uint32_t>(c[q] >> 32)) : -INFINITY;
      m[q] = mass_at(z[q], sh.exp2_tab);
    }
    u64 before, total;
    scan2(m[0], m[1], before, total);
    if (top_p < 1.f) {
      if (want_mass == 0) {
        const u64 w = static_cast<u64>(ceil(fmax(static_cast<double>(top_p), 0.0) * static_cast<double>(total)));
        want_mass = w < 1 ? 1 : w;
      }
      if (before + m[0] >= want_mass) m[1] = 0, z[1] = -INFINITY;
      if (before >= want_mass) m[0] = 0, z[0] = -INFINITY;
    }
#pragma unroll
    for (int q = 0; q < 2; ++q)
      if (!(z[q] >= z_min)) m[q] = 0;
    // the draw in vocabulary order: sort what holds mass by index (largest ~index first)
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int i = 2 * tid + q;
      if (i < n2) {
        sh.cand[i] = m[q] > 0 ? (c[q] << 32) | static_cast<uint32_t>(i) : 0;
        sh.mass_of[i] = m[q];
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
    scan2(m[0], m[1], before, total);
    const u64 target = static_cast<u64>(static_cast<double>(u) * static_cast<double>(total));
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if (before <= target && target < before + m[q]) {
        const uint32_t id = 0xFFFFFFFFu - static_cast<uint32_t>(c[q] >> 32);
        p.tokens[row] = static_cast<int32_t>(id);
        if (p.logprobs != nullptr)
          p.logprobs[row] = static_cast<float>(
              log(static_cast<double>(m[q]) / static_cast<double>(total)));
      }
      before += m[q];
    }
  };

  // Narrows to the key at which the running count (by_mass false) or mass
  // reaches `want`, over the keys >= floor_key; want_p: want is that share of
  // the total, known after the first level. True if the gathered form finished
  // the row.
  auto narrow = [&](bool by_mass, u64 want, double want_p, uint32_t floor_key) -> bool {
    u64 above = 0;        // count or mass above the range
    int b1 = 0;           // first-level bin
    uint32_t klo = 0, khi = 0;
    for (int step = 0; step < 8; ++step) {  // at most six levels: 1 + ceil(32 / 8) + the last key
      Hist& h = sh.h[level & 1];
      const uint32_t width = khi - klo;
      const int shift = step == 0 ? 0 : max(0, 32 - __clz(width) - 8);
      __syncthreads();  // h is zeroed
      if (step == 0) {
        uint32_t far_n = 0;
        u64 far_m = 0;
        each([&](uint32_t k, int) {
          if (k < floor_key) return;
          const int b = bin1(k);
          if (b == kBins - 1) {  // the bulk of a cold row: counted in registers
            ++far_n;
            if (by_mass) far_m += mass_at(sc.z(k), sh.exp2_tab);
            return;
          }
          atomicAdd(&h.n[b], 1u);
          if (by_mass) {
            const u64 m = mass_at(sc.z(k), sh.exp2_tab);
            if (m != 0) add_mass(h, b, m);
          }
        });
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          far_n += __shfl_xor_sync(0xffffffffu, far_n, o);
          far_m += __shfl_xor_sync(0xffffffffu, far_m, o);
        }
        if (lane == 0 && far_n != 0) {
          atomicAdd(&h.n[kBins - 1], far_n);
          if (by_mass) add_mass(h, kBins - 1, far_m);
        }
      } else {
        each([&](uint32_t k, int) {
          if (k < klo || k > khi || bin1(k) != b1) return;
          const int b = static_cast<int>((khi - k) >> shift);
          atomicAdd(&h.n[b], 1u);
          if (by_mass) add_mass(h, b, mass_at(sc.z(k), sh.exp2_tab));
        });
      }
      cl.sync();
      // every CTA sums all histograms and finds the bin; the other buffer is free again
      Hist& nx = sh.h[(level + 1) & 1];
      uint32_t cnt = 0, cnt_inc = 0;
      u64 val = 0, inc = 0;
      if (tid < kBins) {
        nx.n[tid] = nx.lo[tid] = nx.hi[tid] = 0;
        u64 m = 0;
        for (int c = 0; c < C; ++c) {
          const Hist* r = cl.map_shared_rank(&h, c);
          cnt += r->n[tid];
          if (by_mass) m += (static_cast<u64>(r->hi[tid]) << 32) + r->lo[tid];
        }
        val = by_mass ? m : cnt;
        inc = warp_incl(val, lane);
        cnt_inc = cnt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t x = __shfl_up_sync(0xffffffffu, cnt_inc, o);
          if (lane >= o) cnt_inc += x;
        }
        if (lane == 31) {
          sh.wsum[warp] = inc;
          sh.wcnt[warp] = cnt_inc;
        }
      }
      __syncthreads();
      if (tid < kBins) {
        u64 all = 0;
        for (int w = 0; w < kBins / 32; ++w) {
          if (w < warp) {
            inc += sh.wsum[w];
            cnt_inc += sh.wcnt[w];
          }
          all += sh.wsum[w];
        }
        if (step == 0 && by_mass) {
          // ties at the floor beyond those that top-k keeps hold no mass
          if (cut_key != 0) all -= static_cast<u64>(cut_count - cut_ties) * mass_at(sc.z(cut_key), sh.exp2_tab);
          want = static_cast<u64>(ceil(want_p * static_cast<double>(all)));
          want = want < 1 ? 1 : want > all ? all : want;  // `all` may round up as a double
        }
        if (above + inc >= want && above + inc - val < want) {
          sh.pick_bin = tid;
          sh.pick_n = step == 0 ? cnt_inc : cnt;
          sh.pick_above = above + inc - val;
          sh.want = want;
        }
      }
      __syncthreads();
      const int b = static_cast<int>(sh.pick_bin);
      const uint32_t in_bin = sh.pick_n;
      above = sh.pick_above;
      want = sh.want;
      ++level;
      if (step == 0) {
        if (in_bin <= kCand) {
          gathered(floor_key, b, static_cast<int>(in_bin), by_mass ? want : 0);
          return true;
        }
        b1 = b;
        // the keys that can lie in bin b: d = (x_max - x) bin_inv in [b, b + 1), with room for rounding
        const double inv = static_cast<double>(bin_inv), x_max = static_cast<double>(sc.x_max);
        khi = max_key;
        if (b > 0 && inv > 0.0)
          khi = min(khi, key_of(__double2float_ru(x_max - static_cast<double>(b) / inv * (1.0 - 0x1p-20))));
        klo = 0;
        if (b < kBins - 1 && inv > 0.0)
          klo = key_of(__double2float_rd(x_max - (static_cast<double>(b) + 1.0) / inv * (1.0 + 0x1p-20)));
        klo = max(klo, floor_key);
        if (klo > khi) klo = khi;
      } else {
        khi -= static_cast<uint32_t>(b) << shift;
        if (shift > 0) klo = max(klo, khi - ((1u << shift) - 1u));
        else klo = khi;
      }
      if (klo == khi && step > 0) {
        uint32_t keep;
        if (by_mass) {
          const u64 w = mass_at(sc.z(khi), sh.exp2_tab);
          keep = w > 0 ? static_cast<uint32_t>(min(static_cast<u64>(in_bin), (want - above + w - 1) / w)) : in_bin;
          if (khi == cut_key) keep = min(keep, cut_ties);
        } else {
          keep = static_cast<uint32_t>(want - above);
        }
        cut_key = khi;
        cut_ties = keep;
        cut_count = in_bin;
        break;
      }
    }
    return false;
  };

  if (top_k > 0 && top_k < p.V && narrow(false, static_cast<u64>(top_k), 0.0, 0u)) return;
  if (top_p < 1.f && narrow(true, 0, fmax(static_cast<double>(top_p), 0.0), cut_key)) return;

  // ---- the draw over the whole row: each thread a run of consecutive tokens
  // (an odd number: conflict-free)
  const int run = ((n + kThreads - 1) / kThreads) | 1;
  const int r0 = min(n, tid * run), r1 = min(n, r0 + run);
  const double z_cut = cut_key != 0 ? sc.z(cut_key) : -INFINITY;
  const u64 m_cut = z_cut >= z_min ? mass_at(z_cut, sh.exp2_tab) : 0;
  auto mass_above = [&](uint32_t k) -> u64 {
    if (k <= cut_key) return 0;
    const double z = sc.z(k);
    return z >= z_min ? mass_at(z, sh.exp2_tab) : 0;
  };
  u64 mass = 0;
  uint32_t ties = 0;
#pragma unroll 4
  for (int i = r0; i < r1; ++i) {
    const uint32_t k = get(i);
    mass += mass_above(k);
    ties += k == cut_key ? 1u : 0u;
  }
  u64 mass_i = warp_incl(mass, lane);
  uint32_t ties_i = ties;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, ties_i, o);
    if (lane >= o) ties_i += x;
  }
  __syncthreads();
  if (lane == 31) {
    sh.wsum[warp] = mass_i;
    sh.wcnt[warp] = ties_i;
  }
  __syncthreads();
  u64 cta_mass = 0;
  uint32_t cta_ties = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) {
      mass_i += sh.wsum[w];
      ties_i += sh.wcnt[w];
    }
    cta_mass += sh.wsum[w];
    cta_ties += sh.wcnt[w];
  }
  if (tid == 0) {
    sh.mass = cta_mass;
    sh.ties = cta_ties;
  }
  cl.sync();
  // kept mass in front of this CTA, and of the row
  u64 before = 0, total = 0;
  uint32_t ties_before = 0, t_seen = 0;
  for (int c = 0; c < C; ++c) {
    const u64 m = *cl.map_shared_rank(&sh.mass, c);
    const uint32_t t = *cl.map_shared_rank(&sh.ties, c);
    if (c == rank) {
      before = total;
      ties_before = t_seen;
    }
    const uint32_t keep = t_seen < cut_ties ? min(t, cut_ties - t_seen) : 0;
    total += m + keep * m_cut;
    t_seen += t;
  }
  cl.sync();  // the last read of another CTA's shared memory
  const u64 target = static_cast<u64>(static_cast<double>(u) * static_cast<double>(total));
  // this thread's interval of the running mass
  const uint32_t my_ties0 = ties_before + ties_i - ties;
  const uint32_t k0 = min(cut_ties, my_ties0), k1 = min(cut_ties, my_ties0 + ties);
  const u64 acc = before + (mass_i - mass) + static_cast<u64>(k0 - min(cut_ties, ties_before)) * m_cut;
  const u64 end = acc + mass + static_cast<u64>(k1 - k0) * m_cut;
  // exactly one thread of the cluster holds the target; its warp looks through its run
  const unsigned hit = __ballot_sync(0xffffffffu, acc <= target && target < end);
  if (hit == 0) return;
  const int owner = __ffs(hit) - 1;
  u64 at = __shfl_sync(0xffffffffu, acc, owner);
  uint32_t seen = __shfl_sync(0xffffffffu, my_ties0, owner);
  const int e0 = __shfl_sync(0xffffffffu, r0, owner), e1 = __shfl_sync(0xffffffffu, r1, owner);
  for (int i0 = e0; i0 < e1; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t k = i < e1 ? get(i) : 0;
    const bool tie = i < e1 && k == cut_key;
    const unsigned tie_mask = __ballot_sync(0xffffffffu, tie);
    u64 m = i < e1 ? mass_above(k) : 0;
    if (tie && seen + __popc(tie_mask & ((1u << lane) - 1u)) < cut_ties) m = m_cut;
    const u64 inc = at + warp_incl(m, lane);
    if (inc - m <= target && target < inc) {
      p.tokens[row] = base + i;
      if (p.logprobs != nullptr)
        p.logprobs[row] = static_cast<float>(log(static_cast<double>(m) / static_cast<double>(total)));
    }
    seen += __popc(tie_mask);
    at = __shfl_sync(0xffffffffu, inc, 31);
    if (at > target) break;
  }
}

template <typename TL, bool kResident>
cudaError_t launch(const SampleParams& p, int rows, int cluster, size_t smem, cudaStream_t st) {
  auto kern = k_sample<TL, kResident>;
  cudaError_t e = flint_ensure_smem(reinterpret_cast<const void*>(kern));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(rows) * cluster);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cluster;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
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
        reinterpret_cast<uintptr_t>(tokens) | reinterpret_cast<uintptr_t>(logprobs)) & 3u))
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
  int cluster = 1;
  while (cluster < kMaxCluster && vocab > cluster * 4096) cluster *= 2;
  p.slice = ((vocab + cluster - 1) / cluster + 7) & ~7;  // whole 16-byte vectors of either type
  int lg = 0;
  while ((1 << lg) < vocab) ++lg;
  p.mass_bits = 62 - lg < 44 ? 62 - lg : 44;  // the row's mass stays below 2^62
  const bool resident = p.slice <= kMaxSlice;
  const size_t smem = resident ? static_cast<size_t>(p.slice) * 4 : 0;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (logits_dtype == FLINT_LOGITS_F32)
    e = resident ? launch<float, true>(p, rows, cluster, smem, st) : launch<float, false>(p, rows, cluster, smem, st);
  else
    e = resident ? launch<uint16_t, true>(p, rows, cluster, smem, st)
                 : launch<uint16_t, false>(p, rows, cluster, smem, st);
  if (e != cudaSuccess) return flint_fail_external(FLINT_ERR_CUDA, cudaGetErrorString(e));
  return FLINT_OK;
}
