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
// No sort: top-k and top-p both keep a prefix of the order, which is known by
// its last logit value t and how many ties at t it holds. t is found by
// narrowing: a histogram of 256 bins over the range that still holds it (first
// linear in the logit, 1/8 nat a bin, then over the bit patterns in order,
// 8 bits a level) gives the bin it lies in.
//
// One thread-block cluster per row: each CTA keeps its share of the row in
// shared memory as order-preserving integer keys (one pass over HBM: 4 bytes a
// logit, the floor), the CTAs' histograms meet through distributed shared
// memory, and every CTA draws the same conclusion from them.
//
// Masses are sums of rint(w 2^s) in 64-bit integers (s = 44 for 150,144
// tokens): exact and the same in any order, so a run's result does not depend
// on the order of the shared-memory atomics; a token below 2^-45 of the
// largest is never drawn, far below what a 24-bit u can reach.
#include <cooperative_groups.h>

#include "common.cuh"

namespace cg = cooperative_groups;

namespace flint {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 256;
constexpr int kMaxCluster = 8;
constexpr int kMaxSlice = 48 * 1024;     // keys of a CTA's share held in shared memory
constexpr uint32_t kNegInfKey = 0x007FFFFFu;  // key of -inf; NaN counts as -inf

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
  u64 key[2];          // best (key, index) of this CTA
  u64 mass[2];         // final pass: this CTA's kept mass above t, ties at t
  uint32_t ties[2];
  // block-local scratch
  u64 wsum[kWarps];
  uint32_t wcnt[kWarps];
  u64 pick_mass;
  uint32_t pick_bin, pick_above, pick_n;
  u64 total;
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

template <typename TL, bool kResident>
__global__ void __launch_bounds__(kThreads, 1) k_sample(SampleParams p) {
  extern __shared__ __align__(16) uint32_t s_keys[];
  __shared__ Shared sh;
  cg::cluster_group cl = cg::this_cluster();
  const int C = static_cast<int>(cl.num_blocks()), rank = static_cast<int>(cl.block_rank());
  const int row = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int base = rank * p.slice;
  const int n = max(0, min(p.slice, p.V - base));
  const TL* src = static_cast<const TL*>(p.logits) + static_cast<size_t>(row) * p.stride + base;

  auto from_global = [&](int i) {
    if constexpr (sizeof(TL) == 4) return key_of(__ldg(reinterpret_cast<const float*>(src) + i));
    else return key_of(bf16_bits_to_f32(__ldg(reinterpret_cast<const uint16_t*>(src) + i)));
  };
  auto get = [&](int i) -> uint32_t {
    if constexpr (kResident) return s_keys[i];
    else return from_global(i);
  };

  // ---- the row's share into shared memory; the largest (key, lowest index)
  u64 best = 0;
  for (int i = tid; i < n; i += kThreads) {
    const uint32_t k = from_global(i);
    if constexpr (kResident) s_keys[i] = k;
    const u64 c = (static_cast<u64>(k) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(base + i));
    best = c > best ? c : best;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const u64 x = __shfl_xor_sync(0xffffffffu, best, o);
    best = x > best ? x : best;
  }
  if (lane == 0) sh.wsum[warp] = best;
  for (int i = tid; i < kBins; i += kThreads) sh.h[0].n[i] = sh.h[0].lo[i] = sh.h[0].hi[i] = 0;
  __syncthreads();
  if (warp == 0) {
    best = sh.wsum[lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const u64 x = __shfl_xor_sync(0xffffffffu, best, o);
      best = x > best ? x : best;
    }
    if (lane == 0) sh.key[0] = best;
  }
  cl.sync();
  best = 0;
  for (int c = 0; c < C; ++c) {
    const u64 x = *cl.map_shared_rank(&sh.key[0], c);
    best = x > best ? x : best;
  }
  const uint32_t max_key = static_cast<uint32_t>(best >> 32);
  const int arg_max = static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(best));
  const float T = p.temperature != nullptr ? __ldg(p.temperature + row) : 1.f;
  const float u = __ldg(p.u + row);
  const int top_k = p.top_k != nullptr ? __ldg(p.top_k + row) : 0;
  const float top_p = p.top_p != nullptr ? __ldg(p.top_p + row) : 1.f;
  const double min_p = p.min_p != nullptr ? fmin(static_cast<double>(__ldg(p.min_p + row)), 1.0) : 0.0;

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

  const float x_max = value_of(max_key);
  const double inv_t = 1.0 / static_cast<double>(T);
  const double mass_one = static_cast<double>(1ull << p.mass_bits);
  auto weight = [&](uint32_t k) -> double {
    if (k == max_key) return 1.0;  // also where max x is infinite
    if (k <= kNegInfKey) return 0.0;
    return exp((static_cast<double>(value_of(k)) - static_cast<double>(x_max)) * inv_t);
  };
  auto mass_of = [&](double w) -> u64 { return __double2ull_rn(w * mass_one); };

  const float bin_inv = 8.f / T;
  auto bin1 = [&](uint32_t k) -> int {
    if (k == max_key) return 0;
    const float d = (x_max - value_of(k)) * bin_inv;
    return d < static_cast<float>(kBins - 1) ? static_cast<int>(d) : kBins - 1;
  };

  uint32_t cut_key = 0;       // the prefix ends at this key (0: it is the whole row) ...
  uint32_t cut_ties = 0;      // ... with this many of the keys equal to it
  uint32_t cut_count = 0;     // how many are equal to it
  int level = 0;              // histogram buffer in use

  // Narrows to the key at which the running count (by_mass false) or mass
  // reaches `want`, over the keys >= floor_key; want_p: want is that share of
  // the total, known after the first level.
  auto narrow = [&](bool by_mass, u64 want, double want_p, uint32_t floor_key) {
    u64 above = 0;        // count or mass above the range
    uint32_t b1 = 0;      // first-level bin
    uint32_t klo = 0, khi = 0;
    for (int step = 0; step < 8; ++step) {  // at most six levels: 1 + ceil(32 / 8) + the last key
      Hist& h = sh.h[level & 1];
      const uint32_t width = khi - klo;
      const int shift = step == 0 ? 0 : max(0, 32 - __clz(width) - 8);
      __syncthreads();  // h is zeroed
      uint32_t far_n = 0;
      u64 far_m = 0;
      for (int i = tid; i < n; i += kThreads) {
        const uint32_t k = get(i);
        if (k < floor_key) continue;
        int b;
        if (step == 0) {
          b = bin1(k);
          if (b == kBins - 1) {  // the bulk of a cold row: counted in registers
            ++far_n;
            if (by_mass) far_m += mass_of(weight(k));
            continue;
          }
        } else {
          if (k < klo || k > khi || bin1(k) != static_cast<int>(b1)) continue;
          b = static_cast<int>((khi - k) >> shift);
        }
        atomicAdd(&h.n[b], 1u);
        if (by_mass) add_mass(h, b, mass_of(weight(k)));
      }
      if (step == 0) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          far_n += __shfl_xor_sync(0xffffffffu, far_n, o);
          far_m += __shfl_xor_sync(0xffffffffu, far_m, o);
        }
        if (lane == 0 && far_n != 0) {
          atomicAdd(&h.n[kBins - 1], far_n);
          if (by_mass) add_mass(h, kBins - 1, far_m);
        }
      }
      cl.sync();
      // every CTA sums all histograms and finds the bin; the other buffer is free again
      Hist& nx = sh.h[(level + 1) & 1];
      uint32_t cnt = 0;
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
        if (lane == 31) sh.wsum[warp] = inc;
      }
      __syncthreads();
      if (tid < kBins) {
        u64 all = 0;
        for (int w = 0; w < kBins / 32; ++w) {
          if (w < warp) inc += sh.wsum[w];
          all += sh.wsum[w];
        }
        if (step == 0 && by_mass) {
          // ties at the floor beyond those that top-k keeps hold no mass
          if (cut_key != 0) all -= static_cast<u64>(cut_count - cut_ties) * mass_of(weight(cut_key));
          want = static_cast<u64>(ceil(want_p * static_cast<double>(all)));
          want = want < 1 ? 1 : want > all ? all : want;  // `all` may round up as a double
        }
        if (above + inc >= want && above + inc - val < want) {
          sh.pick_bin = tid;
          sh.pick_n = cnt;
          sh.pick_mass = above + inc - val;
          sh.total = want;
        }
      }
      __syncthreads();
      const uint32_t b = sh.pick_bin;
      const uint32_t in_bin = sh.pick_n;
      above = sh.pick_mass;
      want = sh.total;
      ++level;
      if (step == 0) {
        b1 = b;
        // the keys that can lie in bin b: d = (x_max - x) bin_inv in [b, b + 1), with room for rounding
        const double inv = static_cast<double>(bin_inv);
        khi = max_key;
        if (b > 0 && inv > 0.0 && x_max < INFINITY) {
          const double d = static_cast<double>(b) / inv * (1.0 - 0x1p-20);
          const uint32_t k = key_of(__double2float_ru(static_cast<double>(x_max) - d));
          khi = k < max_key ? k : max_key;
        }
        klo = 0;
        if (b < kBins - 1 && inv > 0.0 && x_max < INFINITY) {
          const double d = (static_cast<double>(b) + 1.0) / inv * (1.0 + 0x1p-20);
          klo = key_of(__double2float_rd(static_cast<double>(x_max) - d));
        }
        klo = max(klo, floor_key);
        if (klo > khi) klo = khi;
      } else {
        khi -= b << shift;
        if (shift > 0) klo = max(klo, khi - ((1u << shift) - 1u));
        else klo = khi;
      }
      if (klo == khi && step > 0) {
        uint32_t keep;
        if (by_mass) {
          const u64 w = mass_of(weight(khi));
          keep = w > 0 ? static_cast<uint32_t>(min(static_cast<u64>(in_bin), (want - above + w - 1) / w)) : in_bin;
          if (khi == cut_key) keep = min(keep, cut_ties);
        } else {
          keep = static_cast<uint32_t>(want - above);
        }
        cut_key = khi;
        cut_ties = keep;
        cut_count = in_bin;
        return;
      }
    }
  };

  if (top_k > 0 && top_k < p.V) narrow(false, static_cast<u64>(top_k), 0.0, 0u);
  if (top_p < 1.f) narrow(true, 0, fmax(static_cast<double>(top_p), 0.0), cut_key);

  // ---- the draw: each thread a run of consecutive tokens (an odd number: conflict-free)
  const int run = ((n + kThreads - 1) / kThreads) | 1;
  const int r0 = min(n, tid * run), r1 = min(n, r0 + run);
  const double w_cut = cut_key != 0 ? weight(cut_key) : 0.0;
  const u64 m_cut = w_cut >= min_p ? mass_of(w_cut) : 0;
  u64 mass = 0;
  uint32_t ties = 0;
  for (int i = r0; i < r1; ++i) {
    const uint32_t k = get(i);
    if (k > cut_key) {
      const double w = weight(k);
      if (w >= min_p) mass += mass_of(w);
    } else if (k == cut_key) {
      ++ties;
    }
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
    sh.mass[0] = cta_mass;
    sh.ties[0] = cta_ties;
  }
  cl.sync();
  // kept mass in front of this CTA, and of the row
  u64 before = 0, total = 0;
  uint32_t ties_before = 0, t_seen = 0;
  for (int c = 0; c < C; ++c) {
    const u64 m = *cl.map_shared_rank(&sh.mass[0], c);
    const uint32_t t = *cl.map_shared_rank(&sh.ties[0], c);
    if (c == rank) {
      before = total;
      ties_before = t_seen;
    }
    const uint32_t keep = t_seen < cut_ties ? min(t, cut_ties - t_seen) : 0;
    total += m + keep * m_cut;
    t_seen += t;
  }
  const u64 target = static_cast<u64>(static_cast<double>(u) * static_cast<double>(total));
  // this thread's interval of the running mass
  const uint32_t my_ties0 = ties_before + ties_i - ties;
  const uint32_t cta_kept0 = min(cut_ties, ties_before);
  const uint32_t k0 = min(cut_ties, my_ties0), k1 = min(cut_ties, my_ties0 + ties);
  u64 acc = before + (mass_i - mass) + static_cast<u64>(k0 - cta_kept0) * m_cut;
  const u64 end = acc + mass + static_cast<u64>(k1 - k0) * m_cut;
  if (acc <= target && target < end) {  // exactly one thread of the cluster
    uint32_t seen = my_ties0;
    for (int i = r0; i < r1; ++i) {
      const uint32_t k = get(i);
      double w = 0.0;
      if (k > cut_key) w = weight(k);
      else if (k == cut_key && seen++ < cut_ties) w = w_cut;
      if (w >= min_p) acc += mass_of(w);
      if (acc > target) {
        p.tokens[row] = base + i;
        if (p.logprobs != nullptr) p.logprobs[row] = static_cast<float>(log(w / (static_cast<double>(total) / mass_one)));
        break;
      }
    }
  }
  cl.sync();
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
  p.slice = (vocab + cluster - 1) / cluster;
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
