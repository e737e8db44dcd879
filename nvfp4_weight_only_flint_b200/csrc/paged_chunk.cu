// paged_chunk.cu -- attention of many new tokens per sequence (prompt pieces,
// whole prompts, mixed steps) over the paged cache, on the 5th-generation
// tensor cores ("[Model] Add Flint (RecursiveSI/flint)", section "What
// happened": 8K-token prefill; heads from "Recursive Flint: 125 tok/s on an M4
// Pro", architecture table).
//
// k_chunk_plan (one CTA) turns the lengths it finds on the device into a work
// list; k_paged_chunk (one CTA per SM) takes (entry, kv head) items off it;
// k_chunk_combine joins the entries that were split over keys.
//
// An item is a pair of query tiles against a run of 128-key tiles. A query tile
// is 128 rows = floor(128 / group) tokens x the group of query heads that share
// the kv head: K and V are fetched once for 2 x 128 rows, and a causal edge
// cuts at most 128 / group tokens. Per key tile and query tile
//   S = Q K^T     tcgen05.mma, both operands in shared memory (TMA, 128-byte swizzle)
//   P = 2^(S c - m c)   by the tile's own warpgroup: thread = row, S read from
//                 tensor memory into registers, P rounded and written back over S
//   O += P V      tcgen05.mma, P from tensor memory, V as it lies in the cache
//                 (keys x dims: MN-major)
// with the two tiles' softmax and MMAs alternating. O is rescaled only when a
// row's maximum grew by more than 2^8 since the last time (P then stays below
// 2^8; O / l is the same), by the softmax warps themselves, so no correction
// warps stand in the chain. Tensor memory: S0 S1 O0 O1, 128 columns each.
//   bf16 cache: five 32 KB stages of K and V by TMA, one box per page (or 128 rows).
//   E4M3 cache: three raw 16 KB stages; a further warpgroup turns them into f16
//     tiles (exact), and Q into f16 after a power-of-two scale per row.
// Keys past a sequence's end: S is masked by column, and V rows are zeroed in
// shared memory, so whatever unused cache rows hold stays out of the sums.
#include <cuda.h>

#include "paged_attn.cuh"
#include "tcgen05.cuh"

namespace flint {

int flint_encode_map_sw128(CUtensorMap* m, CUtensorMapDataType dt, int rank, const void* base, const cuuint64_t* dims,
                           const cuuint64_t* strides, const cuuint32_t* box);

namespace {

constexpr int kDh = kPagedHeadDim;
constexpr int kTile = 128;                 // query rows and keys per tile
constexpr int kTileBytes = kTile * kDh * 2;
constexpr int kHalfBytes = kTileBytes / 2; // 64 dims of a tile
constexpr int kRawBytes = kTile * kDh;
constexpr int kCtas = 148;
constexpr int kMaxSplit = 4 * kCtas;       // partial slots over all kv heads
constexpr float kRescale = 8.f;            // log2 units

template <bool kE4M3>
struct Cfg {
  static constexpr int kThreads = kE4M3 ? 512 : 384;
  static constexpr int kStages = kE4M3 ? 3 : 5;
  static constexpr int kRaw = kE4M3 ? 3 : 0;
  static constexpr int kFullCount = kE4M3 ? 128 : 1;
};

// One tile pair of one sequence; entries add a key range and a partial slot.
struct Tile {
  int s, tok0, kt0, kt1;
};
struct Entry {
  int s, tok0, kt0, kt1, slot, pad0, pad1, pad2;  // slot -1: the whole range
};
struct Split {
  int s, tok0, slot, parts;
};
struct Plan {
  int n_entries, n_split, counter, flags;
};
struct Ws {
  Plan* plan;
  int* tile_off;  // [B + 1]
  Tile* tiles;
  Entry* entries;
  Split* splits;
  float* ml;      // [slot][2 * 128][2]
  float* po;      // [slot][2 * 128][128]
};
__host__ __device__ inline size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
__host__ __device__ inline int split_cap(int Hkv) { return Hkv >= kMaxSplit ? 1 : kMaxSplit / Hkv; }
// Tile pairs of T tokens in B sequences, at most.
__host__ __device__ inline size_t max_pairs(int T, int B, int group) {
  return static_cast<size_t>(T) / (2 * (kTile / group)) + B;
}
__host__ __device__ inline int slot_rows(int max_q, int group) {
  const long long r = static_cast<long long>(max_q) * group;
  return r >= 2 * kTile ? 2 * kTile : r > kTile ? 2 * kTile : kTile;
}
__host__ __device__ inline size_t carve(Ws* w, char* ws, int T, int B, int Hkv, int group, int rows) {
  char* p = ws;
  w->plan = reinterpret_cast<Plan*>(p);
  p += 256;
  w->tile_off = reinterpret_cast<int*>(p);
  p += up256((static_cast<size_t>(B) + 1) * sizeof(int));
  const size_t nt = max_pairs(T, B, group), sc = split_cap(Hkv);
  w->tiles = reinterpret_cast<Tile*>(p);
  p += up256(nt * sizeof(Tile));
  w->entries = reinterpret_cast<Entry*>(p);
  p += up256((nt + sc) * sizeof(Entry));
  w->splits = reinterpret_cast<Split*>(p);
  p += up256(sc * sizeof(Split));
  w->ml = reinterpret_cast<float*>(p);
  p += up256(sc * Hkv * rows * 2 * sizeof(float));
  w->po = reinterpret_cast<float*>(p);
  p += sc * Hkv * rows * kDh * sizeof(float);
  return static_cast<size_t>(p - ws);
}

__device__ __forceinline__ PagedSeq chunk_seq(const PagedAttnParams& p, int s, bool* bad) {
  PagedSeq q = paged_seq(p.b, s, bad);
  if (q.n > p.max_q) {
    q.kv = 0;
    *bad = true;
  }
  return q;
}

// ------------------------------------------------------------------- the plan
constexpr int kPlanThreads = 1024;

// Exclusive scan of one value per thread; *total is the sum.
__device__ __forceinline__ int block_scan(int v, int* s_warp, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w < warp) before += s_warp[w];
    all += s_warp[w];
  }
  *total = all;
  return before + inc - v;
}

__global__ void __launch_bounds__(kPlanThreads) k_chunk_plan(PagedAttnParams p, Ws w) {
  __shared__ int s_warp[kPlanThreads / 32];
  __shared__ unsigned long long s_sum[4];
  __shared__ int s_max;
  const int tid = threadIdx.x;
  pdl_trigger();
  const int pair = 2 * (kTile / p.group);  // tokens of a tile pair
  if (tid < 4) s_sum[tid] = 0;
  if (tid == 0) s_max = 0;
  // tile pairs of each sequence
  int n_tiles = 0;
  for (int s0 = 0; s0 < p.b.B; s0 += kPlanThreads) {
    const int s = s0 + tid;
    int c = 0;
    if (s < p.b.B) {
      bool bad;
      const PagedSeq q = chunk_seq(p, s, &bad);
      if (bad && p.status != nullptr) atomicOr(p.status, FLINT_DEVCHECK_INDEX);
      c = q.kv > 0 ? (q.n + pair - 1) / pair : 0;
    }
    int tot;
    const int at = n_tiles + block_scan(c, s_warp, &tot);
    if (s < p.b.B) w.tile_off[s] = at;
    n_tiles += tot;
  }
  // overlapping token ranges could promise more tiles than the list holds
  const int cap = static_cast<int>(max_pairs(p.b.T, p.b.B, p.group));
  if (n_tiles > cap) {
    n_tiles = cap;
    if (tid == 0 && p.status != nullptr) atomicOr(p.status, FLINT_DEVCHECK_INDEX);
  }
  __syncthreads();
  unsigned long long sum = 0;
  int longest = 0;
  for (int i = tid; i < n_tiles; i += kPlanThreads) {
    int lo = 0, hi = p.b.B;  // the last sequence whose tiles start at or before i
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (w.tile_off[mid] <= i) lo = mid;
      else hi = mid;
    }
    bool bad;
    const PagedSeq q = chunk_seq(p, lo, &bad);
    const int tok0 = (i - w.tile_off[lo]) * pair;
    const int last = min(q.n, tok0 + pair);
    const int end = q.kv - q.n + last;
    const int first = p.window > 0 ? max(0, q.kv - q.n + tok0 - p.window + 1) : 0;
    const Tile t{lo, tok0, first / kTile, (end + kTile - 1) / kTile};
    w.tiles[i] = t;
    sum += t.kt1 - t.kt0;
    longest = max(longest, t.kt1 - t.kt0);
  }
  if (sum != 0) atomicAdd(&s_sum[0], sum);
  if (longest != 0) atomicMax(&s_max, longest);
  __syncthreads();
  // Run length: whole ranges, or pieces of about one or half a CTA's even
  // share. Estimated time in key tiles: the even share of all work, 2 tiles of
  // fill and drain per item, 2 more per piece of a split, and half the longest
  // item (the tail of the last one).
  const int Hkv = p.Hkv;
  const unsigned long long W = s_sum[0] * Hkv;
  const int even = static_cast<int>(min((W + kCtas - 1) / kCtas, 1ull << 24));
  const int c1 = max(4, even), c2 = max(4, (even + 1) / 2);
  unsigned long long n1 = 0, n2 = 0;
  for (int i = tid; i < n_tiles; i += kPlanThreads) {
    const int len = w.tiles[i].kt1 - w.tiles[i].kt0;
    if (len > c1) n1 += (len + c1 - 1) / c1;
    if (len > c2) n2 += (len + c2 - 1) / c2;
  }
  if (n1 != 0) atomicAdd(&s_sum[1], n1);
  if (n2 != 0) atomicAdd(&s_sum[2], n2);
  __syncthreads();
  const int sc = split_cap(Hkv);
  auto est = [&](unsigned long long pieces, int len) {
    return (static_cast<float>(W) + Hkv * (2.f * n_tiles + 4.f * pieces)) / kCtas + 0.5f * len;
  };
  int run = 1 << 30;
  float best = est(0, s_max);
  if (s_sum[1] > 0 && s_sum[1] <= sc && est(s_sum[1], c1) < best) {
    best = est(s_sum[1], c1);
    run = c1;
  }
  if (s_sum[2] > 0 && s_sum[2] <= sc && est(s_sum[2], c2) < best) run = c2;
  // the list, last tiles (the longest of a sequence) first
  int n_entries = 0, n_pieces = 0, n_split = 0;
  for (int i0 = 0; i0 < n_tiles; i0 += kPlanThreads) {
    const int i = n_tiles - 1 - (i0 + tid);
    Tile t{0, 0, 0, 0};
    int parts = 0;
    if (i >= 0) {
      t = w.tiles[i];
      parts = max(1, (t.kt1 - t.kt0 + run - 1) / run);
    }
    const bool split = parts > 1;
    int te, tp, ts;
    const int e = n_entries + block_scan(parts, s_warp, &te);
    const int slot = n_pieces + block_scan(split ? parts : 0, s_warp, &tp);
    const int si = n_split + block_scan(split ? 1 : 0, s_warp, &ts);
    if (i >= 0) {
      const int len = t.kt1 - t.kt0;
      for (int k = 0; k < parts; ++k)
        w.entries[e + k] = Entry{t.s, t.tok0, t.kt0 + static_cast<int>(static_cast<long long>(len) * k / parts),
                                 t.kt0 + static_cast<int>(static_cast<long long>(len) * (k + 1) / parts),
                                 split ? slot + k : -1, 0, 0, 0};
      if (split) w.splits[si] = Split{t.s, t.tok0, slot, parts};
    }
    n_entries += te;
    n_pieces += tp;
    n_split += ts;
  }
  if (tid == 0) *w.plan = Plan{n_entries, n_split, 0, 0};
}

// ------------------------------------------------------------------- main kernel
struct Item {
  int row0, tok0, live, n, kv, kt0, kt1, g, slot, s, end, pad;  // live: tokens from tok0 on, at most a pair's
};

template <bool kE4M3>
struct Ctl {
  uint64_t q_full[2], q_empty[2], qc_full[2], kv_full[5], kv_empty[5], raw_full[3], raw_empty[3], s_full[2], p_full[2][2],
      o_done[2], it_full[2], it_empty[2];
  Item item[2];
  uint32_t tmem;
  volatile int abort_flag;
  float inv_sig[kE4M3 ? 2 : 1][2][kE4M3 ? kTile : 1];  // [item parity][tile][row]: 1 / Q scale
};

template <bool kE4M3>
constexpr size_t smem_bytes() {
  return 2 * kTileBytes + Cfg<kE4M3>::kStages * kTileBytes + Cfg<kE4M3>::kRaw * kRawBytes +
         sizeof(Ctl<kE4M3>);
}
static_assert(smem_bytes<true>() <= 232448 && smem_bytes<false>() <= 232448, "shared memory");

template <int kRegs>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs)); }
template <int kRegs>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs)); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Two fp32 at a time (sm_100's packed arithmetic).
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(f32x2 x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

template <bool kE4M3>
__global__ void __launch_bounds__(Cfg<kE4M3>::kThreads, 1)
    k_paged_chunk(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                  const __grid_constant__ CUtensorMap mv, PagedAttnParams p, Ws w, int rows_per_slot) {
  using C = Cfg<kE4M3>;
  extern __shared__ __align__(1024) uint8_t sq[];  // the 128-byte swizzle repeats every 1024 bytes
  uint8_t* skv = sq + 2 * kTileBytes;
  uint8_t* sraw = skv + C::kStages * kTileBytes;
  Ctl<kE4M3>& ctl = *reinterpret_cast<Ctl<kE4M3>*>(sraw + C::kRaw * kRawBytes);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int* status = p.status != nullptr ? p.status : &w.plan->flags;

  if (warp == 0) tmem_alloc(&ctl.tmem, 512);
  if (tid == 32) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl.q_full[i], 1);
      mbar_init(&ctl.q_empty[i], 1);
      mbar_init(&ctl.qc_full[i], 128);
      mbar_init(&ctl.s_full[i], 1);
      mbar_init(&ctl.p_full[i][0], 128);
      mbar_init(&ctl.p_full[i][1], 128);
      mbar_init(&ctl.o_done[i], 1);
      mbar_init(&ctl.it_full[i], 1);
      mbar_init(&ctl.it_empty[i], 1 + 8 + (kE4M3 ? 4 : 0));
    }
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&ctl.kv_full[i], C::kFullCount);
      mbar_init(&ctl.kv_empty[i], 1);
    }
    for (int i = 0; i < C::kRaw; ++i) {
      mbar_init(&ctl.raw_full[i], 1);
      mbar_init(&ctl.raw_empty[i], 128);
    }
    ctl.abort_flag = 0;
    fence_barrier_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem;
  pdl_wait();  // the plan
  pdl_trigger();
  volatile int* ab = &ctl.abort_flag;
  const int tok_t = kTile / p.group;  // tokens of one query tile

  // Next item of the list, for the roles that follow the loader.
  auto next_item = [&](int it, Item& out) -> bool {
    if (!mma_wait(&ctl.it_full[it & 1], (it >> 1) & 1, ab, status)) return false;
    out = ctl.item[it & 1];
    return out.end == 0;
  };
  auto done_item = [&](int it) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctl.it_empty[it & 1]);
  };

  if (warp < 8) {
    // =============================================================== softmax
    regs_inc<kE4M3 ? 184 : 208>();
    const int t = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + t * 128 + lane_off, to = tmem + 256 + t * 128 + lane_off;
    uint32_t cnt = 0;  // S tiles seen: parity of s_full, p_full, o_done
    uint32_t qn = 0;
    bool ok = true;
    Item im;
    for (int it = 0; ok && next_item(it, im); ++it) {
      if (t == 1 && im.live <= tok_t) {  // a lone first tile
        done_item(it);
        continue;
      }
      const int tok = t * tok_t + row / p.group;
      const bool live = row < tok_t * p.group && tok < im.live;
      const int first = im.kv - im.n + im.tok0 + t * tok_t;  // position of the tile's first token
      const int last = im.kv - im.n + im.tok0 + min(im.live, (t + 1) * tok_t) - 1;
      const int hi = live ? im.kv - im.n + im.tok0 + tok + 1 : 0;
      const int lo = p.window > 0 ? hi - p.window : 0;
      float c = p.scale * kLog2e;
      if constexpr (kE4M3) {
        if (!(ok = mma_wait(&ctl.qc_full[t], qn & 1, ab, status))) break;
        ++qn;
        c *= ctl.inv_sig[it & 1][t][row] * __ldg(p.k_scale + im.g);
      }
      done_item(it);
      float m = -INFINITY, l = 0.f;
      for (int kt = im.kt0; kt < im.kt1; ++kt) {
        if (!(ok = mma_wait(&ctl.s_full[t], cnt & 1, ab, status))) break;
        tc_fence_after();
        float s[128];
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld32(ts + 32 * i, s + 32 * i);
        tmem_wait_ld();
        const int k0 = kt * kTile;
        if (k0 + kTile > first + 1 || (p.window > 0 && k0 < last + 1 - p.window)) {
          const int h = hi - k0, q = lo - k0;
#pragma unroll
          for (int i = 0; i < 128; ++i)
            if (i >= h || i < q) s[i] = -INFINITY;
        }
        float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int i = 4; i < 128; i += 4) {
          mx[0] = fmaxf(mx[0], s[i]);
          mx[1] = fmaxf(mx[1], s[i + 1]);
          mx[2] = fmaxf(mx[2], s[i + 2]);
          mx[3] = fmaxf(mx[3], s[i + 3]);
        }
        const float mn = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        if (kt == im.kt0) {
          m = mn;
        } else {
          const bool grow = (mn - m) * c > kRescale || (m == -INFINITY && mn > m);
          if (__any_sync(0xffffffffu, grow)) {
            // P V of the previous tile has to be in O before O is rescaled
            if (!(ok = mma_wait(&ctl.o_done[t], (cnt - 1) & 1, ab, status))) break;
            tc_fence_after();
            const float mu = fmaxf(m, mn);
            const float f = m == -INFINITY ? 0.f : exp2_ftz((m - mu) * c);
            m = mu;
            l *= f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float o[16];
              tmem_ld16(to + 16 * i, o);
              uint32_t r[16];
#pragma unroll
              for (int j = 0; j < 16; ++j) r[j] = __float_as_uint(o[j] * f);
              tmem_st16(to + 16 * i, r);
            }
          }
        }
        const float mc = m == -INFINITY ? 0.f : m * c;
        const f32x2 c2 = pack2(c, c), mc2 = pack2(-mc, -mc);
        f32x2 sum[2] = {pack2(0.f, 0.f), pack2(0.f, 0.f)};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t r[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float a, b;
            unpack2(fma2(pack2(s[32 * i + 2 * j], s[32 * i + 2 * j + 1]), c2, mc2), a, b);
            a = exp2_ftz(a);
            b = exp2_ftz(b);
            sum[j & 1] = add2(sum[j & 1], pack2(a, b));
            if constexpr (kE4M3) {
              r[j] = pack_f16x2(a, b);
            } else {
              const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
              r[j] = *reinterpret_cast<const uint32_t*>(&v);
            }
          }
          tmem_st16(ts + 16 * i, r);
          if (i == 1) {  // P V of the first 64 keys starts while the others are weighed (prompt of 8,192: 524 -> 512 us)
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&ctl.p_full[t][0]);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&ctl.p_full[t][1]);
        float s0, s1, s2, s3;
        unpack2(sum[0], s0, s1);
        unpack2(sum[1], s2, s3);
        l += (s0 + s1) + (s2 + s3);
        ++cnt;
      }
      if (!ok) break;
      // ---- O of the last tile, out
      if (!(ok = mma_wait(&ctl.o_done[t], (cnt - 1) & 1, ab, status))) break;
      tc_fence_after();
      float o[128];
#pragma unroll
      for (int i = 0; i < 4; ++i) tmem_ld32(to + 32 * i, o + 32 * i);
      tmem_wait_ld();
      tc_fence_before();
      if (live) {
        if (im.slot < 0) {
          const float f = (l > 0.f ? 1.f / l : 0.f) * (kE4M3 ? __ldg(p.v_scale + im.g) : 1.f);
          uint4* dst = reinterpret_cast<uint4*>(
              p.out + (static_cast<size_t>(im.row0 + im.tok0 + tok) * p.Hq + im.g * p.group + row % p.group) * kDh);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            uint32_t r[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const __nv_bfloat162 v = __floats2bfloat162_rn(o[8 * i + 2 * j] * f, o[8 * i + 2 * j + 1] * f);
              r[j] = *reinterpret_cast<const uint32_t*>(&v);
            }
            dst[i] = make_uint4(r[0], r[1], r[2], r[3]);
          }
        } else {
          const size_t at = (static_cast<size_t>(im.slot) * p.Hkv + im.g) * rows_per_slot + t * kTile + row;
          *reinterpret_cast<float2*>(w.ml + at * 2) = make_float2(m == -INFINITY ? -INFINITY : m * c, l);
          float4* dst = reinterpret_cast<float4*>(w.po + at * kDh);
#pragma unroll
          for (int i = 0; i < 32; ++i) dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        }
      }
    }
  } else if (warp == 8) {
    // =================================================================== MMA
    regs_dec<kE4M3 ? 64 : 88>();
    const uint32_t idesc_s = mma_idesc(kTile, kTile, !kE4M3);
    const uint32_t idesc_o = idesc_s | kIdescBMn;
    uint32_t kvi = 0, cnt[2] = {0, 0}, qn[2] = {0, 0};
    bool ok = true;
    Item im;
    auto stage = [&](uint32_t i) { return smem_addr(skv) + (i % C::kStages) * kTileBytes; };
    auto wait_kv = [&](uint32_t i) {
      return ok = ok && mma_wait(&ctl.kv_full[i % C::kStages], (i / C::kStages) & 1, ab, status);
    };
    auto issue_s = [&](int t, uint32_t k_addr) {
      if (lane == 0) {
        const uint32_t qa = smem_addr(sq) + t * kTileBytes;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t off = (k >> 2) * kHalfBytes + (k & 3) * 32;
          mma_f16(tmem + t * 128, sw128_desc(qa + off), sw128_desc(k_addr + off), idesc_s, k > 0);
        }
        mma_commit(&ctl.s_full[t]);
      }
      __syncwarp();
    };
    auto issue_o = [&](int t, int half, uint32_t v_addr, bool acc) {
      if (lane == 0) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_f16_ts(tmem + 256 + t * 128, tmem + t * 128 + 32 * half + 8 * k,
                     sw128_mn_desc(v_addr + (4 * half + k) * 2048, kHalfBytes), idesc_o, acc || half + k > 0);
        if (half == 1) mma_commit(&ctl.o_done[t]);
      }
      __syncwarp();
    };
    auto commit = [&](uint64_t* bar) {
      if (lane == 0) mma_commit(bar);
      __syncwarp();
    };
    for (int it = 0; ok && next_item(it, im); ++it) {
      done_item(it);
      const int nt = im.live > tok_t ? 2 : 1, nk = im.kt1 - im.kt0;
      for (int t = 0; t < nt && ok; ++t) {
        ok = mma_wait(kE4M3 ? &ctl.qc_full[t] : &ctl.q_full[t], qn[t] & 1, ab, status);
        ++qn[t];
      }
      if (!ok || !wait_kv(kvi)) break;
      tc_fence_after();
      for (int t = 0; t < nt; ++t) issue_s(t, stage(kvi));
      commit(&ctl.kv_empty[kvi % C::kStages]);
      if (nk == 1)
        for (int t = 0; t < nt; ++t) commit(&ctl.q_empty[t]);
      for (int j = 0; j < nk; ++j) {
        const uint32_t vi = kvi + 2 * j + 1, ki = vi + 1;
        if (!wait_kv(vi)) break;
        if constexpr (!kE4M3) {
          // V rows past the sequence's end hold anything: zeros, for 0 x NaN is NaN
          const int valid = im.kv - (im.kt0 + j) * kTile;
          if (valid < kTile) {
            uint8_t* v = skv + (vi % C::kStages) * kTileBytes;
            for (int i = valid * 8 + lane; i < kTile * 8; i += 32) {
              reinterpret_cast<uint4*>(v)[i] = make_uint4(0, 0, 0, 0);
              reinterpret_cast<uint4*>(v + kHalfBytes)[i] = make_uint4(0, 0, 0, 0);
            }
            fence_async_smem();
            __syncwarp();
          }
        }
        for (int t = 0; t < nt; ++t) {
          for (int half = 0; half < 2 && ok; ++half) {
            if (!(ok = mma_wait(&ctl.p_full[t][half], cnt[t] & 1, ab, status))) break;
            tc_fence_after();
            issue_o(t, half, stage(vi), j > 0);
          }
          if (!ok) break;
          ++cnt[t];
          if (j + 1 < nk) {
            if (t == 0 && !wait_kv(ki)) break;
            tc_fence_after();
            issue_s(t, stage(ki));
            if (j + 2 == nk) commit(&ctl.q_empty[t]);
          }
        }
        if (!ok) break;
        commit(&ctl.kv_empty[vi % C::kStages]);
        if (j + 1 < nk) commit(&ctl.kv_empty[ki % C::kStages]);
      }
      kvi += 2 * nk;
    }
  } else if (warp == 9) {
    // ================================================================ loader
    regs_dec<kE4M3 ? 64 : 88>();
    const int n_items = w.plan->n_entries * p.Hkv;
    const int ps = 1 << p.b.page_shift;
    const int box = min(ps, kTile), n_box = kTile / box;
    const int my_box = kE4M3 ? lane : lane >> 1, half = kE4M3 ? 0 : lane & 1;
    const bool mine = my_box < n_box;
    const int bad_row = static_cast<int>(p.b.n_pages << p.b.page_shift);  // past the pool: zeros
    const uint32_t box_bytes = box * (kE4M3 ? kDh : kDh * 2);
    uint32_t li = 0, qn[2] = {0, 0};
    constexpr int kRing = kE4M3 ? C::kRaw : C::kStages;
    bool ok = true;
    for (int it = 0; ok; ++it) {
      if (!(ok = mma_wait(&ctl.it_empty[it & 1], ((it >> 1) & 1) ^ 1, ab, status))) break;
      Item im{};
      if (lane == 0) {
        const int i = atomicAdd(&w.plan->counter, 1);
        if (i < n_items) {
          const Entry e = w.entries[i / p.Hkv];
          bool bad;
          const PagedSeq q = chunk_seq(p, e.s, &bad);
          im.row0 = q.row0;
          im.tok0 = e.tok0;
          im.live = min(q.n - e.tok0, 2 * tok_t);
          im.n = q.n;
          im.kv = q.kv;
          im.kt0 = e.kt0;
          im.kt1 = e.kt1;
          im.g = i % p.Hkv;
          im.slot = e.slot;
          im.s = e.s;
          im.end = 0;
        } else {
          im.end = 1;
        }
        ctl.item[it & 1] = im;
        mbar_arrive(&ctl.it_full[it & 1]);
      }
      __syncwarp();
      im = ctl.item[it & 1];
      if (im.end) break;
      const int nt = im.live > tok_t ? 2 : 1;
      for (int t = 0; t < nt && ok; ++t) {
        if (!(ok = mma_wait(&ctl.q_empty[t], (qn[t] & 1) ^ 1, ab, status))) break;
        ++qn[t];
        if (lane == 0) mbar_arrive_expect_tx(&ctl.q_full[t], 2u * tok_t * p.group * 128);
        __syncwarp();
        if (lane < 2)
          tma_load_3d(sq + t * kTileBytes + lane * kHalfBytes, &mq, 64 * lane, im.g * p.group,
                      im.row0 + im.tok0 + t * tok_t, &ctl.q_full[t]);
        __syncwarp();
      }
      if (!ok) break;
      const int32_t* table = p.b.block_table + static_cast<size_t>(im.s) * p.b.max_pages;
      // pool row of this lane's box of key tile kt, -1 past the sequence
      auto box_row = [&](int kt) {
        const int key = kt * kTile + my_box * box;
        if (!mine || kt >= im.kt1 || key >= im.kv) return -1;
        const int page = __ldg(table + (key >> p.b.page_shift));
        if (page < 0 || page >= p.b.n_pages) {
          if (half == 0) atomicOr(status, FLINT_DEVCHECK_INDEX);
          return bad_row;
        }
        return (page << p.b.page_shift) + (key & (ps - 1));
      };
      int r = box_row(im.kt0);
      for (int kt = im.kt0; kt < im.kt1 && ok; ++kt) {
        const int nxt = box_row(kt + 1);
        const int boxes = min(n_box, (im.kv - kt * kTile + box - 1) / box);
        for (int v = 0; v < 2; ++v, ++li) {
          const uint32_t st = li % kRing;
          uint64_t* empty = kE4M3 ? &ctl.raw_empty[st] : &ctl.kv_empty[st];
          uint64_t* full = kE4M3 ? &ctl.raw_full[st] : &ctl.kv_full[st];
          if (!(ok = mma_wait(empty, ((li / kRing) & 1) ^ 1, ab, status))) break;
          if (lane == 0) mbar_arrive_expect_tx(full, boxes * box_bytes);
          __syncwarp();
          if (r >= 0) {
            uint8_t* dst = kE4M3 ? sraw + st * kRawBytes + my_box * box * kDh
                                 : skv + st * kTileBytes + half * kHalfBytes + my_box * box * 128;
            tma_load_3d(dst, v ? &mv : &mk, 64 * half, im.g, r, full);
          }
          __syncwarp();
        }
        r = nxt;
      }
    }
    // copies in flight land before the CTA ends (only after a wait gave up)
    if (!ok) {
      const long long t0 = clock64();
      while (clock64() - t0 < 2000000) {
      }
    }
  } else if (warp >= 12) {
    if constexpr (kE4M3) {
      // ============================================================= converter
      regs_dec<80>();
      const int row = tid - 384;
      uint32_t li = 0, qn[2] = {0, 0};
      bool ok = true;
      Item im;
      for (int it = 0; ok && next_item(it, im); ++it) {
        const int nt = im.live > tok_t ? 2 : 1;
        for (int t = 0; t < nt && ok; ++t) {
          if (!(ok = mma_wait(&ctl.q_full[t], qn[t] & 1, ab, status))) break;
          ++qn[t];
          uint8_t* q = sq + t * kTileBytes + row * 128;
          float amax = 0.f;
  #pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint4 v = *reinterpret_cast<const uint4*>(q + (i >> 3) * kHalfBytes + (((i & 7) ^ (row & 7)) << 4));
            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
  #pragma unroll
            for (int j = 0; j < 4; ++j)
              amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(u[j] << 16)), fabsf(__uint_as_float(u[j] & 0xFFFF0000u))));
          }
          const float sig = pow2_scale_for(amax);
  #pragma unroll
          for (int i = 0; i < 16; ++i) {
            uint4* at = reinterpret_cast<uint4*>(q + (i >> 3) * kHalfBytes + (((i & 7) ^ (row & 7)) << 4));
            const uint4 v = *at;
            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
            uint32_t f[4];
  #pragma unroll
            for (int j = 0; j < 4; ++j)
              f[j] = pack_f16x2(__uint_as_float(u[j] << 16) * sig, __uint_as_float(u[j] & 0xFFFF0000u) * sig);
            *at = make_uint4(f[0], f[1], f[2], f[3]);
          }
          ctl.inv_sig[it & 1][t][row] = 1.f / sig;
          fence_async_smem();
          mbar_arrive(&ctl.qc_full[t]);
        }
        for (int kt = im.kt0; kt < im.kt1 && ok; ++kt) {
          const bool in = row < im.kv - kt * kTile;
          for (int v = 0; v < 2; ++v, ++li) {
            const uint32_t rs = li % C::kRaw, st = li % C::kStages;
            if (!(ok = mma_wait(&ctl.raw_full[rs], (li / C::kRaw) & 1, ab, status))) break;
            if (!(ok = mma_wait(&ctl.kv_empty[st], ((li / C::kStages) & 1) ^ 1, ab, status))) break;
            const uint8_t* src = sraw + rs * kRawBytes + row * kDh;
            uint8_t* dst = skv + st * kTileBytes + row * 128;
  #pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint4 x = in ? *reinterpret_cast<const uint4*>(src + ((i ^ (row & 7)) << 4)) : make_uint4(0, 0, 0, 0);
              uint8_t* d = dst + (i >> 2) * kHalfBytes;
              const int cc = 2 * (i & 3);
              *reinterpret_cast<uint4*>(d + ((cc ^ (row & 7)) << 4)) =
                  make_uint4(e4m3x2_to_f16x2(x.x), e4m3x2_to_f16x2(x.x >> 16), e4m3x2_to_f16x2(x.y),
                             e4m3x2_to_f16x2(x.y >> 16));
              *reinterpret_cast<uint4*>(d + (((cc + 1) ^ (row & 7)) << 4)) =
                  make_uint4(e4m3x2_to_f16x2(x.z), e4m3x2_to_f16x2(x.z >> 16), e4m3x2_to_f16x2(x.w),
                             e4m3x2_to_f16x2(x.w >> 16));
            }
            fence_async_smem();
            mbar_arrive(&ctl.kv_full[st]);
            mbar_arrive(&ctl.raw_empty[rs]);
          }
        }
        done_item(it);
      }
    }
  } else {
    regs_dec<kE4M3 ? 64 : 88>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// One warp per query row of a split entry: joins its pieces in key order. The
// same grid writes zeros for the tokens of invalid sequences.
constexpr int kCombineThreads = 256;

__global__ void __launch_bounds__(kCombineThreads) k_chunk_combine(PagedAttnParams p, Ws w, int rows_per_slot) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long long warps = static_cast<long long>(gridDim.x) * (kCombineThreads / 32);
  const long long me = static_cast<long long>(blockIdx.x) * (kCombineThreads / 32) + (threadIdx.x >> 5);
  const int tok_t = kTile / p.group;
  const long long n = static_cast<long long>(__ldcg(&w.plan->n_split)) * p.Hkv * rows_per_slot;
  for (long long i = me; i < n; i += warps) {
    const int r = static_cast<int>(i % rows_per_slot);
    const long long x = i / rows_per_slot;
    const int g = static_cast<int>(x % p.Hkv);
    const int4 sv = __ldcg(reinterpret_cast<const int4*>(w.splits + x / p.Hkv));
    const Split sp{sv.x, sv.y, sv.z, sv.w};
    bool bad;
    const PagedSeq q = chunk_seq(p, sp.s, &bad);
    const int rt = r % kTile, tok = sp.tok0 + (r / kTile) * tok_t + rt / p.group;
    if (rt >= tok_t * p.group || tok >= q.n) continue;
    float M = -INFINITY;
    for (int k = lane; k < sp.parts; k += 32)
      M = fmaxf(M, __ldcg(w.ml + ((static_cast<size_t>(sp.slot + k) * p.Hkv + g) * rows_per_slot + r) * 2));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < sp.parts; ++k) {
      const size_t at = (static_cast<size_t>(sp.slot + k) * p.Hkv + g) * rows_per_slot + r;
      const float2 ml = __ldcg(reinterpret_cast<const float2*>(w.ml + at * 2));
      const float4 o = __ldcg(reinterpret_cast<const float4*>(w.po + at * kDh) + lane);
      const float f = ml.x == -INFINITY ? 0.f : exp2_ftz(ml.x - M);
      l = fmaf(ml.y, f, l);
      acc.x = fmaf(o.x, f, acc.x);
      acc.y = fmaf(o.y, f, acc.y);
      acc.z = fmaf(o.z, f, acc.z);
      acc.w = fmaf(o.w, f, acc.w);
    }
    const float f = (l > 0.f ? 1.f / l : 0.f) * (p.v_scale != nullptr ? __ldg(p.v_scale + g) : 1.f);
    const __nv_bfloat162 a = __floats2bfloat162_rn(acc.x * f, acc.y * f), b = __floats2bfloat162_rn(acc.z * f, acc.w * f);
    reinterpret_cast<uint2*>(p.out + (static_cast<size_t>(q.row0 + tok) * p.Hq + g * p.group + rt % p.group) * kDh)[lane] =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
  for (long long s = me; s < p.b.B; s += warps) {
    bool bad;
    const PagedSeq q = chunk_seq(p, static_cast<int>(s), &bad);
    if (q.n <= 0 || q.kv > 0) continue;
    uint4* dst = reinterpret_cast<uint4*>(p.out + static_cast<size_t>(q.row0) * p.Hq * kDh);
    const long long m = static_cast<long long>(q.n) * p.Hq * (kDh / 8);
    for (long long i = lane; i < m; i += 32) dst[i] = make_uint4(0, 0, 0, 0);
  }
}

template <typename... Args>
cudaError_t launch_pdl(void (*kern)(Args...), int grid, int block, size_t smem, cudaStream_t st,
                       const std::common_type_t<Args>&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace

size_t paged_chunk_workspace(int T, int B, int n_q_heads, int n_kv_heads, int max_q) {
  Ws w;
  const int group = n_q_heads / n_kv_heads;
  return carve(&w, nullptr, T, B, n_kv_heads, group, slot_rows(max_q, group));
}

int paged_chunk_launch(const PagedAttnParams& p, int cache_dtype, size_t ws_bytes, cudaStream_t st) {
  const bool e4m3 = cache_dtype == FLINT_KV_E4M3;
  const int rows = slot_rows(p.max_q, p.group);
  Ws w;
  const size_t need = carve(&w, p.ws, p.b.T, p.b.B, p.Hkv, p.group, rows);
  if (p.ws == nullptr || ws_bytes < need)
    return flint_fail_external(FLINT_ERR_WORKSPACE, "flint_paged_attention: workspace too small");
  CUtensorMap mq, mk, mv;
  const int tok_t = kTile / p.group;
  {
    const cuuint64_t dims[3] = {kDh, static_cast<cuuint64_t>(p.Hq), static_cast<cuuint64_t>(p.b.T)};
    const cuuint64_t str[2] = {kDh * 2, static_cast<cuuint64_t>(p.Hq) * kDh * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(p.group), static_cast<cuuint32_t>(tok_t)};
    const int rc = flint_encode_map_sw128(&mq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, p.q, dims, str, box);
    if (rc != FLINT_OK) return rc;
  }
  {
    const cuuint64_t es = e4m3 ? 1 : 2;
    const cuuint64_t dims[3] = {kDh, static_cast<cuuint64_t>(p.Hkv),
                                static_cast<cuuint64_t>(p.b.n_pages) << p.b.page_shift};
    const cuuint64_t str[2] = {kDh * es, static_cast<cuuint64_t>(p.Hkv) * kDh * es};
    const cuuint32_t box[3] = {e4m3 ? 128u : 64u, 1,
                               static_cast<cuuint32_t>(p.b.page_shift >= 7 ? kTile : 1 << p.b.page_shift)};
    const auto dt = e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    int rc = flint_encode_map_sw128(&mk, dt, 3, p.k, dims, str, box);
    if (rc == FLINT_OK) rc = flint_encode_map_sw128(&mv, dt, 3, p.v, dims, str, box);
    if (rc != FLINT_OK) return rc;
  }
  const void* kern = e4m3 ? reinterpret_cast<const void*>(k_paged_chunk<true>)
                          : reinterpret_cast<const void*>(k_paged_chunk<false>);
  cudaError_t e = flint_ensure_smem(kern);
  if (e != cudaSuccess) return flint_fail_external(FLINT_ERR_CUDA, cudaGetErrorString(e));
  k_chunk_plan<<<1, kPlanThreads, 0, st>>>(p, w);
  e = cudaGetLastError();
  if (e == cudaSuccess)
    e = e4m3 ? launch_pdl(k_paged_chunk<true>, kCtas, Cfg<true>::kThreads, smem_bytes<true>(), st, mq, mk, mv, p, w, rows)
             : launch_pdl(k_paged_chunk<false>, kCtas, Cfg<false>::kThreads, smem_bytes<false>(), st, mq, mk, mv, p, w,
                          rows);
  if (e == cudaSuccess) e = launch_pdl(k_chunk_combine, 2 * kCtas, kCombineThreads, 0, st, p, w, rows);
  if (e != cudaSuccess) return flint_fail_external(FLINT_ERR_CUDA, cudaGetErrorString(e));
  return FLINT_OK;
}

}  // namespace flint
