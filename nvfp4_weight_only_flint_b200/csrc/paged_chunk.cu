// paged_chunk.cu -- attention of many new tokens per sequence (prompt pieces,
// whole prompts, mixed steps) over the paged cache, on the 5th-generation
// tensor cores ("[Model] Add Flint (RecursiveSI/flint)", section "What
// happened": 8K-token prefill; heads from "Recursive Flint: 125 tok/s on an M4
// Pro", architecture table).
//
// k_paged_chunk works through pieces: a pair of query tiles against a run of
// 128-key tiles. A query tile is 128 rows = floor(128 / group) tokens x the
// group of query heads that share the kv head: K and V are fetched once for 2 x
// 128 rows, and a causal edge cuts at most 128 / group tokens. All tile pairs of
// all sequences in turn, each as long as its key tiles and two more for the fill
// and drain of the pipeline, form one line that 148 / Hkv CTAs per kv head cut
// into equal parts; each CTA finds its part from the lengths (a scan over the
// sequences and one over the tile pairs, 1-2 us), so a captured graph stays
// balanced when the lengths change. A pair that spans parts leaves partials, at
// most two per CTA, that k_chunk_combine joins. (A list of whole pairs made by a
// kernel of its own and taken longest first: 1,024 tokens over 31,000 601 us
// against 503, since 128 items do not fill 148 CTAs, and a mixed step 66 us
// against 60, 10 of them the list.) Where pairs are many and short beside a part
// (deal_whole), they are dealt out whole instead, from the last one of the line
// (a prompt's longest) and back and forth, without partials.
// Times here are of calls replayed from a graph; one by one they take up to 10 %
// longer.
//
// Per key tile and query tile
//   S = Q K^T     tcgen05.mma, both operands in shared memory (TMA, 128-byte swizzle)
//   P = 2^(S c - m c)   by the tile's own warpgroup: thread = row, S read from
//                 tensor memory into registers, P rounded and written back over S
//   O += P V      tcgen05.mma, P from tensor memory, V as it lies in the cache
//                 (keys x dims: MN-major)
// with the two tiles' softmax and MMAs alternating. O is rescaled only when a
// row's maximum grew by more than kGrow since the last time (P then stays below
// 2^kGrow; O / l is the same; a published form of the running softmax), by the
// softmax warps themselves, so no correction warps stand in the chain. Tensor
// memory: S0 S1 O0 O1, 128 columns each.
//   bf16 cache: five 32 KB stages of K and V by TMA, one box per page (or 128 rows).
//   E4M3 cache: three raw 16 KB stages; a further warpgroup turns them into f16
//     tiles (exact), and Q into f16 after a power-of-two scale per row; P is f16
//     times 2^kShift.
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
constexpr int kFill = 2;                   // length of a tile pair on the line beyond its key tiles
constexpr int kMinPart = 6;                // a line has at most total / kMinPart parts, rounded up
// So no part is shorter than kMinPart / 2, and each reaches past a pair's first kFill places.
static_assert(kMinPart / 2 > kFill, "a part within a pair's first kFill places would leave no partial, but be joined");
constexpr int kMaxSeqs = 32768;            // the scan over sequences lives in the stages' shared memory

template <bool kE4M3>
struct Cfg {
  static constexpr int kThreads = kE4M3 ? 512 : 384;
  static constexpr int kStages = kE4M3 ? 3 : 5;
  static constexpr int kRaw = kE4M3 ? 3 : 0;
  static constexpr int kFullCount = kE4M3 ? 128 : 1;
  // log2: a row's maximum may grow by 2^kGrow before O is rescaled, and P is 2^kShift times the weight, at most
  // 2^(kGrow + kShift). f16 weights keep 11 bits from 2^-14 on, that is down to 2^-25 of the largest (growth by 2^8 and
  // no shift, as for bf16: 2^-14 to 2^-22, and the keys behind a dominating one lost theirs). 1,024 tokens over 31,000:
  // 531 us, as with 2^8 unshifted (531 to 540); growth by 2^2 and a shift of 2^13 534 to 542.
  static constexpr float kGrow = kE4M3 ? 4.f : 8.f;
  static constexpr float kShift = kE4M3 ? 11.f : 0.f;
};

// A tile pair cut by part boundaries: its pieces are in parts first .. last.
struct Split {
  int s, tok0, first, last;  // s -1: none
};
struct Ws {
  int* flags;     // stands in for a null status
  Split* splits;  // [parts]: the pair that part leaves unfinished
  float* ml;      // [slot][rows][2]: maximum (log2 units), sum
  float* po;      // [slot][rows][128]
};
__host__ __device__ inline size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
__host__ __device__ inline int parts_per_head(int Hkv) { return Hkv >= kCtas ? 1 : kCtas / Hkv; }
__host__ __device__ inline int slot_rows(int max_q, int group) {
  return static_cast<long long>(max_q) * group > kTile ? 2 * kTile : kTile;
}
__host__ __device__ inline size_t carve(Ws* w, char* ws, int Hkv, int rows) {
  char* p = ws;
  w->flags = reinterpret_cast<int*>(p);
  p += 256;
  // a kv head of one part cuts no pair
  const size_t parts = parts_per_head(Hkv), slots = parts > 1 ? parts * Hkv * 2 : 0;
  w->splits = reinterpret_cast<Split*>(p);
  p += up256(parts * sizeof(Split));
  w->ml = reinterpret_cast<float*>(p);
  p += up256(slots * rows * 2 * sizeof(float));
  w->po = reinterpret_cast<float*>(p);
  p += slots * rows * kDh * sizeof(float);
  return static_cast<size_t>(p - ws);
}
// Piece of part i: the pair ends there (0) or goes on (1).
__device__ __forceinline__ size_t slot_of(int part, int Hkv, int g, bool goes_on) {
  return (static_cast<size_t>(part) * Hkv + g) * 2 + (goes_on ? 1 : 0);
}

__device__ __forceinline__ PagedSeq chunk_seq(const PagedAttnParams& p, int s, bool* bad) {
  PagedSeq q = paged_seq(p.b, s, bad);
  if (q.n > p.max_q) {
    q.kv = 0;
    *bad = true;
  }
  return q;
}

// ------------------------------------------------------------------- the line
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Key tiles [kt0, kt1) that the tile pair from token tok0 of a sequence attends.
struct Keys {
  int kt0, kt1;
  __device__ __forceinline__ int length() const { return kt1 - kt0 + kFill; }
};
__device__ __forceinline__ Keys pair_keys(const PagedSeq& q, int tok0, int pair, int window) {
  const int end = q.kv - q.n + min(q.n, tok0 + pair);
  const int first = window > 0 ? max(0, q.kv - q.n + tok0 - window + 1) : 0;
  return Keys{first / kTile, (end + kTile - 1) / kTile};
}
__device__ __forceinline__ int pairs_of(const PagedSeq& q, int pair) { return q.kv > 0 ? (q.n + pair - 1) / pair : 0; }

// Where a part of the line begins.
constexpr int kDealSeqs = 64;  // sequences whose first pairs are kept for it
struct Start {
  long long base, total;  // of the pair that holds the part's first place; length of the line
  int s, tok0;
  int n_pairs, longest, deal;
  int first_pair[kDealSeqs];
};

// Exclusive scan of one value per thread over the block; *total is the sum.
template <int kThreads>
__device__ __forceinline__ long long block_scan(long long v, long long* s_warp, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll 4
  for (int w = 0; w < kThreads / 32; ++w) {
    const long long x = s_warp[w];
    if (w < warp) before += x;
    all += x;
  }
  *total = all;
  return before + inc - v;
}

// Whole pairs, dealt back and forth: four or more a CTA, none longer than a
// third of a part; that is even for one sequence, whose pairs grow steadily, and
// for several if no pair is longer than 1.6 times the mean. Dealt / cut, us (in
// brackets the longest pair over the mean): a prompt of 8,192 502 to 517 / 522 to
// 528, 16 prompts of 512 [1.3] 85 / 91, 8 of 1,024 [1.5] 114 to 117 / 119 to 123,
// 64 pieces of 128 over up to 1,000 keys [1.7] 136 / 129, 5 prompts of 1,500 to
// 1,777 [1.7] 165 / 152 to 166, 32 pieces of 256 over up to 2,000 [1.9] 218 / 191,
// 16 of 512 over up to 4,000 [2.3] 352 / 256.
__device__ __forceinline__ bool deal_whole(int B, long long n_pairs, int longest, long long total, int n_parts) {
  return B <= kDealSeqs && n_pairs >= 4ll * n_parts && 3ll * longest * n_parts <= total &&
         (B == 1 || 5ll * longest * n_pairs <= 8 * total);
}

// All threads of the CTA. first_pair: scratch for B ints. Parts: place i of n is
// total i / n; n is chosen here, at most total / kMinPart (rounded up).
template <int kThreads>
__device__ __forceinline__ void find_start(const PagedAttnParams& p, int part, int* n_parts, int* first_pair,
                                           long long* s_warp, Start* start) {
  const int tid = threadIdx.x;
  const int pair = 2 * (kTile / p.group);
  const int per = (p.b.B + kThreads - 1) / kThreads;
  const int sb = min(p.b.B, tid * per), se = min(p.b.B, sb + per);
  long long mine = 0, n_pairs;
  if (tid == 0) start->longest = 0;
  for (int s = sb; s < se; ++s) {
    bool bad;
    const PagedSeq q = chunk_seq(p, s, &bad);
    if (bad && blockIdx.x == 0 && p.status != nullptr) atomicOr(p.status, FLINT_DEVCHECK_INDEX);
    mine += pairs_of(q, pair);
  }
  long long at = block_scan<kThreads>(mine, s_warp, &n_pairs);
  // overlapping token ranges could promise more pairs than 32 bits count
  if (n_pairs > (1 << 30)) n_pairs = 0;
  for (int s = sb; s < se; ++s) {
    bool bad;
    first_pair[s] = static_cast<int>(min(at, 1ll << 30));
    at += pairs_of(chunk_seq(p, s, &bad), pair);
  }
  __syncthreads();
  // each thread a run of pairs: their length
  const int q_per = static_cast<int>((n_pairs + kThreads - 1) / kThreads);
  const int i0 = static_cast<int>(min(n_pairs, static_cast<long long>(tid) * q_per));
  const int i1 = static_cast<int>(min(n_pairs, static_cast<long long>(i0) + q_per));
  int s0 = 0;
  if (i0 < i1) {
    int hi = p.b.B;  // the last sequence whose pairs start at or before i0
    while (hi - s0 > 1) {
      const int mid = (s0 + hi) >> 1;
      if (first_pair[mid] <= i0) s0 = mid;
      else hi = mid;
    }
  }
  // f(sequence, first token, length) over the run, until it returns true
  auto walk = [&](auto&& f) {
    int s = s0;
    bool bad;
    PagedSeq q = chunk_seq(p, s, &bad);
    int tok = i0 < i1 ? (i0 - first_pair[s]) * pair : 0;
    for (int i = i0; i < i1; ++i) {
      while (q.kv <= 0 || tok >= q.n) {  // the next sequence with new tokens
        q = chunk_seq(p, ++s, &bad);
        tok = 0;
      }
      if (f(s, tok, pair_keys(q, tok, pair, p.window).length())) return;
      tok += pair;
    }
  };
  long long len = 0, total;
  int longest = 0;
  walk([&](int, int, int l) {
    len += l;
    longest = max(longest, l);
    return false;
  });
  longest = __reduce_max_sync(0xffffffffu, longest);
  if ((tid & 31) == 0 && longest != 0) atomicMax(&start->longest, longest);
  long long base = block_scan<kThreads>(len, s_warp, &total);
  *n_parts = static_cast<int>(min(static_cast<long long>(parts_per_head(p.Hkv)), (total + kMinPart - 1) / kMinPart));
  if (tid == 0) {
    start->total = total;
    start->n_pairs = static_cast<int>(n_pairs);
    start->deal = deal_whole(p.b.B, n_pairs, start->longest, total, *n_parts);
  }
  if (tid < kDealSeqs && tid < p.b.B) start->first_pair[tid] = first_pair[tid];
  if (part < *n_parts) {
    const long long a = total * part / *n_parts;
    if (a >= base && a < base + len)
      walk([&](int s, int tok, int l) {
        if (a < base + l) {
          start->base = base;
          start->s = s;
          start->tok0 = tok;
          return true;
        }
        base += l;
        return false;
      });
  }
  fence_async_smem();  // the scratch becomes a destination of TMA copies
  __syncthreads();
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
  Start start;
  long long scan[16];
  uint32_t tmem;
  volatile int abort_flag;
  float inv_sig[kE4M3 ? 2 : 1][2][kE4M3 ? kTile : 1];  // [item parity][tile][row]: 1 / Q scale
};

template <bool kE4M3>
constexpr size_t smem_bytes() {
  return 2 * kTileBytes + Cfg<kE4M3>::kStages * kTileBytes + Cfg<kE4M3>::kRaw * kRawBytes +
         sizeof(Ctl<kE4M3>);
}
static_assert(kMaxSeqs * sizeof(int) <= Cfg<false>::kStages * kTileBytes &&
                  kMaxSeqs * sizeof(int) <= Cfg<true>::kStages * kTileBytes + Cfg<true>::kRaw * kRawBytes,
              "find_start's scratch");
static_assert(smem_bytes<true>() <= 232448 && smem_bytes<false>() <= 232448, "shared memory");

// One 32-byte store (dst 32-byte aligned): whole sectors from a thread that owns a row.
__device__ __forceinline__ void store32(void* dst, const uint32_t (&r)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

template <int kRegs>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs)); }
template <int kRegs>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs)); }

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
  int* status = p.status != nullptr ? p.status : w.flags;
  const int g = blockIdx.x % p.Hkv, part = blockIdx.x / p.Hkv;

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
  pdl_wait();
  pdl_trigger();
  int n_parts;
  find_start<C::kThreads>(p, part, &n_parts, reinterpret_cast<int*>(skv), ctl.scan, &ctl.start);
  if (part >= n_parts && tid == 0 && g == 0) w.splits[part] = Split{-1, 0, 0, 0};
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
      // what is subtracted from the scores; rounded up, no f16 weight passes 2^(kGrow + kShift)
      auto base_of = [&](float mx) {
        if (mx == -INFINITY) return 0.f;
        return kE4M3 ? __fadd_ru(__fmul_ru(mx, c), -C::kShift) : mx * c;
      };
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
          const bool grow = (mn - m) * c > C::kGrow || (m == -INFINITY && mn > m);
          if (__any_sync(0xffffffffu, grow)) {
            // P V of the previous tile has to be in O before O is rescaled
            if (!(ok = mma_wait(&ctl.o_done[t], (cnt - 1) & 1, ab, status))) break;
            tc_fence_after();
            const float mu = fmaxf(m, mn);
            const float f = m == -INFINITY ? 0.f : exp2_ftz(base_of(m) - base_of(mu));
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
        const float base = base_of(m);
        const f32x2 c2 = pack2(c, c), mc2 = pack2(-base, -base);
        // The sum is of the fp32 weights; adding them as rounded, as the decode kernel does, would take two more
        // instructions a pair. Either is within the weights' rounding.
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
          const float f = (l == 0.f ? 0.f : 1.f / l) * (kE4M3 ? __ldg(p.v_scale + im.g) : 1.f);
          uint16_t* dst =
              p.out + (static_cast<size_t>(im.row0 + im.tok0 + tok) * p.Hq + im.g * p.group + row % p.group) * kDh;
          // out is 16-byte aligned: 32-byte stores where it is 32-byte aligned too
          const bool wide = (reinterpret_cast<uintptr_t>(dst) & 31u) == 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint32_t r[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const __nv_bfloat162 v = __floats2bfloat162_rn(o[16 * i + 2 * j] * f, o[16 * i + 2 * j + 1] * f);
              r[j] = *reinterpret_cast<const uint32_t*>(&v);
            }
            if (wide) {
              store32(dst + 16 * i, r);
            } else {
              reinterpret_cast<uint4*>(dst)[2 * i] = make_uint4(r[0], r[1], r[2], r[3]);
              reinterpret_cast<uint4*>(dst)[2 * i + 1] = make_uint4(r[4], r[5], r[6], r[7]);
            }
          }
        } else {
          const size_t at = static_cast<size_t>(im.slot) * rows_per_slot + t * kTile + row;
          *reinterpret_cast<float2*>(w.ml + at * 2) = make_float2(m == -INFINITY ? -INFINITY : base_of(m), l);
          float* dst = w.po + at * kDh;  // 256-byte aligned in a workspace that is 32-byte aligned
          const bool wide = (reinterpret_cast<uintptr_t>(dst) & 31u) == 0;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            uint32_t r[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) r[j] = __float_as_uint(o[8 * i + j]);
            if (wide) {
              store32(dst + 8 * i, r);
            } else {
              reinterpret_cast<uint4*>(dst)[2 * i] = make_uint4(r[0], r[1], r[2], r[3]);
              reinterpret_cast<uint4*>(dst)[2 * i + 1] = make_uint4(r[4], r[5], r[6], r[7]);
            }
          }
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
    const int ps = 1 << p.b.page_shift;
    const int box = min(ps, kTile), n_box = kTile / box;
    const int my_box = kE4M3 ? lane : lane >> 1, half = kE4M3 ? 0 : lane & 1;
    const bool mine = my_box < n_box;
    const int bad_row = static_cast<int>(p.b.n_pages << p.b.page_shift);  // past the pool: zeros
    const uint32_t box_bytes = box * (kE4M3 ? kDh : kDh * 2);
    uint32_t li = 0, qn[2] = {0, 0};
    constexpr int kRing = kE4M3 ? C::kRaw : C::kStages;
    bool ok = true;
    // the part [pos, end) of the line; the pair at its first place
    const int pair = 2 * tok_t;
    const long long total = ctl.start.total;
    long long base = ctl.start.base, pos = part < n_parts ? total * part / n_parts : 0,
              end = part < n_parts ? total * (part + 1) / n_parts : 0;
    int s = ctl.start.s, tok0 = ctl.start.tok0;
    bool bad;
    PagedSeq q{0, 0, 0};
    const bool deal = ctl.start.deal != 0 && part < n_parts;
    if (!deal && pos < end) q = chunk_seq(p, s, &bad);
    Split left{-1, 0, 0, 0};
    for (int it = 0; ok; ++it) {
      Item im{};
      im.end = 1;
      if (deal) {
        const int i = ctl.start.n_pairs - 1 - (it * n_parts + ((it & 1) ? n_parts - 1 - part : part));
        if (i >= 0) {
          s = 0;
          for (int x = 1; x < p.b.B; ++x)
            if (ctl.start.first_pair[x] <= i) s = x;
          q = chunk_seq(p, s, &bad);
          tok0 = (i - ctl.start.first_pair[s]) * pair;
          const Keys k = pair_keys(q, tok0, pair, p.window);
          im.row0 = q.row0;
          im.tok0 = tok0;
          im.live = min(q.n - tok0, pair);
          im.n = q.n;
          im.kv = q.kv;
          im.kt0 = k.kt0;
          im.kt1 = k.kt1;
          im.g = g;
          im.slot = -1;
          im.s = s;
          im.end = 0;
        }
      } else if (pos < end) {
        while (tok0 >= q.n || q.kv <= 0) {  // the next sequence with new tokens
          q = chunk_seq(p, ++s, &bad);
          tok0 = 0;
        }
        const Keys k = pair_keys(q, tok0, pair, p.window);
        const int len = k.length();
        // a boundary within a pair's first kFill places is one in front of it
        if (pos - base <= kFill) pos = base;
        if (end > base + kFill) {
          const bool whole = pos == base && end >= base + len, goes_on = end < base + len;
          im.row0 = q.row0;
          im.tok0 = tok0;
          im.live = min(q.n - tok0, pair);
          im.n = q.n;
          im.kv = q.kv;
          im.kt0 = k.kt0 + (pos == base ? 0 : static_cast<int>(pos - base) - kFill);
          im.kt1 = goes_on ? k.kt0 + static_cast<int>(end - base) - kFill : k.kt1;
          im.g = g;
          im.slot = whole ? -1 : static_cast<int>(slot_of(part, p.Hkv, g, goes_on));
          im.s = s;
          im.end = 0;
          if (goes_on && pos == base)  // ends in the part that holds the pair's last place
            left = Split{s, tok0, part, static_cast<int>(((base + len) * n_parts - 1) / total)};
          pos = base += len;
          tok0 += pair;
        }
      }
      if (!(ok = mma_wait(&ctl.it_empty[it & 1], ((it >> 1) & 1) ^ 1, ab, status))) break;
      if (lane == 0) {
        ctl.item[it & 1] = im;
        mbar_arrive(&ctl.it_full[it & 1]);
      }
      __syncwarp();
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
      // pool row of this lane's box of key tile kt, -1 past the sequence; a box
      // wholly in front of the pair's window is zeros (its page may be gone)
      const int reach = p.window > 0 ? im.kv - im.n + im.tok0 - p.window + 1 : 0;
      auto box_row = [&](int kt) {
        const int key = kt * kTile + my_box * box;
        if (!mine || kt >= im.kt1 || key >= im.kv) return -1;
        if (key + box <= reach) return bad_row;
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
    if (lane == 0 && g == 0 && part < n_parts) w.splits[part] = left;
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

// Joins the pieces of the pairs that parts cut, in key order: a CTA takes 32
// rows of the pair that one part left unfinished in one kv head, a warp four of
// them at once. The last CTA writes zeros for the tokens of invalid sequences.
constexpr int kCombineThreads = 256;
constexpr int kCombineRows = 4 * kCombineThreads / 32;

__global__ void __launch_bounds__(kCombineThreads) k_chunk_combine(PagedAttnParams p, Ws w, int rows_per_slot) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x + 1 == gridDim.x) {
    for (int s = warp; s < p.b.B; s += kCombineThreads / 32) {
      bool bad;
      const PagedSeq q = chunk_seq(p, s, &bad);
      if (q.n <= 0 || q.kv > 0) continue;
      uint4* dst = reinterpret_cast<uint4*>(p.out + static_cast<size_t>(q.row0) * p.Hq * kDh);
      const long long m = static_cast<long long>(q.n) * p.Hq * (kDh / 8);
      for (long long i = lane; i < m; i += 32) dst[i] = make_uint4(0, 0, 0, 0);
    }
    return;
  }
  const int blocks = rows_per_slot / kCombineRows;
  const int x = blockIdx.x / blocks, part = x / p.Hkv, g = x - part * p.Hkv;
  const int4 sv = __ldcg(reinterpret_cast<const int4*>(w.splits + part));
  if (sv.x < 0) return;
  const Split sp{sv.x, sv.y, sv.z, sv.w};
  const int tok_t = kTile / p.group;
  bool bad;
  const PagedSeq q = chunk_seq(p, sp.s, &bad);
  const int r0 = (blockIdx.x - x * blocks) * kCombineRows + 4 * warp;
  float M[4], l[4];
  float4 acc[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    M[i] = -INFINITY;
    l[i] = 0.f;
    acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
#pragma unroll 2
  for (int k = sp.first; k <= sp.last; ++k) {
    const size_t at = slot_of(k, p.Hkv, g, k < sp.last) * rows_per_slot + r0;
    float2 ml[4];
    float4 o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      ml[i] = __ldcg(reinterpret_cast<const float2*>(w.ml + (at + i) * 2));
      o[i] = __ldcg(reinterpret_cast<const float4*>(w.po + (at + i) * kDh) + lane);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // rows past the pair's tokens were not written: what is read for them is dropped below. A piece without a
      // maximum (-inf) adds zeros, or the NaN of a query.
      const float mx = fmaxf(M[i], ml[i].x);
      const float f0 = M[i] == -INFINITY ? 0.f : exp2_ftz(M[i] - mx);
      const float f1 = ml[i].x == -INFINITY ? 0.f : exp2_ftz(ml[i].x - mx);
      M[i] = mx;
      l[i] = fmaf(l[i], f0, ml[i].y * f1);
      acc[i].x = fmaf(acc[i].x, f0, o[i].x * f1);
      acc[i].y = fmaf(acc[i].y, f0, o[i].y * f1);
      acc[i].z = fmaf(acc[i].z, f0, o[i].z * f1);
      acc[i].w = fmaf(acc[i].w, f0, o[i].w * f1);
    }
  }
  const float vs = p.v_scale != nullptr ? __ldg(p.v_scale + g) : 1.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + i, rt = r % kTile, tok = sp.tok0 + (r / kTile) * tok_t + rt / p.group;
    if (rt >= tok_t * p.group || tok >= q.n) continue;
    const float f = (l[i] == 0.f ? 0.f : 1.f / l[i]) * vs;
    const __nv_bfloat162 a = __floats2bfloat162_rn(acc[i].x * f, acc[i].y * f),
                         b = __floats2bfloat162_rn(acc[i].z * f, acc[i].w * f);
    reinterpret_cast<uint2*>(p.out + (static_cast<size_t>(q.row0 + tok) * p.Hq + g * p.group + rt % p.group) * kDh)[lane] =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
}

}  // namespace

size_t paged_chunk_workspace(int n_q_heads, int n_kv_heads, int max_q) {
  Ws w;
  return carve(&w, nullptr, n_kv_heads, slot_rows(max_q, n_q_heads / n_kv_heads));
}

int paged_chunk_launch(const PagedAttnParams& p, int cache_dtype, size_t ws_bytes, cudaStream_t st) {
  const bool e4m3 = cache_dtype == FLINT_KV_E4M3;
  const int rows = slot_rows(p.max_q, p.group);
  Ws w;
  const size_t need = carve(&w, p.ws, p.Hkv, rows);
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
  const int grid = parts_per_head(p.Hkv) * p.Hkv;
  e = e4m3 ? launch_pdl(k_paged_chunk<true>, grid, Cfg<true>::kThreads, smem_bytes<true>(), st, mq, mk, mv, p, w, rows)
           : launch_pdl(k_paged_chunk<false>, grid, Cfg<false>::kThreads, smem_bytes<false>(), st, mq, mk, mv, p, w,
                        rows);
  if (e == cudaSuccess)
    e = launch_pdl(k_chunk_combine, grid * (rows / kCombineRows) + 1, kCombineThreads, 0, st, p, w, rows);
  if (e != cudaSuccess) return flint_fail_external(FLINT_ERR_CUDA, cudaGetErrorString(e));
  return FLINT_OK;
}

}  // namespace flint
