// paged_decode.cu -- attention of few new tokens per sequence (tokens x query
// heads per kv head <= 16, the rows of one register-fragment MMA tile) over the
// paged cache ("[Model] Add Flint (RecursiveSI/flint)", section "What
// happened": the attention step of the per-layer decode chain; heads from
// "Recursive Flint: 125 tok/s on an M4 Pro", architecture table).
//
//   o = sum_j w_j v_j,  w = softmax_j(scale q . k_j), j in the token's range
//
// HBM-bound: each cached row is read once per kv head (512 bytes of bf16 key
// and value, 256 of E4M3), so the split is over keys and is even: the keys of
// all sequences, in quanta of 64, form one line that G = 296 / Hkv CTAs per kv
// head cut into equal parts (2 CTAs per SM). A CTA walks its part sequence by
// sequence. A sequence wholly inside one part is finished there; one that
// spans parts leaves a (max, sum, O) partial per part -- at most two per CTA,
// at its part's ends -- that k_paged_combine joins in part order. The cut is
// made on the device from the lengths it finds there, so a captured graph
// stays balanced when the lengths change.
//
// Inside a part the four warps take a quarter of the keys each, streaming
// blocks of 16 keys through a cp.async ring; page ids are read 32 at a time,
// one batch ahead. Rows of a block past the end are filled with zeros, so
// whatever an unused cache row holds never reaches the sums.
// The products are taken transposed, keys and dimensions as the 16 rows of an
// MMA and the query rows as its 8 columns (two column tiles above 8 rows), so
// that no half of a tile is empty for a group of 8:
//   S^T [16 keys][8] = K Q^T      8 MMAs per 16 keys
//   O^T [16 dims][8] += V^T P^T   8 MMAs, P^T by movmatrix from S^T's layout
//   bf16 cache: K by ldmatrix on key rows, V by ldmatrix.trans (rows padded to
//     272 bytes: conflict-free), P rounded to bf16.
//   E4M3 cache: codes become f16 (exact) on the way into the fragments. The
//     order of the 128 terms of q . k and of the output's dimensions is free, so
//     a thread reads 16-byte runs of a key row (K) and 16-byte runs of the four
//     keys it holds weights for (V) and needs no transpose; Q is f16 after an
//     exact power-of-two scale per row, P is f16 times 2^15 (kShift), so that
//     weights down to 2^-29 of the largest keep f16's 11 bits (unshifted: 2^-14;
//     the keys behind a dominating one, as attention sinks are, lost theirs).
//     128-byte rows whose 16-byte pieces are permuted by the row number
//     (piece_of): conflict-free for both reads without padding.
// (Query rows as the 16 rows of a tile: twice the MMAs and accumulators; 8 x
// 32K of E4M3 58.9 us against 53.5, 64 ragged bf16 sequences 98.8 with both.)
// 8 x 32K of E4M3: 4.8 TB/s from a graph, 4.7 call by call. Two blocks a step
// 53.9 us, three CTAs an SM 53.8 (both 52.9): the warps then wait for memory,
// and the SMs are active for 80 to 88 % of the kernel's time.
// A last 3/16 of the line in short parts for whichever SM comes free gives bf16
// batches 0 to 4 % (64 ragged sequences 97.3 -> 95.2 us) and costs E4M3 12 %
// (53.8 -> 60.5): not kept.
// The running sum adds the rounded weights, so the output stays a convex
// combination of the values.
#include "paged_attn.cuh"

namespace flint {
namespace {

constexpr int kDh = kPagedHeadDim;
constexpr int kWarps = 4;
constexpr int kBlock = 16;
constexpr int kQuantum = kWarps * kBlock;
constexpr int kCtaSlots = 2 * 148;  // two CTAs per SM
constexpr int kRowsMax = kDecodeRows;
constexpr float kShift = 15.f;         // log2 of the largest weight in f16 (65,504 is the type's largest number)

template <bool kE4M3>
struct Ring;
template <>
struct Ring<false> {
  static constexpr int kStages = 3;
  static constexpr int kRowBytes = (kDh + 8) * 2;
};
template <>
struct Ring<true> {
  static constexpr int kStages = 6;
  static constexpr int kRowBytes = kDh;
};
template <bool kE4M3>
constexpr int stage_bytes() { return 2 * kBlock * Ring<kE4M3>::kRowBytes; }
template <bool kE4M3>
constexpr int ring_bytes() { return Ring<kE4M3>::kStages * stage_bytes<kE4M3>(); }

__device__ __forceinline__ uint32_t bf2(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr));
}
// 8 x 8 transpose of 16-bit values across the warp (a thread's register: row lane / 4, columns 2 (lane % 4) ..)
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
template <bool kF16>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (kF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void cp16z(uint32_t dst, const void* src, int src_bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}

// Place of 16-byte piece c of an E4M3 row: key reads (rows 2i, 2i + 1, half a
// row each) and value reads (rows 0, 2, 4, 6, two pieces each) hit all banks once.
__device__ __forceinline__ uint32_t piece_of(int r, int c) {
  return static_cast<uint32_t>(c ^ ((((r >> 1) & 3) << 1) ^ ((r & 1) << 2))) << 4;
}

// Place of dimension d of row r where the warps meet: the four row pairs that a
// warp stores at once take different banks.
template <bool kE4M3>
__device__ __forceinline__ int met_at(int r, int d) { return d ^ (((r >> 1) & 3) * (kE4M3 ? 4 : 8)); }

// A sequence on the line: its keys [first, kv) in quanta of 64.
struct Line {
  PagedSeq sq;
  int first, quanta;
};
__device__ __forceinline__ Line line_of(const PagedAttnParams& p, int s, bool record) {
  Line r;
  bool bad;
  r.sq = paged_seq(p.b, s, &bad);
  if (r.sq.n > p.max_q) {
    bad = true;
    r.sq.kv = 0;
  }
  if (bad && record && p.status != nullptr) atomicOr(p.status, FLINT_DEVCHECK_INDEX);
  r.first = paged_first_key(r.sq.kv, r.sq.n, p.window);
  r.quanta = (r.sq.n > 0 && r.sq.kv > 0) ? (r.sq.kv - r.first + kQuantum - 1) / kQuantum : 0;
  return r;
}

// Workspace: the line's prefix sums (one per sequence, then the total), then
// two partials per CTA: (max, sum) per row, O per row.
struct Ws {
  long long* pre;
  float* ml;
  float* po;
};
__host__ __device__ inline size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
__host__ __device__ inline int ctas_per_head(int Hkv) { return Hkv >= kCtaSlots ? 1 : kCtaSlots / Hkv; }
// Partials; a kv head of one CTA cuts no sequence.
__host__ __device__ inline size_t slots_of(int Hkv) {
  const int g = ctas_per_head(Hkv);
  return g > 1 ? static_cast<size_t>(g) * Hkv * 2 : 0;
}
__host__ __device__ inline Ws carve(char* ws, int B, int Hkv) {
  Ws w;
  const size_t slots = slots_of(Hkv);
  w.pre = reinterpret_cast<long long*>(ws);
  ws += up256((static_cast<size_t>(B) + 1) * sizeof(long long));
  w.ml = reinterpret_cast<float*>(ws);
  ws += up256(slots * kRowsMax * 2 * sizeof(float));
  w.po = reinterpret_cast<float*>(ws);
  return w;
}

// Parts: CTA i of n takes quanta [W i / n, W (i + 1) / n); n <= W, so none is empty.
__device__ __forceinline__ int parts_of(long long W, int Hkv) {
  const int g = ctas_per_head(Hkv);
  return W < g ? static_cast<int>(W) : g;
}

template <bool kE4M3, bool kTall>
__global__ void __launch_bounds__(kWarps * 32, 2) k_paged_decode(PagedAttnParams p) {
  using R = Ring<kE4M3>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float s_m[kWarps][kRowsMax], s_l[kWarps][kRowsMax];
  __shared__ long long s_sum[kWarps], s_pre;
  __shared__ int s_seq;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = blockIdx.x % p.Hkv, part = blockIdx.x / p.Hkv;
  const Ws ws = carve(p.ws, p.b.B, p.Hkv);
  pdl_wait();
  pdl_trigger();

  // ---- the line: thread j sums a run of sequences, the block scans the sums
  const int per = (p.b.B + kWarps * 32 - 1) / (kWarps * 32);
  const int sb = min(p.b.B, tid * per), se = min(p.b.B, sb + per);
  const bool lead = blockIdx.x == 0;
  long long mine = 0;
  for (int s = sb; s < se; ++s) mine += line_of(p, s, lead).quanta;
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) s_sum[warp] = inc;
  __syncthreads();
  long long W = 0, pre = inc - mine;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) pre += s_sum[w];
    W += s_sum[w];
  }
  if (lead) {
    long long a = pre;
    for (int s = sb; s < se; ++s) {
      ws.pre[s] = a;
      a += line_of(p, s, false).quanta;
    }
    if (tid == 0) ws.pre[p.b.B] = W;
  }
  const int n_parts = parts_of(W, p.Hkv);
  if (part >= n_parts) return;
  long long a = W * part / n_parts;
  const long long a_end = W * (part + 1) / n_parts;
  if (a >= pre && a < pre + mine) {
    long long x = pre;
    for (int s = sb; s < se; ++s) {
      const int q = line_of(p, s, false).quanta;
      if (a < x + q) {
        s_seq = s;
        s_pre = x;
        break;
      }
      x += q;
    }
  }
  __syncthreads();
  int s = s_seq;
  long long base = s_pre;  // the line position of sequence s

  const int gq = lane >> 2, t4 = lane & 3;
  const uint32_t ring = smem_addr(smem) + warp * ring_bytes<kE4M3>();
  const int es = kE4M3 ? 1 : 2;  // bytes per element
  const size_t row_stride = static_cast<size_t>(p.Hkv) * kDh * es;
  const uint8_t* kp = static_cast<const uint8_t*>(p.k) + static_cast<size_t>(g) * kDh * es;
  const uint8_t* vp = static_cast<const uint8_t*>(p.v) + static_cast<size_t>(g) * kDh * es;
  const int page_mask = (1 << p.b.page_shift) - 1;

  while (a < a_end) {
    const Line ln = line_of(p, s, false);
    if (a >= base + ln.quanta) {
      base += ln.quanta;
      ++s;
      continue;
    }
    const int q0 = static_cast<int>(a - base);
    const int q1 = static_cast<int>(min(a_end - base, static_cast<long long>(ln.quanta)));
    const int n = ln.sq.n, kv = ln.sq.kv;
    const int k0 = ln.first + q0 * kQuantum, k1 = min(kv, ln.first + q1 * kQuantum);
    const int per_warp = (q1 - q0) * kBlock;
    const int w0 = min(k1, k0 + warp * per_warp), w1 = min(k1, w0 + per_warp);
    const int n_blocks = (w1 - w0 + kBlock - 1) / kBlock;

    // ---- page ids of the warp's run, 32 pages a batch, one batch ahead
    const int32_t* table = p.b.block_table + static_cast<size_t>(s) * p.b.max_pages;
    const int pg_last = w1 > w0 ? (w1 - 1) >> p.b.page_shift : 0;
    int pg_base = w0 >> p.b.page_shift;
    auto page_batch = [&](int b0) {
      const int i = b0 + lane;
      if (n_blocks == 0 || i > pg_last) return -1;
      const int page = __ldg(table + i);
      const bool ok = page >= 0 && page < p.b.n_pages;
      if (!ok && p.status != nullptr) atomicOr(p.status, FLINT_DEVCHECK_INDEX);
      return ok ? page : -1;
    };
    int pg_cur = page_batch(pg_base), pg_nxt = page_batch(pg_base + 32);
    auto load_block = [&](int b) {
      const int kb = w0 + b * kBlock;
      const int i = kb >> p.b.page_shift;
      if (i - pg_base >= 32) {
        pg_base += 32;
        pg_cur = pg_nxt;
        pg_nxt = page_batch(pg_base + 32);
      }
      const int page = __shfl_sync(0xffffffffu, pg_cur, i - pg_base);
      const uint32_t st = ring + (b % R::kStages) * stage_bytes<kE4M3>();
      const size_t off =
          ((static_cast<size_t>(max(page, 0)) << p.b.page_shift) + (kb & page_mask)) * row_stride;
      if constexpr (kE4M3) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int c = lane + 32 * x, r = c >> 3, piece = c & 7;
          const int in = page >= 0 && kb + r < w1 ? 16 : 0;
          const size_t src = off + (in ? r * row_stride : 0) + piece * 16;
          const uint32_t dst = st + r * kDh + piece_of(r, piece);
          cp16z(dst, kp + src, in);
          cp16z(dst + kBlock * kDh, vp + src, in);
        }
      } else {
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const int c = lane + 32 * x, r = c >> 4, piece = c & 15;
          const int in = page >= 0 && kb + r < w1 ? 16 : 0;
          const size_t src = off + (in ? r * row_stride : 0) + piece * 16;
          const uint32_t dst = st + r * R::kRowBytes + piece * 16;
          cp16z(dst, kp + src, in);
          cp16z(dst + kBlock * R::kRowBytes, vp + src, in);
        }
      }
    };
#pragma unroll
    for (int b = 0; b < R::kStages - 1; ++b) {
      if (b < n_blocks) load_block(b);
      cp_commit();
    }

    // ---- Q^T fragments: this lane's column gq of column tile x is row 8 x + gq; row r is token r / group, head r %
    // group. Softmax state: rows 8 x + 2 t4 + {0, 1}, as in the accumulators.
    constexpr int kNt = kTall ? 2 : 1;
    uint32_t qb[8][kNt][2];
    float sc[kNt][2];
    int lim[kNt][2];  // keys below lim and from lim - window on are attended
#pragma unroll
    for (int x = 0; x < kNt; ++x) {
      const int r = gq + 8 * x;
      const int tok = r / p.group, h = r - tok * p.group;
      const bool live = tok < n;
      const uint16_t* qh =
          p.q + (static_cast<size_t>(ln.sq.row0 + (live ? tok : 0)) * p.Hq + g * p.group + (live ? h : 0)) * kDh;
      float scale = p.scale * kLog2e;
      if constexpr (kE4M3) {
        uint4 w[4];  // 64h + 16 t4 + 0..7 and 8..15 of both halves
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = live ? __ldg(reinterpret_cast<const uint4*>(qh + 64 * (i >> 1) + 16 * t4 + 8 * (i & 1)))
                      : make_uint4(0, 0, 0, 0);
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(u[j] << 16)), fabsf(__uint_as_float(u[j] & 0xFFFF0000u))));
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const float sig = pow2_scale_for(amax);
        scale = scale * __ldg(p.k_scale + g) / sig;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
          uint32_t f[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            f[j] = pack_f16x2(__uint_as_float(u[j] << 16) * sig, __uint_as_float(u[j] & 0xFFFF0000u) * sig);
          // k-step 4 (i / 2) + 2 (i % 2) + {0, 1}: elements 4w .. 4w + 3 of the run
          const int ks = 4 * (i >> 1) + 2 * (i & 1);
          qb[ks][x][0] = f[0];
          qb[ks][x][1] = f[1];
          qb[ks + 1][x][0] = f[2];
          qb[ks + 1][x][1] = f[3];
        }
      } else {
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          qb[ks][x][0] = live ? __ldg(reinterpret_cast<const uint32_t*>(qh + 16 * ks + 2 * t4)) : 0u;
          qb[ks][x][1] = live ? __ldg(reinterpret_cast<const uint32_t*>(qh + 16 * ks + 8 + 2 * t4)) : 0u;
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int ri = 8 * x + 2 * t4 + i, ti = ri / p.group;
        sc[x][i] = __shfl_sync(0xffffffffu, scale, (2 * t4 + i) * 4);
        lim[x][i] = ti < n ? kv - n + ti + 1 : 0;
      }
    }
    float m[kNt][2], l[kNt][2];  // l: this lane's keys only, until the end
    float o[8][kNt][4];
#pragma unroll
    for (int x = 0; x < kNt; ++x) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        m[x][i] = -INFINITY;
        l[x][i] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[j][x][c] = 0.f;
    }

    for (int b = 0; b < n_blocks; ++b) {
      if (b + R::kStages - 1 < n_blocks) load_block(b + R::kStages - 1);
      cp_commit();
      cp_wait<R::kStages - 1>();
      __syncwarp();
      const uint32_t kr = ring + (b % R::kStages) * stage_bytes<kE4M3>();
      const uint32_t vr = kr + kBlock * R::kRowBytes;
      // two accumulators a column tile: shorter chains
      float st[kNt][2][4];
#pragma unroll
      for (int x = 0; x < kNt; ++x)
#pragma unroll
        for (int c = 0; c < 4; ++c) st[x][0][c] = st[x][1][c] = 0.f;
      if constexpr (kE4M3) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          // key rows gq and gq + 8 (permuted alike): the run of 16 codes at 64 half + 16 t4
          const uint32_t at = piece_of(gq, 4 * half + t4);
          const uint4 ka = lds16(kr + gq * kDh + at), kc = lds16(kr + (gq + 8) * kDh + at);
          const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wc[4] = {kc.x, kc.y, kc.z, kc.w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t a[4] = {e4m3x2_to_f16x2(wa[w]), e4m3x2_to_f16x2(wc[w]), e4m3x2_to_f16x2(wa[w] >> 16),
                                   e4m3x2_to_f16x2(wc[w] >> 16)};
#pragma unroll
            for (int x = 0; x < kNt; ++x)
              mma16<true>(st[x][w & 1], a, qb[4 * half + w][x][0], qb[4 * half + w][x][1]);
          }
        }
      } else {
        // matrices: (keys 0-7, dims 0-7), (keys 8-15, dims 0-7), (keys 0-7, dims 8-15), (keys 8-15, dims 8-15)
        const int mr = (lane & 7) + ((lane >> 3) & 1) * 8, mc = (lane >> 4) * 16;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          uint32_t a[4];
          ldsm4(kr + mr * R::kRowBytes + 32 * ks + mc, a[0], a[1], a[2], a[3]);
#pragma unroll
          for (int x = 0; x < kNt; ++x) mma16<false>(st[x][ks & 1], a, qb[ks][x][0], qb[ks][x][1]);
        }
      }
      // this lane: keys gq (c 0, 1) and gq + 8 (c 2, 3) of rows 8 x + 2 t4 + {0, 1}
      const int kb = w0 + b * kBlock;
      const bool edge = kb + kBlock > min(w1, kv - n + 1) || (p.window > 0 && kb < kv - p.window);
      uint32_t pb[kNt][2];
      float alpha[kNt][2];
      bool moved = false;
#pragma unroll
      for (int x = 0; x < kNt; ++x) {
        float v[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] = (st[x][0][c] + st[x][1][c]) * sc[x][c & 1];
        if (edge) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int key = kb + gq + 8 * (c >> 1), hi = min(lim[x][c & 1], w1);
            if (key >= hi || (p.window > 0 && key < lim[x][c & 1] - p.window)) v[c] = -INFINITY;
          }
        }
        float e[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float bm = fmaxf(v[i], v[2 + i]);
          bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 4));
          bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 8));
          bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 16));
          // what is subtracted from the scores stands for the maximum; rounded up, no weight passes 2^kShift
          if constexpr (kE4M3) bm = __fadd_ru(bm, -kShift);
          const float mn = fmaxf(m[x][i], bm);
          const float ms = mn == -INFINITY ? 0.f : mn;  // a row that has seen no key yet
          alpha[x][i] = exp2_ftz(m[x][i] - ms);
          moved = moved || mn != m[x][i];
          m[x][i] = mn;
          e[i] = exp2_ftz(v[i] - ms);
          e[2 + i] = exp2_ftz(v[2 + i] - ms);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {  // keys gq + 8 k
          uint32_t pk;
          float p0, p1;
          if constexpr (kE4M3) {
            // 11 significant bits; weights below 2^-40 of the largest vanish
            pk = pack_f16x2(e[2 * k], e[2 * k + 1]);
            const float2 u = __half22float2(*reinterpret_cast<const __half2*>(&pk));
            p0 = u.x;
            p1 = u.y;
          } else {
            pk = bf2(e[2 * k], e[2 * k + 1]);
            p0 = __uint_as_float(pk << 16);
            p1 = __uint_as_float(pk & 0xFFFF0000u);
          }
          l[x][0] = k == 0 ? fmaf(l[x][0], alpha[x][0], p0) : l[x][0] + p0;
          l[x][1] = k == 0 ? fmaf(l[x][1], alpha[x][1], p1) : l[x][1] + p1;
          pb[x][k] = transpose8(pk);
        }
      }
      // the maxima rarely move after the first blocks
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int x = 0; x < kNt; ++x)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[j][x][c] *= alpha[x][c & 1];
      }
      if constexpr (kE4M3) {
        // codes 16 gq .. 16 gq + 15 of keys 2 t4, 2 t4 + 1, 8 + 2 t4, 9 + 2 t4: rows gq and gq + 8 of MMA tile j are
        // dimensions 16 gq + 2 j and 16 gq + 2 j + 1
        const uint32_t pe = piece_of(2 * t4, gq), po = piece_of(2 * t4 + 1, gq);
        const uint4 v0 = lds16(vr + (2 * t4) * kDh + pe), v1 = lds16(vr + (2 * t4 + 1) * kDh + po);
        const uint4 v2 = lds16(vr + (8 + 2 * t4) * kDh + pe), v3 = lds16(vr + (9 + 2 * t4) * kDh + po);
        const uint32_t a0[4] = {v0.x, v0.y, v0.z, v0.w}, a1[4] = {v1.x, v1.y, v1.z, v1.w};
        const uint32_t a2[4] = {v2.x, v2.y, v2.z, v2.w}, a3[4] = {v3.x, v3.y, v3.z, v3.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) {  // bytes 2 (j % 2), 2 (j % 2) + 1 of both keys of a pair
          const uint32_t x0 = __byte_perm(a0[j >> 1], a1[j >> 1], j & 1 ? 0x7362 : 0x5140);
          const uint32_t x1 = __byte_perm(a2[j >> 1], a3[j >> 1], j & 1 ? 0x7362 : 0x5140);
          const uint32_t a[4] = {e4m3x2_to_f16x2(x0), e4m3x2_to_f16x2(x0 >> 16), e4m3x2_to_f16x2(x1),
                                 e4m3x2_to_f16x2(x1 >> 16)};
#pragma unroll
          for (int x = 0; x < kNt; ++x) mma16<true>(o[j][x], a, pb[x][0], pb[x][1]);
        }
      } else {
        // matrices: (keys 0-7, dims 0-7), (keys 0-7, dims 8-15), (keys 8-15, dims 0-7), (keys 8-15, dims 8-15)
        const int vrow = (lane & 7) + (lane >> 4) * 8, vcol = ((lane >> 3) & 1) * 16;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          uint32_t a[4];
          ldsm4t(vr + vrow * R::kRowBytes + 32 * j + vcol, a[0], a[1], a[2], a[3]);
#pragma unroll
          for (int x = 0; x < kNt; ++x) mma16<false>(o[j][x], a, pb[x][0], pb[x][1]);
        }
      }
      __syncwarp();
    }
    cp_wait<0>();
    __syncwarp();

    // ---- the warps meet: (max, sum, O) of each through its own ring
    float* s_o = reinterpret_cast<float*>(smem + warp * ring_bytes<kE4M3>());
#pragma unroll
    for (int x = 0; x < kNt; ++x) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 8 * x + 2 * t4 + i;
        float sum = l[x][i];
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        if (gq == 0) {
          s_m[warp][r] = m[x][i];
          s_l[warp][r] = sum;
        }
        if constexpr (kE4M3) {
#pragma unroll
          for (int j = 0; j < 8; j += 2)
            *reinterpret_cast<float4*>(s_o + r * kDh + met_at<kE4M3>(r, 16 * gq + 2 * j)) =
                make_float4(o[j][x][i], o[j][x][2 + i], o[j + 1][x][i], o[j + 1][x][2 + i]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            s_o[r * kDh + met_at<kE4M3>(r, 16 * j + gq)] = o[j][x][i];
            s_o[r * kDh + met_at<kE4M3>(r, 16 * j + gq + 8)] = o[j][x][2 + i];
          }
        }
      }
    }
    __syncthreads();
    const bool whole = q0 == 0 && q1 == ln.quanta;
    const size_t slot = (static_cast<size_t>(part) * p.Hkv + g) * 2 + (q1 < ln.quanta ? 1 : 0);
    const float vs = kE4M3 ? __ldg(p.v_scale + g) : 1.f;
    const int rows = n * p.group;
    for (int r = 0; r < rows; ++r) {  // thread d owns dimension d
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][r]);
      float tot = 0.f, acc = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = s_m[w][r] == -INFINITY ? 0.f : exp2_ftz(s_m[w][r] - M);
        tot = fmaf(s_l[w][r], f, tot);
        const float* o_w = reinterpret_cast<const float*>(smem + w * ring_bytes<kE4M3>()) + r * kDh;
        acc = fmaf(o_w[met_at<kE4M3>(r, tid)], f, acc);
      }
      if (whole) {
        const int tok = r / p.group, h = r - tok * p.group;
        // a sum of 0: the row saw no key. NaN (from the query) stays.
        const __nv_bfloat16 bv = __float2bfloat16_rn(tot == 0.f ? 0.f : acc / tot * vs);
        p.out[(static_cast<size_t>(ln.sq.row0 + tok) * p.Hq + g * p.group + h) * kDh + tid] =
            *reinterpret_cast<const uint16_t*>(&bv);
      } else {
        if (tid == 0) *reinterpret_cast<float2*>(ws.ml + (slot * kRowsMax + r) * 2) = make_float2(M, tot);
        ws.po[(slot * kRowsMax + r) * kDh + tid] = acc;
      }
    }
    __syncthreads();  // the rings are free again
    a = base + q1;
  }
}

// Joins the partials of the sequences that parts cut, in part order, and writes
// zeros for sequences whose tokens see nothing. Two forms:
//   kByRow: a CTA per (kv head, sequence), a warp per row of the tile. For
//     batches: few sequences are cut, into two or three parts, and what counts
//     is how fast the CTAs of the others are gone.
//   else: a CTA per (query head, sequence), its warps sharing the parts, eight
//     partials in flight each. For a few long sequences cut into many parts.
// 64 sequences of up to 8,192: 106 us in the second form, 97 in the first.
constexpr int kCombineWarps = 8;
constexpr int kCombineBatch = 8;

struct Joined {
  float m, l;
  float4 o;
};
// Partials of row r in parts c0, c0 + step, ... up to i1; lane: four dimensions. A partial without a maximum (-inf)
// adds its sums times 0: zeros of a row that saw no key there, or the NaN of a query.
template <int kStep>
__device__ __forceinline__ Joined join_parts(const Ws& ws, int Hkv, int g, int c_first, int i1, int r, int lane) {
  Joined a{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  for (int c0 = c_first; c0 <= i1; c0 += kStep * kCombineBatch) {
    float2 mlv[kCombineBatch];
    float4 ov[kCombineBatch];
#pragma unroll
    for (int i = 0; i < kCombineBatch; ++i) {
      const int c = c0 + i * kStep;
      mlv[i] = make_float2(-INFINITY, 0.f);
      ov[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c <= i1) {
        const size_t row = ((static_cast<size_t>(c) * Hkv + g) * 2 + (c < i1 ? 1 : 0)) * kRowsMax + r;
        mlv[i] = __ldcg(reinterpret_cast<const float2*>(ws.ml + row * 2));
        ov[i] = __ldcg(reinterpret_cast<const float4*>(ws.po + row * kDh) + lane);
      }
    }
    float mb = a.m;
#pragma unroll
    for (int i = 0; i < kCombineBatch; ++i) mb = fmaxf(mb, mlv[i].x);
    const float fo = a.m == -INFINITY ? 0.f : exp2_ftz(a.m - mb);
    a.l *= fo;
    a.o.x *= fo;
    a.o.y *= fo;
    a.o.z *= fo;
    a.o.w *= fo;
#pragma unroll
    for (int i = 0; i < kCombineBatch; ++i) {
      const float f = mlv[i].x == -INFINITY ? 0.f : exp2_ftz(mlv[i].x - mb);
      a.l = fmaf(mlv[i].y, f, a.l);
      a.o.x = fmaf(ov[i].x, f, a.o.x);
      a.o.y = fmaf(ov[i].y, f, a.o.y);
      a.o.z = fmaf(ov[i].z, f, a.o.z);
      a.o.w = fmaf(ov[i].w, f, a.o.w);
    }
    a.m = mb;
  }
  return a;
}

template <bool kByRow>
__global__ void __launch_bounds__(kCombineWarps * 32) k_paged_combine(PagedAttnParams p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per_seq = kByRow ? p.Hkv : p.Hq;
  const int s = blockIdx.x / per_seq, x = blockIdx.x - s * per_seq;
  const int g = kByRow ? x : x / p.group;
  const Ws ws = carve(p.ws, p.b.B, p.Hkv);
  pdl_wait();
  pdl_trigger();
  const Line ln = line_of(p, s, false);
  const long long base = __ldcg(ws.pre + s), W = __ldcg(ws.pre + p.b.B);
  if (ln.sq.n <= 0) return;
  if (ln.quanta == 0) {
    const int heads = kByRow ? p.group : 1, h0 = kByRow ? g * p.group : x, per_tok = heads * (kDh / 8);
    for (int i = threadIdx.x; i < ln.sq.n * per_tok; i += kCombineWarps * 32) {
      const int tok = i / per_tok, j = i - tok * per_tok;
      reinterpret_cast<uint4*>(p.out + (static_cast<size_t>(ln.sq.row0 + tok) * p.Hq + h0) * kDh)[j] =
          make_uint4(0, 0, 0, 0);
    }
    return;
  }
  const int np = parts_of(W, p.Hkv);
  // the part that holds line position x: the largest i with floor(W i / np) <= x
  const int i0 = static_cast<int>(((base + 1) * np - 1) / W);
  const int i1 = static_cast<int>(((base + ln.quanta) * np - 1) / W);
  if (i0 == i1) return;  // finished by its only part
  const float vs = p.v_scale != nullptr ? __ldg(p.v_scale + g) : 1.f;
  if constexpr (kByRow) {
    for (int r = warp; r < ln.sq.n * p.group; r += kCombineWarps) {
      const Joined a = join_parts<1>(ws, p.Hkv, g, i0, i1, r, lane);
      const int tok = r / p.group, h = r - tok * p.group;
      const float f = a.l == 0.f ? 0.f : vs / a.l;
      reinterpret_cast<uint2*>(p.out + (static_cast<size_t>(ln.sq.row0 + tok) * p.Hq + g * p.group + h) * kDh)[lane] =
          make_uint2(bf2(a.o.x * f, a.o.y * f), bf2(a.o.z * f, a.o.w * f));
    }
  } else {
    __shared__ float s_m[kCombineWarps], s_l[kCombineWarps];
    __shared__ __align__(16) float s_acc[kCombineWarps][kDh];
    for (int tok = 0; tok < ln.sq.n; ++tok) {
      const Joined a =
          join_parts<kCombineWarps>(ws, p.Hkv, g, i0 + warp, i1, tok * p.group + x - g * p.group, lane);
      if (lane == 0) {
        s_m[warp] = a.m;
        s_l[warp] = a.l;
      }
      *reinterpret_cast<float4*>(&s_acc[warp][4 * lane]) = a.o;
      __syncthreads();
      if (threadIdx.x < kDh) {
        const int d = threadIdx.x;
        float Mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < kCombineWarps; ++w) Mx = fmaxf(Mx, s_m[w]);
        float den = 0.f, num = 0.f;
#pragma unroll
        for (int w = 0; w < kCombineWarps; ++w) {
          const float f = s_m[w] == -INFINITY ? 0.f : exp2_ftz(s_m[w] - Mx);
          den = fmaf(s_l[w], f, den);
          num = fmaf(s_acc[w][d], f, num);
        }
        const __nv_bfloat16 bv = __float2bfloat16_rn(den == 0.f ? 0.f : num / den * vs);
        p.out[(static_cast<size_t>(ln.sq.row0 + tok) * p.Hq + x) * kDh + d] = *reinterpret_cast<const uint16_t*>(&bv);
      }
      __syncthreads();
    }
  }
}

template <bool kE4M3, bool kTall>
cudaError_t launch(const PagedAttnParams& p, cudaStream_t st) {
  auto kern = k_paged_decode<kE4M3, kTall>;
  cudaError_t e = flint_ensure_smem(reinterpret_cast<const void*>(kern));
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, ctas_per_head(p.Hkv) * p.Hkv, kWarps * 32, kWarps * ring_bytes<kE4M3>(), st, p);
}

}  // namespace

size_t paged_decode_workspace(int B, int n_kv_heads) {
  const Ws w = carve(nullptr, B, n_kv_heads);
  return reinterpret_cast<size_t>(w.po) + slots_of(n_kv_heads) * kRowsMax * kDh * sizeof(float);
}

int paged_decode_launch(const PagedAttnParams& p, int cache_dtype, size_t ws_bytes, cudaStream_t st) {
  if (p.ws == nullptr || ws_bytes < paged_decode_workspace(p.b.B, p.Hkv))
    return flint_fail_external(FLINT_ERR_WORKSPACE, "flint_paged_attention: workspace too small");
  const bool tall = p.max_q * p.group > 8;
  cudaError_t e = cache_dtype == FLINT_KV_E4M3 ? (tall ? launch<true, true>(p, st) : launch<true, false>(p, st))
                                               : (tall ? launch<false, true>(p, st) : launch<false, false>(p, st));
  if (e != cudaSuccess) return flint_fail_external(FLINT_ERR_CUDA, cudaGetErrorString(e));
  // by row / by head, us, bf16 sequences of up to 8,192 keys: Hkv B = 16 17.1 / 14.4, 32 24.3 / 22.2, 64 29.1 / 29.6,
  // 128 50.6 / 54.1, 256 90 / 98; of 16,000 keys each 32 54.6 / 53.2, 64 95.3 / 96.7, 128 176 / 181
  const bool by_row = static_cast<long long>(p.Hkv) * p.b.B >= 128;
  e = by_row ? launch_pdl(k_paged_combine<true>, static_cast<unsigned>(p.Hkv) * p.b.B, kCombineWarps * 32, 0, st, p)
             : launch_pdl(k_paged_combine<false>, static_cast<unsigned>(p.Hq) * p.b.B, kCombineWarps * 32, 0, st, p);
  if (e != cudaSuccess) return flint_fail_external(FLINT_ERR_CUDA, cudaGetErrorString(e));
  return FLINT_OK;
}

}  // namespace flint
