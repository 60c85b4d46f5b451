// fa_fwd_cache for few query rows: the kernel that reads the cache at HBM speed.
//
// A work item is a sequence, a K / V head and up to 8 NT of the rows that share
// it (query token i, group member j: row i * group + j). One pass over the
// item's keys forms O and the softmax sums, so what counts is that the codes
// stream in without a pause: every warp owns a ring of kStages tiles (4 KB of K
// and of V each), filled by TMA straight from the blocks that the table lists
// and emptied by the same warp. So a slot needs no "empty" barrier, no warp
// waits for another one inside an item, and the ring runs on across items.
//
// Products: mma.sync m16n8k16 with the keys as M and the rows as N. Few rows
// would leave most of a 128-row tcgen05 tile empty, and the operands come
// straight from registers: codes are widened there to fp16, exactly. S^T =
// K Q^T: a lane's 16-byte chunk of a K row is the four (k-step, half) pieces of
// a fragment under a permutation of d, which Q's fragments follow. O^T += V^T
// P^T: bytes of two neighbouring keys are paired by byte permutes before they
// are widened, so no transposition goes through shared memory; the rows of O^T
// are a permutation of d that the epilogue undoes.
//
// Both scales go into the exponent. With c = scale log2 e, and K and V scales
// ks, vs of the key's block,
//     e_j = c ks (q . k8_j) + log2 vs,   P'_j = 2^(e_j - m),
//     O = sum P'_j v8_j / sum (P'_j / vs),   LSE = ln 2 (m + log2 sum (P'_j / vs)),
// so V is used as stored. P' goes into the product as fp16, whose values have 11
// bits from 2^-14 on, and below that a step of 2^-24; l and the reference m are
// fp32. So that little of a small weight is lost, m is kept kWeightLift below
// the e that it was taken from, near the top of fp16's range: with W = max w_j
// vs_j (w the softmax weights), w vs is off by at most 2^-11 of itself (half a step
// of 11 bits), or, where it is below 2^-22 W, by 2^-33 W. m moves (and O, l are
// rescaled) only when an e_j exceeds it by more than kWeightMost.
// Not m at the largest e itself: there a weight of 2^-14 W loses bits and one of
// 2^-25 W all, which l, the sum of the unrounded weights, would still count.
//
// Splitting: the items' tiles form one list, cut into equal shares for the
// persistent CTAs (two or three on each SM). A share that begins or ends inside an item
// writes a partial result (O, m, l), which fa_cache_join_kernel joins in order.
//
// Measured, all launches of captured calls (a call by itself takes 1 to 2 us more):
// two sequences of 131071 keys, 32 heads on 8, d 128: 95 us (5.7 TB/s, 85 % of a
// copy's rate); 96 sequences of up to 16384 keys, the same heads: 235 us (5.8
// TB/s); four of 4096 keys, 16 heads: 21.4 us, 3 of them the join. What bounds it
// stands at step_ctas.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_cache.cuh"
#include "fa_common.cuh"

namespace fa {

constexpr int kStepWarps = 4;
constexpr int kStepThreads = 32 * kStepWarps;
// CTAs on an SM and stages of a ring, by the rows of an item. What bounds the
// kernel is the latency of its instructions (a warp issues one in 5 cycles and
// hardly ever waits for a copy), so 8 rows, which leave room for three CTAs'
// registers, run on 12 warps with two stages each. Against 8 warps with three
// stages: B128 H16 1000 keys, d 64, 60 us (76), B4 H16 4096 keys 21.3 (22.1),
// ragged B96 236 (240), but B2 131071 keys 95 (92).
__host__ __device__ constexpr int step_ctas(int nt) { return nt == 1 ? 3 : 2; }
__host__ __device__ constexpr int step_stages(int nt) { return nt == 1 ? 2 : 3; }
constexpr int kStepTileBytes = 4096;  // of K, and of V
constexpr int kStepMaxRows = 16;      // rows of an item: 8 NT, NT = 1 or 2

// P' = 2^(e - m) is at most fp16's largest power of two, and m is taken so far
// below the largest e. The closer the two, the more of small weights is kept, and
// the oftener m moves: us of the chunk kernel with m 0 / 7 / 8 / 9 / 11 below, P' at
// most 2^8 / 2^15 ..: 2048 x 16384 chunk 371.4 / 371.9 / 373.3 / 374.4 / 376.8, drafts
// 59.5 / 59.7 / 59.7 / 59.8 / 60.6 (few rows: no difference).
constexpr float kWeightMost = 15.f;
constexpr float kWeightLift = 8.f;

// Keys of a tile.
__host__ __device__ constexpr int step_keys(int d) { return kStepTileBytes / d; }

// Floats of a partial result of `rows` rows: O, m, l.
__host__ __device__ constexpr int partial_floats(int rows, int d) { return rows * (d + 2); }

// The first sequence from b on that a launch computes, or -1. Called by whole
// warps, which look at 32 sequences at a time: a large batch may have many of the
// other launch's, or without rows, in a row. (The chunk kernel, whose sequences
// are the long ones, looks at them one by one: there the search's code alone
// cost 5 %.)
__device__ __forceinline__ int next_taken(const CacheAttnArgs& a, int b) {
  if (a.cu_q == nullptr) return -1;  // all sequences alike
  const int lane = static_cast<int>(threadIdx.x & 31);
  for (; b < a.B; b += 32) {
    const bool taken = b + lane < a.B && takes_seq(a, seq_rows(a, b + lane));
    const uint32_t mask = __ballot_sync(0xffffffffu, taken);
    if (mask != 0u) return b + __ffs(static_cast<int>(mask)) - 1;
  }
  return -1;
}

// Position of a CTA's share in the list of tiles. An item with no keys counts
// as one (empty) tile, so that its rows are written.
template <int KT>
struct StepWalk {
  int b = 0, hk = 0, rb = 0;
  int n_rb = 0, real = 0, tiles = 0;  // row blocks, tiles with keys, tiles counted
  int t0 = 0, t1 = 0;                 // the share's tiles of this item
  long long left = 0;                 // tiles of the share from t0 on
  SeqRows s{};

  __device__ __forceinline__ static int row_blocks(const CacheAttnArgs& a, const SeqRows& s,
                                                   int rows) {
    return takes_seq(a, s)
               ? static_cast<int>((static_cast<long long>(s.count) * a.group + rows - 1) / rows)
               : 0;
  }
  __device__ __forceinline__ static long long units(const CacheAttnArgs& a, const SeqRows& s,
                                                    int rows, bool whole) {
    const int t = whole ? 1 : max(1, (s.kv_len + KT - 1) / KT);
    return static_cast<long long>(a.Hkv) * row_blocks(a, s, rows) * t;
  }
  __device__ __forceinline__ void load(const CacheAttnArgs& a, int rows, bool whole) {
    s = seq_rows(a, b);
    n_rb = row_blocks(a, s, rows);
    real = (s.kv_len + KT - 1) / KT;
    tiles = whole ? 1 : max(1, real);
  }
  // Tiles [first, last) of the item that hold keys and belong to the share.
  __device__ __forceinline__ int first(bool whole) const { return whole ? 0 : t0; }
  __device__ __forceinline__ int last(bool whole) const { return whole ? real : min(t1, real); }

  __device__ __forceinline__ void start(const CacheAttnArgs& a, int rows, bool whole, int b_,
                                        long long off, long long n) {
    b = b_;
    load(a, rows, whole);
    const long long item = off / tiles;
    t0 = static_cast<int>(off - item * tiles);
    hk = static_cast<int>(item / n_rb);
    rb = static_cast<int>(item - static_cast<long long>(hk) * n_rb);
    left = n;
    t1 = static_cast<int>(min(static_cast<long long>(tiles), t0 + left));
  }
  // To the next item; false if the share ends. Called by whole warps.
  __device__ __forceinline__ bool next(const CacheAttnArgs& a, int rows, bool whole) {
    left -= t1 - t0;
    if (left <= 0) return false;
    if (++rb == n_rb) {
      rb = 0;
      if (++hk == a.Hkv) {
        hk = 0;
        ++b;
        load(a, rows, whole);
        if (n_rb == 0) {
          b = next_taken(a, b + 1);
          if (b < 0) return false;  // (no tiles are left then)
          load(a, rows, whole);
        }
      }
    }
    t0 = 0;
    t1 = static_cast<int>(min(static_cast<long long>(tiles), left));
    return true;
  }
};

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transposes an 8 x 8 matrix of 16-bit values held as an mma fragment.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}

__device__ __forceinline__ uint32_t widen_lo(uint32_t w) {
  return ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(w));
}
__device__ __forceinline__ uint32_t widen_hi(uint32_t w) {
  return ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(w >> 16));
}

// Bytes of w that hold NaN codes (0x7F without the sign), as 0x80 in each.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

// Two fp32 values as fp16, lo in the low half.
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) { return pack2<false>(lo, hi); }

// Two weights as fp16. Where scores are so large that the exponent's fp32 steps are
// whole numbers, one may pass fp16's range: it becomes the largest number, not infinity.
__device__ __forceinline__ uint32_t pack_weights(float lo, float hi) {
  uint32_t u;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %2, %1;" : "=r"(u) : "f"(lo), "f"(hi));
  return u;
}

__device__ __forceinline__ float2 unpack_f16(uint32_t w) {
  __half2 h;
  __builtin_memcpy(&h, &w, 4);
  return __half22float2(h);
}

// N packed pairs of a query row, as fp16 values of `fac` (returned), a power of
// two that brings the row into fp16's range (bf16 queries; 1 for fp16): the
// conversion loses nothing that fp32 sums of the products would keep. kShare:
// lanes xor 1 .. kShare / 2 hold the other parts of the row. A bf16 row with an
// infinity becomes NaN: its scores might all be -inf, which looks like a row
// without keys. (fp16: inf_to_nan.)
template <int N, int kShare, bool BF16>
__device__ __forceinline__ float rows_to_f16(uint32_t (&w)[N]) {
  if constexpr (!BF16) {
    return 1.f;
  } else {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) m = max(m, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
#pragma unroll
    for (int o = 1; o < kShare; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    // exponent of the row's largest magnitude less 14, within normal fp32
    const int e = (m == 0u || m >= 0x7F80u) ? 0 : max(static_cast<int>(m >> 7) - 127 - 14, -126);
    const float fac = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
    const float inv = m >= 0x7F80u ? __int_as_float(0x7FFFFFFF) : 1.f / fac;
#pragma unroll
    for (int i = 0; i < N; ++i)
      w[i] = pack_f16(__uint_as_float(w[i] << 16) * inv, __uint_as_float(w[i] & 0xFFFF0000u) * inv);
    return fac;
  }
}

// Infinities among N packed pairs of fp16 values become NaN: w 0 + w.
template <int N>
__device__ __forceinline__ void inf_to_nan(uint32_t (&w)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    __half2 h;
    __builtin_memcpy(&h, &w[i], 4);
    h = __hfma2(h, __half2half2(__ushort_as_half(0)), h);
    __builtin_memcpy(&w[i], &h, 4);
  }
}

// Whether a row with the reference m and the sum l saw no key. (The maximum of
// scores that are all NaN is -inf too, but their sum is NaN: that row is NaN.)
__device__ __forceinline__ bool no_weight(float m, float l) { return m == -INFINITY && l == 0.f; }

// Shared memory (all of it dynamic: a static array would be padded to the
// ring's alignment).
template <int D, int NT>
struct StepLayout {
  static constexpr int kStages = step_stages(NT);
  static constexpr int kBoxes = step_keys(D) / 16;  // blocks of a tile, at most
  static constexpr int kRing = kStepWarps * kStages * 2 * kStepTileBytes;
  static constexpr int kOffMerge = kRing;  // merged rows: [warp][8][64] floats
  static constexpr int kOffStats = kOffMerge + kStepWarps * 8 * 64 * 4;  // m, l: [2][warp][8]
  static constexpr int kOffBar = kOffStats + 2 * kStepWarps * 8 * 4;
  static constexpr int kOffIdx = kOffBar + kStepWarps * kStages * 8;  // [warp][stage][box]
  static constexpr int kOffNan = kOffIdx + kStepWarps * kStages * kBoxes * 4;  // [D]
  static constexpr int kOffWords = kOffNan + D * 4;
  static constexpr int kSmem = kOffWords + 8;
  // 228 KB on an SM, 1 KB of it reserved for each CTA
  static_assert(step_ctas(NT) * (kSmem + 1024) <= 228 * 1024, "CTAs on an SM");
};

// Results are merged 64 columns at a time. Place (in pairs of floats) in merged
// row r of the columns of part h that lane group g holds in O^T tile i of its
// kI ones: the exclusive ors spread the 16 lanes of a store over all banks.
template <int D>
__device__ __forceinline__ int merge_pair(int r, int g, int i) {
  constexpr int kI = 4;  // tiles of O^T in 64 columns of each lane group's share
  return (kI * g + (i ^ ((g >> 1) & (kI / 2 - 1)))) ^ (r & 6);
}

// D: head dimension; BF16: type of q and o; NT: 8-row groups of an item; TREE: rows
// see the drafted keys that their masks tell (fa_fwd_cache_tree).
template <int D, bool BF16, int NT, bool TREE>
__global__ void __launch_bounds__(kStepThreads, step_ctas(NT))
    fa_cache_step_kernel(const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, const CacheAttnArgs a,
                         const int whole_items) {
  using L = StepLayout<D, NT>;
  constexpr int kStages = L::kStages;
  constexpr int KT = step_keys(D);
  constexpr int kSub = KT / 16;      // 16-key groups of a tile
  constexpr int kMt = D / 16;        // 16-row tiles of O^T
  constexpr int kRows = 8 * NT;
  constexpr int kQWords = D / 8;     // packed pairs of q a lane holds for one 8-row group
  extern __shared__ __align__(1024) uint8_t smem[];
  static_assert(L::kBoxes <= 4, "a lane of the first four for each block of a tile");
  const bool whole = whole_items != 0;
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t base = ptx::smem_u32(smem);
  const uint32_t ring = base + static_cast<uint32_t>(warp * kStages * 2 * kStepTileBytes);
  const uint32_t bars = base + L::kOffBar + static_cast<uint32_t>(warp * kStages * 8);
  int* const s_idx = reinterpret_cast<int*>(smem + L::kOffIdx) + warp * kStages * L::kBoxes;
  float* const s_merge = reinterpret_cast<float*>(smem + L::kOffMerge);
  float* const s_m = reinterpret_cast<float*>(smem + L::kOffStats);
  float* const s_l = s_m + kStepWarps * 8;
  long long* const s_scan = reinterpret_cast<long long*>(smem + L::kOffStats);  // before the items
  // smallest key whose V is NaN in a column, of keys that not all rows see
  int* const s_nan = reinterpret_cast<int*>(smem + L::kOffNan);
  volatile uint32_t* const s_abort = reinterpret_cast<volatile uint32_t*>(smem + L::kOffWords);
  volatile int* const s_any_nan = reinterpret_cast<volatile int*>(smem + L::kOffWords + 4);
  const AbortCtx ab{s_abort, a.status};
  // the join kernel may be set up while this one runs; it waits for its end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) ptx::mbar_init(bars + 8u * i, 1);
    ptx::fence_mbar_init();
    if (warp == 0) {
      ptx::prefetch_tmap(&tm_k);
      ptx::prefetch_tmap(&tm_v);
    }
  }
  for (int c = tid; c < D; c += kStepThreads) s_nan[c] = 0x7FFFFFFF;
  if (tid == 0) {
    *s_abort = 0u;
    *s_any_nan = 0;
  }

  // The share of this CTA: the list's length is a sum over the sequences.
  const int run = (a.B + kStepThreads - 1) / kStepThreads;
  const int b0 = min(tid * run, a.B), b1 = min(b0 + run, a.B);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += StepWalk<KT>::units(a, seq_rows(a, b), kRows, whole);
  long long upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += u;
  }
  if (lane == 31) s_scan[warp] = upto;
  __syncthreads();
  long long total = 0, before = 0;
#pragma unroll
  for (int w = 0; w < kStepWarps; ++w) {
    if (w < warp) before += s_scan[w];
    total += s_scan[w];
  }
  upto += before;
  // at least a tile for each warp, so that a small problem is not cut finer
  // than the CTA can use
  const long long fair = (total + gridDim.x - 1) / gridDim.x;
  const long long share = max(fair, static_cast<long long>(whole ? 1 : kStepWarps));
  const long long u0 = share * blockIdx.x, u1 = min(u0 + share, total);
  JoinItem* const join = a.join + blockIdx.x;
  float* const parts = a.parts;
  if (tid == 0 && !whole) *join = JoinItem{0, 0, 0, 0};
  if (u0 >= u1) return;
  if (u0 >= upto - mine && u0 < upto) {
    long long at = upto - mine;
    int b = b0;
    for (;; ++b) {
      const long long n = StepWalk<KT>::units(a, seq_rows(a, b), kRows, whole);
      if (u0 < at + n) break;
      at += n;
    }
    s_scan[kStepWarps] = b;
    s_scan[kStepWarps + 1] = u0 - at;
  }
  __syncthreads();

  const int box_keys = min(1 << a.block_shift, KT), boxes = KT / box_keys;
  StepWalk<KT> ahead, now;  // of the copies, and of the products
  now.start(a, kRows, whole, static_cast<int>(s_scan[kStepWarps]), s_scan[kStepWarps + 1], u1 - u0);
  __syncthreads();
  ahead = now;

  // ---- the ring. prepare() finds the next tile to copy and loads its block
  // id (lane j: the tile's j-th block), fire() starts the copy into a slot.
  int at_tile = ahead.first(whole) + warp;
  bool more = true;
  int id = -1, fire_tile = 0, fire_hk = 0;
  const int32_t* table = nullptr;  // of the item that is copied, and its blocks that hold keys
  int held = 0;
  auto enter = [&] {
    table = a.table + static_cast<long long>(ahead.b) * a.table_width;
    held = (ahead.s.kv_len + (1 << a.block_shift) - 1) >> a.block_shift;
  };
  enter();
  auto prepare = [&] {
    while (more && at_tile >= ahead.last(whole)) {
      more = ahead.next(a, kRows, whole);
      at_tile = ahead.first(whole) + warp;
      enter();
    }
    if (!more) return;
    id = -1;
    const int bi = ((at_tile * KT) >> a.block_shift) + lane;
    if (lane < boxes && bi < held) id = __ldg(table + bi);
    fire_tile = at_tile;
    fire_hk = ahead.hk;
    at_tile += kStepWarps;
  };
  auto fire = [&](int slot) {
    const bool ok = id >= 0 && id < a.num_blocks;
    const uint32_t have = __ballot_sync(0xffffffffu, ok);
    const uint32_t bar = bars + 8u * slot;
    if (lane < L::kBoxes) s_idx[slot * L::kBoxes + lane] = ok ? id * a.Hkv + fire_hk : -1;
    if (lane == 0)
      ptx::mbar_arrive_expect_tx(bar, static_cast<uint32_t>(__popc(have) * 2 * box_keys * D));
    __syncwarp();
    if (ok) {
      const uint32_t dst = ring + static_cast<uint32_t>(slot * 2 * kStepTileBytes + lane * box_keys * D);
      const int row = (fire_tile * KT) & ((1 << a.block_shift) - 1);
      ptx::tma_load_4d(dst, &tm_k, bar, 0, row, fire_hk, id);
      ptx::tma_load_4d(dst + kStepTileBytes, &tm_v, bar, 0, row, fire_hk, id);
    }
  };
  uint32_t fired = 0, used = 0;  // tiles copied into and taken from the ring
  for (int i = 0; i < kStages; ++i) {
    prepare();
    if (!more) break;
    fire(i);
    ++fired;
  }
  __syncwarp();
  // scales of the next tile: lane j < 4 the K scale of its j-th block, lanes
  // 4 - 7 the V scales; the index is < 0 where the block is hidden
  float scale_next = 1.f;
  int idx_next = -1;
  auto load_scales = [&](uint32_t n) {
    idx_next = s_idx[(n % kStages) * L::kBoxes + (t & (L::kBoxes - 1))];
    scale_next = 1.f;
    if (lane < 8 && idx_next >= 0) scale_next = __ldg((lane < 4 ? a.ks : a.vs) + idx_next);
  };
  if (used < fired) load_scales(0);

  bool alive = true;
  for (;;) {
    // ---- an item: its rows, their limits and Q
    const int row0 = now.rb * kRows;
    const int rows = min(kRows, now.s.count * a.group - row0);
    const int behind = now.s.kv_len - now.s.count;  // causal: row of query i sees behind + i + 1 keys
    int lim[NT][2];    // keys that rows 8 nt + 2 t and + 1 see (TREE: their masks' rows, or -1)
    float cs[NT][2];   // scale log2 e times the row's factor
    uint32_t q[NT][kQWords];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = row0 + 8 * nt + g;
      const bool there = 8 * nt + g < rows;
      const int i = there ? r / a.group : 0, j = there ? r - i * a.group : 0;
      const uint16_t* p = static_cast<const uint16_t*>(a.q) +
                          q_offset(a, now.b, now.s, i, now.hk * a.group + j) + t * (D / 4);
#pragma unroll
      for (int w = 0; w < kQWords / 4; ++w) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (there) v = *reinterpret_cast<const uint4*>(p + 8 * w);
        q[nt][4 * w] = v.x;
        q[nt][4 * w + 1] = v.y;
        q[nt][4 * w + 2] = v.z;
        q[nt][4 * w + 3] = v.w;
      }
      const float fac = rows_to_f16<kQWords, 4, BF16>(q[nt]);
      int sees = 0;
      if (there) sees = a.causal ? min(max(behind + i + 1, 0), now.s.kv_len) : now.s.kv_len;
      if constexpr (TREE) sees = there ? now.s.first + i : -1;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        lim[nt][h] = __shfl_sync(0xffffffffu, sees, (2 * t + h) * 4);
        cs[nt][h] = a.scale_log2 * __shfl_sync(0xffffffffu, fac, (2 * t + h) * 4);
      }
    }
    // keys that every row of the item sees
    const int all_see = TREE ? min(max(behind, 0), now.s.kv_len)
                        : a.causal ? min(max(behind + row0 / a.group + 1, 0), now.s.kv_len)
                                   : now.s.kv_len;
    float o[NT][kMt][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int i = 0; i < kMt; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.f;
    }

    const int last = now.last(whole);
    for (int tile = now.first(whole) + warp; tile < last; tile += kStepWarps) {
      const int slot = static_cast<int>(used % kStages);
      const float sc = scale_next;
      const int idx = idx_next;
      prepare();
      const bool refill = more && alive;
      if (used + 1 < fired) load_scales(used + 1);
      if (alive) alive = wait_bounded_warp(bars + 8u * slot, (used / kStages) & 1u, ab,
                                           kStatusSoftmax);
      if constexpr (!BF16) {
        // (here and not where Q is loaded: there it would wait for the rows)
        if (tile == now.first(whole) + warp) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) inf_to_nan<kQWords>(q[nt]);
        }
      }
      const uint32_t sk = ring + static_cast<uint32_t>(slot * 2 * kStepTileBytes);
      const uint32_t sv = sk + kStepTileBytes;
      const int key0 = tile * KT;
      const uint32_t hidden = __ballot_sync(0xffffffffu, lane < boxes && idx < 0);
      const bool edge = key0 + KT > all_see || hidden != 0u;
      const float lv_all = ptx::lg2(sc), iv_all = ptx::rcp(sc);  // (lanes 4 - 7: of the V scales)

      // S^T = K Q^T for the tile's keys
      float s[kSub][NT][4];
#pragma unroll
      for (int u = 0; u < kSub; ++u) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[u][nt][e] = 0.f;
        const int ra = 16 * u + g;
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
          uint4 x, y;  // rows ra and ra + 8
          if constexpr (D == 128) {
            const uint32_t ch = static_cast<uint32_t>((2 * t + j) ^ (ra & 7)) << 4;
            x = lds128(sk + static_cast<uint32_t>(ra) * 128u + ch);
            y = lds128(sk + static_cast<uint32_t>(ra + 8) * 128u + ch);
          } else {
            const uint32_t ch = static_cast<uint32_t>(t ^ ((ra >> 1) & 3)) << 4;
            x = lds128(sk + static_cast<uint32_t>(ra) * 64u + ch);
            y = lds128(sk + static_cast<uint32_t>(ra + 8) * 64u + ch);
          }
          const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t a0 = widen_lo(xw[w]), a2 = widen_hi(xw[w]);
            const uint32_t a1 = widen_lo(yw[w]), a3 = widen_hi(yw[w]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_16816(s[u][nt], a0, a1, a2, a3, q[nt][8 * j + 2 * w], q[nt][8 * j + 2 * w + 1]);
          }
        }
      }

      // trees: which of the tile's keys the rows see
      [[maybe_unused]] unsigned long long see[NT][2];
      if constexpr (TREE) {
        static_assert(KT <= 64, "a word of bits");
        if (edge) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              see[nt][h] = lim[nt][h] < 0
                               ? 0ull
                               : tree_seen64(a, now.s.kv_len, behind, lim[nt][h], key0);
        }
      }

      // e = S (c ks) + log2 vs, its largest per row
      float iv[kSub];
      float top[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) top[nt][0] = top[nt][1] = -INFINITY;
#pragma unroll
      for (int u = 0; u < kSub; ++u) {
        const int box = (16 * u) >> a.block_shift;
        const float ks = __shfl_sync(0xffffffffu, sc, box);
        const float lv = __shfl_sync(0xffffffffu, lv_all, 4 + box);
        iv[u] = __shfl_sync(0xffffffffu, iv_all, 4 + box);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float f0 = cs[nt][0] * ks, f1 = cs[nt][1] * ks;
          s[u][nt][0] = fmaf(s[u][nt][0], f0, lv);
          s[u][nt][1] = fmaf(s[u][nt][1], f1, lv);
          s[u][nt][2] = fmaf(s[u][nt][2], f0, lv);
          s[u][nt][3] = fmaf(s[u][nt][3], f1, lv);
          if (edge) {
            const int ka = key0 + 16 * u + g;
            const bool no = ((hidden >> box) & 1u) != 0u;
            if constexpr (TREE) {
              const int at = 16 * u + g;
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (no || ((see[nt][e & 1] >> (at + 4 * (e & 2))) & 1ull) == 0ull)
                  s[u][nt][e] = -INFINITY;
            } else {
              if (no || ka >= lim[nt][0]) s[u][nt][0] = -INFINITY;
              if (no || ka >= lim[nt][1]) s[u][nt][1] = -INFINITY;
              if (no || ka + 8 >= lim[nt][0]) s[u][nt][2] = -INFINITY;
              if (no || ka + 8 >= lim[nt][1]) s[u][nt][3] = -INFINITY;
            }
          }
          top[nt][0] = fmaxf(top[nt][0], fmaxf(s[u][nt][0], s[u][nt][2]));
          top[nt][1] = fmaxf(top[nt][1], fmaxf(s[u][nt][1], s[u][nt][3]));
        }
      }
      bool grow = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        grow = grow || top[nt][0] > m[nt][0] + kWeightMost || top[nt][1] > m[nt][1] + kWeightMost;
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float v = top[nt][h];
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, x));
            const float ref = fmaxf(m[nt][h], v - kWeightLift);
            const float keep = ref == -INFINITY ? 1.f : ptx::ex2(m[nt][h] - ref);
            m[nt][h] = ref;
            l[nt][h] *= keep;
#pragma unroll
            for (int i = 0; i < kMt; ++i) {
              o[nt][i][h] *= keep;
              o[nt][i][2 + h] *= keep;
            }
          }
      }

      // P' and the sums; P'^T as B fragments
      // (for fp16 queries in two parts: a weight's rounding to 11 bits would add
      // as much to the error as the rounding of O itself; bf16's O hides it)
      uint32_t p[kSub][NT][2], p_low[BF16 ? 1 : kSub][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float n0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0];
        const float n1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
#pragma unroll
        for (int u = 0; u < kSub; ++u) {
          const float p0 = ptx::ex2(s[u][nt][0] - n0), p1 = ptx::ex2(s[u][nt][1] - n1);
          const float p2 = ptx::ex2(s[u][nt][2] - n0), p3 = ptx::ex2(s[u][nt][3] - n1);
          l[nt][0] = fmaf(p0 + p2, iv[u], l[nt][0]);
          l[nt][1] = fmaf(p1 + p3, iv[u], l[nt][1]);
          const uint32_t h0 = pack_weights(p0, p1), h1 = pack_weights(p2, p3);
          p[u][nt][0] = transpose_8x8(h0);
          p[u][nt][1] = transpose_8x8(h1);
          if constexpr (!BF16) {
            const float2 b0 = unpack_f16(h0), b1 = unpack_f16(h1);
            p_low[u][nt][0] = transpose_8x8(pack_f16(p0 - b0.x, p1 - b0.y));
            p_low[u][nt][1] = transpose_8x8(pack_f16(p2 - b1.x, p3 - b1.y));
          }
        }
      }

      // O^T += V^T P'^T
#pragma unroll
      for (int u = 0; u < kSub; ++u) {
        uint32_t v[4][D / 32];  // keys 2t, 2t + 1, 2t + 8, 2t + 9; D / 8 columns from D / 8 * g
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int row = 16 * u + 2 * t + (k & 1) + (k >> 1) * 8;
          if constexpr (D == 128) {
            const uint4 w = lds128(sv + static_cast<uint32_t>(row) * 128u +
                                   (static_cast<uint32_t>(g ^ (row & 7)) << 4));
            v[k][0] = w.x;
            v[k][1] = w.y;
            v[k][2] = w.z;
            v[k][3] = w.w;
          } else {
            const uint2 w = lds64(sv + static_cast<uint32_t>(row) * 64u +
                                  (static_cast<uint32_t>((g >> 1) ^ ((row >> 1) & 3)) << 4) +
                                  static_cast<uint32_t>(g & 1) * 8u);
            v[k][0] = w.x;
            v[k][1] = w.y;
          }
        }
        if (edge) {
          // keys that no row sees (their V may be anything), and NaN in keys
          // that only some rows see: weight 0 times NaN must not reach the others
          const int box = (16 * u) >> a.block_shift;
          const bool no = ((hidden >> box) & 1u) != 0u;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int key = key0 + 16 * u + 2 * t + (k & 1) + (k >> 1) * 8;
            const bool out = no || key >= now.s.kv_len;
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
              if (out) v[k][w] = 0u;
              const uint32_t bad = key >= all_see ? nan_bytes(v[k][w]) : 0u;
              if (bad) {
                for (int y = 0; y < 4; ++y)
                  if ((bad >> (8 * y)) & 0x80u) {
                    atomicMin(&s_nan[D / 8 * g + 4 * w + y], key);
                    v[k][w] &= ~(0xFFu << (8 * y));
                  }
                *s_any_nan = 1;
              }
            }
          }
        }
#pragma unroll
        for (int i = 0; i < kMt; ++i) {
          const uint32_t sel = (i & 1) ? 0x7362u : 0x5140u;
          const uint32_t x = __byte_perm(v[0][i / 2], v[1][i / 2], sel);
          const uint32_t y = __byte_perm(v[2][i / 2], v[3][i / 2], sel);
          const uint32_t a0 = widen_lo(x), a1 = widen_hi(x), a2 = widen_lo(y), a3 = widen_hi(y);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_16816(o[nt][i], a0, a1, a2, a3, p[u][nt][0], p[u][nt][1]);
            if constexpr (!BF16)
              mma_16816(o[nt][i], a0, a1, a2, a3, p_low[u][nt][0], p_low[u][nt][1]);
          }
        }
      }
      __syncwarp();  // the slot is read by every lane
      ++used;
      if (refill) {
        fire(slot);
        ++fired;
      }
    }

    // ---- the four warps' results together, 8 rows at a time
    bool any_nan = false;
    const bool begins = whole || now.t0 == 0, ends = whole || now.t1 == now.tiles;
    float* part = nullptr;  // where a partial result goes
    if (!begins) part = parts + 2LL * blockIdx.x * partial_floats(kRows, D);
    else if (!ends) part = parts + (2LL * blockIdx.x + 1) * partial_floats(kRows, D);
    if (part != nullptr && begins && tid == 0)
      *join = join_item(now.b, now.hk, now.rb, rows,
                        1 + static_cast<int>((now.tiles - now.t1 + share - 1) / share));
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v = l[nt][h];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) v += __shfl_xor_sync(0xffffffffu, v, x);
        if (g == 0) {
          s_m[warp * 8 + 2 * t + h] = m[nt][h];
          s_l[warp * 8 + 2 * t + h] = v;
        }
      }
#pragma unroll
      for (int half = 0; half < D / 64; ++half) {  // tiles 4 half .. 4 half + 3 of O^T
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float2* row = reinterpret_cast<float2*>(s_merge + (warp * 8 + 2 * t + h) * 64);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            row[merge_pair<D>(2 * t + h, g, i)] =
                make_float2(o[nt][4 * half + i][h], o[nt][4 * half + i][2 + h]);
        }
        __syncthreads();
        any_nan = *s_any_nan != 0;  // (no warp is at another item's tiles here)
        for (int e = tid; e < 8 * 32; e += kStepThreads) {
          const int r = e >> 5, gg = (e >> 2) & 7, i = e & 3;
          const int c = D / 8 * gg + 2 * (4 * half + i);  // columns c and c + 1
          const int rr = 8 * nt + r;                      // row of the item
          if (rr >= rows) break;
          float top = -INFINITY;
#pragma unroll
          for (int w = 0; w < kStepWarps; ++w) top = fmaxf(top, s_m[w * 8 + r]);
          const int pair = merge_pair<D>(r, gg, i);
          float sum = 0.f;
          float2 acc = make_float2(0.f, 0.f);
#pragma unroll
          for (int w = 0; w < kStepWarps; ++w) {
            const float mw = s_m[w * 8 + r];
            const float f = mw == -INFINITY ? 0.f : ptx::ex2(mw - top);
            const float2 v = reinterpret_cast<const float2*>(s_merge + (w * 8 + r) * 64)[pair];
            sum = fmaf(s_l[w * 8 + r], f, sum);
            acc.x = fmaf(v.x, f, acc.x);
            acc.y = fmaf(v.y, f, acc.y);
          }
          const int i_q = (row0 + rr) / a.group, j_q = (row0 + rr) - i_q * a.group;
          if (any_nan) {
            if constexpr (TREE) {
#pragma unroll 1
              for (int x = 0; x < 2; ++x)
                if (s_nan[c + x] < now.s.kv_len &&
                    tree_nan(a, now.b, now.hk, now.s, now.s.first + i_q, c + x))
                  (x ? acc.y : acc.x) = __int_as_float(0x7FFFFFFF);
            } else {
              const int sees = a.causal ? min(behind + i_q + 1, now.s.kv_len) : now.s.kv_len;
              if (s_nan[c] < sees) acc.x = __int_as_float(0x7FFFFFFF);
              if (s_nan[c + 1] < sees) acc.y = __int_as_float(0x7FFFFFFF);
            }
          }
          if (part != nullptr) {
            *reinterpret_cast<float2*>(part + rr * D + c) = acc;
            if (c == 0) {
              part[kRows * D + rr] = top;
              part[kRows * D + kRows + rr] = sum;
            }
          } else {
            const bool none = no_weight(top, sum);
            const float inv = none ? 0.f : 1.f / sum;
            const int h = now.hk * a.group + j_q;
            *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.o) +
                                         o_offset(a, now.b, now.s, i_q, h) + c) =
                pack2<BF16>(acc.x * inv, acc.y * inv);
            if (c == 0)
              a.lse[lse_index(a, now.b, now.s, i_q, h)] =
                  none ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
          }
        }
        __syncthreads();
      }
    }
    if (any_nan) {
      for (int c = tid; c < D; c += kStepThreads) s_nan[c] = 0x7FFFFFFF;
      __syncthreads();
      if (tid == 0) *s_any_nan = 0;
      __syncthreads();
    }
    if (!now.next(a, kRows, whole)) break;
  }
  // (every copy has been waited for, unless a wait gave up: then those in
  // flight land before the CTA ends, as far as they do)
  if (!alive)
    for (uint32_t n = used > kStages ? used - kStages : 0; n < fired; ++n)
      wait_drain(bars + 8u * (n % kStages), (n / kStages) & 1u, ab, kStatusDrain);
}

// Joins the partial results of the items that the shares of a step or chunk
// launch cut: blocks (c, y) take the rows from y * kJoinRows on of the item that
// begins in share c and ends in a later one. Parts are added in a fixed order.
// (Blocks that first found all items and shared their rows evenly were slower
// by the time of that search, 3 us.)
constexpr int kJoinThreads = 256;
constexpr int kJoinRows = 32;
// Blocks on an SM. Their loads from L2 are what takes time: four in 64 registers
// each, 2048 x 16384 chunk 369.5 us, chunks beside single tokens 38.8; two in 128,
// 374.5 and 40.2; five in 48, 371 and 39.1.
constexpr int kJoinBlocks = 4;

// The chunk kernel's partial results lie column by column ([D][max_rows], then m
// and l): a lane takes a row, a warp D / 8 of its columns, and the joined rows
// go out through shared memory.
template <int D, bool BF16>
__device__ __forceinline__ void join_columns(const CacheAttnArgs& a, const JoinItem& it,
                                             const float* parts, int cta, int max_rows, int first,
                                             int rows, float* s_rows, int warp, int lane) {
  constexpr int kCols = D / (kJoinThreads / 32), kPitch = D + 4;
  const int n = join_parts(it), size = partial_floats(max_rows, D);
  const int r = first + lane;
  const bool there = r < rows;
  auto part = [&](int p) { return parts + (2LL * (cta + p) + (p == 0 ? 1 : 0)) * size + r; };
  float m = -INFINITY, l = 0.f, o[kCols] = {};
  if (there) {
#pragma unroll 4
    for (int p = 0; p < n; ++p) m = fmaxf(m, __ldcg(part(p) + max_rows * D));
#pragma unroll 2
    for (int p = 0; p < n; ++p) {
      const float* q = part(p);
      const float mp = __ldcg(q + max_rows * D);
      const float f = mp == -INFINITY ? 0.f : ptx::ex2(mp - m);
      l = fmaf(__ldcg(q + max_rows * D + max_rows), f, l);
#pragma unroll
      for (int c = 0; c < kCols; ++c)
        o[c] = fmaf(__ldcg(q + (warp * kCols + c) * max_rows), f, o[c]);
    }
    const float inv = no_weight(m, l) ? 0.f : 1.f / l;
#pragma unroll
    for (int c = 0; c < kCols; ++c) s_rows[lane * kPitch + warp * kCols + c] = o[c] * inv;
  }
  __syncthreads();
  const SeqRows s = seq_rows(a, it.b);
  for (int e = static_cast<int>(threadIdx.x); e < kJoinRows * (D / 8); e += kJoinThreads) {
    const int rr = e / (D / 8), c = 8 * (e % (D / 8));
    if (first + rr >= rows) break;
    const long long row = static_cast<long long>(it.rb) * max_rows + first + rr;
    const int i = static_cast<int>(row / a.group);
    const int h = it.hk * a.group + static_cast<int>(row - static_cast<long long>(i) * a.group);
    const float* v = s_rows + rr * kPitch + c;
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) + o_offset(a, it.b, s, i, h) + c) =
        make_uint4(pack2<BF16>(v[0], v[1]), pack2<BF16>(v[2], v[3]), pack2<BF16>(v[4], v[5]),
                   pack2<BF16>(v[6], v[7]));
  }
  if (warp == 0 && there) {
    const long long row = static_cast<long long>(it.rb) * max_rows + r;
    const int i = static_cast<int>(row / a.group);
    const int h = it.hk * a.group + static_cast<int>(row - static_cast<long long>(i) * a.group);
    a.lse[lse_index(a, it.b, s, i, h)] =
        no_weight(m, l) ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
  }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kJoinThreads, kJoinBlocks)
    fa_cache_join_kernel(const CacheAttnArgs a, const JoinSides sides) {
  constexpr int kWarps = kJoinThreads / 32, kPer = D / 32;
  __shared__ float s_rows[kJoinRows * (D + 4)];
  __shared__ float s_l[kWarps];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const bool second = static_cast<int>(blockIdx.x) >= sides.ctas[0];
  const int cta = static_cast<int>(blockIdx.x) - (second ? sides.ctas[0] : 0);
  const int4 word = __ldcg(reinterpret_cast<const int4*>(second ? sides.join[1] : sides.join[0]) + cta);
  const JoinItem it{word.x, word.y, word.z, word.w};
  const int first = static_cast<int>(blockIdx.y) * kJoinRows;
  const int n = join_parts(it), rows = min(join_rows(it), first + kJoinRows);
  if (first >= rows) return;
  const int max_rows = second ? sides.rows[1] : sides.rows[0];
  const float* parts = second ? sides.parts[1] : sides.parts[0];
  const int size = partial_floats(max_rows, D);
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  if (second) {
    join_columns<D, BF16>(a, it, parts, cta, max_rows, first, rows, s_rows, warp, lane);
    return;
  }
  // the step kernel's lie row by row; warps share a row's parts when there are
  // fewer rows than warps
  float (*const s_o)[D] = reinterpret_cast<float(*)[D]>(s_rows);
  int per_row = 1;  // warps for a row: a power of two
  while (per_row * 2 * (rows - first) <= kWarps) per_row *= 2;
  auto part = [&](int p) { return parts + (2LL * (cta + p) + (p == 0 ? 1 : 0)) * size; };
  const SeqRows s = seq_rows(a, it.b);
  for (int r0 = first; r0 < rows; r0 += kWarps / per_row) {
    const int r = r0 + warp / per_row, k = warp % per_row;
    float m = -INFINITY, l = 0.f, o[kPer] = {};
    if (r < rows) {
      // the largest reference of all of the row's parts first, so that nothing is rescaled
      for (int p = lane; p < n; p += 32) m = fmaxf(m, __ldcg(part(p) + max_rows * D + r));
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
#pragma unroll 8
      for (int p = k; p < n; p += per_row) {
        const float* q = part(p);
        const float mp = __ldcg(q + max_rows * D + r);
        const float f = mp == -INFINITY ? 0.f : ptx::ex2(mp - m);
        l = fmaf(__ldcg(q + max_rows * D + max_rows + r), f, l);
        if constexpr (kPer == 4) {
          const float4 v = __ldcg(reinterpret_cast<const float4*>(q + r * D + 4 * lane));
          o[0] = fmaf(v.x, f, o[0]);
          o[1] = fmaf(v.y, f, o[1]);
          o[2] = fmaf(v.z, f, o[2]);
          o[3] = fmaf(v.w, f, o[3]);
        } else {
          const float2 v = __ldcg(reinterpret_cast<const float2*>(q + r * D + 2 * lane));
          o[0] = fmaf(v.x, f, o[0]);
          o[1] = fmaf(v.y, f, o[1]);
        }
      }
    }
    if (per_row > 1) {  // (one turn of the loop: each row has its warps)
#pragma unroll
      for (int e = 0; e < kPer; ++e) s_o[warp][kPer * lane + e] = o[e];
      if (lane == 0) s_l[warp] = l;
      __syncthreads();
      if (k == 0) {
        for (int w = 1; w < per_row; ++w) {
          l += s_l[warp + w];
#pragma unroll
          for (int e = 0; e < kPer; ++e) o[e] += s_o[warp + w][kPer * lane + e];
        }
      }
    }
    if (r < rows && k == 0) {
      const bool none = no_weight(m, l);
      const float inv = none ? 0.f : 1.f / l;
      const long long row = static_cast<long long>(it.rb) * max_rows + r;
      const int i = static_cast<int>(row / a.group);
      const int h = it.hk * a.group + static_cast<int>(row - static_cast<long long>(i) * a.group);
      uint16_t* out = static_cast<uint16_t*>(a.o) + o_offset(a, it.b, s, i, h) + kPer * lane;
      if constexpr (kPer == 4)
        *reinterpret_cast<uint2*>(out) = make_uint2(pack2<BF16>(o[0] * inv, o[1] * inv),
                                                    pack2<BF16>(o[2] * inv, o[3] * inv));
      else
        *reinterpret_cast<uint32_t*>(out) = pack2<BF16>(o[0] * inv, o[1] * inv);
      if (lane == 0)
        a.lse[lse_index(a, it.b, s, i, h)] =
            none ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
    }
  }
}

}  // namespace fa
