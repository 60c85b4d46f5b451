// fa_fwd_cache for many query rows: S = Q K^T and O += P V on tcgen05 with S, P
// and O in tensor memory, from the cache's 8-bit blocks.
//
// A work item is a sequence, a K / V head and up to 256 of the rows that share
// it (query token i, group member j: row i * group + j, so later rows see at
// least as many keys). More than 128 rows: two tiles of 128 that share every
// KV tile of 128 keys, and the softmax of one runs while the tensor core works
// for the other (pair mode). At most 128 rows, a group's drafts or the last
// rows of a chunk: one Q tile, S in two buffers; of every KV tile one warpgroup
// takes the first and the other the second 64 keys, each with a maximum, a sum
// and an O of its own, which are merged at the end (split mode). So S of a tile
// is formed while the softmax is at the one before.
//
// The operands are fp16 (kind::f16) whatever the queries' type: every e4m3 code
// is an fp16 value, so K and V lose nothing, and bf16 queries are brought into
// fp16's range row by row with a power of two (rows_to_f16). TMA brings the blocks
// that the table lists into a ring of 8-bit tiles; converter warps widen them
// into the swizzled operand tiles, and zero what no row may see.
// PARTS > 0 (split mode only, d 128): Q is written as the sum of PARTS e4m3 tiles
// (query_parts), and K goes from the cache into the product as it is
// (kind::f8f6f4). That leaves the converters half of their work for some more
// time of the tensor core. P cannot be cut up in that way: e4m3's smallest step,
// 2^-9, would take away the weights of a flat row beside one large one.
//
// Both scales go into the exponent, as in fa_cache_step.cuh: e = c ks s + log2
// vs, P' = 2^(e - m), O = sum P' v8, l = sum P' / vs.
//
// Warp roles (16 warps):
//   warp 0       issues the MMAs (elected lane), owns the tensor memory
//   warp 1       copies: table entries, scales, TMA
//   warps 4-7    softmax and epilogue of tile 0 (split mode: the first 64 keys)
//   warps 8-11   softmax and epilogue of tile 1 (split mode: the others)
//   warps 12-15  converters
// Tensor memory: S0 0-127, S1 128-255, O0 256.., O1 256 + D..; P_i goes over the
// first 64 columns of S_i (split mode: 32 columns of each half).
//
// Splitting: as in fa_cache_step.cuh, the items' tiles form one list that is
// cut into equal shares, one for each SM; fa_cache_join_kernel joins the
// partial results of cut items.
//
// What bounds it. Pair mode: the chain S - softmax - P V - S of each Q tile, as in
// the forward kernel of whole matrices; tensor memory is full, so S has no second
// buffer. 2048 tokens behind 14336 others, 32 heads of d 128 on 8: 371 us, 1.39
// PFLOP/s (72 % of a matrix product's burst rate), tensor pipe active 61 %. Split
// mode: 16 x 40 rows, 4 K / V heads, 8192 keys: 60 us a call of equal sequences, 70
// a ragged one, whose launch of the step kernel finds nothing to do (9 us less than
// with all of K widened, too, and whole tiles for each warpgroup); a KV tile takes
// 2400 cycles, 1700 of them the MMAs (shared-memory traffic, 208 KB a tile) and 1700
// a warpgroup's softmax, whose warps stand alone on their schedulers. The other
// third of the 60 us is the launch, Q, the epilogues and the join.
#pragma once

#include "fa_cache_step.cuh"

namespace fa {

constexpr int kChunkThreads = 512;
constexpr int kChunkRows = 256;
constexpr int kChunkKeys = 128;
constexpr int kChunkMinShare = 2;  // tiles
// Registers a thread after setmaxnreg (sum 512 = 4 x 128): MMA and copy
// warpgroup, each softmax warpgroup, converters.
constexpr uint32_t kChunkRegsMma = 64, kChunkRegsSoftmax = 184, kChunkRegsConvert = 80;
static_assert(kChunkRegsMma + 2 * kChunkRegsSoftmax + kChunkRegsConvert == 512, "register split");

// PARTS = 0: items of up to 256 rows, K and V widened. PARTS > 0: items of up to
// 128 rows, Q in PARTS e4m3 tiles, V widened.
template <int D, int PARTS>
struct ChunkLayout {
  static constexpr int kPanels = D / 64;
  static constexpr int kTileBytes = kPanels * kPanelBytes;  // 128 rows of fp16
  static constexpr int kRawBytes = kChunkKeys * D;          // 128 rows of codes
  static constexpr int kQBytes = PARTS > 0 ? PARTS * kRawBytes : kTileBytes;
  static constexpr int kHalves = PARTS > 0 ? 1 : 2;  // of a tile that are widened: V, or K and V
  static constexpr int kStages = PARTS > 0 ? 2 : D == 128 ? 3 : 6;            // fp16 slots
  static constexpr int kRaw = PARTS > 0 ? 3 : D == 128 ? 3 : 6;  // slots of codes
  static constexpr int kDirect = PARTS > 0 ? 3 : 0;                            // K slots
  static constexpr int kOffQ = 0;                                              // Q0, Q1
  static constexpr int kOffKV = (PARTS > 0 ? 1 : 2) * kQBytes;
  static constexpr int kOffRaw = kOffKV + kStages * kTileBytes;
  static constexpr int kOffK = kOffRaw + kRaw * kRawBytes;
  // scales of a tile's 16-key groups: [16 tiles][8] {ks, log2 vs, 1 / vs, 0}
  static constexpr int kOffScale = kOffK + kDirect * kRawBytes;
  static constexpr int kOffNan = kOffScale + 16 * 8 * 16;    // [8 items][D] uint64
  static constexpr int kOffStats = kOffNan + 8 * D * 8;      // [2][128] m, l of the second halves
  static constexpr int kOffShelf = kOffStats + 1024;  // [8 warps] 64 bytes
  static constexpr int kOffBar = kOffShelf + 512;
  static constexpr int kSmem = kOffBar + 544 + 1024;  // barriers, alignment slack
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kColS = 0, kColO = 256;
  static_assert(kSmem <= 232448, "shared memory budget");
  static_assert(kRaw <= 8 && kStages + kRaw + kDirect <= 12, "barrier block");
  static_assert(kQBytes >= kTileBytes, "the epilogue stages its rows there");
};

enum ChunkBar : int {
  kCbQFull = 0,       // [2] 128 softmax threads: Q_i in shared memory
  kCbSFull = 2,       // [2] MMA: S_i ready
  kCbPFull = 4,       // [2] 128 softmax threads: P_i written, O_i rescaled
  kCbOFull = 6,       // [2] MMA: the item's last O_i += P_i V done
  kCbStats = 8,       // 128 threads of tile 1: its m, l in shared memory (split mode)
  kCbMerged = 9,      // 128 threads of tile 0: O1 and the stats read (split mode)
  kCbDrain = 10,      // MMA: every tcgen05 op completed
  kCbPSplit = 11,     // [2] 256 softmax threads: both halves of P_b written (split mode)
  kCbOStep = 13,      // MMA: a tile's products with V done (split mode)
  kCbScaleFull = 14,  // [16] copy warp: scales of tile n in entry n % 16
  kCbVDone = 30,      // [8] converter warps: V of tile n converted (its NaN recorded)
  // [stages] converter warps: operand slot filled; [stages] MMA: slot free;
  // [raw] TMA: raw slot filled; [raw] converter warps: slot free;
  // [direct] TMA: K slot filled; [direct] MMA: slot free
  kCbKVFull = 38,
};
constexpr int kChunkSlotTmem = 496, kChunkSlotAbort = 500, kChunkSlotStart = 504;
constexpr int kChunkSlotHidden = 520;  // [raw] bytes: bit g: 16-key group g is hidden
constexpr int kChunkSlotAnyNan = 528;  // not 0: a converter has noted NaN

// Keys that query token i of a sequence sees.
__device__ __forceinline__ int keys_seen(const CacheAttnArgs& a, const SeqRows& s, int i) {
  return a.causal ? min(max(s.kv_len - s.count + i + 1, 0), s.kv_len) : s.kv_len;
}

// Row blocks of a sequence, and the tiles that one of them reads (counted: at
// least one, so that rows without keys are written).
__device__ __forceinline__ int chunk_row_blocks(const CacheAttnArgs& a, const SeqRows& s) {
  const long long rows = static_cast<long long>(s.count) * a.group;
  return takes_seq(a, s) ? static_cast<int>((rows + a.item_rows - 1) / a.item_rows) : 0;
}
__device__ __forceinline__ int chunk_real_tiles(const CacheAttnArgs& a, const SeqRows& s, int rb) {
  const long long last = min((rb + 1LL) * a.item_rows, static_cast<long long>(s.count) * a.group) - 1;
  return (keys_seen(a, s, static_cast<int>(last / a.group)) + kChunkKeys - 1) / kChunkKeys;
}
// Tiles of one head of a sequence.
__device__ __forceinline__ long long chunk_head_tiles(const CacheAttnArgs& a, const SeqRows& s) {
  const int n = chunk_row_blocks(a, s);
  if (!a.causal) return static_cast<long long>(n) * max(1, (s.kv_len + kChunkKeys - 1) / kChunkKeys);
  long long sum = 0;
  for (int rb = 0; rb < n; ++rb) sum += max(1, chunk_real_tiles(a, s, rb));
  return sum;
}

// A CTA's share, item by item (every role walks a copy of its own).
struct ChunkWalk {
  int b, hk, rb, n_rb;
  int tiles;     // counted tiles of the item
  int t0, t1;    // the share's tiles of it
  int real_end;  // end of those that hold keys: tiles t0 .. real_end - 1 are read
  long long left;
  int item;      // items with tiles to read so far
  SeqRows s;

  __device__ __forceinline__ void item_tiles(const CacheAttnArgs& a) {
    const int real = chunk_real_tiles(a, s, rb);
    tiles = max(1, real);
    t1 = static_cast<int>(min(static_cast<long long>(tiles), t0 + left));
    real_end = min(t1, real);
  }
  __device__ __forceinline__ void start(const CacheAttnArgs& a, int b_, int hk_, int rb_, int t0_,
                                        long long n) {
    b = b_;
    hk = hk_;
    rb = rb_;
    t0 = t0_;
    left = n;
    item = 0;
    s = seq_rows(a, b);
    n_rb = chunk_row_blocks(a, s);
    item_tiles(a);
  }
  __device__ __forceinline__ bool next(const CacheAttnArgs& a) {
    left -= t1 - t0;
    if (left <= 0) return false;
    item += n() > 0 ? 1 : 0;
    if (++rb == n_rb) {
      rb = 0;
      if (++hk == a.Hkv) {
        hk = 0;
        do {
          ++b;
          s = seq_rows(a, b);
          n_rb = chunk_row_blocks(a, s);
        } while (n_rb == 0);  // ends: tiles are left
      }
    }
    t0 = 0;
    item_tiles(a);
    return true;
  }
  __device__ __forceinline__ int rows(const CacheAttnArgs& a) const {
    return static_cast<int>(min(static_cast<long long>(a.item_rows),
                                static_cast<long long>(s.count) * a.group -
                                    static_cast<long long>(rb) * a.item_rows));
  }
  __device__ __forceinline__ int n() const { return max(0, real_end - t0); }
};

// ---- copies: warp 1. Lane j < 128 / block handles the j-th block of a tile,
// lane g < 8 the scales of the g-th 16-key group.
template <int D, int PARTS>
__device__ __forceinline__ void chunk_copy_role(const CUtensorMap* tm_k, const CUtensorMap* tm_v,
                                                const CacheAttnArgs& a, ChunkWalk w, uint8_t* sgen,
                                                uint32_t sbase, uint32_t bars, const AbortCtx& ab,
                                                int lane) {
  using L = ChunkLayout<D, PARTS>;
  constexpr int R = L::kRaw;
  constexpr int kRawFull = kCbKVFull + 2 * L::kStages, kRawFree = kRawFull + R;
  constexpr int kKFull = kRawFree + R, kKFree = kKFull + L::kDirect;
  auto bar = [&](int i) { return bars + 8u * static_cast<uint32_t>(i); };
  float4* const s_scale = reinterpret_cast<float4*>(sgen + L::kOffScale);
  uint8_t* const s_hidden = sgen + L::kOffBar + kChunkSlotHidden;
  const int boxes = kChunkKeys >> a.block_shift, box_bytes = D << a.block_shift;
  if (lane == 0) {
    ptx::prefetch_tmap(tm_k);
    ptx::prefetch_tmap(tm_v);
  }
  uint32_t ring = 0, count = 0, asked = 0;  // V (K and V), tiles, K
  bool ok = true;
  do {
    // Table entries and scales are read for four tiles at a time (lane 8 q + g:
    // 16-key group g of tile q), entries two rounds and scales one round ahead:
    // two trips to memory one after another for each tile would take longer
    // than its products.
    auto entries = [&](int t) {  // block of this lane's group, or -1
      const long long key = (static_cast<long long>(t) + (lane >> 3)) * kChunkKeys +
                            ((16 * (lane & 7)) & -(1 << a.block_shift));  // the block's first
      int id = -1;
      if (t + (lane >> 3) < w.real_end && key < w.s.kv_len)
        id = __ldg(a.table + static_cast<long long>(w.b) * a.table_width + (key >> a.block_shift));
      return id >= 0 && id < a.num_blocks ? id : -1;
    };
    auto scales = [&](int id) {
      float2 f = make_float2(1.f, 0.f);
      if (id >= 0) {
        const long long at = static_cast<long long>(id) * a.Hkv + w.hk;
        f = make_float2(__ldg(a.ks + at), __ldg(a.vs + at));
      }
      return f;
    };
    int ids = entries(w.t0), ids_next = entries(w.t0 + 4);
    float2 sc = scales(ids), sc_next = make_float2(0.f, 0.f);
    for (int t = w.t0; t < w.real_end; ++t) {
      const int q = (t - w.t0) & 3;
      if (q == 0) {
        if (t > w.t0) {
          ids = ids_next;
          sc = sc_next;
          ids_next = entries(t + 4);
        }
        sc_next = scales(ids_next);
      }
      const uint32_t hidden = (__ballot_sync(0xffffffffu, ids < 0) >> (8 * q)) & 0xFFu;
      // lane j: the tile's j-th block
      const int jd = __shfl_sync(0xffffffffu, ids, 8 * q + ((lane << (a.block_shift - 4)) & 7));
      const int id = lane < boxes ? jd : -1;
      const uint32_t have = __ballot_sync(0xffffffffu, id >= 0);
      if constexpr (L::kDirect > 0) {
        // K in the MMA's layout; keys that no row may see become zeros here
        const uint32_t slot = asked % L::kDirect;
        if (!(ok = wait_spin_warp(bar(kKFree + slot), ((asked / L::kDirect) & 1u) ^ 1u, ab,
                                  kStatusProducer)))
          break;
        const uint32_t to = sbase + L::kOffK + slot * L::kRawBytes;
        if (hidden != 0u) {
          for (int at = 16 * lane; at < L::kRawBytes; at += 512)
            if ((hidden >> (at / (16 * D))) & 1u) ptx::st_shared_v4(to + at, 0u, 0u, 0u, 0u);
          ptx::fence_proxy_async_smem();
          __syncwarp();
        }
        if (lane == 0)
          ptx::mbar_arrive_expect_tx(bar(kKFull + slot),
                                     static_cast<uint32_t>(__popc(have) * box_bytes));
        __syncwarp();
        if (id >= 0)
          ptx::tma_load_4d(to + static_cast<uint32_t>(lane * box_bytes), tm_k, bar(kKFull + slot), 0,
                           0, w.hk, id);
        ++asked;
      }
#pragma unroll
      for (int is_v = 2 - L::kHalves; is_v < 2; ++is_v) {
        const uint32_t slot = ring % R;
        if (!(ok = wait_spin_warp(bar(kRawFree + slot), ((ring / R) & 1u) ^ 1u, ab,
                                  kStatusProducer)))
          break;
        if (lane == 0) {
          s_hidden[slot] = static_cast<uint8_t>(hidden);
          ptx::mbar_arrive_expect_tx(bar(kRawFull + slot),
                                     static_cast<uint32_t>(__popc(have) * box_bytes));
        }
        __syncwarp();
        if (id >= 0)
          ptx::tma_load_4d(sbase + L::kOffRaw + slot * L::kRawBytes +
                               static_cast<uint32_t>(lane * box_bytes),
                           is_v ? tm_v : tm_k, bar(kRawFull + slot), 0, 0, w.hk, id);
        ++ring;
      }
      if (!ok) break;
      if ((lane >> 3) == q)
        s_scale[(count & 15) * 8 + (lane & 7)] =
            make_float4(sc.x, log2f(sc.y), ids >= 0 ? 1.f / sc.y : 0.f, 0.f);
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(kCbScaleFull + (count & 15)));
      ++count;
    }
  } while (ok && w.next(a));
  if (!ok)  // let the copies in flight land before the CTA exits
    for (uint32_t n = ring > R ? ring - R : 0; n < ring; ++n)
      wait_drain(bar(kRawFull + n % R), (n / R) & 1u, ab, kStatusDrain);
  if constexpr (L::kDirect > 0) {
    constexpr uint32_t N = L::kDirect;
    if (!ok)
      for (uint32_t n = asked > N ? asked - N : 0; n < asked; ++n)
        wait_drain(bar(kKFull + n % N), (n / N) & 1u, ab, kStatusDrain);
  }
}

// ---- converters: warps 12-15. A thread takes 16 codes of a row at a time: 32
// bytes in two chunks of one of the row's 128-byte panels.
template <int D, int PARTS>
__device__ __forceinline__ void chunk_convert_role(const CacheAttnArgs& a, ChunkWalk w,
                                                   uint8_t* sgen, uint32_t sbase, uint32_t bars,
                                                   const AbortCtx& ab, int warp, int lane) {
  using L = ChunkLayout<D, PARTS>;
  constexpr int S = L::kStages, R = L::kRaw;
  constexpr int kRawFull = kCbKVFull + 2 * S, kRawFree = kRawFull + R;
  constexpr int kLanesPerRow = D / 16;
  constexpr int kRowsPerLoad = 4 * 32 / kLanesPerRow;  // of the four warps together
  constexpr int kLoads = kChunkKeys / kRowsPerLoad;
  auto bar = [&](int i) { return bars + 8u * static_cast<uint32_t>(i); };
  const int cw = warp & 3;
  // Row and chunk of a lane. d = 128: 16 lanes take two rows, eight of them the
  // first half of one row and the second half of the other, which conflicts
  // neither on the 128-byte rows read nor on the swizzled panels written. d = 64:
  // eight lanes take two rows of 64 bytes, one after another.
  const int l16 = lane & 15;
  const int r0 = D == 128 ? cw * 4 + (lane >> 4) * 2 + (((l16 >> 2) ^ (l16 >> 3)) & 1)
                          : cw * 8 + (lane >> 2);
  const int c = D == 128 ? (l16 & 7) : (lane & 3);
  const int panel = c >> 2;
  static_assert(kRowsPerLoad % 8 == 0, "one swizzle for all rows of a thread");
  const uint32_t row_at = static_cast<uint32_t>(panel * kPanelBytes + r0 * 128);
  const uint32_t ch = static_cast<uint32_t>(2 * (c & 3)), x7 = static_cast<uint32_t>(r0 & 7);
  const uint32_t to0 = row_at + ((ch ^ x7) << 4), to1 = row_at + (((ch + 1u) ^ x7) << 4);
  unsigned long long* const s_nan = reinterpret_cast<unsigned long long*>(sgen + L::kOffNan);
  volatile uint32_t* const s_any =
      reinterpret_cast<volatile uint32_t*>(sgen + L::kOffBar + kChunkSlotAnyNan);
  const uint8_t* const s_hidden = sgen + L::kOffBar + kChunkSlotHidden;
  uint32_t ring = 0, count = 0;  // slots filled, tiles done
  bool ok = true;
  do {
    const int first_seen = keys_seen(
        a, w.s, static_cast<int>(static_cast<long long>(w.rb) * a.item_rows / a.group));
    const int halves = L::kHalves * max(0, w.real_end - w.t0);  // (K and) V of each tile
#pragma unroll 1
    for (int h = 0; h < halves; ++h, ++ring) {
      const bool is_v = PARTS > 0 || (h & 1) != 0;
      const int key0 = (w.t0 + h / L::kHalves) * kChunkKeys;
      const uint32_t slot = ring % S, raw = ring % R;
      if (!(ok = wait_bounded_warp(bar(kRawFull + raw), (ring / R) & 1u, ab, kStatusProducer) &&
                 wait_bounded_warp(bar(kCbKVFull + S + slot), ((ring / S) & 1u) ^ 1u, ab,
                                   kStatusProducer)))
        break;
      const uint32_t src = sbase + L::kOffRaw + raw * L::kRawBytes +
                           static_cast<uint32_t>(r0 * D + 16 * c);
      const uint32_t dst = sbase + L::kOffKV + slot * L::kTileBytes;
      const uint32_t hidden = s_hidden[raw];
      const bool edge = hidden != 0u || (is_v && key0 + kChunkKeys > first_seen);
      if (edge) {
        // put right in the raw tile, each thread the codes that it reads below
#pragma unroll 1
        for (int l = 0; l < kLoads; ++l) {
          const int row = r0 + l * kRowsPerLoad, key = key0 + row;
          const uint32_t at = src + static_cast<uint32_t>(l * kRowsPerLoad * D);
          if (((hidden >> (row >> 4)) & 1u) || (is_v && key >= w.s.kv_len)) {
            ptx::st_shared_v4(at, 0u, 0u, 0u, 0u);
          } else if (is_v && key >= first_seen) {
            // seen by later rows only: a weight of 0 times NaN must not reach
            // the others, so NaN is taken out and its key noted per column
            const uint4 x = lds128(at);
            uint32_t v[4] = {x.x, x.y, x.z, x.w};
            if (nan_bytes(v[0]) | nan_bytes(v[1]) | nan_bytes(v[2]) | nan_bytes(v[3])) {
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const uint32_t bad = nan_bytes(v[q]);
                for (int y = 0; y < 4; ++y)
                  if ((bad >> (8 * y)) & 0x80u) {
                    *s_any = 1;
                    atomicMax(s_nan + (w.item & 7) * D + 16 * c + 4 * q + y,
                              (static_cast<unsigned long long>(w.item + 1) << 32) |
                                  static_cast<unsigned>(0x7FFFFFFF - key));
                    v[q] &= ~(0xFFu << (8 * y));
                  }
              }
              ptx::st_shared_v4(at, v[0], v[1], v[2], v[3]);
            }
          }
        }
      }
      uint4 x[kLoads];
#pragma unroll
      for (int l = 0; l < kLoads; ++l)
        x[l] = lds128(src + static_cast<uint32_t>(l * kRowsPerLoad * D));
#pragma unroll
      for (int l = 0; l < kLoads; ++l) {
        const uint32_t at = dst + static_cast<uint32_t>(l * kRowsPerLoad * 128);
        ptx::st_shared_v4(at + to0, widen_lo(x[l].x), widen_hi(x[l].x), widen_lo(x[l].y),
                          widen_hi(x[l].y));
        ptx::st_shared_v4(at + to1, widen_lo(x[l].z), widen_hi(x[l].z), widen_lo(x[l].w),
                          widen_hi(x[l].w));
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        ptx::mbar_arrive(bar(kRawFree + raw));
        ptx::mbar_arrive(bar(kCbKVFull + slot));
        if (is_v) ptx::mbar_arrive(bar(kCbVDone + (count & 7)));
      }
      count += is_v ? 1u : 0u;
    }
  } while (ok && w.next(a));
}

// S[tmem] = Q K^T with Q in PARTS tiles of e4m3 (K-major SW128, one after
// another) that add up to its rows, and K as the cache holds it.
template <int D, int PARTS>
__device__ __forceinline__ void issue_qk_parts(uint32_t d_tmem, uint64_t dq, uint64_t dk) {
  static_assert(D == 128, "a row is one 128-byte panel");
  constexpr uint32_t id = ptx::idesc_f8(128, 128);
#pragma unroll
  for (int p = 0; p < PARTS; ++p) {
    uint64_t k = dk;
#pragma unroll
    for (int kk = 0; kk < D / 32; ++kk) {
      ptx::umma_f8_ss_elect(d_tmem, dq, k, id, p + kk > 0 ? 1u : 0u);
      dq = desc_add(dq, kk + 1 < D / 32 ? 32u : static_cast<uint32_t>(kChunkKeys * D - 96));
      k = desc_add(k, 32u);
      asm volatile("" : "+l"(dq), "+l"(k));  // advance in place: three live descriptors
    }
  }
}

// O[tmem] (+)= P V over half `h` of a tile's keys: 64 keys of P in tensor memory.
template <int D>
__device__ __forceinline__ void issue_pv_half(uint32_t d_tmem, uint32_t p_tmem, uint64_t dv, int h,
                                              bool accumulate) {
  constexpr uint32_t id = ptx::idesc_f16(false, true, 128, D);
  dv = desc_add(dv, static_cast<uint32_t>(4 * 2048 * h));
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) {
    ptx::umma_f16_ts_elect(d_tmem, p_tmem + 8u * kk, dv, id, accumulate || kk > 0 ? 1u : 0u);
    dv = desc_add(dv, 2048u);
    asm volatile("" : "+l"(dv));
  }
}

// ---- MMA issue: warp 0
template <int D, int PARTS>
__device__ __forceinline__ void chunk_mma_role(const CacheAttnArgs& a, ChunkWalk w, uint32_t sbase,
                                               uint32_t bars, uint32_t tmem, const AbortCtx& ab) {
  using L = ChunkLayout<D, PARTS>;
  constexpr int S = L::kStages;
  auto bar = [&](int i) { return bars + 8u * static_cast<uint32_t>(i); };
  constexpr int N = PARTS > 0 ? L::kDirect : S;  // slots of K
  constexpr int kKFull = PARTS > 0 ? kCbKVFull + 2 * S + 2 * L::kRaw : kCbKVFull;
  const uint64_t dQ[2] = {desc_kmajor(sbase + L::kOffQ), desc_kmajor(sbase + L::kOffQ + L::kQBytes)};
  const uint64_t dK0 = desc_kmajor(sbase + (PARTS > 0 ? L::kOffK : L::kOffKV));
  const uint64_t dV0 = desc_v(sbase + L::kOffKV);
  const uint32_t tS[2] = {tmem + L::kColS, tmem + L::kColS + 128};
  const uint32_t tO[2] = {tmem + L::kColO, tmem + L::kColO + D};
  // K and V of tile t (of all that this CTA reads) as they were filled
  auto k_at = [](uint32_t t) { return PARTS > 0 ? t : 2u * t; };
  auto v_at = [](uint32_t t) { return PARTS > 0 ? t : 2u * t + 1u; };
  auto k_wait = [&](uint32_t t) {
    return wait_spin_warp(bar(kKFull + k_at(t) % N), (k_at(t) / N) & 1u, ab, kStatusMma);
  };
  auto v_wait = [&](uint32_t t) {
    return wait_spin_warp(bar(kCbKVFull + v_at(t) % S), (v_at(t) / S) & 1u, ab, kStatusMma);
  };
  auto k_free = [&](uint32_t t) { ptx::umma_commit_elect(bar(kKFull + N + k_at(t) % N)); };
  auto v_free = [&](uint32_t t) { ptx::umma_commit_elect(bar(kCbKVFull + S + v_at(t) % S)); };
  auto qk = [&](int q, int i, uint32_t t) {
    const uint64_t dk = desc_add(
        dK0, (k_at(t) % N) * static_cast<uint32_t>(PARTS > 0 ? L::kRawBytes : L::kTileBytes));
    if constexpr (PARTS > 0) issue_qk_parts<D, PARTS>(tS[i], dQ[q], dk);
    else issue_qk_desc<D, false, true>(tS[i], dQ[q], dk);
    ptx::umma_commit_elect(bar(kCbSFull + i));
  };
  auto v_desc = [&](uint32_t t) {
    return desc_add(dV0, (v_at(t) % S) * static_cast<uint32_t>(L::kTileBytes));
  };
  auto pv = [&](int i, uint32_t t, bool acc) {
    issue_pv_ts_desc<D, false, true>(tO[i], tS[i], v_desc(t), acc);
  };
  uint32_t done = 0, qn[2] = {0u, 0u}, pn[2] = {0u, 0u}, hn[2] = {0u, 0u};  // tiles, Q, P, P in halves
  bool ok = true;
  do {
    const int n = w.n();
    if (n == 0) continue;
    const bool pair = PARTS == 0 && w.rows(a) > 128;
    ok = wait_spin_warp(bar(kCbQFull + 0), (qn[0]++) & 1u, ab, kStatusMma) &&
         (!(pair || PARTS > 0) ||
          wait_spin_warp(bar(kCbQFull + 1), (qn[1]++) & 1u, ab, kStatusMma));
    if (!ok) break;
    if (pair) {
      if (!(ok = k_wait(done))) break;
      ptx::tc_fence_after();
      qk(0, 0, done);
      qk(1, 1, done);
      k_free(done);
      for (int j = 0; j < n && ok; ++j) {
        const uint32_t t = done + static_cast<uint32_t>(j);
        const bool more = j + 1 < n;
        if (!(ok = v_wait(t))) break;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (!(ok = wait_spin_warp(bar(kCbPFull + i), (pn[i]++) & 1u, ab, kStatusMma))) break;
          ptx::tc_fence_after();
          pv(i, t, j > 0);
          if (!more) {
            ptx::umma_commit_elect(bar(kCbOFull + i));
            continue;
          }
          if (i == 0) {
            if (!(ok = k_wait(t + 1u))) break;
            ptx::tc_fence_after();
          }
          qk(i, i, t + 1u);
        }
        if (!ok) break;
        v_free(t);
        if (more) k_free(t + 1u);
      }
    } else {
      for (int i = 0; i < 2 && i < n && ok; ++i) {
        if (!(ok = k_wait(done + i))) break;
        ptx::tc_fence_after();
        qk(0, i, done + i);
        k_free(done + i);
      }
      for (int j = 0; j < n && ok; ++j) {
        const int i = j & 1;
        const uint32_t t = done + static_cast<uint32_t>(j);
        if (!(ok = v_wait(t))) break;
        if (!(ok = wait_spin_warp(bar(kCbPSplit + i), (hn[i]++) & 1u, ab, kStatusMma))) break;
        ptx::tc_fence_after();
#pragma unroll
        for (int h = 0; h < 2; ++h) issue_pv_half<D>(tO[h], tS[i] + 64u * h, v_desc(t), h, j > 0);
        ptx::umma_commit_elect(bar(kCbOStep));
        v_free(t);
        if (j + 2 < n) {
          if (!(ok = k_wait(t + 2u))) break;
          ptx::tc_fence_after();
          qk(0, i, t + 2u);
          k_free(t + 2u);
        } else if (j + 1 == n) {
          ptx::umma_commit_elect(bar(kCbOFull + 0));
        }
      }
    }
    if (!ok) break;
    done += static_cast<uint32_t>(n);
  } while (w.next(a));
  ptx::umma_commit_elect(bar(kCbDrain));
  wait_drain(bar(kCbDrain), 0u, ab, kStatusDrain);
}

// ---- softmax and epilogue: warps 4-7 (tile 0) and 8-11 (tile 1)

// What a softmax warp needs between its tile loops only, kept in shared memory
// meanwhile (16 words a warp): the loop holds 128 scores in registers.
struct ChunkShelf {
  ChunkWalk w;
  uint32_t flags;  // parities: bits 0-1 items with O_i, bit 2 split items
  int share;
};
static_assert(sizeof(ChunkWalk) == 56 && sizeof(ChunkShelf) == 64, "16 words");

__device__ __forceinline__ void shelve(uint32_t at, const ChunkShelf& k, int lane) {
  uint32_t u[16];
  __builtin_memcpy(u, &k, 64);
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < 16; i += 4) ptx::st_shared_v4(at + 4u * i, u[i], u[i + 1], u[i + 2], u[i + 3]);
  }
  __syncwarp();
}
__device__ __forceinline__ ChunkShelf unshelve(uint32_t at) {
  uint32_t u[16];
#pragma unroll
  for (int i = 0; i < 16; i += 4) {
    const uint4 v = lds128(at + 4u * i);
    u[i] = v.x;
    u[i + 1] = v.y;
    u[i + 2] = v.z;
    u[i + 3] = v.w;
  }
  __syncwarp();
  ChunkShelf k;
  __builtin_memcpy(&k, u, 64);
  return k;
}

// Query token and head of row `r` of an item.
struct RowAt {
  int i, head;
};
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  __half2 x, y;
  __builtin_memcpy(&x, &a, 4);
  __builtin_memcpy(&y, &b, 4);
  x = __hsub2(x, y);
  __builtin_memcpy(&a, &x, 4);
  return a;
}

__device__ __forceinline__ RowAt row_at(const CacheAttnArgs& a, const ChunkWalk& w, int r) {
  const int row = w.rb * a.item_rows + r;  // (T * H is in int range)
  const int i = row / a.group;
  return {i, w.hk * a.group + row - i * a.group};
}

// The power of two that is 1 / 256 to 1 / 128 of the largest of the magnitudes whose
// 16-bit patterns `top` bounds (NaN if there is an infinity or NaN among them).
template <bool BF16>
__device__ __forceinline__ float e4m3_step(uint32_t top) {
  const float big = BF16 ? __uint_as_float(top << 16) : unpack_f16(top).x;
  const int e = max(static_cast<int>(__float_as_uint(big) >> 23) - 127 - 7, -126);
  const float fac = top == 0u ? 1.f : __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
  return top >= (BF16 ? 0x7F80u : 0x7C00u) ? __int_as_float(0x7FFFFFFF) : fac;
}

// Chunks e0 .. e1 - 1 (16 elements each) of this thread's query row p as PARTS
// e4m3 rows at `to` (row r of tiles of kChunkKeys rows) that add up to row / fac,
// whose largest magnitude is 128 to 256. bf16's 8-bit significands are the sum of
// two parts, fp16's 11 bits of three, as long as their last bit is not below e4m3's
// smallest step, 2^-9: for elements from 2^-9 (bf16) or 2^-6 (fp16) of the largest
// one on. Of smaller ones the last part is rounded, by 2^-10 at most, 2^-17 of the
// largest. A row with a few very large elements pays for it with its small ones.
template <int D, bool BF16, int PARTS>
__device__ __forceinline__ void query_parts(const uint16_t* p, float fac, uint32_t to, int r, int e0,
                                            int e1) {
  const float inv = 1.f / fac;
#pragma unroll 1  // (unrolled, it took longer to fetch than to run)
  for (int e = e0; e < e1; ++e) {
    const uint4 u0 = *reinterpret_cast<const uint4*>(p + 16 * e);
    const uint4 u1 = *reinterpret_cast<const uint4*>(p + 16 * e + 8);
    uint32_t h[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      float2 f;
      if constexpr (BF16)
        f = make_float2(__uint_as_float(h[x] << 16), __uint_as_float(h[x] & 0xFFFF0000u));
      else
        f = unpack_f16(h[x]);
      h[x] = pack_f16(f.x * inv, f.y * inv);
    }
#pragma unroll
    for (int q = 0; q < PARTS; ++q) {
      uint32_t code[4];
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const uint16_t c = ptx::f16x2_to_e4m3x2(h[x]);
        code[x >> 1] = x & 1 ? code[x >> 1] | (static_cast<uint32_t>(c) << 16) : c;
        if (q + 1 < PARTS) h[x] = sub_f16x2(h[x], ptx::e4m3x2_to_f16x2(c));
      }
      ptx::st_shared_v4(to + static_cast<uint32_t>(q * kChunkKeys * D + r * D) +
                            (static_cast<uint32_t>(e ^ (r & 7)) << 4),
                        code[0], code[1], code[2], code[3]);
    }
  }
}

// The first key of a block that exists in the share's tiles of the item (2^31 - 1:
// none). Called by whole warps.
__device__ __forceinline__ int first_key(const CacheAttnArgs& a, const ChunkWalk& w, int lane) {
  const int32_t* const table = a.table + static_cast<long long>(w.b) * a.table_width;
  const long long keys = min(static_cast<long long>(w.s.kv_len), 1LL * w.real_end * kChunkKeys);
  const int end = static_cast<int>((keys + (1 << a.block_shift) - 1) >> a.block_shift);
  for (int at = (w.t0 * kChunkKeys) >> a.block_shift; at < end; at += 32) {
    const int id = at + lane < end ? __ldg(table + at + lane) : -1;
    const uint32_t there = __ballot_sync(0xffffffffu, id >= 0 && id < a.num_blocks);
    if (there != 0u) return (at + __ffs(static_cast<int>(there)) - 1) << a.block_shift;
  }
  return 0x7FFFFFFF;
}

// The tiles of one item for a warpgroup: NC = 128, all keys of a tile for the rows
// of Q tile `wg` (pair mode), or NC = 64, half `wg` of the keys (split mode).
// S of tile j is in S_wg, or in that half of S_(j mod 2); P goes over it.
struct TileLoop {
  uint32_t tl, phase;  // tensor memory of the warp's lanes; parities (chunk_softmax_role)
  int wg, n, k0;       // tiles of the item, first key
  uint32_t count;      // tiles before the item
  int lim, lim0;       // keys that the row and that all rows see
  float crow;
  bool idle;
};
template <int D, int NC, int PARTS>
__device__ __forceinline__ bool softmax_tiles(const CacheAttnArgs& a, const TileLoop& x,
                                              const uint8_t* sgen, uint32_t bars,
                                              const AbortCtx& ab, float& m_ref, float& l) {
  using L = ChunkLayout<D, PARTS>;
  constexpr bool kHalf = NC == 64;
  constexpr int G = NC / 16;
  auto bar = [&](int i) { return bars + 8u * static_cast<uint32_t>(i); };
  const uint32_t tO = x.tl + L::kColO + static_cast<uint32_t>(D * x.wg);
  const bool one_scale = a.block_shift == 7;  // a tile is one block
  int k0 = x.k0 + (kHalf ? 64 * x.wg : 0);
  for (int j = 0; j < x.n; ++j, k0 += kChunkKeys) {
    const int b = kHalf ? j & 1 : x.wg;
    const uint32_t tix = x.count + static_cast<uint32_t>(j);
    const uint32_t tS = x.tl + L::kColS + static_cast<uint32_t>(128 * b + (kHalf ? 64 * x.wg : 0));
    if (!(wait_bounded_warp(bar(kCbSFull + b),
                            ((x.phase >> b) ^ static_cast<uint32_t>(kHalf ? j >> 1 : j)) & 1u, ab,
                            kStatusSoftmax) &&
          wait_bounded_warp(bar(kCbScaleFull + (tix & 15u)), (tix >> 4) & 1u, ab, kStatusSoftmax)))
      return false;
    ptx::tc_fence_after();
    const uint32_t p_bar = bar(kHalf ? kCbPSplit + b : kCbPFull + x.wg);
    if (x.idle) {
      ptx::tc_fence_before();
      ptx::mbar_arrive(p_bar);
      continue;
    }
    uint32_t sr[NC / 64][2][32];
    float mx_lo, mx_hi;
    ptx::tmem_ld64_max(tS, sr[0], mx_lo);
    if constexpr (kHalf) {
      ptx::tmem_ld_wait(sr[0][0]);
      ptx::tmem_ld_wait(sr[0][1]);
      mx_hi = mx_lo;
    } else {
      ptx::tmem_ld64_max(tS + 64u, sr[NC / 64 - 1], mx_hi);
      ptx::tmem_ld_wait64x2(sr[0], sr[NC / 64 - 1]);
    }
    ptx::tmem_ld_wait_f2(mx_lo, mx_hi);
    float s[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) s[c] = __uint_as_float(sr[c >> 6][(c >> 5) & 1][c & 31]);
    const float4* const sc = reinterpret_cast<const float4*>(sgen + L::kOffScale) +
                             (tix & 15u) * 8 + (kHalf ? 4 * x.wg : 0);
    auto scales = [&](int g) {  // {ks, log2 vs, 1 / vs} of a 16-key group
      const float4 v = sc[g];
      return make_float3(v.x * x.crow, v.y, v.z);
    };
    const bool need_mask = k0 + NC > x.lim0;
    float m_tile;
    if (one_scale && !need_mask) {
      const float3 f = scales(0);
      m_tile = fmaf(fmaxf(mx_lo, mx_hi), f.x, f.y);
    } else {
      if (need_mask) {
        const int see = x.lim - k0;
#pragma unroll
        for (int c = 0; c < NC; ++c) s[c] = c < see ? s[c] : -INFINITY;
      }
      m_tile = -INFINITY;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const float3 f = scales(g);
        float t0 = fmaxf(s[16 * g], s[16 * g + 1]), t1 = fmaxf(s[16 * g + 2], s[16 * g + 3]);
#pragma unroll
        for (int c = 4; c < 16; c += 4) {
          t0 = ptx::fmax3(t0, s[16 * g + c], s[16 * g + c + 1]);
          t1 = ptx::fmax3(t1, s[16 * g + c + 2], s[16 * g + c + 3]);
        }
        m_tile = fmaxf(m_tile, fmaf(fmaxf(t0, t1), f.x, f.y));
      }
    }
    float alpha = 1.f;
    if (m_tile > m_ref + kWeightMost) {
      m_tile -= kWeightLift;
      alpha = ptx::ex2(m_ref - m_tile);  // (0 for the first visible tile)
      m_ref = m_tile;
    }
    const float neg = m_ref == -INFINITY ? 0.f : -m_ref;
    l *= alpha;
    uint32_t pk[NC / 64][32];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const float3 f = scales(g);
      const float add = f.y + neg;
      const float2 f2 = make_float2(f.x, f.x), a2 = make_float2(add, add);
      float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float2 t = ptx::ffma2(make_float2(s[16 * g + 2 * c], s[16 * g + 2 * c + 1]), f2, a2);
        const float p0 = ptx::ex2(t.x), p1 = ptx::ex2(t.y);
        // (one fp16 value, for fp16 queries too: a second part, which the step kernel
        // keeps for them, would double the products with V here. Relative error of
        // fp16 drafts against 64 bits 2.9e-4, of which rounding O is 2.1e-4.)
        pk[g >> 2][(g & 3) * 8 + c] = pack_weights(p0, p1);
        if (c & 1) sum1 = ptx::fadd2(sum1, make_float2(p0, p1));
        else sum0 = ptx::fadd2(sum0, make_float2(p0, p1));
      }
      sum0 = ptx::fadd2(sum0, sum1);
      l = fmaf(sum0.x + sum0.y, f.z, l);
    }
    ptx::tmem_st32(tS, pk[0]);
    if constexpr (!kHalf) ptx::tmem_st32(tS + 32u, pk[NC / 64 - 1]);
    if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
      // O has to hold the products so far. Pair mode: S_wg's commit came after the
      // last of them. Split mode: S of this tile was formed before them.
      if constexpr (kHalf) {
        if (!wait_bounded_warp(bar(kCbOStep), ((x.phase >> 2) + static_cast<uint32_t>(j - 1)) & 1u, ab,
                               kStatusSoftmax))
          return false;
        ptx::tc_fence_after();
      }
      const float2 a2 = make_float2(alpha, alpha);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        ptx::tmem_ld32(tO + 32u * c, o);
        ptx::tmem_ld_wait(o);
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const float2 v =
              ptx::fmul2(make_float2(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), a2);
          o[e] = __float_as_uint(v.x);
          o[e + 1] = __float_as_uint(v.y);
        }
        ptx::tmem_st32(tO + 32u * c, o);
      }
    }
    ptx::tmem_st_wait();
    ptx::tc_fence_before();
    ptx::mbar_arrive(p_bar);
  }
  return true;
}

template <int D, bool BF16, int PARTS>
__device__ __forceinline__ void chunk_softmax_role(const CacheAttnArgs& a, const ChunkWalk& start,
                                                   int share, uint8_t* sgen, uint32_t sbase,
                                                   uint32_t bars, uint32_t tmem, const AbortCtx& ab,
                                                   int warp, int lane) {
  using L = ChunkLayout<D, PARTS>;
  constexpr int kLanes = D / 8, kRowsPerTurn = 32 / kLanes;  // 16 bytes of a 16-bit row each
  auto bar = [&](int i) { return bars + 8u * static_cast<uint32_t>(i); };
  const int wg = (warp >> 2) - 1;
  const int r = (warp & 3) * 32 + lane;
  const uint32_t tl = ptx::tmem_lane_base(tmem, warp);
  const uint32_t shelf = sbase + L::kOffShelf + static_cast<uint32_t>(warp - 4) * 64u;
  uint32_t phase = 0, count = 0;  // parities (bits 0, 1: S_i; 2: O steps); tiles before the item
  shelve(shelf, ChunkShelf{start, 0u, share}, lane);
  for (;;) {
    // ---- an item: Q, and what its tile loop needs
    int n;
    bool in_pairs;
    TileLoop x;
    x.crow = a.scale_log2;
    {
      const ChunkShelf k = unshelve(shelf);
      const ChunkWalk& w = k.w;
      n = w.n();
      const int rows = w.rows(a);
      const bool pair = PARTS == 0 && rows > 128;
      const int base = pair ? 128 * wg : 0;  // the tile's first row
      in_pairs = pair;
      x.tl = tl;
      x.phase = phase;
      x.wg = wg;
      x.n = n;
      x.count = count;
      x.k0 = w.t0 * kChunkKeys;
      x.lim = keys_seen(a, w.s, row_at(a, w, base + r < rows ? base + r : 0).i);
      x.lim0 = keys_seen(a, w.s, row_at(a, w, base).i);
      // (a warp without rows hands P over as it is: its rows of O are not read)
      x.idle = base + r - lane >= rows;
      if (n > 0) {
        // this thread's row of Q into the swizzled layout. (A row for each thread,
        // not 16 lanes to a row, which reads whole lines but has to loop over the
        // rows: 2048 x 16384 chunk 387 us, 378 so. Unrolled, that loop's code alone
        // took longer to fetch than the rows: 415 us.)
        const bool there = base + r < rows;
        const RowAt at = row_at(a, w, there ? base + r : 0);
        const uint16_t* p = static_cast<const uint16_t*>(a.q) + q_offset(a, w.b, w.s, at.i, at.head);
        float fac;
        if constexpr (PARTS > 0) {
          uint32_t top = 0;
          if (there) {
#pragma unroll
            for (int e = 0; e < D / 8; ++e) {
              const uint4 v = *reinterpret_cast<const uint4*>(p + 8 * e);
              constexpr uint32_t kAbs = 0x7FFF7FFFu;
              top = __vmaxu2(__vmaxu2(top, __vmaxu2(v.x & kAbs, v.y & kAbs)),
                             __vmaxu2(v.z & kAbs, v.w & kAbs));
            }
          }
          fac = e4m3_step<BF16>(max(top & 0xFFFFu, top >> 16));
          // each warpgroup writes half of the row
          if (there)
            query_parts<D, BF16, PARTS>(p, fac, sbase + L::kOffQ, r, wg * (D / 32),
                                        (wg + 1) * (D / 32));
        } else {
          uint32_t q[D / 2];
#pragma unroll
          for (int e = 0; e < D / 8; ++e) {
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (there) v = *reinterpret_cast<const uint4*>(p + 8 * e);
            q[4 * e] = v.x;
            q[4 * e + 1] = v.y;
            q[4 * e + 2] = v.z;
            q[4 * e + 3] = v.w;
          }
          if constexpr (!BF16) inf_to_nan<D / 2>(q);
          fac = rows_to_f16<D / 2, 1, BF16>(q);
          if (pair || wg == 0) {
            const uint32_t to = sbase + L::kOffQ +
                                static_cast<uint32_t>((pair ? wg : 0) * L::kQBytes + r * 128);
#pragma unroll
            for (int e = 0; e < D / 8; ++e)
              ptx::st_shared_v4(to + (e >> 3) * kPanelBytes +
                                    (static_cast<uint32_t>((e & 7) ^ (r & 7)) << 4),
                                q[4 * e], q[4 * e + 1], q[4 * e + 2], q[4 * e + 3]);
          }
        }
        // (so that c ks does not underflow to 0, and -inf times it to NaN, for a hidden
        // key: at 2^-80 the scores are nothing, S being 2^32 at most. A row without a
        // value has NaN in Q, and a factor that leaves its hidden keys hidden.)
        x.crow = fmaxf(x.crow * fac, 0x1p-80f);
        if (PARTS > 0 || pair || wg == 0) {
          ptx::fence_proxy_async_smem();
          ptx::mbar_arrive(bar(kCbQFull + wg));
        }
      }
    }
    float m_ref = -INFINITY, l = 0.f;
    if (PARTS == 0 && in_pairs) {
      if (!softmax_tiles<D, 128, PARTS>(a, x, sgen, bars, ab, m_ref, l)) return;
      phase ^= n & 1 ? 3u : 0u;
    } else {
      if (!softmax_tiles<D, 64, PARTS>(a, x, sgen, bars, ab, m_ref, l)) return;
      phase ^= static_cast<uint32_t>((((n + 1) >> 1) & 1) | (n & 2) | ((n & 1) << 2));
    }

    // ---- epilogue
    ChunkShelf k = unshelve(shelf);
    ChunkWalk& w = k.w;
    const int rows = w.rows(a);
    const bool pair = PARTS == 0 && rows > 128;
    const int base = pair ? 128 * wg : 0;
    const bool there = base + r < rows;
    const bool works = n > 0;
    const bool begins = w.t0 == 0, ends = w.t1 == w.tiles;
    float* part = nullptr;
    if (!begins || !ends)
      part = a.parts + (2LL * blockIdx.x + (begins ? 1 : 0)) * partial_floats(a.item_rows, D);
    if (!ends && begins && wg == 0 && r == 0)
      a.join[blockIdx.x] =
          join_item(w.b, w.hk, w.rb, rows, 1 + (w.tiles - w.t1 + k.share - 1) / k.share);
    const bool two = !pair;  // results of two warpgroups
    float* const s_m = reinterpret_cast<float*>(sgen + L::kOffStats);
    if (two && wg == 1) {
      s_m[r] = m_ref;
      s_m[128 + r] = l;
      ptx::mbar_arrive(bar(kCbStats));
    }
    if (pair || wg == 0) {
      // the last V of the item has been converted: its NaN columns are known
      if (n > 0) {
        const uint32_t tix = count + static_cast<uint32_t>(n - 1);
        if (!wait_bounded_warp(bar(kCbVDone + (tix & 7u)), (tix >> 3) & 1u, ab, kStatusEpilogue))
          return;
      }
      float f0 = 1.f, f1 = 0.f;  // factors of O of this and of the other warpgroup
      if (works &&
          !wait_bounded_warp(bar(kCbOFull + wg), (k.flags >> wg) & 1u, ab, kStatusEpilogue))
        return;
      if (two) {
        if (!wait_bounded_warp(bar(kCbStats), (k.flags >> 2) & 1u, ab, kStatusEpilogue)) return;
        const float m1 = s_m[r], l1 = s_m[128 + r];
        const float top = fmaxf(m_ref, m1);
        f0 = m_ref == -INFINITY ? 0.f : ptx::ex2(m_ref - top);
        f1 = m1 == -INFINITY ? 0.f : ptx::ex2(m1 - top);
        l = l * f0 + l1 * f1;
        m_ref = top;
      }
      ptx::tc_fence_after();
      // Scores of NaN, which a row without a value has against the zeros of hidden
      // blocks too: where it sees no other keys they count for nothing.
      if (__any_sync(0xffffffffu, l != l)) {
        const int first = first_key(a, w, lane);
        if (l != l && x.lim <= first) {
          m_ref = -INFINITY;
          l = 0.f;
        }
      }
      const bool none = no_weight(m_ref, l);
      if (part == nullptr) {
        const float inv = none ? 0.f : 1.f / l;
        f0 *= inv;
        f1 *= inv;
        if (there) {
          const RowAt at = row_at(a, w, base + r);
          a.lse[lse_index(a, w.b, w.s, at.i, at.head)] =
              none ? -INFINITY : (m_ref + log2f(l)) * 0.69314718055994531f;
        }
      } else if (there) {
        part[a.item_rows * D + base + r] = m_ref;
        part[a.item_rows * D + a.item_rows + base + r] = l;
      }
      const uint32_t sQ = sbase + L::kOffQ + static_cast<uint32_t>((pair ? wg : 0) * L::kQBytes);
      const uint32_t tO0 = tl + L::kColO + static_cast<uint32_t>(D) * wg;
      const unsigned long long* nan =
          reinterpret_cast<const unsigned long long*>(sgen + L::kOffNan) + (w.item & 7) * D;
      const bool any_nan = *reinterpret_cast<const volatile uint32_t*>(sgen + L::kOffBar +
                                                                       kChunkSlotAnyNan) != 0u;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        float v[32];
        if (works) {
          uint32_t o[32];
          ptx::tmem_ld32(tO0 + 32u * c, o);
          ptx::tmem_ld_wait(o);
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = none ? 0.f : __uint_as_float(o[e]) * f0;
          if (two) {
            ptx::tmem_ld32(tO0 + D + 32u * c, o);
            ptx::tmem_ld_wait(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = none ? 0.f : fmaf(__uint_as_float(o[e]), f1, v[e]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = 0.f;
        }
        if (any_nan) {
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const unsigned long long u = nan[32 * c + e];
            if (static_cast<int>(u >> 32) == w.item + 1 &&
                0x7FFFFFFF - static_cast<int>(u & 0xFFFFFFFFu) < x.lim)
              v[e] = __int_as_float(0x7FFFFFFF);
          }
        }
        if (part == nullptr) {
          // through the Q tile, whose products are done: the rows' chunks, swizzled
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            const uint32_t ch = static_cast<uint32_t>(4 * c + e / 8);
            ptx::st_shared_v4(sQ + static_cast<uint32_t>(r) * 128u + (ch >> 3) * kPanelBytes +
                                  (((ch & 7u) ^ static_cast<uint32_t>(r & 7)) << 4),
                              pack2<BF16>(v[e], v[e + 1]), pack2<BF16>(v[e + 2], v[e + 3]),
                              pack2<BF16>(v[e + 4], v[e + 5]), pack2<BF16>(v[e + 6], v[e + 7]));
          }
        } else if (there) {
          // partial results column by column: neighbouring rows are neighbours
#pragma unroll
          for (int e = 0; e < 32; ++e) part[(32 * c + e) * a.item_rows + base + r] = v[e];
        }
        __syncwarp();
      }
      if (part == nullptr) {
        const int e = lane % kLanes, tr0 = (warp & 3) * 32 + lane / kLanes;
        RowAt at = row_at(a, w, base + tr0);
        int j = at.head - w.hk * a.group;
#pragma unroll 1
        for (int tr = tr0; tr < tr0 + 32 && base + tr < rows; tr += kRowsPerTurn) {
          const uint4 x = lds128(sQ + (e >> 3) * kPanelBytes + static_cast<uint32_t>(tr) * 128u +
                                 (static_cast<uint32_t>((e & 7) ^ (tr & 7)) << 4));
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) +
                                    o_offset(a, w.b, w.s, at.i, w.hk * a.group + j) + 8 * e) = x;
          for (j += kRowsPerTurn; j >= a.group; j -= a.group) ++at.i;
        }
        __syncwarp();
      }
      ptx::tc_fence_before();
      if (two) ptx::mbar_arrive(bar(kCbMerged));
    } else if (two) {
      // O1 and the stats are free for the next item only when they have been read
      if (!wait_bounded_warp(bar(kCbMerged), (k.flags >> 2) & 1u, ab, kStatusEpilogue)) return;
      ptx::tc_fence_after();
    }
    k.flags ^= (n > 0 ? 1u | (pair ? 2u : 0u) : 0u) | (two ? 4u : 0u);
    count += static_cast<uint32_t>(n);
    if (!w.next(a)) return;
    shelve(shelf, k, lane);
  }
}

template <int D, bool BF16, int PARTS>
__global__ void __launch_bounds__(kChunkThreads, 1)
    fa_cache_chunk_kernel(const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v, const CacheAttnArgs a) {
  using L = ChunkLayout<D, PARTS>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* sgen = smem_raw + (sbase - raw);
  const uint32_t bars = sbase + L::kOffBar;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sgen + L::kOffBar + kChunkSlotTmem);
  volatile uint32_t* abort_flag =
      reinterpret_cast<volatile uint32_t*>(sgen + L::kOffBar + kChunkSlotAbort);
  int* const s_start = reinterpret_cast<int*>(sgen + L::kOffBar + kChunkSlotStart);  // b, hk, rb, t0
  long long* const s_scan = reinterpret_cast<long long*>(sgen);  // (before Q)
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const AbortCtx ab{abort_flag, a.status};
  auto bar = [&](int i) { return bars + 8u * static_cast<uint32_t>(i); };
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(bar(kCbQFull + i), 128);
      ptx::mbar_init(bar(kCbSFull + i), 1);
      ptx::mbar_init(bar(kCbPFull + i), 128);
      ptx::mbar_init(bar(kCbOFull + i), 1);
    }
    ptx::mbar_init(bar(kCbStats), 128);
    ptx::mbar_init(bar(kCbMerged), 128);
    ptx::mbar_init(bar(kCbDrain), 1);
    ptx::mbar_init(bar(kCbPSplit), 256);
    ptx::mbar_init(bar(kCbPSplit + 1), 256);
    ptx::mbar_init(bar(kCbOStep), 1);
    for (int i = 0; i < 16; ++i) ptx::mbar_init(bar(kCbScaleFull + i), 1);
    for (int i = 0; i < 8; ++i) ptx::mbar_init(bar(kCbVDone + i), 4);
    for (int i = 0; i < L::kStages; ++i) {
      ptx::mbar_init(bar(kCbKVFull + i), 4);
      ptx::mbar_init(bar(kCbKVFull + L::kStages + i), 1);
    }
    for (int i = 0; i < L::kRaw; ++i) {
      ptx::mbar_init(bar(kCbKVFull + 2 * L::kStages + i), 1);
      ptx::mbar_init(bar(kCbKVFull + 2 * L::kStages + L::kRaw + i), 4);
    }
    for (int i = 0; i < 2 * L::kDirect; ++i)
      ptx::mbar_init(bar(kCbKVFull + 2 * L::kStages + 2 * L::kRaw + i), 1);
    *abort_flag = 0u;
    *reinterpret_cast<uint32_t*>(sgen + L::kOffBar + kChunkSlotAnyNan) = 0u;
    ptx::fence_mbar_init();
    a.join[blockIdx.x] = JoinItem{0, 0, 0, 0};
  }
  for (int i = tid; i < 8 * D; i += kChunkThreads)
    reinterpret_cast<unsigned long long*>(sgen + L::kOffNan)[i] = 0ull;

  // this CTA's share of the list of tiles
  constexpr int kWarps = kChunkThreads / 32;
  const int run = (a.B + kChunkThreads - 1) / kChunkThreads;
  const int b0 = min(tid * run, a.B), b1 = min(b0 + run, a.B);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += a.Hkv * chunk_head_tiles(a, seq_rows(a, b));
  long long upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += u;
  }
  if (lane == 31) s_scan[warp] = upto;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int k = 0; k < kWarps; ++k) {
    if (k < warp) upto += s_scan[k];
    total += s_scan[k];
  }
  const long long share = max((total + gridDim.x - 1) / gridDim.x,
                              static_cast<long long>(kChunkMinShare));
  const long long u0 = share * blockIdx.x, u1 = min(u0 + share, total);
  if (u0 >= u1) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  if (u0 >= upto - mine && u0 < upto) {
    long long at = upto - mine, head_tiles;
    int b = b0;
    SeqRows s;
    for (;; ++b) {
      s = seq_rows(a, b);
      head_tiles = chunk_head_tiles(a, s);
      if (u0 < at + a.Hkv * head_tiles) break;
      at += a.Hkv * head_tiles;
    }
    const int hk = static_cast<int>((u0 - at) / head_tiles);
    long long rest = u0 - at - hk * head_tiles;
    int rb = 0;
    for (;; ++rb) {
      const int n = max(1, chunk_real_tiles(a, s, rb));
      if (rest < n) break;
      rest -= n;
    }
    s_start[0] = b;
    s_start[1] = hk;
    s_start[2] = rb;
    s_start[3] = static_cast<int>(rest);
  }
  if (warp == 0) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), L::kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  ChunkWalk w;
  w.start(a, s_start[0], s_start[1], s_start[2], s_start[3], u1 - u0);

  const int wgrp = warp >> 2;
  if (wgrp == 0) {
    ptx::setmaxnreg_dec<kChunkRegsMma>();
    if (warp == 0) chunk_mma_role<D, PARTS>(a, w, sbase, bars, tmem, ab);
    else if (warp == 1) chunk_copy_role<D, PARTS>(&tm_k, &tm_v, a, w, sgen, sbase, bars, ab, lane);
  } else if (wgrp < 3) {
    ptx::setmaxnreg_inc<kChunkRegsSoftmax>();
    chunk_softmax_role<D, BF16, PARTS>(a, w, static_cast<int>(share), sgen, sbase, bars, tmem, ab, warp,
                                lane);
  } else {
    ptx::setmaxnreg_dec<kChunkRegsConvert>();
    chunk_convert_role<D, PARTS>(a, w, sgen, sbase, bars, ab, warp, lane);
  }
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 0) ptx::tmem_dealloc(tmem, L::kTmemCols);
  // This launch may run beside the step kernel's last CTAs. It ends behind it,
  // so that the join, which waits for this one, finds both complete.
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

}  // namespace fa
