// fa_fwd_cache for many query rows: S = Q K^T and O += P V on tcgen05 with S, P
// and O in tensor memory, from the cache's 8-bit blocks.
//
// A work item is a sequence, a K / V head and up to 256 of the rows that share
// it (query token i, group member j: row i * group + j, so later rows see at
// least as many keys). More than 128 rows: two tiles of 128 that share every
// KV tile of 128 keys, and the softmax of one runs while the tensor core works
// for the other (pair mode). At most 128 rows, a group's drafts or the last
// rows of a chunk: both halves of the machine work on the same rows, one on
// the even KV tiles and one on the odd ones, and their results are merged
// from tensor memory at the end (split mode).
//
// kind::f16 on fp16 operands whatever the queries' type: every e4m3 code is an
// fp16 value, so K and V lose nothing (the 8-bit kind would need Q and P in 8
// bits, 2^-4 each), and bf16 queries are brought into fp16's range row by row
// with a power of two (rows_to_f16). TMA brings the blocks that the table lists
// into a ring of 8-bit tiles; converter warps widen them into the swizzled
// operand tiles, and zero what no row may see.
//
// Both scales go into the exponent, as in fa_cache_step.cuh: e = c ks s + log2
// vs, P' = 2^(e - m), O = sum P' v8, l = sum P' / vs.
//
// Warp roles (16 warps):
//   warp 0       issues the MMAs (elected lane), owns the tensor memory
//   warp 1       copies: table entries, scales, TMA
//   warps 4-7    softmax and epilogue of tile 0 (split mode: even KV tiles)
//   warps 8-11   softmax and epilogue of tile 1 (split mode: odd KV tiles)
//   warps 12-15  converters
// Tensor memory: S0 0-127, S1 128-255, O0 256.., O1 256 + D..; P_i goes over the
// first 64 columns of S_i.
//
// Splitting: as in fa_cache_step.cuh, the items' tiles form one list that is
// cut into equal shares, one for each SM; fa_cache_join_kernel joins the
// partial results of cut items.
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

template <int D>
struct ChunkLayout {
  static constexpr int kPanels = D / 64;
  static constexpr int kTileBytes = kPanels * kPanelBytes;  // 128 rows of fp16
  static constexpr int kRawBytes = kChunkKeys * D;          // 128 rows of codes
  static constexpr int kStages = D == 128 ? 3 : 6;          // K / V slots (fp16)
  static constexpr int kRaw = D == 128 ? 3 : 6;             // K / V slots (codes)
  static constexpr int kOffQ = 0;                           // Q0, Q1
  static constexpr int kOffKV = 2 * kTileBytes;
  static constexpr int kOffRaw = kOffKV + kStages * kTileBytes;
  // scales of a tile's 16-key groups: [16 tiles][8] {ks, log2 vs, 1 / vs, 0}
  static constexpr int kOffScale = kOffRaw + kRaw * kRawBytes;
  static constexpr int kOffNan = kOffScale + 16 * 8 * 16;    // [8 items][D] uint64
  static constexpr int kOffStats = kOffNan + 8 * D * 8;      // [2][128] m, l of the odd tiles
  static constexpr int kOffShelf = kOffStats + 1024;  // [8 warps] 64 bytes
  static constexpr int kOffBar = kOffShelf + 512;
  static constexpr int kSmem = kOffBar + 512 + 1024;  // barriers, alignment slack
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kColS = 0, kColO = 256;
  static_assert(kSmem <= 232448, "shared memory budget");
  static_assert(kRaw <= 8 && kStages + kRaw <= 12, "barrier block");
};

enum ChunkBar : int {
  kCbQFull = 0,       // [2] 128 softmax threads: Q_i in shared memory
  kCbSFull = 2,       // [2] MMA: S_i ready
  kCbPFull = 4,       // [2] 128 softmax threads: P_i written, O_i rescaled
  kCbOFull = 6,       // [2] MMA: the item's last O_i += P_i V done
  kCbStats = 8,       // 128 threads of tile 1: its m, l in shared memory (split mode)
  kCbMerged = 9,      // 128 threads of tile 0: O1 and the stats read (split mode)
  kCbDrain = 10,      // MMA: every tcgen05 op completed
  kCbScaleFull = 11,  // [16] copy warp: scales of tile n in entry n % 16
  kCbVDone = 27,      // [8] converter warps: V of tile n converted (its NaN recorded)
  // [stages] converter warps: operand slot filled; [stages] MMA: slot free;
  // [raw] TMA: raw slot filled; [raw] converter warps: slot free
  kCbKVFull = 35,
};
constexpr int kChunkSlotTmem = 480, kChunkSlotAbort = 484, kChunkSlotStart = 488;
constexpr int kChunkSlotHidden = 504;  // [raw] bytes: bit g: 16-key group g is hidden

// Keys that query token i of a sequence sees.
__device__ __forceinline__ int keys_seen(const CacheAttnArgs& a, const SeqRows& s, int i) {
  return a.causal ? min(max(s.kv_len - s.count + i + 1, 0), s.kv_len) : s.kv_len;
}

// Row blocks of a sequence, and the tiles that one of them reads (counted: at
// least one, so that rows without keys are written).
__device__ __forceinline__ int chunk_row_blocks(const CacheAttnArgs& a, const SeqRows& s) {
  return takes_seq(a, s) ? static_cast<int>(
                               (static_cast<long long>(s.count) * a.group + kChunkRows - 1) / kChunkRows)
                         : 0;
}
__device__ __forceinline__ int chunk_real_tiles(const CacheAttnArgs& a, const SeqRows& s, int rb) {
  const long long last = min((rb + 1LL) * kChunkRows, static_cast<long long>(s.count) * a.group) - 1;
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
    return static_cast<int>(min(static_cast<long long>(kChunkRows),
                                static_cast<long long>(s.count) * a.group -
                                    static_cast<long long>(rb) * kChunkRows));
  }
  __device__ __forceinline__ int n() const { return max(0, real_end - t0); }
};

// ---- copies: warp 1. Lane j < 128 / block handles the j-th block of a tile,
// lane g < 8 the scales of the g-th 16-key group.
template <int D>
__device__ __forceinline__ void chunk_copy_role(const CUtensorMap* tm_k, const CUtensorMap* tm_v,
                                                const CacheAttnArgs& a, ChunkWalk w, uint8_t* sgen,
                                                uint32_t sbase, uint32_t bars, const AbortCtx& ab,
                                                int lane) {
  using L = ChunkLayout<D>;
  constexpr int R = L::kRaw;
  constexpr int kRawFull = kCbKVFull + 2 * L::kStages, kRawFree = kRawFull + R;
  auto bar = [&](int i) { return bars + 8u * static_cast<uint32_t>(i); };
  float4* const s_scale = reinterpret_cast<float4*>(sgen + L::kOffScale);
  uint8_t* const s_hidden = sgen + L::kOffBar + kChunkSlotHidden;
  const int boxes = kChunkKeys >> a.block_shift, box_bytes = D << a.block_shift;
  if (lane == 0) {
    ptx::prefetch_tmap(tm_k);
    ptx::prefetch_tmap(tm_v);
  }
  uint32_t ring = 0, count = 0;
  bool ok = true;
  do {
    // the table entry of this lane's block in tile t, or -1
    auto entry = [&](int t) {
      const long long key = static_cast<long long>(t) * kChunkKeys + (lane << a.block_shift);
      int id = -1;
      if (lane < boxes && key < w.s.kv_len)
        id = __ldg(a.table + static_cast<long long>(w.b) * a.table_width + (key >> a.block_shift));
      return id >= 0 && id < a.num_blocks ? id : -1;
    };
    int next = w.t0 < w.real_end ? entry(w.t0) : -1;
    for (int t = w.t0; t < w.real_end; ++t) {
      const int id = next;
      const uint32_t have = __ballot_sync(0xffffffffu, id >= 0);
      // this lane's 16-key group
      const int gid = __shfl_sync(0xffffffffu, id, (lane & 7) >> (a.block_shift - 4));
      const uint32_t hidden = __ballot_sync(0xffffffffu, lane < 8 && gid < 0);
      float ks = 1.f, vs = 1.f;
      if (lane < 8 && gid >= 0) {
        const long long at = static_cast<long long>(gid) * a.Hkv + w.hk;
        ks = __ldg(a.ks + at);
        vs = __ldg(a.vs + at);
      }
      if (t + 1 < w.real_end) next = entry(t + 1);
#pragma unroll
      for (int is_v = 0; is_v < 2; ++is_v) {
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
      if (lane < 8)
        s_scale[(count & 15) * 8 + lane] = gid >= 0
                                               ? make_float4(ks, log2f(vs), 1.f / vs, 0.f)
                                               : make_float4(1.f, -INFINITY, 0.f, 0.f);
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(kCbScaleFull + (count & 15)));
      ++count;
    }
  } while (ok && w.next(a));
  if (!ok)  // let the copies in flight land before the CTA exits
    for (uint32_t n = ring > R ? ring - R : 0; n < ring; ++n)
      wait_drain(bar(kRawFull + n % R), (n / R) & 1u, ab, kStatusDrain);
}

// ---- converters: warps 12-15. A thread takes 16 codes of a row at a time: 32
// bytes in two chunks of one of the row's 128-byte panels.
template <int D>
__device__ __forceinline__ void chunk_convert_role(const CacheAttnArgs& a, ChunkWalk w,
                                                   uint8_t* sgen, uint32_t sbase, uint32_t bars,
                                                   const AbortCtx& ab, int warp, int lane) {
  using L = ChunkLayout<D>;
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
  const uint8_t* const s_hidden = sgen + L::kOffBar + kChunkSlotHidden;
  uint32_t ring = 0, count = 0;  // slots filled, tiles done
  bool ok = true;
  do {
    const int first_seen = keys_seen(
        a, w.s, static_cast<int>(static_cast<long long>(w.rb) * kChunkRows / a.group));
    const int halves = 2 * max(0, w.real_end - w.t0);  // K and V of each tile
#pragma unroll 1
    for (int h = 0; h < halves; ++h, ++ring) {
      const bool is_v = (h & 1) != 0;
      const int key0 = (w.t0 + (h >> 1)) * kChunkKeys;
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

// ---- MMA issue: warp 0
template <int D>
__device__ __forceinline__ void chunk_mma_role(const CacheAttnArgs& a, ChunkWalk w, uint32_t sbase,
                                               uint32_t bars, uint32_t tmem, const AbortCtx& ab) {
  using L = ChunkLayout<D>;
  constexpr int S = L::kStages;
  auto bar = [&](int i) { return bars + 8u * static_cast<uint32_t>(i); };
  const uint64_t dQ[2] = {desc_kmajor(sbase + L::kOffQ),
                          desc_kmajor(sbase + L::kOffQ + L::kTileBytes)};
  const uint64_t dK0 = desc_kmajor(sbase + L::kOffKV);
  const uint64_t dV0 = desc_v(sbase + L::kOffKV);
  const uint32_t tS[2] = {tmem + L::kColS, tmem + L::kColS + 128};
  const uint32_t tO[2] = {tmem + L::kColO, tmem + L::kColO + D};
  auto off = [](uint32_t idx) { return (idx % S) * static_cast<uint32_t>(L::kTileBytes); };
  auto kv_wait = [&](uint32_t idx) {
    return wait_spin_warp(bar(kCbKVFull + idx % S), (idx / S) & 1u, ab, kStatusMma);
  };
  auto kv_free = [&](uint32_t idx) { ptx::umma_commit_elect(bar(kCbKVFull + S + idx % S)); };
  auto qk = [&](int q, int i, uint32_t idx) {
    issue_qk_desc<D, false, true>(tS[i], dQ[q], desc_add(dK0, off(idx)));
    ptx::umma_commit_elect(bar(kCbSFull + i));
  };
  auto pv = [&](int i, uint32_t idx, bool acc) {
    issue_pv_ts_desc<D, false, true>(tO[i], tS[i], desc_add(dV0, off(idx)), acc);
  };
  uint32_t ring = 0, qn[2] = {0u, 0u}, pn[2] = {0u, 0u};
  bool ok = true;
  do {
    const int n = w.n();
    if (n == 0) continue;
    const bool pair = w.rows(a) > 128;
    ok = wait_spin_warp(bar(kCbQFull + 0), (qn[0]++) & 1u, ab, kStatusMma) &&
         (!pair || wait_spin_warp(bar(kCbQFull + 1), (qn[1]++) & 1u, ab, kStatusMma));
    if (!ok) break;
    // K of tile j is slot ring + 2 j, its V the next one
    if (pair) {
      if (!(ok = kv_wait(ring))) break;
      ptx::tc_fence_after();
      qk(0, 0, ring);
      qk(1, 1, ring);
      kv_free(ring);
      for (int j = 0; j < n && ok; ++j) {
        const uint32_t vj = ring + 2u * j + 1u, kn = vj + 1u;
        const bool more = j + 1 < n;
        if (!(ok = kv_wait(vj))) break;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (!(ok = wait_spin_warp(bar(kCbPFull + i), (pn[i]++) & 1u, ab, kStatusMma))) break;
          ptx::tc_fence_after();
          pv(i, vj, j > 0);
          if (!more) {
            ptx::umma_commit_elect(bar(kCbOFull + i));
            continue;
          }
          if (i == 0) {
            if (!(ok = kv_wait(kn))) break;
            ptx::tc_fence_after();
          }
          qk(i, i, kn);
        }
        if (!ok) break;
        kv_free(vj);
        if (more) kv_free(kn);
      }
    } else {
      for (int i = 0; i < 2 && i < n && ok; ++i) {
        if (!(ok = kv_wait(ring + 2u * i))) break;
        ptx::tc_fence_after();
        qk(0, i, ring + 2u * i);
        kv_free(ring + 2u * i);
      }
      for (int j = 0; j < n && ok; ++j) {
        const int i = j & 1;
        const uint32_t vj = ring + 2u * j + 1u, kn = vj + 3u;
        if (!(ok = kv_wait(vj))) break;
        if (!(ok = wait_spin_warp(bar(kCbPFull + i), (pn[i]++) & 1u, ab, kStatusMma))) break;
        ptx::tc_fence_after();
        pv(i, vj, j > 1);
        kv_free(vj);
        if (j + 2 < n) {
          if (!(ok = kv_wait(kn))) break;
          ptx::tc_fence_after();
          qk(0, i, kn);
          kv_free(kn);
        } else {
          ptx::umma_commit_elect(bar(kCbOFull + i));
        }
      }
    }
    if (!ok) break;
    ring += 2u * static_cast<uint32_t>(n);
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
__device__ __forceinline__ RowAt row_at(const CacheAttnArgs& a, const ChunkWalk& w, int r) {
  const int row = w.rb * kChunkRows + r;  // (T * H is in int range)
  const int i = row / a.group;
  return {i, w.hk * a.group + row - i * a.group};
}

template <int D, bool BF16>
__device__ __forceinline__ void chunk_softmax_role(const CacheAttnArgs& a, const ChunkWalk& start,
                                                   int share, uint8_t* sgen, uint32_t sbase,
                                                   uint32_t bars, uint32_t tmem, const AbortCtx& ab,
                                                   int warp, int lane) {
  using L = ChunkLayout<D>;
  constexpr int kLanes = D / 8, kRowsPerTurn = 32 / kLanes;  // 16 bytes of a 16-bit row each
  auto bar = [&](int i) { return bars + 8u * static_cast<uint32_t>(i); };
  const int wg = (warp >> 2) - 1;
  const int r = (warp & 3) * 32 + lane;
  const uint32_t tl = ptx::tmem_lane_base(tmem, warp);
  const uint32_t shelf = sbase + L::kOffShelf + static_cast<uint32_t>(warp - 4) * 64u;
  uint32_t sn = 0, count = 0;  // S tiles taken; tiles before the item
  shelve(shelf, ChunkShelf{start, 0u, share}, lane);
  for (;;) {
    // ---- an item: Q, and what its tile loop needs
    int n, step, k0, lim, lim0;  // tiles, step, first key; keys that the row and that all rows see
    bool idle;
    float crow = a.scale_log2;
    {
      const ChunkShelf k = unshelve(shelf);
      const ChunkWalk& w = k.w;
      n = w.n();
      const int rows = w.rows(a);
      const bool pair = rows > 128;
      const int base = pair ? 128 * wg : 0;  // the tile's first row
      step = pair ? 1 : 2;
      k0 = (w.t0 + (pair ? 0 : wg)) * kChunkKeys;
      lim = keys_seen(a, w.s, row_at(a, w, base + r < rows ? base + r : 0).i);
      lim0 = keys_seen(a, w.s, row_at(a, w, base).i);
      // (a warp without rows hands P over as it is: its rows of O are not read)
      idle = base + r - lane >= rows;
      if (n > 0) {
        // this thread's row of Q, widened or rescaled to fp16, into the swizzled
        // layout. (A row for each thread, not 16 lanes to a row, which reads
        // whole lines but has to loop over the rows: 2048 x 16384 chunk 387 us,
        // drafts 70.6 us; 378 and 68.7 us so. Unrolled, its code alone took
        // longer to fetch than the rows: 415 us.)
        const bool there = base + r < rows;
        const RowAt at = row_at(a, w, there ? base + r : 0);
        const uint16_t* p = static_cast<const uint16_t*>(a.q) + q_offset(a, w.b, w.s, at.i, at.head);
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
        const float fac = rows_to_f16<D / 2, 1, BF16>(q);
        if (pair || wg == 0) {
          const uint32_t to = sbase + L::kOffQ +
                              static_cast<uint32_t>((pair ? wg : 0) * L::kTileBytes + r * 128);
#pragma unroll
          for (int e = 0; e < D / 8; ++e)
            ptx::st_shared_v4(to + (e >> 3) * kPanelBytes + (static_cast<uint32_t>((e & 7) ^ (r & 7)) << 4),
                              q[4 * e], q[4 * e + 1], q[4 * e + 2], q[4 * e + 3]);
        }
        crow *= fac;
        if (pair || wg == 0) {
          ptx::fence_proxy_async_smem();
          ptx::mbar_arrive(bar(kCbQFull + (pair ? wg : 0)));
        }
      }
    }
    const uint32_t tS = tl + L::kColS + 128u * wg;
    const uint32_t tO = tl + L::kColO + static_cast<uint32_t>(D) * wg;
    const bool one_scale = a.block_shift == 7;  // a tile is one block
    float m_ref = -INFINITY, l = 0.f;
    bool first = true, ok = true;
    for (int j = step == 1 ? 0 : wg; j < n; j += step, k0 += step * kChunkKeys) {
      const uint32_t tix = count + static_cast<uint32_t>(j);
      if (!(ok = wait_bounded_warp(bar(kCbSFull + wg), sn & 1u, ab, kStatusSoftmax) &&
                 wait_bounded_warp(bar(kCbScaleFull + (tix & 15u)), (tix >> 4) & 1u, ab,
                                   kStatusSoftmax)))
        break;
      ++sn;
      ptx::tc_fence_after();
      if (idle) {
        ptx::tc_fence_before();
        ptx::mbar_arrive(bar(kCbPFull + wg));
        continue;
      }
      uint32_t sr[2][2][32];
      float mx_lo, mx_hi;
      ptx::tmem_ld64_max(tS, sr[0], mx_lo);
      ptx::tmem_ld64_max(tS + 64u, sr[1], mx_hi);
      ptx::tmem_ld_wait64x2(sr[0], sr[1]);
      ptx::tmem_ld_wait_f2(mx_lo, mx_hi);
      float s[128];
#pragma unroll
      for (int c = 0; c < 128; ++c) s[c] = __uint_as_float(sr[c >> 6][(c >> 5) & 1][c & 31]);
      const float4* const sc = reinterpret_cast<const float4*>(sgen + L::kOffScale) + (tix & 15u) * 8;
      auto scales = [&](int g) {  // {ks, log2 vs, 1 / vs} of a 16-key group
        const float4 v = sc[g];
        return make_float3(v.x * crow, v.y, v.z);
      };
      const bool need_mask = k0 + kChunkKeys > lim0;
      float m_tile;
      if (one_scale && !need_mask) {
        const float3 f = scales(0);
        m_tile = fmaf(fmaxf(mx_lo, mx_hi), f.x, f.y);
      } else {
        if (need_mask) {
          const int see = lim - k0;
#pragma unroll
          for (int c = 0; c < 128; ++c) s[c] = c < see ? s[c] : -INFINITY;
        }
        m_tile = -INFINITY;
#pragma unroll
        for (int g = 0; g < 8; ++g) {
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
      if (m_tile > m_ref + 8.f) {
        alpha = ptx::ex2(m_ref - m_tile);  // (0 for the first visible tile)
        m_ref = m_tile;
      }
      const float neg = m_ref == -INFINITY ? 0.f : -m_ref;
      l *= alpha;
      uint32_t pk[2][32];
#pragma unroll
      for (int g = 0; g < 8; ++g) {
        const float3 f = scales(g);
        const float add = f.y + neg;
        const float2 f2 = make_float2(f.x, f.x), a2 = make_float2(add, add);
        float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float2 t = ptx::ffma2(make_float2(s[16 * g + 2 * c], s[16 * g + 2 * c + 1]), f2, a2);
          const float p0 = ptx::ex2(t.x), p1 = ptx::ex2(t.y);
          pk[g >> 2][(g & 3) * 8 + c] = pack_f16(p0, p1);
          if (c & 1) sum1 = ptx::fadd2(sum1, make_float2(p0, p1));
          else sum0 = ptx::fadd2(sum0, make_float2(p0, p1));
        }
        sum0 = ptx::fadd2(sum0, sum1);
        l = fmaf(sum0.x + sum0.y, f.z, l);
      }
      ptx::tmem_st32(tS, pk[0]);
      ptx::tmem_st32(tS + 32u, pk[1]);
      // O_i holds the products so far: S_i's commit came after the last of them
      if (!first && __any_sync(0xffffffffu, alpha != 1.f)) {
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
      ptx::mbar_arrive(bar(kCbPFull + wg));
      first = false;
    }
    if (!ok) return;

    // ---- epilogue
    ChunkShelf k = unshelve(shelf);
    ChunkWalk& w = k.w;
    const int rows = w.rows(a);
    const bool pair = rows > 128;
    const int base = pair ? 128 * wg : 0;
    const bool there = base + r < rows;
    const bool works = n > 0 && (pair || n > wg);  // this warpgroup had tiles
    const bool begins = w.t0 == 0, ends = w.t1 == w.tiles;
    float* part = nullptr;
    if (!begins || !ends)
      part = a.parts + (2LL * blockIdx.x + (begins ? 1 : 0)) * partial_floats(kChunkRows, D);
    if (!ends && begins && wg == 0 && r == 0)
      a.join[blockIdx.x] =
          join_item(w.b, w.hk, w.rb, rows, 1 + (w.tiles - w.t1 + k.share - 1) / k.share);
    const bool two = !pair && n > 1;  // results of two warpgroups
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
        if (!(wait_bounded_warp(bar(kCbOFull + 1), (k.flags >> 1) & 1u, ab, kStatusEpilogue) &&
              wait_bounded_warp(bar(kCbStats), (k.flags >> 2) & 1u, ab, kStatusEpilogue)))
          return;
        const float m1 = s_m[r], l1 = s_m[128 + r];
        const float top = fmaxf(m_ref, m1);
        f0 = m_ref == -INFINITY ? 0.f : ptx::ex2(m_ref - top);
        f1 = m1 == -INFINITY ? 0.f : ptx::ex2(m1 - top);
        l = l * f0 + l1 * f1;
        m_ref = top;
      }
      ptx::tc_fence_after();
      const bool none = m_ref == -INFINITY;
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
        part[kChunkRows * D + base + r] = m_ref;
        part[kChunkRows * D + kChunkRows + base + r] = l;
      }
      const uint32_t sQ = sbase + L::kOffQ + static_cast<uint32_t>((pair ? wg : 0) * L::kTileBytes);
      const uint32_t tO0 = tl + L::kColO + static_cast<uint32_t>(D) * wg;
      const unsigned long long* nan =
          reinterpret_cast<const unsigned long long*>(sgen + L::kOffNan) + (w.item & 7) * D;
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
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const unsigned long long u = nan[32 * c + e];
          if (static_cast<int>(u >> 32) == w.item + 1 &&
              0x7FFFFFFF - static_cast<int>(u & 0xFFFFFFFFu) < lim)
            v[e] = __int_as_float(0x7FFFFFFF);
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
          for (int e = 0; e < 32; ++e) part[(32 * c + e) * kChunkRows + base + r] = v[e];
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
    if (n > 0) k.flags ^= 1u | (pair || n > 1 ? 2u : 0u) | (two ? 4u : 0u);
    count += static_cast<uint32_t>(n);
    if (!w.next(a)) return;
    shelve(shelf, k, lane);
  }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kChunkThreads, 1)
    fa_cache_chunk_kernel(const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v, const CacheAttnArgs a) {
  using L = ChunkLayout<D>;
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
    *abort_flag = 0u;
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
    if (warp == 0) chunk_mma_role<D>(a, w, sbase, bars, tmem, ab);
    else if (warp == 1) chunk_copy_role<D>(&tm_k, &tm_v, a, w, sgen, sbase, bars, ab, lane);
  } else if (wgrp < 3) {
    ptx::setmaxnreg_inc<kChunkRegsSoftmax>();
    chunk_softmax_role<D, BF16>(a, w, static_cast<int>(share), sgen, sbase, bars, tmem, ab, warp,
                                lane);
  } else {
    ptx::setmaxnreg_dec<kChunkRegsConvert>();
    chunk_convert_role<D>(a, w, sgen, sbase, bars, ab, warp, lane);
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
