// Upkeep of the block cache (include/fa_pages.h): kernels, argument checks, launches.
#include <initializer_list>

#include "fa_cache.cuh"
#include "fa_cache_scale.cuh"
#include "fa_check.h"
#include "fa_pages.h"

namespace fa {
namespace {

// ------------------------------------------------------------ keep
//
// A warp takes a plane (K or V of a head) of one sequence, a CTA kKeepWarps of its
// planes, which share the list of kept tokens. Kept token k of the last n ones
// goes from place path[k] >= k to place k, and path rises: so a row that has been
// written is no later token's source, and the rows move in order, kRows at a
// time (all read before any is written), with no copy in between. Blocks are done
// one after another, each with its own new scale.
//
// A chain of loads (lengths and words - table - scales - rows), so what counts is how
// many warps are in it. Half of up to 96 tokens of 256 requests, 32 heads, blocks of 128, d
// 128: 97 MB of kept tokens, and 49 MB of older rows whose block's scale grows, which are
// re-coded one load and store after another: 49.5 us on a cache as it comes (2.9 TB/s). On
// a cache that has been through it, so without older rows, 26.7, in L2 22.8; in that form,
// 32 rows of a warp under way, 8 warps to a CTA and 3 CTAs 29.7, 16 rows, 5 CTAs of 8
// warps 23.6, 64 rows 40. Paths of up to 64 tokens in place of halves 31.6 (as it
// comes); a path of 16 requests, 4 heads: 4.5, repeated 3.6.

constexpr int kKeepWarps = 4;
constexpr int kKeepThreads = 32 * kKeepWarps;
constexpr int kKeepCtas = 10;  // on an SM
constexpr int kMostKept = 64 * kMaxWords;
constexpr int kMostBlocks = kMostKept / 16 + 1;  // that the kept tokens lie in
constexpr int kRows = 16;                        // rows of a warp under way together

struct PageArgs {
  uint8_t* k;
  uint8_t* v;
  float* k_scales;
  float* v_scales;
  long long block_stride, head_stride, token_stride;
  int Hkv, num_blocks, block_shift;
  const int32_t* table;
  const int32_t* kv_lens;
  const int32_t* cu;
  const unsigned long long* keep;
  int32_t* lens_out;
  int table_width, words, B;
};

// A scale as it counts: a power of two, 0 for one that is not above 0.
__device__ __forceinline__ float counted(float s) { return s > 0.f ? pow2_above(s) : 0.f; }

template <int D>
__global__ void __launch_bounds__(kKeepThreads, kKeepCtas) fa_cache_keep_kernel(const PageArgs a, const int groups) {
  constexpr int kLanes = D / 16;            // of a row, 16 codes each
  constexpr int kPerLoad = 32 / kLanes;     // rows
  constexpr int kLoads = kRows / kPerLoad;
  __shared__ unsigned long long s_words[kMaxWords];
  __shared__ short s_path[kMostKept];
  __shared__ int s_ids[kMostBlocks];
  __shared__ float s_old[kKeepWarps][kMostBlocks];
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const int b = static_cast<int>(blockIdx.x) / groups;
  const int group = static_cast<int>(blockIdx.x) - b * groups;
  const int bs = 1 << a.block_shift;

  const int len = __ldg(a.kv_lens + b);
  const long long n_all = static_cast<long long>(__ldg(a.cu + b + 1)) - __ldg(a.cu + b);
  if (tid < kMaxWords) {
    unsigned long long w = tid < a.words ? __ldg(a.keep + static_cast<long long>(b) * a.words + tid) : 0ull;
    const long long left = n_all - 64 * tid;
    if (left < 64) w = left <= 0 ? 0ull : w & ((1ull << left) - 1ull);
    s_words[tid] = w;
  }
  __syncthreads();
  int kept = 0;
#pragma unroll
  for (int w = 0; w < kMaxWords; ++w) kept += __popcll(s_words[w]);
  bool ok = n_all >= 0 && n_all <= len && len <= (static_cast<long long>(a.table_width) << a.block_shift);
  const int base = ok ? len - static_cast<int>(n_all) : 0;  // tokens before the last n
  // the blocks of all of the last n tokens have to exist; those of the first ones are noted
  const int j0 = base >> a.block_shift, j1 = ok && n_all > 0 ? (len - 1) >> a.block_shift : j0 - 1;
  bool bad = false;
  for (int j = j0 + tid; j <= j1; j += kKeepThreads) {
    const int id = __ldg(a.table + static_cast<long long>(b) * a.table_width + j);
    bad = bad || id < 0 || id >= a.num_blocks;
    if (j - j0 < kMostBlocks) s_ids[j - j0] = id;
  }
  ok = __syncthreads_or(bad) == 0 && ok;
  if (group == 0 && tid == 0) a.lens_out[b] = ok ? base + kept : len;
  if (!ok || kept == 0) return;
  for (int c = tid; c < 64 * a.words; c += kKeepThreads) {
    const unsigned long long w = s_words[c >> 6];
    if ((w >> (c & 63)) & 1ull) {
      int k = __popcll(w & ((1ull << (c & 63)) - 1ull));
      for (int x = 0; x < (c >> 6); ++x) k += __popcll(s_words[x]);
      s_path[k] = static_cast<short>(c);
    }
  }
  __syncthreads();
  if (s_path[kept - 1] == kept - 1) return;  // all stay where they are

  const int plane = group * kKeepWarps + warp;
  if (plane >= 2 * a.Hkv) return;
  const int head = plane >> 1, is_v = plane & 1;
  uint8_t* const codes = (is_v ? a.v : a.k) + head * a.head_stride;
  float* const scales = (is_v ? a.v_scales : a.k_scales) + head;
  float* const old = s_old[warp];
  const int last = (base + s_path[kept - 1]) >> a.block_shift;  // block of the last kept token
  for (int j = j0 + lane; j <= last; j += 32)
    old[j - j0] = scales[static_cast<long long>(s_ids[j - j0]) * a.Hkv];
  __syncwarp();
  const int r = lane / kLanes, at = 16 * (lane % kLanes);
  auto row = [&](int place) {  // of the place-th token from the start
    return codes + s_ids[(place >> a.block_shift) - j0] * a.block_stride +
           (place & (bs - 1)) * a.token_stride + at;
  };
  for (int j = j0; (j << a.block_shift) < base + kept; ++j) {
    const int first = j << a.block_shift;
    const int k0 = max(first - base, 0), k1 = min(first + bs - base, kept);
    if (s_path[k1 - 1] == k1 - 1) continue;
    const int older = max(base - first, 0);  // rows of tokens before the last n
    float now = 0.f;
    for (int k = k0 + lane; k < k1; k += 32)
      now = fmaxf(now, counted(old[((base + s_path[k]) >> a.block_shift) - j0]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, o));
    const float mine = old[j - j0];
    if (older > 0) now = fmaxf(now, counted(mine));
    if (!(now > 0.f)) now = __uint_as_float(static_cast<uint32_t>(kCacheMinScaleExp + 127) << 23);
    auto factor = [&](float s) { return s > 0.f ? s / now : 0.f; };
    const float again = factor(mine);
    if (older > 0 && again != 1.f) {
      for (int i = r; i < older; i += kPerLoad) {
        uint4* const p = reinterpret_cast<uint4*>(row(first + i));
        *p = rescale16(*p, again);
      }
    }
    for (int k = k0; k < k1; k += kRows) {
      uint4 x[kLoads];
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int kk = k + i * kPerLoad + r;
        if (kk < k1) x[i] = *reinterpret_cast<const uint4*>(row(base + s_path[kk]));
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int kk = k + i * kPerLoad + r;
        if (kk >= k1) continue;
        const int from = base + s_path[kk];
        const float f = factor(old[(from >> a.block_shift) - j0]);
        if (f != 1.f) x[i] = rescale16(x[i], f);
        else if (from == base + kk) continue;
        *reinterpret_cast<uint4*>(row(base + kk)) = x[i];
      }
      __syncwarp();
    }
    if (lane == 0) scales[static_cast<long long>(s_ids[j - j0]) * a.Hkv] = now;
  }
}

// ------------------------------------------------------------ release
//
// Entries are numbered through all requests; a cluster of CTAs takes equal ranges of
// them, a thread kEntries at a time. With counts of holders three passes: every entry
// lowers its block's count; entries of a block that nobody holds any more leave the
// smallest of their numbers in its place; that one entry puts the block on the
// list, at its rank among them (a scan over the threads, and over the CTAs through
// their shared memory), and clears the count. So the list does not depend on which
// request came first in time. Up to 4096 entries are the first CTA's alone. Latency:
// the blocks behind the kept tokens of 256 requests 5.9 us, with counts 8.1; all 128 blocks of
// 256 requests, in random order, 9.3 and 24.2 (one CTA for any number: 40 and 152), of 4096
// requests 182 and 440.

constexpr int kReleaseThreads = 1024;
constexpr int kEntries = 4;
constexpr int kReleaseCtas = 8;

struct ReleaseArgs {
  const int32_t* table;
  const int32_t* lens;
  const int32_t* new_lens;
  int32_t* shares;
  int32_t* free_blocks;
  const int32_t* free_pos;
  int32_t* free_next;
  int table_width, num_blocks, n_free, B, block_shift;
};

struct Given {
  int first, count;  // entries of a request's table row
};
__device__ __forceinline__ Given given(const ReleaseArgs& a, int b) {
  const int len = __ldg(a.lens + b), left = __ldg(a.new_lens + b);
  const long long most = static_cast<long long>(a.table_width) << a.block_shift;
  if (left < 0 || left > len || len > most) return {0, 0};
  const int bs1 = (1 << a.block_shift) - 1;
  const int first = static_cast<int>((static_cast<long long>(left) + bs1) >> a.block_shift);
  return {first, static_cast<int>((static_cast<long long>(len) + bs1) >> a.block_shift) - first};
}

// Sum over the CTA's threads before this one, and all of them.
struct Scan {
  int before, total;
};
__device__ __forceinline__ Scan block_scan(int v, int* s_warp) {
  const int lane = static_cast<int>(threadIdx.x & 31), warp = static_cast<int>(threadIdx.x >> 5);
  int in = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, in, o);
    if (lane >= o) in += u;
  }
  __syncthreads();  // (s_warp may still be read)
  if (lane == 31) s_warp[warp] = in;
  __syncthreads();
  if (warp == 0) {
    int t = lane < static_cast<int>(blockDim.x >> 5) ? s_warp[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += u;
    }
    s_warp[lane] = t;
  }
  __syncthreads();
  return {in - v + (warp > 0 ? s_warp[warp - 1] : 0), s_warp[(blockDim.x >> 5) - 1]};
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// An int of another CTA of the cluster, at the address that it has in this one.
__device__ __forceinline__ int of_cta(const int* own, int cta) {
  uint32_t at;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(ptx::smem_u32(own)), "r"(cta));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

__global__ void __cluster_dims__(kReleaseCtas, 1, 1) __launch_bounds__(kReleaseThreads)
    fa_cache_release_kernel(const ReleaseArgs a) {
  __shared__ int s_first[kReleaseThreads];  // number of the first entry of each thread's requests
  __shared__ int s_warp[32];
  __shared__ int s_count;  // blocks that this CTA puts on the list
  const int tid = static_cast<int>(threadIdx.x), cta = static_cast<int>(blockIdx.x);
  const int pos = __ldg(a.free_pos);
  if (pos < 0 || pos > a.n_free) {
    if (cta == 0 && tid == 0) *a.free_next = pos;
    return;
  }
  const int run = (a.B + kReleaseThreads - 1) / kReleaseThreads;
  const int b0 = min(tid * run, a.B), b1 = min(b0 + run, a.B);
  int mine = 0;
  for (int b = b0; b < b1; ++b) mine += given(a, b).count;
  const Scan s = block_scan(mine, s_warp);
  s_first[tid] = s.before;
  const int total = s.total, step = kReleaseThreads * kEntries;
  const bool alone = total <= step;  // (all CTAs see the same)
  if (alone && cta != 0) return;
  __syncthreads();
  // this CTA's entries [from, to)
  const int per = alone ? step : (total + kReleaseCtas * kEntries - 1) / (kReleaseCtas * kEntries) * kEntries;
  const int from = min(cta * per, total), to = min(from + per, total);
  auto sync = [&] {
    __threadfence();
    if (alone) __syncthreads();
    else cluster_sync();
  };

  // the block of entry e, -1 for one that does not exist
  auto block_of_entry = [&](int e) {
    int lo = 0, hi = kReleaseThreads - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_first[mid] <= e) lo = mid;
      else hi = mid - 1;
    }
    int at = s_first[lo], b = lo * run;
    for (;; ++b) {  // ends: e is below the number of all entries
      const Given g = given(a, b);
      if (e < at + g.count) {
        const int id = __ldg(a.table + static_cast<long long>(b) * a.table_width + g.first + (e - at));
        return id < a.num_blocks ? max(id, -1) : -1;
      }
      at += g.count;
    }
  };
  auto look_up = [&](int e0, int (&id)[kEntries]) {
#pragma unroll
    for (int i = 0; i < kEntries; ++i) id[i] = e0 + i < to ? block_of_entry(e0 + i) : -1;
  };
  // (those of the first round are looked up once for all passes)
  int first_ids[kEntries];
  look_up(from + tid * kEntries, first_ids);
  auto ids_at = [&](int e0, int (&id)[kEntries]) {
    if (e0 >= from + step) {
      look_up(e0, id);
    } else {
#pragma unroll
      for (int i = 0; i < kEntries; ++i) id[i] = first_ids[i];
    }
  };
  const bool counted_blocks = a.shares != nullptr;
  if (counted_blocks) {
    for (int pass = 0; pass < 2; ++pass) {
      for (int e0 = from + tid * kEntries; e0 < to; e0 += step) {
        int id[kEntries], held[kEntries];
        ids_at(e0, id);
        if (pass == 0) {
#pragma unroll
          for (int i = 0; i < kEntries; ++i)
            if (id[i] >= 0) atomicSub(a.shares + id[i], 1);
        } else {
#pragma unroll
          for (int i = 0; i < kEntries; ++i) held[i] = id[i] >= 0 ? __ldcg(a.shares + id[i]) : 0;
#pragma unroll
          for (int i = 0; i < kEntries; ++i)
            if (held[i] < 0) atomicMin(a.shares + id[i], INT32_MIN + e0 + i);
        }
      }
      sync();
    }
  }
  // entries that put their block on the list
  auto winners = [&](int e0, int (&id)[kEntries]) {
    int n = 0;
    ids_at(e0, id);
#pragma unroll
    for (int i = 0; i < kEntries; ++i) {
      if (counted_blocks && id[i] >= 0 && __ldcg(a.shares + id[i]) != INT32_MIN + e0 + i) id[i] = -1;
      n += id[i] >= 0;
    }
    return n;
  };
  int rank = 0, listed = 0;  // blocks of the CTAs before this one, of all
  if (!alone) {
    int id[kEntries], n = 0;
    for (int e0 = from + tid * kEntries; e0 < to; e0 += step) n += winners(e0, id);
    const Scan all = block_scan(n, s_warp);
    if (tid == 0) s_count = all.total;
    cluster_sync();
    for (int c = 0; c < kReleaseCtas; ++c) {
      const int other = of_cta(&s_count, c);
      rank += c < cta ? other : 0;
      listed += other;
    }
    cluster_sync();  // (no CTA clears a count, or ends, before all have seen them)
  }
  for (int at = from; at < to; at += step) {
    int id[kEntries];
    const int n = winners(at + tid * kEntries, id);
    const Scan all = block_scan(n, s_warp);
    int place = pos - 1 - rank - all.before;
#pragma unroll
    for (int i = 0; i < kEntries; ++i) {
      if (id[i] < 0) continue;
      if (counted_blocks) __stcg(a.shares + id[i], 0);
      if (place >= 0) a.free_blocks[place] = id[i];
      --place;
    }
    rank += all.total;
  }
  if (cta == 0 && tid == 0) *a.free_next = max(pos - (alone ? rank : listed), 0);
}

// ------------------------------------------------------------ fork
//
// As in fa_cache_plan: every CTA forms the one prefix sum (new requests that need a
// free block) for itself and writes its share of the rows, neighbouring ones, so that
// the sum goes on from row to row; a warp for a row, or where there are enough CTAs all
// of its warps. Which block a row gets does not depend on order in time, counts go up by
// integer additions. Latency: 4 rows 2.8 us, 512 of up to 5 blocks 5.6. Rows of 7 shared blocks
// and a copied one, eight to a source: 512 9.5, 4096 35, 65536 442. (32 registers a thread,
// 4 bytes of them spilled.)

constexpr int kForkThreads = 256;

struct ForkArgs {
  const int32_t* table;
  const int32_t* lens;
  const int32_t* src;
  int32_t* shares;
  const int32_t* free_blocks;
  const int32_t* free_pos;
  int32_t* new_table;
  int32_t* new_lens;
  int32_t* copies;
  int32_t* free_next;
  int table_width, B, n, num_blocks, n_free, block_shift;
};

struct Source {
  int row, len;  // len 0: refused, or nothing to copy
  int last;      // its last block, if that is not full and exists; -1
};
__device__ __forceinline__ Source source(const ForkArgs& a, int k) {
  Source s{__ldg(a.src + k), 0, -1};
  if (s.row < 0 || s.row >= a.B) return s;
  const int len = __ldg(a.lens + s.row);
  if (len <= 0 || len > (static_cast<long long>(a.table_width) << a.block_shift)) return s;
  s.len = len;
  if ((len & ((1 << a.block_shift) - 1)) != 0) {
    const int id = __ldcg(a.table + static_cast<long long>(s.row) * a.table_width + (len >> a.block_shift));
    if (id >= 0 && id < a.num_blocks) s.last = id;
  }
  return s;
}

__global__ void __launch_bounds__(kForkThreads) fa_cache_fork_kernel(const ForkArgs a) {
  __shared__ int s_need[kForkThreads / 32];
  __shared__ int s_before[kForkThreads];  // free blocks needed before each thread's requests
  __shared__ int s_warp[32];
  const int tid = static_cast<int>(threadIdx.x);
  const int run = (a.n + kForkThreads - 1) / kForkThreads;
  const int k0 = min(tid * run, a.n), k1 = min(k0 + run, a.n);
  const int pos = __ldg(a.free_pos);
  const int left = pos >= 0 ? max(a.n_free - pos, 0) : 0;  // (a free_pos out of range offers none)
  int mine = 0;
#pragma unroll 4
  for (int k = k0; k < k1; ++k) mine += source(a, k).last >= 0;
  const Scan s = block_scan(mine, s_warp);
  s_before[tid] = s.before;
  if (blockIdx.x == 0 && tid == 0) *a.free_next = pos + min(s.total, left);
  __syncthreads();
  // this CTA's rows [from, to), and the free blocks needed before them
  constexpr int kWarps = kForkThreads / 32;
  const int ctas = static_cast<int>(gridDim.x), per = (a.n + ctas - 1) / ctas;
  const int from = min(static_cast<int>(blockIdx.x) * per, a.n), to = min(from + per, a.n);
  if (from >= to) return;
  int before = s_before[from / run];
  for (int x = from / run * run; x < from; x += kForkThreads)
    before += __syncthreads_count(x + tid < from && source(a, x + tid).last >= 0);
  const int warps = per == 1 ? kWarps : 1;  // of a row
  const int team = tid / (32 * warps), lane = tid - team * 32 * warps;
  for (int k0 = from; k0 < to; k0 += kWarps / warps) {
    const int k = k0 + team;
    const bool there = k < to;
    const Source f = there ? source(a, k) : Source{0, 0, -1};
    __syncthreads();  // (s_need may still be read)
    if (lane == 0) s_need[team] = f.last >= 0;
    __syncthreads();
    int mine_before = before;
    for (int x = 0; x < kWarps / warps; ++x) {
      mine_before += x < team ? s_need[x] : 0;
      before += s_need[x];
    }
    if (!there) continue;
    const bool ok = f.len > 0 && (f.last < 0 || mine_before < left);
    const int full = f.len >> a.block_shift, rows = f.len & ((1 << a.block_shift) - 1);
    const int fresh = ok && f.last >= 0 ? __ldg(a.free_blocks + pos + mine_before) : -1;
    const int32_t* const src = a.table + static_cast<long long>(f.row) * a.table_width;
    int32_t* const dst = a.new_table + static_cast<long long>(k) * a.table_width;
#pragma unroll 4
    for (int j = lane; j < a.table_width; j += 32 * warps) {
      int id = -1;
      if (ok && j < full + (rows != 0)) {
        id = j == full && f.last >= 0 ? fresh : __ldcg(src + j);
        if (j < full && id >= 0 && id < a.num_blocks) atomicAdd(a.shares + id, 1);
      }
      dst[j] = id;
    }
    if (lane == 0) {
      a.new_lens[k] = ok ? f.len : 0;
      const bool copy = ok && f.last >= 0;
      a.copies[3LL * k] = copy ? f.last : -1;
      a.copies[3LL * k + 1] = copy ? fresh : -1;
      a.copies[3LL * k + 2] = copy ? rows : 0;
    }
  }
}

// ------------------------------------------------------------ copy
//
// A CTA for a copy and head at a time: 16 bytes a thread and load, K and V. Two trips to
// memory, the entry and the rows, so many small CTAs: a beam of 512 copies of 128-token
// blocks, 32 heads, d 128, 537 MB: 64 us (8.4 TB/s, the eight copies of a block are read
// from L2) with 8 CTAs on an SM, 74 with 4 that request four rows at a time, 108 with 2
// and eight rows. (Eight CTAs leave 32 registers a thread, 52 bytes of which are spilled.)

constexpr int kCopyThreads = 256, kCopyCtas = 8;

template <int D>
__global__ void __launch_bounds__(kCopyThreads, kCopyCtas)
    fa_cache_copy_kernel(const PageArgs a, const int32_t* copies, const long long units) {
  constexpr int kLanes = D / 16;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const long long c = u / a.Hkv;
    const int head = static_cast<int>(u - c * a.Hkv);
    const int from = __ldg(copies + 3 * c), to = __ldg(copies + 3 * c + 1);
    const int rows = min(__ldg(copies + 3 * c + 2), 1 << a.block_shift);
    if (from < 0 || from >= a.num_blocks || to < 0 || to >= a.num_blocks || from == to || rows <= 0)
      continue;
    const long long src = from * a.block_stride + head * a.head_stride;
    const long long dst = to * a.block_stride + head * a.head_stride;
#pragma unroll 1
    for (int e = static_cast<int>(threadIdx.x); e < rows * kLanes; e += kCopyThreads) {
      const long long at = (e / kLanes) * a.token_stride + 16 * (e % kLanes);
      const uint4 k = *reinterpret_cast<const uint4*>(a.k + src + at);
      const uint4 v = *reinterpret_cast<const uint4*>(a.v + src + at);
      *reinterpret_cast<uint4*>(a.k + dst + at) = k;
      *reinterpret_cast<uint4*>(a.v + dst + at) = v;
    }
    if (threadIdx.x < 2) {
      float* const s = threadIdx.x ? a.v_scales : a.k_scales;
      s[static_cast<long long>(to) * a.Hkv + head] = s[static_cast<long long>(from) * a.Hkv + head];
    }
  }
}

PageArgs of_cache(const fa_cache& c) {
  PageArgs a{};
  a.k = static_cast<uint8_t*>(c.k);
  a.v = static_cast<uint8_t*>(c.v);
  a.k_scales = c.k_scales;
  a.v_scales = c.v_scales;
  a.block_stride = c.block_stride;
  a.head_stride = c.head_stride;
  a.token_stride = c.token_stride;
  a.Hkv = c.Hkv;
  a.num_blocks = c.num_blocks;
  a.block_shift = block_shift(c.block);
  return a;
}

fa_status launched() { return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

// Written arrays: there, aligned, none of them twice or among the read ones.
bool apart(std::initializer_list<const void*> written, std::initializer_list<const void*> read) {
  for (const void* const* w = written.begin(); w != written.end(); ++w) {
    for (const void* const* x = written.begin(); x != w; ++x)
      if (*x && *x == *w) return false;
    for (const void* r : read)
      if (r && r == *w) return false;
  }
  return true;
}
bool there(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!p || !aligned(p, 4)) return false;
  return true;
}

}  // namespace
}  // namespace fa

extern "C" {

fa_status fa_cache_keep(const fa_cache* cache, const int32_t* block_table, int table_width,
                        const int32_t* kv_lens, const int32_t* cu, const uint64_t* keep, int words,
                        int32_t* lens_out, int B, void* stream) {
  const fa_status cs = fa::check_cache(cache);
  if (cs == FA_ERR_INVALID_ARG) return cs;
  if (!fa::there({block_table, kv_lens, cu, keep, lens_out}) || !fa::aligned(keep, 8))
    return FA_ERR_INVALID_ARG;
  if (!fa::apart({lens_out}, {block_table, kv_lens, cu, keep})) return FA_ERR_INVALID_ARG;
  if (B <= 0 || words <= 0 || table_width <= 0) return FA_ERR_INVALID_ARG;
  if (cs != FA_OK) return cs;
  if (B > (1 << 20) || words > fa::kMaxWords ||
      static_cast<long long>(table_width) * cache->block > (1LL << 30))
    return FA_ERR_UNSUPPORTED;
  const int groups = (2 * cache->Hkv + fa::kKeepWarps - 1) / fa::kKeepWarps;
  if (static_cast<long long>(B) * groups > 0x7FFFFFFFLL) return FA_ERR_UNSUPPORTED;
  int sms = 0;
  const fa_status ds = fa::device_facts(&sms, nullptr);
  if (ds != FA_OK) return ds;
  fa::PageArgs a = fa::of_cache(*cache);
  a.table = block_table;
  a.kv_lens = kv_lens;
  a.cu = cu;
  a.keep = reinterpret_cast<const unsigned long long*>(keep);
  a.lens_out = lens_out;
  a.table_width = table_width;
  a.words = words;
  a.B = B;
  (void)cudaGetLastError();
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cache->d == 64) fa::fa_cache_keep_kernel<64><<<B * groups, fa::kKeepThreads, 0, s>>>(a, groups);
  else fa::fa_cache_keep_kernel<128><<<B * groups, fa::kKeepThreads, 0, s>>>(a, groups);
  return fa::launched();
}

fa_status fa_cache_release(const int32_t* block_table, int table_width, const int32_t* lens,
                           const int32_t* new_lens, int32_t* shares, int num_blocks,
                           int32_t* free_blocks, int n_free, const int32_t* free_pos,
                           int32_t* free_next, int B, int block, void* stream) {
  if (!fa::there({block_table, lens, new_lens, free_pos, free_next}) || !fa::aligned(shares, 4) ||
      !fa::aligned(free_blocks, 4))
    return FA_ERR_INVALID_ARG;
  if (B <= 0 || table_width <= 0 || n_free < 0 || (n_free > 0 && !free_blocks) ||
      (shares && num_blocks <= 0))
    return FA_ERR_INVALID_ARG;
  // (an empty array has no address of its own)
  const int32_t* const list = n_free > 0 ? free_blocks : nullptr;
  if (!fa::apart({free_next, shares, list}, {block_table, lens, new_lens, free_pos}))
    return FA_ERR_INVALID_ARG;
  const int shift = fa::block_shift(block);
  if (shift < 0 || B > (1 << 20) || static_cast<long long>(B) * table_width > (1LL << 30))
    return FA_ERR_UNSUPPORTED;
  int sms = 0;
  const fa_status ds = fa::device_facts(&sms, nullptr);
  if (ds != FA_OK) return ds;
  fa::ReleaseArgs a{};
  a.table = block_table;
  a.lens = lens;
  a.new_lens = new_lens;
  a.shares = shares;
  a.free_blocks = free_blocks;
  a.free_pos = free_pos;
  a.free_next = free_next;
  a.table_width = table_width;
  a.num_blocks = shares ? num_blocks : 0x7FFFFFFF;
  a.n_free = n_free;
  a.B = B;
  a.block_shift = shift;
  (void)cudaGetLastError();
  fa::fa_cache_release_kernel<<<fa::kReleaseCtas, fa::kReleaseThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return fa::launched();
}

fa_status fa_cache_fork(const int32_t* block_table, int table_width, const int32_t* lens, int B,
                        const int32_t* src, int n, int32_t* shares, int num_blocks,
                        const int32_t* free_blocks, int n_free, const int32_t* free_pos,
                        int32_t* new_table, int32_t* new_lens, int32_t* copies, int32_t* free_next,
                        int block, void* stream) {
  if (!fa::there({block_table, lens, src, shares, free_pos, new_table, new_lens, copies, free_next}) ||
      !fa::aligned(free_blocks, 4))
    return FA_ERR_INVALID_ARG;
  if (B <= 0 || n <= 0 || table_width <= 0 || n_free < 0 || (n_free > 0 && !free_blocks) ||
      num_blocks <= 0)
    return FA_ERR_INVALID_ARG;
  const int32_t* const list = n_free > 0 ? free_blocks : nullptr;
  if (!fa::apart({shares, new_table, new_lens, copies, free_next}, {block_table, lens, src, list, free_pos}))
    return FA_ERR_INVALID_ARG;
  const int shift = fa::block_shift(block);
  if (shift < 0 || B > (1 << 20) || n > (1 << 20) || static_cast<long long>(table_width) * block > (1LL << 30))
    return FA_ERR_UNSUPPORTED;
  int sms = 0;
  const fa_status ds = fa::device_facts(&sms, nullptr);
  if (ds != FA_OK) return ds;
  fa::ForkArgs a{};
  a.table = block_table;
  a.lens = lens;
  a.src = src;
  a.shares = shares;
  a.free_blocks = free_blocks;
  a.free_pos = free_pos;
  a.new_table = new_table;
  a.new_lens = new_lens;
  a.copies = copies;
  a.free_next = free_next;
  a.table_width = table_width;
  a.B = B;
  a.n = n;
  a.num_blocks = num_blocks;
  a.n_free = n_free;
  a.block_shift = shift;
  (void)cudaGetLastError();
  const int most = 4 * sms;
  fa::fa_cache_fork_kernel<<<n < most ? n : most, fa::kForkThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return fa::launched();
}

fa_status fa_cache_copy(const fa_cache* cache, const int32_t* copies, int n, void* stream) {
  const fa_status cs = fa::check_cache(cache);
  if (cs == FA_ERR_INVALID_ARG) return cs;
  if (!fa::there({copies}) || n < 0) return FA_ERR_INVALID_ARG;
  if (cs != FA_OK) return cs;
  if (n > (1 << 20)) return FA_ERR_UNSUPPORTED;
  int sms = 0;
  const fa_status ds = fa::device_facts(&sms, nullptr);
  if (ds != FA_OK) return ds;
  if (n == 0) return FA_OK;
  const fa::PageArgs a = fa::of_cache(*cache);
  const long long units = static_cast<long long>(n) * cache->Hkv, most = 8LL * fa::kCopyCtas * sms;
  const int grid = static_cast<int>(units < most ? units : most);
  (void)cudaGetLastError();
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cache->d == 64) fa::fa_cache_copy_kernel<64><<<grid, fa::kCopyThreads, 0, s>>>(a, copies, units);
  else fa::fa_cache_copy_kernel<128><<<grid, fa::kCopyThreads, 0, s>>>(a, copies, units);
  return fa::launched();
}

}  // extern "C"
