// fa_cache_plan: block table entries and slots of new tokens.
//
// Two prefix sums over the requests (new tokens, blocks that they open) decide
// everything: a request's rows start at the first, its blocks at the second
// in the free list, and both are monotone, so "does it still fit" needs no
// sequential pass even though requests are served in order: once one request
// is refused for want of blocks, every later one that needs a block sees a
// larger sum and is refused too.
//
// One launch. Every CTA forms both sums for itself (its kThreads threads each
// take a run of requests, then a scan over the threads), because the sums cost
// 8 bytes a request from L2 while handing them over would cost a second launch
// or a grid-wide barrier; then each CTA fills its own share of the slots, and
// the first one writes the per-request results (where there is more than one
// CTA it does only that). Latency bound at every size: 8 requests of one token
// 4 us, 4096 requests with 259075 tokens 8 us.
#include "fa_cache.cuh"

namespace fa {
namespace {

constexpr int kThreads = 512;
constexpr int kSlotsPerThread = 4;

struct Request {
  long long tokens;  // rows it takes in cu_new
  long long opens;   // blocks that it needs (0 for one that is refused for its own numbers)
  bool valid;        // lengths in range and its table row is long enough
  int len;           // cached tokens (0 for a negative length)
  int have;          // blocks that it holds
};

__device__ __forceinline__ Request request(const CachePlanArgs& a, int b) {
  const int len = __ldg(a.lens + b), add = __ldg(a.new_lens + b);
  const int bs1 = (1 << a.block_shift) - 1;
  Request r;
  r.len = max(len, 0);
  r.tokens = max(add, 0);
  const long long have = (static_cast<long long>(r.len) + bs1) >> a.block_shift;
  const long long want = (static_cast<long long>(r.len) + r.tokens + bs1) >> a.block_shift;
  r.valid = len >= 0 && add >= 0 && want <= a.table_width && r.len + r.tokens <= 0x7FFFFFFFLL;
  r.opens = r.valid ? want - have : 0;
  r.have = static_cast<int>(min(have, static_cast<long long>(0x7FFFFFFF)));
  return r;
}

// Whether request r, whose rows end at `end` and blocks at `upto` (both
// inclusive sums, `upto` counted from the start of the free list), is served.
__device__ __forceinline__ bool served(const CachePlanArgs& a, const Request& r, long long end,
                                       long long upto) {
  return r.valid && (r.tokens == 0 || end <= a.T) && (r.opens == 0 || upto <= a.n_free);
}

__device__ __forceinline__ long long warp_scan(long long v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

__global__ void __launch_bounds__(kThreads) fa_cache_plan_kernel(const CachePlanArgs a) {
  __shared__ long long s_tok[kThreads], s_open[kThreads];  // sums before each thread's run
  __shared__ long long s_wtok[kThreads / 32], s_wopen[kThreads / 32];
  __shared__ long long s_used[kThreads / 32];
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const int run = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * run, a.B), b1 = min(b0 + run, a.B);
  // a free_pos out of range offers no block
  const int pos0 = __ldg(a.free_pos);
  const long long base = pos0 >= 0 ? pos0 : static_cast<long long>(a.n_free) + 1;

  long long tok = 0, open = 0;
#pragma unroll 4
  for (int b = b0; b < b1; ++b) {
    const Request r = request(a, b);
    tok += r.tokens;
    open += r.opens;
  }
  const long long tok_in = warp_scan(tok, lane), open_in = warp_scan(open, lane);
  if (lane == 31) {
    s_wtok[warp] = tok_in;
    s_wopen[warp] = open_in;
  }
  __syncthreads();
  if (warp == 0) {
    constexpr int kWarps = kThreads / 32;
    const long long t = lane < kWarps ? s_wtok[lane] : 0, p = lane < kWarps ? s_wopen[lane] : 0;
    const long long ti = warp_scan(t, lane), pi = warp_scan(p, lane);
    if (lane < kWarps) {
      s_wtok[lane] = ti;
      s_wopen[lane] = pi;
    }
  }
  __syncthreads();
  const long long tok_ex = tok_in - tok + (warp > 0 ? s_wtok[warp - 1] : 0);
  const long long open_ex = open_in - open + (warp > 0 ? s_wopen[warp - 1] : 0);
  s_tok[tid] = tok_ex;
  s_open[tid] = open_ex;
  const long long total = s_wtok[kThreads / 32 - 1];
  __syncthreads();

  if (blockIdx.x == 0) {  // per-request results
    long long t = tok_ex, p = base + open_ex;
    long long used = 0;
    for (int b = b0; b < b1; ++b) {
      const Request r = request(a, b);
      a.cu_new[b] = static_cast<int32_t>(min(t, static_cast<long long>(a.T)));
      t += r.tokens;
      p += r.opens;
      const bool ok = served(a, r, t, p);
      a.kv_lens[b] = ok ? r.len + static_cast<int>(r.tokens) : r.len;
      if (ok) used += r.opens;
    }
    used = warp_scan(used, lane);
    if (lane == 31) s_used[warp] = used;
    __syncthreads();
    if (tid == 0) {
      long long sum = 0;
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) sum += s_used[w];
      a.cu_new[a.B] = static_cast<int32_t>(min(total, static_cast<long long>(a.T)));
      *a.free_next = pos0 + static_cast<int32_t>(sum);
    }
  }

  // slots: each thread takes kSlotsPerThread consecutive rows at a time (with
  // several CTAs the first one is busy with the per-request results)
  const int fillers = max(static_cast<int>(gridDim.x) - 1, 1);
  const int filler = static_cast<int>(blockIdx.x) - (gridDim.x > 1 ? 1 : 0);
  if (filler < 0) return;
  const int bs1 = (1 << a.block_shift) - 1;
  const long long step = static_cast<long long>(fillers) * kThreads * kSlotsPerThread;
  for (long long row0 = (static_cast<long long>(filler) * kThreads + tid) * kSlotsPerThread;
       row0 < a.T; row0 += step) {
    int out[kSlotsPerThread];
    int b = -1;
    long long end = 0, upto = 0;  // inclusive sums of request b
    Request r{};
    bool ok = false;
#pragma unroll
    for (int i = 0; i < kSlotsPerThread; ++i) {
      const long long row = row0 + i;
      out[i] = -1;
      if (row >= total || row >= a.T) continue;
      if (b < 0) {
        // the last run of requests that starts at or before this row (later
        // runs of the same start hold no row before it), then the request
        int lo = 0, hi = kThreads - 1;
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (s_tok[mid] <= row) lo = mid;
          else hi = mid - 1;
        }
        b = lo * run;
        r = request(a, b);
        end = s_tok[lo] + r.tokens;
        upto = base + s_open[lo] + r.opens;
        ok = served(a, r, end, upto);
      }
      while (row >= end) {  // ends: row < total = the last request's end
        ++b;
        r = request(a, b);
        end += r.tokens;
        upto += r.opens;
        ok = served(a, r, end, upto);
      }
      if (!ok) continue;
      const int at = r.len + static_cast<int>(row - (end - r.tokens));
      const int j = at >> a.block_shift;
      int32_t* entry = a.block_table + static_cast<long long>(b) * a.table_width + j;
      int id;
      if (j >= r.have) {
        id = __ldg(a.free_blocks + (upto - r.opens) + (j - r.have));
        if ((at & bs1) == 0) *entry = id;  // the first token of a block writes its entry
      } else {
        id = *entry;
      }
      const long long slot = (static_cast<long long>(id) << a.block_shift) + (at & bs1);
      out[i] = (id >= 0 && slot <= 0x7FFFFFFFLL) ? static_cast<int>(slot) : -1;
    }
    if (row0 + kSlotsPerThread <= a.T && (reinterpret_cast<uintptr_t>(a.slots) & 15u) == 0) {
      *reinterpret_cast<int4*>(a.slots + row0) = make_int4(out[0], out[1], out[2], out[3]);
    } else {
#pragma unroll
      for (int i = 0; i < kSlotsPerThread; ++i)
        if (row0 + i < a.T) a.slots[row0 + i] = out[i];
    }
  }
}

}  // namespace

cudaError_t launch_cache_plan(const CachePlanArgs& a, int sm_count, cudaStream_t stream) {
  const long long per_cta = static_cast<long long>(kThreads) * kSlotsPerThread;
  const long long want = (a.T + per_cta - 1) / per_cta;
  const int grid = want <= 1 ? 1 : static_cast<int>(want < sm_count ? want + 1 : sm_count);
  fa_cache_plan_kernel<<<grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace fa
