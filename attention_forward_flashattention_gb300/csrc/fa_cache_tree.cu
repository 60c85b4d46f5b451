// Trees of drafted tokens (include/fa_draft.h): the attention's kernels, which
// are fa_fwd_cache's with a mask for the drafted keys, and the masks from the
// tokens' parents.
//
// A mask costs the attention next to nothing: only the tiles that hold a
// sequence's last keys look at it. There the step kernel asks for each score's bit, and
// the chunk kernel forms a row's 64 bits of a half tile at once (tree_seen64).
#include "fa_cache_launch.cuh"
#include "fa_check.h"
#include "fa_draft.h"

namespace fa {
namespace {

constexpr int kTreeThreads = 64;
constexpr int kTreeStaged = 64 * kMaxWords;  // tokens whose parents are kept in shared memory

// A CTA for a request, a thread for a token, which walks to the root: its
// ancestors have falling numbers, so the mask's words are complete one after another.
// (A token without a bit does not walk: a walk has at most 64 * words steps.) Bound by a
// launch, two dependent trips to memory and a walk through shared memory: 16 requests
// of 13 tokens 2.4 us, 32 of up to 64 tokens 2.9. A request has 64 threads, and the last token
// of a chain (a prompt, say) walks all of it: chains of 64 tokens 5.9 us, of 256 61, of
// 1024 911 (binary trees of as many 2.1, 4.9 and 20).
__global__ void __launch_bounds__(kTreeThreads)
    fa_cache_tree_kernel(const int32_t* parents, const int32_t* cu, const int32_t* lens,
                         unsigned long long* masks, int32_t* positions, int T, int words) {
  __shared__ int32_t s_parents[kTreeStaged];
  const int b = static_cast<int>(blockIdx.x);
  const int lo = min(max(__ldg(cu + b), 0), T), hi = min(max(__ldg(cu + b + 1), 0), T);
  const int n = hi - lo, len = max(__ldg(lens + b), 0);
  for (int i = static_cast<int>(threadIdx.x); i < min(n, kTreeStaged); i += kTreeThreads)
    s_parents[i] = __ldg(parents + lo + i);
  __syncthreads();
  for (int i = static_cast<int>(threadIdx.x); i < n; i += kTreeThreads) {
    unsigned long long* const row = masks + static_cast<long long>(lo + i) * words;
    unsigned long long bits = 0;
    int w = words - 1, ancestors = i < 64 * words ? -1 : 0;
    for (int at = i < 64 * words ? i : -1; at >= 0;) {
      ++ancestors;
      for (; w > (at >> 6); --w) {
        row[w] = bits;
        bits = 0;
      }
      bits |= 1ull << (at & 63);
      const int p = s_parents[at];
      at = p < at ? p : -1;  // (below 0: none)
    }
    for (; w >= 0; --w) {
      row[w] = bits;
      bits = 0;
    }
    positions[lo + i] = static_cast<int32_t>(min(static_cast<long long>(len) + ancestors, 0x7FFFFFFFLL));
  }
}

}  // namespace

cudaError_t launch_cache_tree_attn(const CacheAttnArgs& a, const fa_cache& c, bool bf16,
                                   int sm_count, float* ws, cudaStream_t stream, bool* mapped) {
  return launch_attn<true>(a, c, bf16, sm_count, ws, stream, mapped);
}

}  // namespace fa

extern "C" fa_status fa_cache_tree(const int32_t* parents, const int32_t* cu, const int32_t* lens,
                                   uint64_t* masks, int32_t* positions, int B, int T, int words,
                                   void* stream) {
  if (!parents || !cu || !lens || !masks || !positions) return FA_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(parents), static_cast<const void*>(cu),
                        static_cast<const void*>(lens), static_cast<const void*>(positions)})
    if (!fa::aligned(p, 4)) return FA_ERR_INVALID_ARG;
  if (!fa::aligned(masks, 8) || B <= 0 || T < 0 || words <= 0) return FA_ERR_INVALID_ARG;
  for (const int32_t* p : {parents, cu, lens})
    if (p == positions || static_cast<const void*>(p) == static_cast<const void*>(masks))
      return FA_ERR_INVALID_ARG;
  if (static_cast<void*>(positions) == static_cast<void*>(masks)) return FA_ERR_INVALID_ARG;
  if (B > (1 << 20) || words > fa::kMaxWords || static_cast<long long>(T) * words > 0x7FFFFFFFLL)
    return FA_ERR_UNSUPPORTED;
  int sms = 0;
  const fa_status ds = fa::device_facts(&sms, nullptr);
  if (ds != FA_OK) return ds;
  if (T == 0) return FA_OK;
  (void)cudaGetLastError();
  fa::fa_cache_tree_kernel<<<B, fa::kTreeThreads, 0, static_cast<cudaStream_t>(stream)>>>(
      parents, cu, lens, reinterpret_cast<unsigned long long*>(masks), positions, T, words);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}
