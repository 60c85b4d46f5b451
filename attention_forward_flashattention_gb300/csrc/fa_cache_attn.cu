// fa_fwd_cache: its kernels.
#include "fa_cache_launch.cuh"

namespace fa {

long long cache_workspace_floats(int B, int T, int group, int d, int sm_count) {
  // the larger of what a ragged call and one of equal sequences take
  const long long r = plan_floats(plan_attn(B, T, group, true), d, sm_count);
  const long long u = T % B == 0 ? plan_floats(plan_attn(B, T, group, false), d, sm_count) : 0;
  return r > u ? r : u;
}

cudaError_t launch_cache_attn(const CacheAttnArgs& a, const fa_cache& c, bool bf16, int sm_count,
                              float* ws, cudaStream_t stream, bool* mapped) {
  return launch_attn<false>(a, c, bf16, sm_count, ws, stream, mapped);
}

}  // namespace fa
