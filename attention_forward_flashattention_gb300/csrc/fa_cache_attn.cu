// fa_fwd_cache: choice of kernel and launches.
#include "fa_cache_step.cuh"

namespace fa {
namespace {

template <int D, bool BF16, int NT>
cudaError_t launch_step(const CacheAttnArgs& a, const CUtensorMap* maps, int sm_count,
                        cudaStream_t stream) {
  constexpr int kSmem = StepLayout<D>::kSmem;
  auto kern = fa_cache_step_kernel<D, BF16, NT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  const int grid = 2 * sm_count;
  // sequences of at most one round of tiles (a tile for each warp) are never
  // cut: nothing to join, one launch
  const bool whole = (static_cast<long long>(a.table_width) << a.block_shift) <=
                     kStepWarps * step_keys(D);
  kern<<<grid, kStepThreads, kSmem, stream>>>(maps[0], maps[1], a, whole ? 1 : 0);
  e = cudaGetLastError();
  if (e != cudaSuccess || whole) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fa_cache_join_kernel<D, BF16>, a, 8 * NT);
}

template <int D>
cudaError_t pick(const CacheAttnArgs& a, const CUtensorMap* maps, bool bf16, int sm_count,
                 cudaStream_t s) {
  // rows that share a K / V head, on average: they decide only how many rows
  // go through the cache together
  const long long rows = ((static_cast<long long>(a.T) + a.B - 1) / a.B) * a.group;
  if (rows <= 8)
    return bf16 ? launch_step<D, true, 1>(a, maps, sm_count, s)
                : launch_step<D, false, 1>(a, maps, sm_count, s);
  return bf16 ? launch_step<D, true, 2>(a, maps, sm_count, s)
              : launch_step<D, false, 2>(a, maps, sm_count, s);
}

}  // namespace

long long cache_workspace_floats(int d, int sm_count) {
  const long long grid = 2LL * sm_count;
  return 4 * grid + 2 * grid * partial_floats(kStepMaxRows, d);
}

cudaError_t launch_cache_attn(const CacheAttnArgs& a, const fa_cache& c, bool bf16, int sm_count,
                              cudaStream_t stream, bool* mapped) {
  CUtensorMap maps[2];
  const int keys = step_keys(c.d), rows = c.block < keys ? c.block : keys;
  *mapped = encode_cache(&maps[0], c.k, c, rows) && encode_cache(&maps[1], c.v, c, rows);
  if (!*mapped) return cudaErrorUnknown;
  return c.d == 64 ? pick<64>(a, maps, bf16, sm_count, stream)
                   : pick<128>(a, maps, bf16, sm_count, stream);
}

}  // namespace fa
