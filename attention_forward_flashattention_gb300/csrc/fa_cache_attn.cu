// fa_fwd_cache: choice of kernel and launches.
#include "fa_cache_chunk.cuh"

namespace fa {
namespace {

// The join of a launch of `grid` shares with `rows` rows an item, set up while
// that launch still runs.
template <int D, bool BF16>
cudaError_t launch_join(const CacheAttnArgs& a, int grid, int rows, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid),
                     static_cast<unsigned>((rows + kJoinRows - 1) / kJoinRows));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fa_cache_join_kernel<D, BF16>, a, rows);
}

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
  return launch_join<D, BF16>(a, grid, 8 * NT, stream);
}

template <int D, bool BF16>
cudaError_t launch_chunk(const CacheAttnArgs& a, const CUtensorMap* maps, int sm_count,
                         cudaStream_t stream) {
  constexpr int kSmem = ChunkLayout<D>::kSmem;
  auto kern = fa_cache_chunk_kernel<D, BF16>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  kern<<<sm_count, kChunkThreads, kSmem, stream>>>(maps[0], maps[1], a);
  e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_join<D, BF16>(a, sm_count, kChunkRows, stream);
}

// Rows that share a K / V head, on average over the sequences: up to 16 go
// through the step kernel, more through the chunk kernel. Either one computes
// any number of rows.
bool runs_steps(int B, int T, int group) {
  return ((static_cast<long long>(T) + B - 1) / B) * group <= kStepMaxRows;
}

template <int D>
cudaError_t pick(const CacheAttnArgs& a, const CUtensorMap* maps, bool bf16, int sm_count,
                 cudaStream_t s) {
  if (!runs_steps(a.B, a.T, a.group))
    return bf16 ? launch_chunk<D, true>(a, maps, sm_count, s)
                : launch_chunk<D, false>(a, maps, sm_count, s);
  if (((static_cast<long long>(a.T) + a.B - 1) / a.B) * a.group <= 8)
    return bf16 ? launch_step<D, true, 1>(a, maps, sm_count, s)
                : launch_step<D, false, 1>(a, maps, sm_count, s);
  return bf16 ? launch_step<D, true, 2>(a, maps, sm_count, s)
              : launch_step<D, false, 2>(a, maps, sm_count, s);
}

}  // namespace

long long cache_workspace_floats(int B, int T, int group, int d, int sm_count) {
  const bool steps = runs_steps(B, T, group);
  const long long grid = steps ? 2LL * sm_count : sm_count;
  return 4 * grid + 2 * grid * partial_floats(steps ? kStepMaxRows : kChunkRows, d);
}

cudaError_t launch_cache_attn(const CacheAttnArgs& a, const fa_cache& c, bool bf16, int sm_count,
                              cudaStream_t stream, bool* mapped) {
  CUtensorMap maps[2];
  const bool steps = runs_steps(a.B, a.T, a.group);
  const int keys = steps ? step_keys(c.d) : kChunkKeys, rows = c.block < keys ? c.block : keys;
  *mapped = encode_cache(&maps[0], c.k, c, rows, steps) &&
            encode_cache(&maps[1], c.v, c, rows, steps);
  if (!*mapped) return cudaErrorUnknown;
  return c.d == 64 ? pick<64>(a, maps, bf16, sm_count, stream)
                   : pick<128>(a, maps, bf16, sm_count, stream);
}

}  // namespace fa
