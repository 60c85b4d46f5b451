// Choice of kernels and launches of fa_fwd_cache (TREE: of fa_fwd_cache_tree),
// included by the translation unit of each.
#pragma once

#include <climits>

#include "fa_cache_chunk.cuh"

namespace fa {
namespace {

// e4m3 tiles that hold a query tile in the chunk kernel for items of up to 128
// rows (0: there is none; at d = 64 a row is half a swizzled panel): two parts
// are exact for bf16's 8-bit significands, three for fp16's 11 bits.
constexpr int chunk_parts(int d, bool bf16) { return d == 64 ? 0 : bf16 ? 2 : 3; }

// Kernels of a call. The lengths are device memory, so the choice goes by the
// sizes that the host knows. Both kernels compute any number of rows; they
// differ in how many go through the cache together.
struct AttnPlan {
  int nt = 0;          // 8-row groups of the step kernel's instance; 0: not launched
  bool chunk = false;  // the chunk kernel
  int upto = INT_MAX;  // with both: most rows of the step kernel's sequences
  int item_rows = kChunkRows;  // most rows of the chunk kernel's items: 256 or 128
};

AttnPlan plan_attn(int B, int T, int group, bool ragged, bool tree = false) {
  AttnPlan p;
  const long long most = static_cast<long long>(T) * group;  // rows of a sequence to a K / V head
  if (!ragged || B == 1 || T <= B || most <= kStepMaxRows) {
    // sequences of one size, of a token each, or small in any case. Up to 16 rows the
    // step kernel: 16 sequences, 4 K / V heads, 8192 keys, bf16: a call takes 50 us with
    // 16 rows there; the chunk kernel takes 60 for any number from 24 to 64.
    // A ragged batch of at most a token for each sequence need not be one of single
    // tokens, but the host does not see its lengths. Calls of 256 sequences, 8 query
    // heads to a K / V head, here / as a mixture: all with one token, 1000 keys, 58 / 64
    // us (4 heads: 95 / 137); one with 16 tokens behind 8000 keys, the others idle, 31 /
    // 49; but one with 64 tokens 70 / 37, and with 200 tokens 189 / 62.
    const long long rows = !ragged ? most / B : (T <= B && B > 1 ? group : most);
    p.nt = rows <= 8 ? 1 : (rows <= kStepMaxRows ? 2 : 0);
    p.chunk = p.nt == 0;
  } else if (group > kStepMaxRows || (tree && most > static_cast<long long>(kStepMaxRows) * B)) {
    // Trees of more than 16 rows on average are one launch: those of fewer rows cost
    // the chunk kernel hardly more, and the launch before it does not take part in its
    // shares. 32 trees of up to 16 / 32 / 64 tokens, 4 heads to a K / V head, up to
    // 16384 keys, d 128: 153 / 157 / 234 us so, 219 / 180 / 270 as a mixture.
    p.chunk = true;
  } else {
    // a batch of single tokens and longer pieces, in a mixture that only the
    // device knows: each sequence goes to the kernel of its size. Single tokens are
    // faster on the instance of 8 rows; pieces of 9 to 16 rows, two items there, are
    // slower. So it is taken where no draft of up to four tokens has so many rows, or
    // one of two tokens alone. D 128, us on 8 rows / on 16, beside chunks of 300 to 512
    // tokens: 63 single tokens, 8 query heads to a K / V head 117 / 125, 4 heads
    // 151 / 157; 60 drafts of two tokens, 8 heads 134 / 130, of three, 4 heads 227 / 173.
    p.nt = group <= 2 || (group > 4 && group <= 8) ? 1 : 2;
    p.chunk = true;
    p.upto = kStepMaxRows;
  }
  return p;
}

// Rounds of tiles up to which a sequence of a tree batch is not cut. The host knows the
// table's width and not the lengths, so it goes by that: 5 tokens behind 256 keys, d 64, in a
// table of 768 keys 9.3 us, in one of 784 or more 12.5, with the join. Us with 1 / 3 / 6,
// 5 tokens behind 250 keys, 2 heads, d 64: 9.4 / 8.3 / 8.2, 64 x 2 tokens behind 500 keys, 32
// heads on 8: 20.9 / 19.7 / 19.7, the same behind 1000 keys, 6 rounds: 25.1 / 25.0 / 27.4.
constexpr int kTreeRounds = 3;

int step_grid(const AttnPlan& p, int sm_count) { return p.nt == 0 ? 0 : step_ctas(p.nt) * sm_count; }

// Workspace: the join items of both launches, then their partial results.
long long plan_floats(const AttnPlan& p, int d, int sm_count) {
  const long long s = step_grid(p, sm_count), c = p.chunk ? sm_count : 0;
  return 4 * (s + c) + 2 * s * partial_floats(8 * p.nt, d) + 2 * c * partial_floats(kChunkRows, d);
}

// Launches `kern` so that it may be set up while the launch before it ends.
template <typename... Params, typename... Args>
cudaError_t launch_early(void (*kern)(Params...), dim3 grid, int threads, int smem,
                         cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <int D, bool BF16, int NT, bool TREE>
cudaError_t launch_step(const CacheAttnArgs& a, const CUtensorMap* maps, bool whole, int grid,
                        cudaStream_t stream) {
  constexpr int kSmem = StepLayout<D, NT>::kSmem;
  auto kern = fa_cache_step_kernel<D, BF16, NT, TREE>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  kern<<<grid, kStepThreads, kSmem, stream>>>(maps[0], maps[1], a, whole ? 1 : 0);
  return cudaGetLastError();
}

template <int D, bool BF16, int PARTS, bool TREE>
cudaError_t launch_chunk(const CacheAttnArgs& a, const fa_cache& c, const AttnPlan& p, int grid,
                         cudaStream_t stream, bool* mapped) {
  constexpr int kSmem = ChunkLayout<D, PARTS>::kSmem;
  auto kern = fa_cache_chunk_kernel<D, BF16, PARTS, TREE>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  CUtensorMap maps[2];
  *mapped = encode_cache(&maps[0], c.k, c, c.block, PARTS > 0) &&
            encode_cache(&maps[1], c.v, c, c.block, false);
  if (!*mapped) return cudaErrorUnknown;
  // after a step launch it takes the SMs that are done with that one (its
  // CTAs wait for the step launch before they end)
  if (p.nt != 0)
    return launch_early(kern, dim3(grid), kChunkThreads, kSmem, stream, maps[0], maps[1], a);
  kern<<<grid, kChunkThreads, kSmem, stream>>>(maps[0], maps[1], a);
  return cudaGetLastError();
}

template <int D, bool BF16, bool TREE>
cudaError_t launch_all(CacheAttnArgs a, const fa_cache& c, const AttnPlan& p, int sm_count,
                       float* ws, cudaStream_t stream, bool* mapped) {
  const int sgrid = step_grid(p, sm_count), cgrid = p.chunk ? sm_count : 0;
  JoinSides sides{};
  sides.join[0] = reinterpret_cast<JoinItem*>(ws);
  sides.join[1] = sides.join[0] + sgrid;
  sides.parts[0] = ws + 4LL * (sgrid + cgrid);
  sides.parts[1] = sides.parts[0] + 2LL * sgrid * partial_floats(8 * p.nt, D);
  sides.rows[0] = 8 * p.nt;
  sides.rows[1] = p.item_rows;
  sides.ctas[1] = cgrid;
  if (p.nt != 0) {
    // sequences of at most one round of tiles (one for each warp) are not cut:
    // nothing to join. (Trees: of up to kTreeRounds.)
    const bool whole = (static_cast<long long>(a.table_width) << a.block_shift) <=
                       (TREE ? kTreeRounds : 1) * kStepWarps * step_keys(D);
    sides.ctas[0] = whole ? 0 : sgrid;
    a.rows_over = 0;
    a.rows_upto = p.upto;
    a.join = sides.join[0];
    a.parts = sides.parts[0];
    CUtensorMap maps[2];
    const int rows = c.block < step_keys(D) ? c.block : step_keys(D);
    *mapped = encode_cache(&maps[0], c.k, c, rows, true) && encode_cache(&maps[1], c.v, c, rows, true);
    if (!*mapped) return cudaErrorUnknown;
    const cudaError_t e = p.nt == 2 ? launch_step<D, BF16, 2, TREE>(a, maps, whole, sgrid, stream)
                                    : launch_step<D, BF16, 1, TREE>(a, maps, whole, sgrid, stream);
    if (e != cudaSuccess) return e;
  }
  if (p.chunk) {
    a.item_rows = p.item_rows;
    a.rows_over = p.nt != 0 ? p.upto : 0;
    a.rows_upto = INT_MAX;
    a.join = sides.join[1];
    a.parts = sides.parts[1];
    cudaError_t e;
    if constexpr (TREE && chunk_parts(D, BF16) > 0)
      e = launch_chunk<D, BF16, chunk_parts(D, BF16), TREE>(a, c, p, cgrid, stream, mapped);
    else
      e = p.item_rows == kChunkRows
              ? launch_chunk<D, BF16, 0, TREE>(a, c, p, cgrid, stream, mapped)
              : launch_chunk<D, BF16, chunk_parts(D, BF16), TREE>(a, c, p, cgrid, stream, mapped);
    if (e != cudaSuccess) return e;
  }
  const int n = sides.ctas[0] + sides.ctas[1];
  if (n == 0) return cudaSuccess;
  const int rows = cgrid > 0 ? sides.rows[1] : sides.rows[0];
  return launch_early(fa_cache_join_kernel<D, BF16>,
                      dim3(static_cast<unsigned>(n),
                           static_cast<unsigned>((rows + kJoinRows - 1) / kJoinRows)),
                      kJoinThreads, 0, stream, a, sides);
}

template <bool TREE>
cudaError_t launch_attn(const CacheAttnArgs& a, const fa_cache& c, bool bf16, int sm_count,
                        float* ws, cudaStream_t stream, bool* mapped) {
  AttnPlan p = plan_attn(a.B, a.T, a.group, a.cu_q != nullptr, TREE);
  // Items of 128 rows, K unwidened, where sequences have up to 128 rows to a K / V
  // head on average. Us of ragged calls with items of 256 rows beside it, bf16 (fp16),
  // 4 K / V heads, 8192 keys: 16 x 24 rows 70 / 77 (72 / 74), 16 x 64 rows 71 / 77
  // (72 / 75), 16 x 128 rows 78 / 83 (79 / 80). The average counts the sequences of the
  // step kernel too, which the host cannot tell from the others: one chunk of 2048
  // tokens behind 14336 others (behind none) beside 200 single tokens, 8 query heads to
  // a K / V head, takes 524 / 468 us (308 / 207), one of 512 tokens 116 / 123.
  // Trees: always, where there is that kernel.
  if (chunk_parts(c.d, bf16) > 0 && (TREE || static_cast<long long>(a.T) * a.group <= 128LL * a.B))
    p.item_rows = 128;
  *mapped = true;
  if (c.d == 64)
    return bf16 ? launch_all<64, true, TREE>(a, c, p, sm_count, ws, stream, mapped)
                : launch_all<64, false, TREE>(a, c, p, sm_count, ws, stream, mapped);
  return bf16 ? launch_all<128, true, TREE>(a, c, p, sm_count, ws, stream, mapped)
              : launch_all<128, false, TREE>(a, c, p, sm_count, ws, stream, mapped);
}

}  // namespace
}  // namespace fa
