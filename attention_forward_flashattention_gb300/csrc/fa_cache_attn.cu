// fa_fwd_cache: attention over the block cache. One warp per query row: a pass
// over the row's keys with the running maximum and sum, each lane holding
// d / 32 elements of q, K, V and O.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_cache.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

template <int D, bool BF16>
__global__ void __launch_bounds__(128) fa_cache_row_kernel(const CacheAttnArgs a) {
  constexpr int kPer = D / 32;
  const int lane = static_cast<int>(threadIdx.x & 31);
  const int b = static_cast<int>(blockIdx.y);
  const SeqRows s = seq_rows(a, b);
  const long long rows = static_cast<long long>(s.count) * a.H;
  const int bs1 = (1 << a.block_shift) - 1;
  for (long long r = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5); r < rows;
       r += 4LL * gridDim.x) {
    const int i = static_cast<int>(r / a.H), h = static_cast<int>(r % a.H);
    const int hk = h / a.group;
    const int lim = a.causal ? min(s.kv_len, s.kv_len - s.count + i + 1) : s.kv_len;
    float q[kPer], o[kPer];
    const uint16_t* qp = static_cast<const uint16_t*>(a.q) + q_offset(a, b, s, i, h) + kPer * lane;
    for (int e = 0; e < kPer; ++e) {
      if constexpr (BF16) q[e] = __uint_as_float(static_cast<uint32_t>(qp[e]) << 16);
      else q[e] = __half2float(__ushort_as_half(qp[e]));
      o[e] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    for (int j = 0; j < lim; ++j) {
      const int id = __ldg(a.table + static_cast<long long>(b) * a.table_width + (j >> a.block_shift));
      if (id < 0 || id >= a.num_blocks) continue;
      const long long at = id * a.block_stride + hk * a.head_stride + (j & bs1) * a.token_stride;
      const float ks = __ldg(a.ks + static_cast<long long>(id) * a.Hkv + hk);
      const float vs = __ldg(a.vs + static_cast<long long>(id) * a.Hkv + hk);
      float x = 0.f, v[kPer];
      for (int e = 0; e < kPer; e += 2) {
        const int c = kPer * lane + e;
        const float2 kk = ptx::e4m3x2_to_f32(*reinterpret_cast<const uint16_t*>(a.k + at + c));
        const float2 vv = ptx::e4m3x2_to_f32(*reinterpret_cast<const uint16_t*>(a.v + at + c));
        x = fmaf(q[e], kk.x, fmaf(q[e + 1], kk.y, x));
        v[e] = vv.x * vs;
        v[e + 1] = vv.y * vs;
      }
      for (int w = 16; w > 0; w >>= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
      x *= ks * a.scale_log2;
      const float top = fmaxf(m, x);
      const float keep = exp2f(m - top), p = exp2f(x - top);
      l = l * keep + p;
      for (int e = 0; e < kPer; ++e) o[e] = o[e] * keep + p * v[e];
      m = top;
    }
    const bool none = m == -INFINITY && l == 0.f;
    const float inv = none ? 0.f : 1.f / l;
    uint16_t* op = static_cast<uint16_t*>(a.o) + o_offset(a, b, s, i, h) + kPer * lane;
    for (int e = 0; e < kPer; ++e) {
      if constexpr (BF16) op[e] = __bfloat16_as_ushort(__float2bfloat16_rn(o[e] * inv));
      else op[e] = __half_as_ushort(__float2half_rn(o[e] * inv));
    }
    if (lane == 0)
      a.lse[lse_index(a, b, s, i, h)] =
          none ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
  }
}

}  // namespace

cudaError_t launch_cache_attn(const CacheAttnArgs& a, int d, bool bf16, int sm_count,
                              cudaStream_t stream) {
  const long long rows = static_cast<long long>(a.T) * a.H;
  long long x = (rows + 3) / 4;
  if (x > 64LL * sm_count) x = 64LL * sm_count;
  const dim3 grid(static_cast<unsigned>(x), static_cast<unsigned>(a.B));
  if (d == 64) {
    if (bf16) fa_cache_row_kernel<64, true><<<grid, 128, 0, stream>>>(a);
    else fa_cache_row_kernel<64, false><<<grid, 128, 0, stream>>>(a);
  } else {
    if (bf16) fa_cache_row_kernel<128, true><<<grid, 128, 0, stream>>>(a);
    else fa_cache_row_kernel<128, false><<<grid, 128, 0, stream>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace fa
