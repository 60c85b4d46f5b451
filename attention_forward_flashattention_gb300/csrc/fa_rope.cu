// fa_qk_norm_rope and its gradients (include/fa_rope.h): kernels, argument
// checks, launches.
//
// Every element is read and written once, with some ten operations, so HBM
// bounds both directions. d / 8 lanes share a row of d elements: a lane holds
// four elements and the four that they are paired with, so that the rotation
// needs no other lane and the norm one sum over the lanes. A lane group takes
// the same token of several heads, one after another in batches of kBatch rows
// whose loads are under way together: cosines, sines and weights are then read
// once for all of them.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "fa_cache.cuh"
#include "fa_check.h"
#include "fa_rope.h"
#include "ptx.cuh"

namespace fa {
namespace {

// Threads of a CTA, rows of a lane group under way together, CTAs on an SM. What
// counts is the rows under way on an SM, for which the registers have to suffice. Us,
// prompt of 16384 tokens, 32 + 8 heads, d 128 / B4 H16 N4096 d 128 / B2 H32 N8191 d 64.
// Forward, 128 threads, 4 rows, 8 CTAs 56.2 / 43.2 / 26.8 (6.0 / 6.2 / 5.6 TB/s, 87 % of a
// copy's rate for the prompt); 256, 4, 4: 58.0 / 44.9 / 28.0;
// 256, 8, 3: 61.7 / 48.4 / 29.3; 256, 4, 5, whose registers spill, 76.6 / 62.7 / 42.1.
// Backward (- / B4 / B2), 256, 4, 2: 76.0 / 48.3; 128, 4, 4: 76.0 / 49.4; 256, 2, 3: 95.4 /
// 60.4; the next rows requested while these are worked on, 256, 2, 2: 80.0 / 52.3.
constexpr int kFwdThreads = 128, kFwdBatch = 4, kFwdCtas = 8;
constexpr int kBwdThreads = 256, kBwdBatch = 4, kBwdCtas = 2;

struct RowsOf {  // q or k: its heads, and element strides of each operand
  const uint16_t* x;
  const uint16_t* dy;  // backward
  uint16_t* out;       // y, or dx
  fa_strides xs, dys, outs;
  const void* weight;
  int heads;
};

struct RopeArgs {
  RowsOf of[2];  // q, k
  const float* table;
  const int32_t* positions;
  long long positions_b;
  int n_positions, rotary, interleaved, weights_fp32;
  int B, N;
  int per_unit;        // heads that a lane group takes
  int chunks[2];       // units of a token, of q and of k
  int heads_inner;     // neighbouring units: chunks of one token, or tokens of one chunk
  long long units[2];  // B * N * chunks
  int ctas[2];         // the first ones take q's units, the others k's
  float eps;
  float* partial;  // backward: [CTAs][d]
};

template <bool BF16>
__device__ __forceinline__ float2 widen(uint32_t w) {
  if constexpr (BF16) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  } else {
    __half2 h;
    __builtin_memcpy(&h, &w, 4);
    return __half22float2(h);
  }
}
template <bool BF16>
__device__ __forceinline__ uint32_t narrow(float lo, float hi) {
  uint32_t w;
  if constexpr (BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    __builtin_memcpy(&w, &v, 4);
  } else {
    const __half2 v = __floats2half2_rn(lo, hi);
    __builtin_memcpy(&w, &v, 4);
  }
  return w;
}

// Eight elements of a row that a lane holds: four and their partners (half a
// row apart), or four neighbouring pairs.
struct Eight {
  uint2 lo, hi;
};
using Eight32 = float2[4];
template <bool BF16>
__device__ __forceinline__ void widen8(const Eight& e, Eight32& f) {
  f[0] = widen<BF16>(e.lo.x);
  f[1] = widen<BF16>(e.lo.y);
  f[2] = widen<BF16>(e.hi.x);
  f[3] = widen<BF16>(e.hi.y);
}
template <bool BF16>
__device__ __forceinline__ Eight narrow8(const Eight32& f) {
  return {make_uint2(narrow<BF16>(f[0].x, f[0].y), narrow<BF16>(f[1].x, f[1].y)),
          make_uint2(narrow<BF16>(f[2].x, f[2].y), narrow<BF16>(f[3].x, f[3].y))};
}

// Where a lane's two fours lie in a row.
struct Place {
  int lo, hi;
  int pair;  // its first pair's cosine, -1: not turned
};
template <int D>
__device__ __forceinline__ Place place_of(const RopeArgs& a, int lane) {
  const int p = 4 * lane, half = a.rotary >> 1;
  if (a.interleaved) return {2 * p, 2 * p + 4, p < half ? p : -1};
  if (p < half) return {p, p + half, p};
  return {a.rotary + p - half, a.rotary + (D - a.rotary) / 2 + p - half, -1};
}

// Cosines and sines of a lane's four pairs.
struct Turn {
  float4 c, s;
};
__device__ __forceinline__ Turn turn_of(const RopeArgs& a, const Place& w, int b, int n) {
  Turn t{make_float4(1.f, 1.f, 1.f, 1.f), make_float4(0.f, 0.f, 0.f, 0.f)};
  if (w.pair >= 0) {
    const int p = min(max(__ldg(a.positions + b * a.positions_b + n), 0), a.n_positions - 1);
    const float* row = a.table + static_cast<long long>(p) * a.rotary + w.pair;
    t.c = __ldg(reinterpret_cast<const float4*>(row));
    t.s = __ldg(reinterpret_cast<const float4*>(row + (a.rotary >> 1)));
  }
  return t;
}
// The rotation of eight elements as factors of each one (own) and of the one that it
// is paired with (other), two at a time. kBack: by the opposite angles.
struct Factors {
  Eight32 own, other;
};
template <bool INTERLEAVED, bool kBack>
__device__ __forceinline__ Factors factors_of(const Turn& t) {
  Factors f;
  const float sign = kBack ? -1.f : 1.f;
  const float c[4] = {t.c.x, t.c.y, t.c.z, t.c.w};
  const float s[4] = {sign * t.s.x, sign * t.s.y, sign * t.s.z, sign * t.s.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (INTERLEAVED) {
      f.own[i] = make_float2(c[i], c[i]);
      f.other[i] = make_float2(-s[i], s[i]);
    } else {
      const int j = 2 * (i & 1);
      f.own[i] = make_float2(c[j], c[j + 1]);
      f.other[i] = i < 2 ? make_float2(-s[j], -s[j + 1]) : make_float2(s[j], s[j + 1]);
    }
  }
  return f;
}
template <bool INTERLEAVED>
__device__ __forceinline__ float2 partner(const Eight32& f, int i) {
  return INTERLEAVED ? make_float2(f[i].y, f[i].x) : f[i ^ 2];
}
template <bool INTERLEAVED>
__device__ __forceinline__ void rotate(const Eight32& f, const Factors& k, Eight32& out) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    out[i] = ptx::ffma2(partner<INTERLEAVED>(f, i), k.other[i], ptx::fmul2(f[i], k.own[i]));
}

template <bool BF16>
__device__ __forceinline__ void weights_of(const RopeArgs& a, const void* w, const Place& at,
                                           Eight32& f) {
  if (w == nullptr) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = make_float2(1.f, 1.f);
  } else if (a.weights_fp32) {
    const float* p = static_cast<const float*>(w);
    const float4 x = __ldg(reinterpret_cast<const float4*>(p + at.lo));
    const float4 y = __ldg(reinterpret_cast<const float4*>(p + at.hi));
    f[0] = make_float2(x.x, x.y);
    f[1] = make_float2(x.z, x.w);
    f[2] = make_float2(y.x, y.y);
    f[3] = make_float2(y.z, y.w);
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(w);
    widen8<BF16>({__ldg(reinterpret_cast<const uint2*>(p + at.lo)),
                  __ldg(reinterpret_cast<const uint2*>(p + at.hi))}, f);
  }
}

// (plain loads: an output may be its input)
__device__ __forceinline__ Eight load8(const uint16_t* row, const Place& at) {
  return {*reinterpret_cast<const uint2*>(row + at.lo), *reinterpret_cast<const uint2*>(row + at.hi)};
}
__device__ __forceinline__ void store8(uint16_t* row, const Place& at, const Eight& e) {
  *reinterpret_cast<uint2*>(row + at.lo) = e.lo;
  *reinterpret_cast<uint2*>(row + at.hi) = e.hi;
}

// Sum over the L lanes of a group.
template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ float dot8(const Eight32& x, const Eight32& y) {
  float2 s = ptx::fmul2(x[0], y[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) s = ptx::ffma2(x[i], y[i], s);
  return s.x + s.y;
}
__device__ __forceinline__ float squares(const Eight32& x) { return dot8(x, x); }

struct Unit {
  int b, n, h0, h1;  // token, heads h0 .. h1 - 1
};
// (B * N * (H + Hkv), and so everything here, is below 2^31: divisions of 64 bits would take
// as long as a row's work)
__device__ __forceinline__ Unit unit_of(const RopeArgs& a, int which, uint32_t u) {
  uint32_t token, chunk;
  if (a.heads_inner) {
    const uint32_t chunks = static_cast<uint32_t>(a.chunks[which]);
    token = u / chunks;
    chunk = u - token * chunks;
  } else {
    const uint32_t tokens = static_cast<uint32_t>(a.B) * static_cast<uint32_t>(a.N);
    chunk = u / tokens;
    token = u - chunk * tokens;
  }
  const uint32_t b = token / static_cast<uint32_t>(a.N);
  Unit r;
  r.b = static_cast<int>(b);
  r.n = static_cast<int>(token - b * static_cast<uint32_t>(a.N));
  r.h0 = static_cast<int>(chunk) * a.per_unit;
  r.h1 = min(r.h0 + a.per_unit, a.of[which].heads);
  return r;
}
__device__ __forceinline__ long long row_at(const fa_strides& s, const Unit& u, int h) {
  return u.b * s.b + h * s.h + u.n * s.n;
}
// Rows h0 .. h0 + N - 1 of a unit, zeros for those that it does not have.
template <int N>
__device__ __forceinline__ void load_rows(const uint16_t* x, const fa_strides& s, const Unit& u,
                                          bool there, int h0, const Place& at, Eight (&e)[N]) {
  const uint16_t* row = x + row_at(s, u, h0);
#pragma unroll
  for (int i = 0; i < N; ++i, row += s.h) {
    e[i] = {make_uint2(0u, 0u), make_uint2(0u, 0u)};
    if (there && h0 + i < u.h1) e[i] = load8(row, at);
  }
}

template <int D, bool BF16, bool INTERLEAVED>
__global__ void __launch_bounds__(kFwdThreads, kFwdCtas) fa_norm_rope_kernel(const RopeArgs a) {
  constexpr int L = D / 8;
  const int lane = static_cast<int>(threadIdx.x) % L;
  const int which = static_cast<int>(blockIdx.x) >= a.ctas[0];
  const long long u = static_cast<long long>(static_cast<int>(blockIdx.x) - (which ? a.ctas[0] : 0)) *
                          (kFwdThreads / L) + threadIdx.x / L;
  // (a group without a unit takes part in the sums)
  const bool there = u < a.units[which];
  const Unit w = unit_of(a, which, there ? static_cast<uint32_t>(u) : 0u);
  const RowsOf& o = a.of[which];
  const Place at = place_of<D>(a, lane);
  Eight x[kFwdBatch];
  // (the rows first: the table waits for the positions)
  load_rows(o.x, o.xs, w, there, w.h0, at, x);
  Factors k = factors_of<INTERLEAVED, false>(turn_of(a, at, w.b, w.n));
  Eight32 wt;
  weights_of<BF16>(a, o.weight, at, wt);
  // the weights go into the rotation's factors, 1 / rms behind it
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    k.own[i] = ptx::fmul2(k.own[i], wt[i]);
    k.other[i] = ptx::fmul2(k.other[i], partner<INTERLEAVED>(wt, i));
  }
  for (int h0 = w.h0; h0 < w.h0 + a.per_unit; h0 += kFwdBatch) {  // (as often for all groups)
    if (h0 > w.h0) load_rows(o.x, o.xs, w, there, h0, at, x);
    uint16_t* out = o.out + row_at(o.outs, w, h0);
#pragma unroll
    for (int i = 0; i < kFwdBatch; ++i, out += o.outs.h) {
      Eight32 f, y;
      widen8<BF16>(x[i], f);
      const float inv = rsqrtf(fmaf(group_sum<L>(squares(f)), 1.f / D, a.eps));
      rotate<INTERLEAVED>(f, k, y);
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = ptx::fmul2(y[e], make_float2(inv, inv));
      if (there && h0 + i < w.h1) store8(out, at, narrow8<BF16>(y));
    }
  }
}

// dx, and each CTA's sum for the weights of q or k.
template <int D, bool BF16, bool INTERLEAVED>
__global__ void __launch_bounds__(kBwdThreads, kBwdCtas) fa_norm_rope_bwd_kernel(const RopeArgs a) {
  constexpr int L = D / 8, kGroups = kBwdThreads / L;
  __shared__ float s_sum[kGroups][D];
  const int lane = static_cast<int>(threadIdx.x) % L, group = static_cast<int>(threadIdx.x) / L;
  const int which = static_cast<int>(blockIdx.x) >= a.ctas[0];
  const int cta = static_cast<int>(blockIdx.x) - (which ? a.ctas[0] : 0);
  const RowsOf& o = a.of[which];
  const Place at = place_of<D>(a, lane);
  Eight32 wt, dw;
  weights_of<BF16>(a, o.weight, at, wt);
#pragma unroll
  for (int e = 0; e < 4; ++e) dw[e] = make_float2(0.f, 0.f);
  const long long step_units = static_cast<long long>(a.ctas[which]) * kGroups;
  for (long long u0 = static_cast<long long>(cta) * kGroups; u0 < a.units[which]; u0 += step_units) {
    const long long u = u0 + group;
    const bool there = u < a.units[which];
    const Unit w = unit_of(a, which, there ? static_cast<uint32_t>(u) : 0u);
    Eight x[kBwdBatch], dy[kBwdBatch];
    load_rows(o.x, o.xs, w, there, w.h0, at, x);
    load_rows(o.dy, o.dys, w, there, w.h0, at, dy);
    const Factors k = factors_of<INTERLEAVED, true>(turn_of(a, at, w.b, w.n));
    for (int h0 = w.h0; h0 < w.h0 + a.per_unit; h0 += kBwdBatch) {
      if (h0 > w.h0) {
        load_rows(o.x, o.xs, w, there, h0, at, x);
        load_rows(o.dy, o.dys, w, there, h0, at, dy);
      }
      uint16_t* out = o.out + row_at(o.outs, w, h0);
#pragma unroll
      for (int i = 0; i < kBwdBatch; ++i, out += o.outs.h) {
        Eight32 f, t, u;
        widen8<BF16>(x[i], f);
        widen8<BF16>(dy[i], u);
        rotate<INTERLEAVED>(u, k, t);
#pragma unroll
        for (int e = 0; e < 4; ++e) u[e] = ptx::fmul2(t[e], wt[e]);
        const float sum = group_sum<L>(squares(f)), dot = group_sum<L>(dot8(u, f));
        const float inv = rsqrtf(fmaf(sum, 1.f / D, a.eps));
        const float mean = dot * inv * (1.f / D);
        const float2 inv2 = make_float2(inv, inv), mean2 = make_float2(-mean, -mean);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 n = ptx::fmul2(f[e], inv2);
          dw[e] = ptx::ffma2(t[e], n, dw[e]);
          f[e] = ptx::fmul2(ptx::ffma2(n, mean2, u[e]), inv2);
        }
        if (there && h0 + i < w.h1) store8(out, at, narrow8<BF16>(f));
      }
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (a.partial == nullptr) return;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    *reinterpret_cast<float2*>(&s_sum[group][(e < 2 ? at.lo : at.hi) + 2 * (e & 1)]) = dw[e];
  __syncthreads();
  for (int c = static_cast<int>(threadIdx.x); c < D; c += kBwdThreads) {
    float v = 0.f;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) v += s_sum[g][c];
    a.partial[static_cast<long long>(blockIdx.x) * D + c] = v;
  }
}

// The CTAs' sums together: a CTA for 32 columns of dq_weight or dk_weight, eight
// warps that each take every eighth part.
template <int D>
__global__ void __launch_bounds__(256)
    fa_norm_rope_join_kernel(const float* partial, int parts_q, int parts_k, float* dq_weight,
                             float* dk_weight) {
  __shared__ float s_sum[8][32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  const bool of_k = blockIdx.x >= D / 32;
  const int col = (static_cast<int>(blockIdx.x) - (of_k ? D / 32 : 0)) * 32 + lane;
  const int parts = of_k ? parts_k : parts_q;
  const float* const from = partial + (of_k ? static_cast<long long>(parts_q) * D : 0) + col;
  float v = 0.f;
#pragma unroll 8
  for (int p = warp; p < parts; p += 8) v += __ldcg(from + static_cast<long long>(p) * D);
  s_sum[warp][lane] = v;
  __syncthreads();
  if (warp != 0) return;
#pragma unroll
  for (int w = 1; w < 8; ++w) v += s_sum[w][lane];
  float* const out = of_k ? dk_weight : dq_weight;
  if (out != nullptr) out[col] = v;
}

fa_status check_rope(const fa_rope* r, int d) {
  if (!r || !r->table || !r->positions) return FA_ERR_INVALID_ARG;
  if (!aligned(r->table, 16) || !aligned(r->positions, 4) || !aligned(r->q_weight, 16) ||
      !aligned(r->k_weight, 16))
    return FA_ERR_INVALID_ARG;
  if (r->n_positions <= 0 || r->positions_b < 0) return FA_ERR_INVALID_ARG;
  if (r->rotary_dim < 8 || r->rotary_dim > d || (r->rotary_dim & 7) != 0) return FA_ERR_INVALID_ARG;
  if (!(std::isfinite(r->eps) && r->eps > 0.f)) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

fa_status check_shape(int B, int H, int Hkv, int N, int d, fa_dtype dtype, const fa_strides* strides,
                      int n_strides) {
  if (B <= 0 || H <= 0 || Hkv <= 0 || N < 0 || !strides) return FA_ERR_INVALID_ARG;
  if (dtype != FA_DTYPE_FP16 && dtype != FA_DTYPE_BF16) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  for (int i = 0; i < n_strides; ++i)
    for (const long long s : {strides[i].b, strides[i].h, strides[i].n}) {
      const fa_status ss = check_stride(s);
      if (ss != FA_OK) return ss;
    }
  // (each factor is below 2^31, so that no product of two passes 2^63)
  const long long heads = static_cast<long long>(H) + Hkv, tokens = static_cast<long long>(B) * N;
  if (heads > 0x7FFFFFFFLL || tokens > 0x7FFFFFFFLL || tokens * heads > 0x7FFFFFFFLL)
    return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// Whether an output that is one of its own side's inputs has its rows where that has them. (An
// axis of length one has no stride of its own.)
bool in_place(const void* out, const void* in, const fa_strides& x, const fa_strides& y, int B, int heads, int N) {
  return out != in || ((B == 1 || x.b == y.b) && (heads == 1 || x.h == y.h) && (N <= 1 || x.n == y.n));
}

RopeArgs common(const fa_rope& r, int B, int N, int H, int Hkv, const fa_strides& q) {
  RopeArgs a{};
  a.of[0].weight = r.q_weight;
  a.of[1].weight = r.k_weight;
  a.of[0].heads = H;
  a.of[1].heads = Hkv;
  a.table = r.table;
  a.positions = r.positions;
  a.positions_b = r.positions_b;
  a.n_positions = r.n_positions;
  a.rotary = r.rotary_dim;
  a.interleaved = r.interleaved != 0;
  a.weights_fp32 = r.weights_fp32 != 0;
  a.B = B;
  a.N = N;
  a.heads_inner = q.h < q.n;
  a.eps = r.eps;
  return a;
}

// Heads of a unit: as many as leave every SM `groups` lane groups to run.
void split(RopeArgs& a, int most, long long groups) {
  const long long tokens = static_cast<long long>(a.B) * a.N;
  int per = most;
  auto units = [&](int i, int p) { return tokens * ((a.of[i].heads + p - 1) / p); };
  while (per > 1 && units(0, per) + units(1, per) < groups) per >>= 1;
  a.per_unit = per;
  for (int i = 0; i < 2; ++i) {
    a.chunks[i] = (a.of[i].heads + per - 1) / per;
    a.units[i] = units(i, per);
  }
}

template <int D, bool BF16>
cudaError_t launch_forward(RopeArgs a, cudaStream_t s) {
  constexpr int kGroups = kFwdThreads / (D / 8);
  for (int i = 0; i < 2; ++i) a.ctas[i] = static_cast<int>((a.units[i] + kGroups - 1) / kGroups);
  const unsigned grid = static_cast<unsigned>(a.ctas[0]) + static_cast<unsigned>(a.ctas[1]);
  if (a.interleaved) fa_norm_rope_kernel<D, BF16, true><<<grid, kFwdThreads, 0, s>>>(a);
  else fa_norm_rope_kernel<D, BF16, false><<<grid, kFwdThreads, 0, s>>>(a);
  return cudaGetLastError();
}

template <int D, bool BF16>
cudaError_t launch_backward(RopeArgs a, int most, float* dqw, float* dkw, cudaStream_t s) {
  constexpr int kGroups = kBwdThreads / (D / 8);
  // CTAs that run at once, shared out by the units of q and k
  const long long want[2] = {(a.units[0] + kGroups - 1) / kGroups, (a.units[1] + kGroups - 1) / kGroups};
  const long long share = (most * a.units[1] + (a.units[0] + a.units[1]) / 2) / (a.units[0] + a.units[1]);
  const long long k = share < 1 ? 1 : share > most - 1 ? most - 1 : share;
  a.ctas[1] = static_cast<int>(want[1] < k ? want[1] : k);
  a.ctas[0] = static_cast<int>(want[0] < most - k ? want[0] : most - k);
  const unsigned grid = static_cast<unsigned>(a.ctas[0] + a.ctas[1]);
  if (a.interleaved) fa_norm_rope_bwd_kernel<D, BF16, true><<<grid, kBwdThreads, 0, s>>>(a);
  else fa_norm_rope_bwd_kernel<D, BF16, false><<<grid, kBwdThreads, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.partial == nullptr) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2 * D / 32);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fa_norm_rope_join_kernel<D>, static_cast<const float*>(a.partial),
                            a.ctas[0], a.ctas[1], dqw, dkw);
}

}  // namespace
}  // namespace fa

extern "C" {

fa_status fa_qk_norm_rope(const void* q, const void* k, void* q_out, void* k_out, int B, int H,
                          int Hkv, int N, int d, const fa_strides* strides, const fa_rope* rope,
                          fa_dtype dtype, void* stream) {
  for (const void* p : {q, k, static_cast<const void*>(q_out), static_cast<const void*>(k_out)})
    if (!p || !fa::aligned(p, 16)) return FA_ERR_INVALID_ARG;
  const fa_status cs = fa::check_shape(B, H, Hkv, N, d, dtype, strides, 4);
  if (cs == FA_ERR_INVALID_ARG) return cs;
  if (N > 0 && (q_out == k_out || q_out == k || k_out == q ||
                !fa::in_place(q_out, q, strides[2], strides[0], B, H, N) ||
                !fa::in_place(k_out, k, strides[3], strides[1], B, Hkv, N)))
    return FA_ERR_INVALID_ARG;
  const fa_status cr = fa::check_rope(rope, d);
  if (cr != FA_OK) return cr;
  if (cs != FA_OK) return cs;
  int sms = 0;
  const fa_status ds = fa::device_facts(&sms, nullptr);
  if (ds != FA_OK) return ds;
  if (N == 0) return FA_OK;
  fa::RopeArgs a = fa::common(*rope, B, N, H, Hkv, strides[0]);
  const void* in[2] = {q, k};
  void* out[2] = {q_out, k_out};
  for (int i = 0; i < 2; ++i) {
    a.of[i].x = static_cast<const uint16_t*>(in[i]);
    a.of[i].out = static_cast<uint16_t*>(out[i]);
    a.of[i].xs = strides[i];
    a.of[i].outs = strides[2 + i];
  }
  fa::split(a, 8, 2048LL / (d / 8) * sms);
  (void)cudaGetLastError();
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool bf16 = dtype == FA_DTYPE_BF16;
  const cudaError_t e = d == 64 ? (bf16 ? fa::launch_forward<64, true>(a, s) : fa::launch_forward<64, false>(a, s))
                                : (bf16 ? fa::launch_forward<128, true>(a, s) : fa::launch_forward<128, false>(a, s));
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_qk_norm_rope_bwd_workspace_size(int d, size_t* bytes) {
  if (!bytes) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  int sms = 0;
  const fa_status ds = fa::device_facts(&sms, nullptr);
  if (ds != FA_OK) return ds;
  *bytes = sizeof(float) * static_cast<size_t>(d) * static_cast<size_t>(sms * fa::kBwdCtas);
  return FA_OK;
}

fa_status fa_qk_norm_rope_bwd(const void* dq_out, const void* dk_out, const void* q, const void* k,
                              void* dq, void* dk, float* dq_weight, float* dk_weight, int B, int H,
                              int Hkv, int N, int d, const fa_strides* strides, const fa_rope* rope,
                              fa_dtype dtype, void* workspace, size_t workspace_size, void* stream) {
  for (const void* p : {dq_out, dk_out, q, k, static_cast<const void*>(dq), static_cast<const void*>(dk)})
    if (!p || !fa::aligned(p, 16)) return FA_ERR_INVALID_ARG;
  if (!fa::aligned(dq_weight, 4) || !fa::aligned(dk_weight, 4) || !fa::aligned(workspace, 16))
    return FA_ERR_INVALID_ARG;
  const bool sums = dq_weight != nullptr || dk_weight != nullptr;
  if ((sums && !workspace) || (sums && dq_weight == dk_weight)) return FA_ERR_INVALID_ARG;
  const fa_status cs = fa::check_shape(B, H, Hkv, N, d, dtype, strides, 6);
  if (cs == FA_ERR_INVALID_ARG) return cs;
  if (N > 0 && (dq == dk || dq == dk_out || dk == dq_out || dq == k || dk == q ||
                !fa::in_place(dq, dq_out, strides[4], strides[0], B, H, N) ||
                !fa::in_place(dq, q, strides[4], strides[2], B, H, N) ||
                !fa::in_place(dk, dk_out, strides[5], strides[1], B, Hkv, N) ||
                !fa::in_place(dk, k, strides[5], strides[3], B, Hkv, N)))
    return FA_ERR_INVALID_ARG;
  const fa_status cr = fa::check_rope(rope, d);
  if (cr != FA_OK) return cr;
  if (cs != FA_OK) return cs;
  size_t need = 0;
  const fa_status ws = fa_qk_norm_rope_bwd_workspace_size(d, &need);
  if (ws != FA_OK) return ws;
  if (sums && workspace_size < need) return FA_ERR_INVALID_ARG;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  (void)cudaGetLastError();
  if (N == 0) {
    for (float* w : {dq_weight, dk_weight})
      if (w && cudaMemsetAsync(w, 0, sizeof(float) * static_cast<size_t>(d), s) != cudaSuccess) return FA_ERR_CUDA;
    return FA_OK;
  }
  int sms = 0;
  const fa_status ds = fa::device_facts(&sms, nullptr);
  if (ds != FA_OK) return ds;
  fa::RopeArgs a = fa::common(*rope, B, N, H, Hkv, strides[2]);
  const void* x[2] = {q, k};
  const void* dy[2] = {dq_out, dk_out};
  void* out[2] = {dq, dk};
  for (int i = 0; i < 2; ++i) {
    a.of[i].x = static_cast<const uint16_t*>(x[i]);
    a.of[i].dy = static_cast<const uint16_t*>(dy[i]);
    a.of[i].out = static_cast<uint16_t*>(out[i]);
    a.of[i].dys = strides[i];
    a.of[i].xs = strides[2 + i];
    a.of[i].outs = strides[4 + i];
  }
  a.partial = sums ? static_cast<float*>(workspace) : nullptr;
  fa::split(a, 8, 2048LL / (d / 8) * sms);
  const int most = sms * fa::kBwdCtas;
  const bool bf16 = dtype == FA_DTYPE_BF16;
  const cudaError_t e =
      d == 64 ? (bf16 ? fa::launch_backward<64, true>(a, most, dq_weight, dk_weight, s)
                      : fa::launch_backward<64, false>(a, most, dq_weight, dk_weight, s))
              : (bf16 ? fa::launch_backward<128, true>(a, most, dq_weight, dk_weight, s)
                      : fa::launch_backward<128, false>(a, most, dq_weight, dk_weight, s));
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
