// fa_cache_append: new K and V into the cache's e4m3 blocks.
//
// The scale of a block and head is a power of two, s = 2^ceil(log2(amax / 448)),
// so value / s and old code * old s / new s are exact in fp32 and each value is
// rounded once, on conversion (a code that a grown scale makes subnormal twice).
// Against amax / 448 itself this costs no accuracy: e4m3 is a floating format,
// and a factor below 2 in the scale moves only the point where codes become
// subnormal.
//
// A run is the new tokens of one block: consecutive tokens with consecutive
// slots. A team of block / 16 warps owns the runs that start in `block`
// consecutive tokens (a tile) of one head of K or V. It takes them in windows
// of whole runs, at most `block` tokens: each warp holds 16 tokens in
// registers (one read of the input), the largest magnitudes meet in shared
// memory per run, and the codes are written from the same registers. A run's
// scale has one owner, so there are no atomics in global memory and no order
// to depend on.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_cache.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;

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

// Largest finite magnitude of two packed 16-bit values, as the bits of its
// magnitude (the order of magnitudes is that of their bits).
template <bool BF16>
__device__ __forceinline__ uint32_t magnitude(uint32_t w, uint32_t so_far) {
  constexpr uint32_t kInf = BF16 ? 0x7F80u : 0x7C00u;
  const uint32_t lo = w & 0x7FFFu, hi = (w >> 16) & 0x7FFFu;
  so_far = max(so_far, lo < kInf ? lo : 0u);
  return max(so_far, hi < kInf ? hi : 0u);
}

template <bool BF16>
__device__ __forceinline__ float from_bits(uint32_t m) {
  return BF16 ? __uint_as_float(m << 16)
              : __half2float(__ushort_as_half(static_cast<unsigned short>(m)));
}

// The smallest power of two s >= 2^kCacheMinScaleExp with x <= 448 s (x >= 0, finite).
__device__ __forceinline__ float scale_for(float x) {
  // 448 = 1.75 * 2^8: the exponent of x less 8, one more above 1.75
  const uint32_t u = __float_as_uint(x);
  int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = max(e, kCacheMinScaleExp);
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}
// The smallest power of two that is not below x (a positive normal number).
__device__ __forceinline__ float pow2_above(float x) {
  const uint32_t u = __float_as_uint(x);
  return __uint_as_float((u + 0x7FFFFFu) & 0xFF800000u);
}

// x * f, but NaN where x is infinite (f is positive and finite).
__device__ __forceinline__ float scaled(float x, float f) { return fmaf(x, f, x * 0.f); }

// Four codes times f, rounded to codes again.
__device__ __forceinline__ uint32_t rescale4(uint32_t c, float f) {
  const float2 lo = ptx::e4m3x2_to_f32(c & 0xFFFFu), hi = ptx::e4m3x2_to_f32(c >> 16);
  return ptx::pack4_e4m3(lo.x * f, lo.y * f, hi.x * f, hi.y * f);
}

// BLOCK: tokens in a block. D: head dimension.
template <int BLOCK, int D, bool BF16>
__global__ void __launch_bounds__(kThreads) fa_cache_append_kernel(const CacheAppendArgs a) {
  constexpr int kTeamWarps = BLOCK / 16;
  constexpr int kTeams = kWarps / kTeamWarps;
  constexpr int kTeamThreads = kTeamWarps * 32;
  constexpr int kLanesPerRow = D / 8;           // 16 bytes of input per lane
  constexpr int kRowsPerLoad = 32 / kLanesPerRow;
  constexpr int kLoads = 16 / kRowsPerLoad;     // loads that cover a warp's 16 tokens
  constexpr int kWords = BLOCK / 16 + 1;        // start bits of 2 * BLOCK + 1 tokens
  struct Team {
    int slot[2 * BLOCK];      // slots of the tile's tokens and the next BLOCK ones
    uint32_t start[kWords];   // bit p: token t0 + p starts a run (or is in none)
    uint32_t amax[BLOCK];     // per run of the window, at its first token's place
    float inv[BLOCK];         // 1 / scale
    float again[BLOCK];       // old scale / new scale of a run whose block's old codes change
    uint32_t grown[(BLOCK + 31) / 32];  // the runs that have such a block
  };
  __shared__ Team teams[kTeams];

  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  const int team = warp / kTeamWarps, tw = warp % kTeamWarps;
  const int tt = tw * 32 + lane;
  Team& s = teams[team];
  const int hk = static_cast<int>(blockIdx.y) * kTeams + team;  // 2 * head + (0: K, 1: V)
  const bool active = hk < 2 * a.Hkv;
  const int which = hk & 1, head = hk >> 1;
  auto sync = [&] {
    if constexpr (kTeamWarps == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(kTeamThreads) : "memory");
  };
  if (!active) return;  // a whole team leaves together
  const int t0 = static_cast<int>(blockIdx.x) * BLOCK;

  // Slots of the 2 * BLOCK tokens from t0, and where runs start. Bits at and
  // behind the last token are set.
  for (int p = tt; p < 32 * kWords; p += kTeamThreads) {
    const int t = t0 + p;
    const int now = t < a.T ? __ldg(a.slots + t) : -1;
    const bool ok = now >= 0 && now < a.n_slots;
    bool first = true;
    if (ok && t > 0) {
      const int before = __ldg(a.slots + t - 1);
      first = before + 1 != now || before < 0 || (now & (BLOCK - 1)) == 0;
    }
    if (p < 2 * BLOCK) s.slot[p] = ok ? now : -1;
    const uint32_t bits = __ballot_sync(0xffffffffu, first);
    if (lane == 0) s.start[p >> 5] = bits;
  }
  sync();

  // First start at or behind place p (2 * BLOCK if there is none before it).
  auto next_start = [&](int p) {
    while (p < 2 * BLOCK) {
      const uint32_t w = s.start[p >> 5] >> (p & 31);
      if (w) return p + __ffs(static_cast<int>(w)) - 1;
      p = (p | 31) + 1;
    }
    return 2 * BLOCK;
  };
  // Last start at or before place p (the caller knows that there is one).
  auto last_start = [&](int p) {
    int w = p >> 5;
    uint32_t u = s.start[w] & (0xFFFFFFFFu >> (31 - (p & 31)));
    while (u == 0 && w > 0) u = s.start[--w];
    return (w << 5) + 31 - __clz(static_cast<int>(u));
  };

  const uint8_t* xbase = reinterpret_cast<const uint8_t*>(
      which ? a.v + head * a.v_h : a.k + head * a.k_h);
  const long long xrow = 2 * (which ? a.v_n : a.k_n);  // bytes from token to token
  uint8_t* cbase = (which ? a.v_codes : a.k_codes) + head * a.head_stride;
  float* scales = (which ? a.v_scales : a.k_scales) + head;
  const int row_in_load = lane / kLanesPerRow, part = lane % kLanesPerRow;

  int cur = next_start(0);
  while (cur < BLOCK && t0 + cur < a.T) {
    // the window [cur, end): whole runs, at most BLOCK tokens, starts below BLOCK
    // (a run ends with its block, so one starts in (cur, cur + BLOCK])
    int end = last_start(cur + BLOCK);
    if (end > BLOCK) end = next_start(BLOCK);
    for (int p = tt; p < BLOCK; p += kTeamThreads) s.amax[p] = 0u;
    sync();

    uint4 x[kLoads];
    int run[kLoads];  // window place of the row's run, or -1
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int p = cur + tw * 16 + i * kRowsPerLoad + row_in_load;
      run[i] = (p < end && s.slot[p] >= 0) ? last_start(p) - cur : -1;
      x[i] = make_uint4(0u, 0u, 0u, 0u);
      if (run[i] >= 0)
        x[i] = *reinterpret_cast<const uint4*>(
            xbase + (t0 + p) * xrow + 16 * part);
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      uint32_t m = magnitude<BF16>(x[i].x, 0u);
      m = magnitude<BF16>(x[i].y, m);
      m = magnitude<BF16>(x[i].z, m);
      m = magnitude<BF16>(x[i].w, m);
#pragma unroll
      for (int o = kLanesPerRow / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (part == 0 && run[i] >= 0) atomicMax(&s.amax[run[i]], m);
    }
    sync();

    // one thread per run: its scale
    for (int p = tt; p < (BLOCK < 32 ? 32 : BLOCK); p += kTeamThreads) {
      const int at = cur + p;
      bool grew = false;
      if (at < end && s.slot[at] >= 0 && ((s.start[at >> 5] >> (at & 31)) & 1u)) {
        const int slot = s.slot[at];
        float* sc = scales + static_cast<long long>(slot / BLOCK) * a.Hkv;
        float now = scale_for(from_bits<BF16>(s.amax[p]));
        if ((slot & (BLOCK - 1)) != 0) {
          const float old = *sc;
          now = fmaxf(now, pow2_above(old));
          s.again[p] = old / now;
          grew = now != old;
        }
        *sc = now;
        s.inv[p] = 1.f / now;
      }
      const uint32_t bits = __ballot_sync(0xffffffffu, grew);
      if (lane == 0) s.grown[p >> 5] = bits;
    }
    sync();

#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      if (run[i] < 0) continue;
      const int slot = s.slot[cur + tw * 16 + i * kRowsPerLoad + row_in_load];
      const float f = s.inv[run[i]];
      const float2 v0 = widen<BF16>(x[i].x), v1 = widen<BF16>(x[i].y);
      const float2 v2 = widen<BF16>(x[i].z), v3 = widen<BF16>(x[i].w);
      uint2 c;
      c.x = ptx::pack4_e4m3(scaled(v0.x, f), scaled(v0.y, f), scaled(v1.x, f), scaled(v1.y, f));
      c.y = ptx::pack4_e4m3(scaled(v2.x, f), scaled(v2.y, f), scaled(v3.x, f), scaled(v3.y, f));
      *reinterpret_cast<uint2*>(cbase + static_cast<long long>(slot / BLOCK) * a.block_stride +
                                (slot & (BLOCK - 1)) * a.token_stride + 8 * part) = c;
    }
    // blocks whose scale grew: their older rows, 16 codes a thread
    for (int wd = 0; wd < (BLOCK + 31) / 32; ++wd) {
      uint32_t left = s.grown[wd];
      while (left) {
        const int p = 32 * wd + __ffs(static_cast<int>(left)) - 1;
        left &= left - 1;
        const float f = s.again[p];
        const int slot = s.slot[cur + p];
        uint8_t* rows = cbase + static_cast<long long>(slot / BLOCK) * a.block_stride;
        const int older = (slot & (BLOCK - 1)) * (D / 16);
        for (int e = tt; e < older; e += kTeamThreads) {
          uint4* w = reinterpret_cast<uint4*>(rows + (e / (D / 16)) * a.token_stride +
                                              16 * (e % (D / 16)));
          uint4 u = *w;
          u.x = rescale4(u.x, f);
          u.y = rescale4(u.y, f);
          u.z = rescale4(u.z, f);
          u.w = rescale4(u.w, f);
          *w = u;
        }
      }
    }
    cur = next_start(end);
    sync();  // the window's shared values are free
  }
}

template <int BLOCK, int D, bool BF16>
cudaError_t launch(const CacheAppendArgs& a, cudaStream_t stream) {
  constexpr int kTeams = kWarps / (BLOCK / 16);
  const dim3 grid(static_cast<unsigned>((static_cast<long long>(a.T) + BLOCK - 1) / BLOCK),
                  static_cast<unsigned>((2 * a.Hkv + kTeams - 1) / kTeams));
  fa_cache_append_kernel<BLOCK, D, BF16><<<grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

template <int BLOCK>
cudaError_t pick(const CacheAppendArgs& a, int d, bool bf16, cudaStream_t s) {
  if (d == 64) return bf16 ? launch<BLOCK, 64, true>(a, s) : launch<BLOCK, 64, false>(a, s);
  return bf16 ? launch<BLOCK, 128, true>(a, s) : launch<BLOCK, 128, false>(a, s);
}

}  // namespace

cudaError_t launch_cache_append(const CacheAppendArgs& a, int block, int d, bool bf16,
                                cudaStream_t stream) {
  switch (block) {
    case 16: return pick<16>(a, d, bf16, stream);
    case 32: return pick<32>(a, d, bf16, stream);
    case 64: return pick<64>(a, d, bf16, stream);
    default: return pick<128>(a, d, bf16, stream);
  }
}

}  // namespace fa
