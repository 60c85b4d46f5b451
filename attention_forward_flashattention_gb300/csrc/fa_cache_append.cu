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
// consecutive tokens (a tile), for some of the planes (K or V, head). It takes
// them in windows of whole runs, at most `block` tokens: each warp holds 16
// tokens in registers (one read of the input), the largest magnitudes meet in
// shared memory per run, and the codes are written from the same registers. A
// run's scale has one owner, so there are no atomics in global memory and no
// order to depend on. A second team takes a tile's windows behind the first,
// so that a batch of odd lengths does not serialise them.
//
// Bound by HBM for prompts (6 bytes for 2 values), by the chain slots - input -
// scale - codes for single tokens. Measured: two prompts of 16384 tokens, 32
// heads, d 128, 805 MB: 130 us, 6.2 TB/s (93 % of a copy's rate); 32 single
// tokens, 8 heads, d 64: 4.0 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_cache.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
// 64 registers a thread: the instances of blocks of 16, 32 and 64 spill 32 to 36
// bytes at d = 128 (blocks of 32 at d = 64: 4), those of 128 nothing.
constexpr int kCtasPerSm = 4;

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

// Largest magnitudes of two packed 16-bit values each, as their bits: the order
// of magnitudes is that of their bits, infinities and NaN above all numbers.
__device__ __forceinline__ uint32_t magnitudes(uint4 v) {
  constexpr uint32_t kAbs = 0x7FFF7FFFu;
  return __vimax3_u16x2(__vmaxu2(v.x & kAbs, v.y & kAbs), v.z & kAbs, v.w & kAbs);
}
template <bool BF16>
constexpr uint32_t kInfBits = BF16 ? 0x7F80u : 0x7C00u;
// The largest finite one of 8 values.
template <bool BF16>
__device__ __forceinline__ uint32_t finite_magnitude(uint4 v) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
    const uint32_t e = (i & 1 ? w >> 16 : w) & 0x7FFFu;
    if (e < kInfBits<BF16>) m = max(m, e);
  }
  return m;
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

// Codes of 8 values times f; kOdd: infinities and NaN among them become NaN
// (inf * 0 is NaN, a finite value plus its product with 0 is itself).
template <bool BF16, bool kOdd>
__device__ __forceinline__ uint2 encode8(uint4 x, float f) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = widen<BF16>(w[i]);
    v[2 * i] = kOdd ? fmaf(t.x, f, t.x * 0.f) : t.x * f;
    v[2 * i + 1] = kOdd ? fmaf(t.y, f, t.y * 0.f) : t.y * f;
  }
  return make_uint2(ptx::pack4_e4m3(v[0], v[1], v[2], v[3]),
                    ptx::pack4_e4m3(v[4], v[5], v[6], v[7]));
}

// Four codes times f, rounded to codes again.
__device__ __forceinline__ uint32_t rescale4(uint32_t c, float f) {
  const float2 lo = ptx::e4m3x2_to_f32(c & 0xFFFFu), hi = ptx::e4m3x2_to_f32(c >> 16);
  return ptx::pack4_e4m3(lo.x * f, lo.y * f, hi.x * f, hi.y * f);
}

// BLOCK: tokens in a block. D: head dimension. A team takes `planes` of the 2 Hkv
// (K or V, head) planes of its tile, one after another.
template <int BLOCK, int D, bool BF16>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) fa_cache_append_kernel(
    const CacheAppendArgs a, const int planes, const int windows) {
  constexpr int kTeamWarps = BLOCK / 16;
  constexpr int kTeams = kWarps / kTeamWarps;
  constexpr int kTeamThreads = kTeamWarps * 32;
  constexpr int kLanesPerRow = D / 8;           // 16 bytes of input per lane
  constexpr int kRowsPerLoad = 32 / kLanesPerRow;
  constexpr int kLoads = 16 / kRowsPerLoad;     // loads that cover a warp's 16 tokens
  constexpr int kWords = BLOCK / 16 + 1;        // start bits of 2 * BLOCK + 1 tokens
  constexpr int kGrown = (BLOCK + 31) / 32;
  struct Team {
    int slot[2 * BLOCK];      // slots of the tile's tokens and the next BLOCK ones
    short run[BLOCK];         // window place of a token's run, or -1
    uint32_t start[kWords];   // bit p: token t0 + p starts a run (or is in none)
    uint32_t amax[BLOCK];     // per run of the window, at its first token's place
    float inv[BLOCK];         // 1 / scale
    float again[BLOCK];       // old scale / new scale of a run whose block's old codes change
    uint32_t grown[kGrown];   // the runs that have such a block
  };
  __shared__ Team teams[kTeams];

  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  const int team = warp / kTeamWarps, tw = warp % kTeamWarps;
  const int tt = tw * 32 + lane;
  Team& s = teams[team];
  auto sync = [&] {
    if constexpr (kTeamWarps == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(kTeamThreads) : "memory");
  };
  // Teams of one tile are neighbours: they read the same rows of the input.
  const int groups = (2 * a.Hkv + planes - 1) / planes;  // teams of a window
  const long long unit = static_cast<long long>(blockIdx.x) * kTeams + team;
  const long long tile_window = unit / groups;
  const long long tile = tile_window / windows;
  int skip = static_cast<int>(tile_window - tile * windows);  // windows that other teams take
  const bool rest = skip == windows - 1;  // this team takes all windows behind them
  const int plane0 = static_cast<int>(unit - tile_window * groups) * planes;
  const int plane1 = min(plane0 + planes, 2 * a.Hkv);
  if (tile * BLOCK >= a.T) return;  // a whole team leaves together
  const int t0 = static_cast<int>(tile) * BLOCK;

  // Slots of the 2 * BLOCK tokens from t0, and where runs start. Bits at and
  // behind the last token are set.
  for (int p = tt; p < 32 * kWords; p += kTeamThreads) {
    const int t = t0 + p;
    const int now = t < a.T ? __ldg(a.slots + t) : -1;
    const int before = t > 0 && t < a.T ? __ldg(a.slots + t - 1) : -1;
    const bool ok = now >= 0 && now < a.n_slots;
    const bool first = !ok || before < 0 || before + 1 != now || (now & (BLOCK - 1)) == 0;
    if (p < 2 * BLOCK) s.slot[p] = ok ? now : -1;
    const uint32_t bits = __ballot_sync(0xffffffffu, first);
    if (lane == 0) s.start[p >> 5] = bits;
  }
  for (int p = tt; p < BLOCK; p += kTeamThreads) s.amax[p] = 0u;
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
  const int row_in_load = lane / kLanesPerRow, part = lane % kLanesPerRow;

  for (int cur = next_start(0); cur < BLOCK && t0 + cur < a.T;) {
    // the window [cur, end): whole runs, at most BLOCK tokens, starts below BLOCK
    // (a run ends with its block, so one starts in (cur, cur + BLOCK])
    int end = last_start(cur + BLOCK);
    if (end > BLOCK) end = next_start(BLOCK);
    if (skip > 0) {
      --skip;
      cur = next_start(end);
      continue;
    }
    for (int p = tt; p < BLOCK; p += kTeamThreads)
      s.run[p] = static_cast<short>(
          cur + p < end && s.slot[cur + p] >= 0 ? last_start(cur + p) - cur : -1);
    sync();
    const int place = tw * 16 + row_in_load;  // of this lane's first row in the window
    const long long first_row = t0 + cur + place;
    // All of the warp's 16 tokens in one run (the rule in prompts): one
    // reduction, and rows at a constant distance on both sides.
    const int warp_run = s.run[tw * 16];
    const bool together = warp_run >= 0 && s.run[tw * 16 + 15] == warp_run;
    const int warp_slot = together ? s.slot[cur + place] : 0;

    for (int plane = plane0; plane < plane1; ++plane) {
      const bool is_v = plane >= a.Hkv;
      const int head = is_v ? plane - a.Hkv : plane;
      const uint16_t* x_in = is_v ? a.v + head * a.v_h : a.k + head * a.k_h;
      const long long x_n = is_v ? a.v_n : a.k_n;
      uint8_t* codes = (is_v ? a.v_codes : a.k_codes) + head * a.head_stride;
      float* scales = (is_v ? a.v_scales : a.k_scales) + head;

      // the run's present scale, one thread per run (a team has a thread for each place)
      const int at = cur + tt;
      const bool owner = tt < BLOCK && at < end && s.run[tt < BLOCK ? tt : 0] == tt;
      float* sc = nullptr;
      float old = 0.f;
      if (owner) {
        const int slot = s.slot[at];
        sc = scales + static_cast<long long>(slot / BLOCK) * a.Hkv;
        if ((slot & (BLOCK - 1)) != 0) old = *sc;
      }
      uint4 x[kLoads];
      {
        const uint16_t* p = x_in + first_row * x_n + 8 * part;
        const long long step = kRowsPerLoad * x_n;
#pragma unroll
        for (int i = 0; i < kLoads; ++i, p += step) {
          x[i] = make_uint4(0u, 0u, 0u, 0u);
          if (together || s.run[place + i * kRowsPerLoad] >= 0)
            x[i] = __ldcs(reinterpret_cast<const uint4*>(p));
        }
      }
      uint32_t odd = 0;  // bit i: infinities or NaN in x[i]
      if (together) {
        uint32_t two = magnitudes(x[0]);
#pragma unroll
        for (int i = 1; i < kLoads; ++i) two = __vmaxu2(two, magnitudes(x[i]));
        uint32_t m = max(two & 0xFFFFu, two >> 16);
        if (m >= kInfBits<BF16>) {
          odd = (1u << kLoads) - 1u;
          m = 0;
#pragma unroll
          for (int i = 0; i < kLoads; ++i) m = max(m, finite_magnitude<BF16>(x[i]));
        }
        m = __reduce_max_sync(0xffffffffu, m);
        if (lane == 0) atomicMax(&s.amax[warp_run], m);
      } else {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const uint32_t two = magnitudes(x[i]);
          uint32_t m = max(two & 0xFFFFu, two >> 16);
          if (m >= kInfBits<BF16>) {
            odd |= 1u << i;
            m = finite_magnitude<BF16>(x[i]);
          }
#pragma unroll
          for (int o = kLanesPerRow / 2; o > 0; o >>= 1)
            m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
          const int run = s.run[place + i * kRowsPerLoad];
          if (part == 0 && run >= 0) atomicMax(&s.amax[run], m);
        }
      }
      sync();

      bool grew = false;
      if (owner) {
        float now = scale_for(from_bits<BF16>(s.amax[tt]));
        if (old > 0.f) {  // the block holds older tokens
          now = fmaxf(now, pow2_above(old));
          s.again[tt] = old / now;
          grew = now != old;
        }
        *sc = now;
        s.inv[tt] = 1.f / now;
        s.amax[tt] = 0u;
      }
      const uint32_t bits = __ballot_sync(0xffffffffu, grew);
      if (lane == 0 && tt < BLOCK) s.grown[tt >> 5] = bits;
      sync();

      if (together && odd == 0u) {
        const float f = s.inv[warp_run];
        uint8_t* p = codes + static_cast<long long>(warp_slot / BLOCK) * a.block_stride +
                     (warp_slot & (BLOCK - 1)) * a.token_stride + 8 * part;
        const long long step = kRowsPerLoad * a.token_stride;
#pragma unroll
        for (int i = 0; i < kLoads; ++i, p += step)
          *reinterpret_cast<uint2*>(p) = encode8<BF16, false>(x[i], f);
      } else {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const int run = s.run[place + i * kRowsPerLoad];
          if (run < 0) continue;
          const int slot = s.slot[cur + place + i * kRowsPerLoad];
          const float f = s.inv[run];
          const uint2 c = ((odd >> i) & 1u) ? encode8<BF16, true>(x[i], f)
                                            : encode8<BF16, false>(x[i], f);
          *reinterpret_cast<uint2*>(codes + static_cast<long long>(slot / BLOCK) * a.block_stride +
                                    (slot & (BLOCK - 1)) * a.token_stride + 8 * part) = c;
        }
      }
      // blocks whose scale grew: their older rows, 16 codes a thread
      for (int wd = 0; wd < kGrown; ++wd) {
        uint32_t left = s.grown[wd];
        while (left) {
          const int p = 32 * wd + __ffs(static_cast<int>(left)) - 1;
          left &= left - 1;
          const float f = s.again[p];
          const int slot = s.slot[cur + p];
          uint8_t* rows = codes + static_cast<long long>(slot / BLOCK) * a.block_stride;
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
      // (the next plane's shared values are written behind its first barrier)
    }
    if (!rest) break;
    cur = next_start(end);
    sync();  // the window's places are read
  }
}

template <int BLOCK, int D, bool BF16>
cudaError_t launch(const CacheAppendArgs& a, int sm_count, cudaStream_t stream) {
  constexpr int kTeams = kWarps / (BLOCK / 16);
  constexpr int kWindows = 2;  // (a tile owns less than 2 * BLOCK tokens: two windows, rarely three)
  const long long tiles = (static_cast<long long>(a.T) + BLOCK - 1) / BLOCK;
  // Planes for each team: looking for runs costs as much as a plane or two, so
  // it is done once for several planes as soon as there is work for more
  // than the CTAs that run at once. B sequences of 401 tokens, 8 heads, d 128,
  // blocks of 128 (us at 1 / 2 / 4 planes): 0.3 waves 6.1 / 7.9 / 11.2,
  // 3.3 waves 29.3 / 25.8 / 27.5, 26 waves 199 / 157 / 141.
  const long long waves = tiles * 2 * a.Hkv / (static_cast<long long>(kTeams) * kCtasPerSm * sm_count);
  const int planes = waves < 1 ? 1 : (waves < 8 ? 2 : 4);
  const long long groups = (2LL * a.Hkv + planes - 1) / planes;
  const long long grid = (tiles * kWindows * groups + kTeams - 1) / kTeams;
  if (grid > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  fa_cache_append_kernel<BLOCK, D, BF16><<<static_cast<unsigned>(grid), kThreads, 0, stream>>>(
      a, planes, kWindows);
  return cudaGetLastError();
}

template <int BLOCK>
cudaError_t pick(const CacheAppendArgs& a, int d, bool bf16, int n, cudaStream_t s) {
  if (d == 64) return bf16 ? launch<BLOCK, 64, true>(a, n, s) : launch<BLOCK, 64, false>(a, n, s);
  return bf16 ? launch<BLOCK, 128, true>(a, n, s) : launch<BLOCK, 128, false>(a, n, s);
}

}  // namespace

cudaError_t launch_cache_append(const CacheAppendArgs& a, int block, int d, bool bf16,
                                int sm_count, cudaStream_t stream) {
  switch (block) {
    case 16: return pick<16>(a, d, bf16, sm_count, stream);
    case 32: return pick<32>(a, d, bf16, sm_count, stream);
    case 64: return pick<64>(a, d, bf16, sm_count, stream);
    default: return pick<128>(a, d, bf16, sm_count, stream);
  }
}

}  // namespace fa
