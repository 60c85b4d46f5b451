// C ABI of the block cache (include/fa_cache.h): argument checks and launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "fa_cache.cuh"

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int block_shift(int block) {
  switch (block) {
    case 16: return 4;
    case 32: return 5;
    case 64: return 6;
    case 128: return 7;
  }
  return -1;
}

fa_status check_cache(const fa_cache* c) {
  if (!c || !c->k || !c->v || !c->k_scales || !c->v_scales) return FA_ERR_INVALID_ARG;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scales, 4) ||
      !aligned(c->v_scales, 4))
    return FA_ERR_INVALID_ARG;
  if (c->num_blocks <= 0 || c->Hkv <= 0) return FA_ERR_INVALID_ARG;
  for (const long long s : {c->block_stride, c->head_stride, c->token_stride})
    if (s <= 0 || (s & 15) != 0) return FA_ERR_INVALID_ARG;
  if (c->d != 64 && c->d != 128) return FA_ERR_UNSUPPORTED;
  if (c->token_stride < c->d) return FA_ERR_INVALID_ARG;
  if (block_shift(c->block) < 0) return FA_ERR_UNSUPPORTED;
  for (const long long s : {c->block_stride, c->head_stride, c->token_stride})
    if (s >= (1LL << 38)) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(c->num_blocks) * c->block > 0x7FFFFFFFLL || c->Hkv > 32767 ||
      static_cast<long long>(c->num_blocks) * c->Hkv > 0x7FFFFFFFLL)
    return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// Strides of a 16-bit operand: positive multiples of 8 elements below 2^38.
fa_status check_stride(long long s) {
  if (s <= 0 || (s & 7) != 0) return FA_ERR_INVALID_ARG;
  return s >= (1LL << 38) ? FA_ERR_UNSUPPORTED : FA_OK;
}

fa_status done(cudaError_t e) { return e == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

}  // namespace

extern "C" {

fa_status fa_cache_plan(const int32_t* lens, const int32_t* new_lens, int32_t* block_table,
                        int table_width, const int32_t* free_blocks, int n_free,
                        const int32_t* free_pos, int32_t* slots, int T, int32_t* cu_new,
                        int32_t* kv_lens, int32_t* free_next, int B, int block, void* stream) {
  if (!lens || !new_lens || !block_table || !free_pos || !cu_new || !kv_lens || !free_next)
    return FA_ERR_INVALID_ARG;
  if (B <= 0 || T < 0 || table_width <= 0 || n_free < 0) return FA_ERR_INVALID_ARG;
  if ((T > 0 && !slots) || (n_free > 0 && !free_blocks)) return FA_ERR_INVALID_ARG;
  // (an empty array has no address of its own)
  const void* in[4] = {lens, new_lens, n_free > 0 ? free_blocks : nullptr, free_pos};
  const void* out[5] = {block_table, T > 0 ? slots : nullptr, cu_new, kv_lens, free_next};
  for (int i = 0; i < 5; ++i) {
    if (!aligned(out[i], 4) || (i < 4 && !aligned(in[i], 4))) return FA_ERR_INVALID_ARG;
    if (!out[i]) continue;
    for (const void* p : in)
      if (p == out[i]) return FA_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (out[j] == out[i]) return FA_ERR_INVALID_ARG;
  }
  const int shift = block_shift(block);
  if (shift < 0 || B > (1 << 20) || T > (1 << 30)) return FA_ERR_UNSUPPORTED;
  int sms = 0;
  const fa_status ds = fa::device_facts(&sms, nullptr);
  if (ds != FA_OK) return ds;
  fa::CachePlanArgs a{};
  a.lens = lens;
  a.new_lens = new_lens;
  a.block_table = block_table;
  a.free_blocks = free_blocks;
  a.free_pos = free_pos;
  a.slots = slots;
  a.cu_new = cu_new;
  a.kv_lens = kv_lens;
  a.free_next = free_next;
  a.table_width = table_width;
  a.n_free = n_free;
  a.T = T;
  a.B = B;
  a.block_shift = shift;
  (void)cudaGetLastError();
  return done(fa::launch_cache_plan(a, sms, static_cast<cudaStream_t>(stream)));
}

fa_status fa_cache_append(const void* k, const void* v, const fa_strides* strides,
                          const int32_t* slots, int T, const fa_cache* cache, fa_dtype dtype,
                          void* stream) {
  const fa_status cs = check_cache(cache);
  if (cs == FA_ERR_INVALID_ARG) return cs;
  if (!k || !v || !strides || !slots || T < 0) return FA_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 4)) return FA_ERR_INVALID_ARG;
  if (dtype != FA_DTYPE_FP16 && dtype != FA_DTYPE_BF16) return FA_ERR_INVALID_ARG;
  if (cs != FA_OK) return cs;
  for (int i = 0; i < 2; ++i)
    for (const long long s : {strides[i].n, strides[i].h}) {
      const fa_status ss = check_stride(s);
      if (ss != FA_OK) return ss;
    }
  if (T > (1 << 30)) return FA_ERR_UNSUPPORTED;
  int sms = 0;
  const fa_status ds = fa::device_facts(&sms, nullptr);
  if (ds != FA_OK) return ds;
  if (T == 0) return FA_OK;
  fa::CacheAppendArgs a{};
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.k_n = strides[0].n;
  a.k_h = strides[0].h;
  a.v_n = strides[1].n;
  a.v_h = strides[1].h;
  a.k_codes = static_cast<uint8_t*>(cache->k);
  a.v_codes = static_cast<uint8_t*>(cache->v);
  a.k_scales = cache->k_scales;
  a.v_scales = cache->v_scales;
  a.slots = slots;
  a.block_stride = cache->block_stride;
  a.head_stride = cache->head_stride;
  a.token_stride = cache->token_stride;
  a.T = T;
  a.Hkv = cache->Hkv;
  a.n_slots = cache->num_blocks * cache->block;
  (void)cudaGetLastError();
  return done(fa::launch_cache_append(a, cache->block, cache->d, dtype == FA_DTYPE_BF16, sms,
                                      static_cast<cudaStream_t>(stream)));
}

fa_status fa_fwd_cache_workspace_size(int B, int T, int H, int Hkv, int d, size_t* bytes) {
  if (!bytes || B <= 0 || T < 0 || H <= 0 || Hkv <= 0 || H % Hkv != 0) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  int sms = 0;
  const fa_status ds = fa::device_facts(&sms, nullptr);
  if (ds != FA_OK) return ds;
  *bytes = static_cast<size_t>(fa::cache_workspace_floats(B, T, H / Hkv, d, sms)) * sizeof(float);
  return FA_OK;
}

fa_status fa_fwd_cache(const void* q, const fa_cache* cache, const int32_t* block_table,
                       int table_width, const int32_t* kv_lens, const int32_t* cu_q, void* o,
                       float* lse, int B, int T, int H, const fa_strides* strides, int causal,
                       float scale, fa_dtype dtype, void* workspace, size_t workspace_size,
                       void* stream) {
  const fa_status cs = check_cache(cache);
  if (cs == FA_ERR_INVALID_ARG) return cs;
  if (!q || !block_table || !kv_lens || !o || !lse || !strides || !workspace)
    return FA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(workspace, 16) || !aligned(lse, 4) ||
      !aligned(block_table, 4) || !aligned(kv_lens, 4) || !aligned(cu_q, 4))
    return FA_ERR_INVALID_ARG;
  if (!(std::isfinite(scale) && scale > 0.f)) return FA_ERR_INVALID_ARG;
  if (dtype != FA_DTYPE_FP16 && dtype != FA_DTYPE_BF16) return FA_ERR_INVALID_ARG;
  if (B <= 0 || T < 0 || H <= 0 || table_width <= 0 || H % cache->Hkv != 0)
    return FA_ERR_INVALID_ARG;
  if (!cu_q && T % B != 0) return FA_ERR_INVALID_ARG;
  if (cs != FA_OK) return cs;
  for (int i = 0; i < 2; ++i) {
    for (const long long s : {strides[i].n, strides[i].h, cu_q ? 8LL : strides[i].b}) {
      const fa_status ss = check_stride(s);
      if (ss != FA_OK) return ss;
    }
  }
  if (static_cast<long long>(T) * H > 0x7FFFFFFFLL || B > (1 << 20) ||
      static_cast<long long>(table_width) * cache->block > (1LL << 30))
    return FA_ERR_UNSUPPORTED;
  size_t need = 0;
  const fa_status ws = fa_fwd_cache_workspace_size(B, T, H, cache->Hkv, cache->d, &need);
  if (ws != FA_OK) return ws;
  if (workspace_size < need) return FA_ERR_INVALID_ARG;
  int sms = 0;
  fa::CacheAttnArgs a{};
  const fa_status ds = fa::device_facts(&sms, &a.status);
  if (ds != FA_OK) return ds;
  if (T == 0) return FA_OK;
  a.q = q;
  a.o = o;
  a.lse = lse;
  a.k = static_cast<const uint8_t*>(cache->k);
  a.v = static_cast<const uint8_t*>(cache->v);
  a.ks = cache->k_scales;
  a.vs = cache->v_scales;
  a.table = block_table;
  a.kv_lens = kv_lens;
  a.cu_q = cu_q;
  a.q_b = strides[0].b;
  a.q_h = strides[0].h;
  a.q_n = strides[0].n;
  a.o_b = strides[1].b;
  a.o_h = strides[1].h;
  a.o_n = strides[1].n;
  a.block_stride = cache->block_stride;
  a.head_stride = cache->head_stride;
  a.token_stride = cache->token_stride;
  a.B = B;
  a.T = T;
  a.H = H;
  a.Hkv = cache->Hkv;
  a.group = H / cache->Hkv;
  a.n_uniform = cu_q ? 0 : T / B;
  a.table_width = table_width;
  a.num_blocks = cache->num_blocks;
  a.block_shift = block_shift(cache->block);
  a.causal = causal != 0;
  a.scale_log2 = scale * 1.4426950408889634f;
  (void)cudaGetLastError();
  bool mapped = true;
  const cudaError_t e = fa::launch_cache_attn(a, *cache, dtype == FA_DTYPE_BF16, sms,
                                              static_cast<float*>(workspace),
                                              static_cast<cudaStream_t>(stream), &mapped);
  return mapped ? done(e) : FA_ERR_CUDA;
}

}  // extern "C"
