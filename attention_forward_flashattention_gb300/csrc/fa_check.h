// Argument checks that several entry points share (host code).
#pragma once

#include <cstdint>

#include "fa_cache.h"

namespace fa {

// Words of a mask over drafted tokens, at most.
constexpr int kMaxWords = 16;

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

inline int block_shift(int block) {
  switch (block) {
    case 16: return 4;
    case 32: return 5;
    case 64: return 6;
    case 128: return 7;
  }
  return -1;
}

inline fa_status check_cache(const fa_cache* c) {
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
inline fa_status check_stride(long long s) {
  if (s <= 0 || (s & 7) != 0) return FA_ERR_INVALID_ARG;
  return s >= (1LL << 38) ? FA_ERR_UNSUPPORTED : FA_OK;
}

}  // namespace fa
