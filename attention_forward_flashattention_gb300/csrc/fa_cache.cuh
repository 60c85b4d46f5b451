// Shared by the block cache's translation units (include/fa_cache.h): the
// arguments of its kernels and their launch functions.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fa_cache.h"

namespace fa {

// Exponent of the smallest scale that fa_cache_append writes: 2^-40 keeps
// values down to 2^-49, far below any 16-bit activation that matters, and the
// ratio of two scales inside fp32's exponent range.
constexpr int kCacheMinScaleExp = -40;

struct CachePlanArgs {
  const int32_t* lens;
  const int32_t* new_lens;
  int32_t* block_table;
  const int32_t* free_blocks;
  const int32_t* free_pos;
  int32_t* slots;
  int32_t* cu_new;
  int32_t* kv_lens;
  int32_t* free_next;
  int table_width, n_free, T, B;
  int block_shift;  // log2 of the block size
};

struct CacheAppendArgs {
  const uint16_t* k;  // new K and V, their token and head strides in elements
  const uint16_t* v;
  long long k_n, k_h, v_n, v_h;
  uint8_t* k_codes;  // the cache
  uint8_t* v_codes;
  float* k_scales;
  float* v_scales;
  const int32_t* slots;
  long long block_stride, head_stride, token_stride;
  int T, Hkv, n_slots;  // n_slots = num_blocks * block
};

// What the join kernel has to do for CTA c: join the partial results of an item
// (16 bytes; what = rows << 16 | parts, 0: nothing).
struct alignas(16) JoinItem {
  int b, hk, rb, what;
};
__host__ __device__ inline JoinItem join_item(int b, int hk, int rb, int rows, int parts) {
  return JoinItem{b, hk, rb, (rows << 16) | parts};
}
__host__ __device__ inline int join_parts(const JoinItem& j) { return j.what & 0xFFFF; }
__host__ __device__ inline int join_rows(const JoinItem& j) { return j.what >> 16; }

// The partial results of a call's launches: the step kernel's (0), the chunk kernel's (1).
struct JoinSides {
  JoinItem* join[2];
  float* parts[2];
  int ctas[2];  // of the launch; 0: nothing to join
  int rows[2];  // of an item
};

struct CacheAttnArgs {
  const void* q;
  void* o;
  float* lse;
  const uint8_t* k;
  const uint8_t* v;
  const float* ks;
  const float* vs;
  const int32_t* table;
  const int32_t* kv_lens;
  const int32_t* cu_q;  // null: n_uniform rows for each sequence
  long long q_b, q_h, q_n, o_b, o_h, o_n;        // element strides (b: uniform only)
  long long block_stride, head_stride, token_stride;
  int B, T, H, Hkv, group, n_uniform, table_width, num_blocks, block_shift;
  int causal;
  float scale_log2;  // scale * log2(e)
  uint32_t* status;
  // sequences of more than rows_over and at most rows_upto rows to a K / V head
  // are this launch's; the others are left alone
  int rows_over, rows_upto;
  int item_rows;   // of a work item of the chunk kernel: 128 or 256
  JoinItem* join;  // [CTAs of the launch]
  float* parts;    // [CTAs of the launch][2] partial results
};

cudaError_t launch_cache_plan(const CachePlanArgs& a, int sm_count, cudaStream_t stream);
cudaError_t launch_cache_append(const CacheAppendArgs& a, int block, int d, bool bf16,
                                int sm_count, cudaStream_t stream);
// False in *mapped: a tensor map could not be encoded.
cudaError_t launch_cache_attn(const CacheAttnArgs& a, const fa_cache& c, bool bf16, int sm_count,
                              float* ws, cudaStream_t stream, bool* mapped);

// fa_host.cu: a cache's K or V as a 4-D byte map {d, token in block, head,
// block}; box = `rows` tokens of one head and block, swizzled over its d bytes
// or row after row.
bool encode_cache(CUtensorMap* m, const void* codes, const fa_cache& c, int rows, bool swizzle);
// Floats of workspace that the attention of T rows of B sequences needs, `group`
// query heads to a K / V head.
long long cache_workspace_floats(int B, int T, int group, int d, int sm_count);

// fa_host.cu: the current device's SM count and status word (allocated on first use).
fa_status device_facts(int* sm_count, uint32_t** status);

// Rows of one sequence in q, o and lse, and its keys.
struct SeqRows {
  int first, count;  // query rows (count may be 0)
  int kv_len;
};

__device__ __forceinline__ SeqRows seq_rows(const CacheAttnArgs& a, int b) {
  SeqRows s;
  if (a.cu_q != nullptr) {
    const int lo = min(max(__ldg(a.cu_q + b), 0), a.T);
    const int hi = min(max(__ldg(a.cu_q + b + 1), 0), a.T);
    s.first = lo;
    s.count = max(hi - lo, 0);
  } else {
    s.first = b * a.n_uniform;
    s.count = a.n_uniform;
  }
  const long long most = static_cast<long long>(a.table_width) << a.block_shift;
  const int len = max(__ldg(a.kv_lens + b), 0);
  s.kv_len = len < most ? len : static_cast<int>(most);
  return s;
}

// Whether a launch computes a sequence.
__device__ __forceinline__ bool takes_seq(const CacheAttnArgs& a, const SeqRows& s) {
  const long long rows = static_cast<long long>(s.count) * a.group;
  return rows > a.rows_over && rows <= a.rows_upto;
}

// Element offsets of query row i of sequence b, head h, in q / o, and its LSE index.
__device__ __forceinline__ long long q_offset(const CacheAttnArgs& a, int b, const SeqRows& s,
                                              int i, int h) {
  return a.cu_q != nullptr ? (s.first + i) * a.q_n + h * a.q_h : b * a.q_b + i * a.q_n + h * a.q_h;
}
__device__ __forceinline__ long long o_offset(const CacheAttnArgs& a, int b, const SeqRows& s,
                                              int i, int h) {
  return a.cu_q != nullptr ? (s.first + i) * a.o_n + h * a.o_h : b * a.o_b + i * a.o_n + h * a.o_h;
}
__device__ __forceinline__ long long lse_index(const CacheAttnArgs& a, int b, const SeqRows& s,
                                               int i, int h) {
  return a.cu_q != nullptr
             ? static_cast<long long>(s.first + i) * a.H + h
             : (static_cast<long long>(b) * a.H + h) * a.n_uniform + i;
}

}  // namespace fa
