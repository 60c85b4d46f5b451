/*
 * fa_cache.h - C ABI of the 8-bit block cache: attention over keys and values
 * held in e4m3 blocks, and the two calls that fill such a cache.
 *
 * A cache holds K and V of many sequences in blocks of `block` tokens. A
 * block of one head is `block` rows of d e4m3 codes (the 8-bit format of
 * fa_fwd_fp8) with one float32 scale for K and one for V: value = scale *
 * code. A sequence's block table lists its blocks in order, so position j of
 * sequence b is row j % block of block block_table[b][j / block], and its
 * slot is that block's number times `block` plus the row. One step of a
 * serving loop is
 *
 *     fa_cache_plan    block table entries and slots of the step's new tokens
 *     fa_cache_append  their K and V into those slots, in 8 bits
 *     fa_fwd_cache     their attention over everything cached so far
 *
 * Conventions are fa.h's: plain C, device pointers unless said otherwise,
 * asynchronous on `stream`, arguments checked before anything is enqueued,
 * fa_status results. None of these calls allocates device memory but the
 * status word of fa_fwd's first call on a device. Lengths, tables and slots
 * are device memory that the host does not see: values out of range are
 * handled as each call says, and never read or written through.
 */
#ifndef FA_SM103_CACHE_H
#define FA_SM103_CACHE_H

#include "fa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A block cache. Row t of block p of head h starts at
 * k + p * block_stride + h * head_stride + t * token_stride (bytes, which are
 * elements), and the same for v; the d codes of a row are contiguous. */
typedef struct fa_cache {
  void* k;                /* e4m3 codes, 16-byte aligned */
  void* v;
  float* k_scales;        /* [num_blocks][Hkv], contiguous; 2^-60 to 2^120 where fa_fwd_cache
                             reads them (outside: 1 / v_scale and sums of it leave fp32's range) */
  float* v_scales;
  int num_blocks;         /* >= 1, times block and times Hkv at most 2^31 - 1 */
  int block;              /* tokens in a block: 16, 32, 64 or 128 */
  int Hkv;                /* K / V heads */
  int d;                  /* head dimension, 64 or 128 */
  long long block_stride; /* each a positive multiple of 16, below 2^38; */
  long long head_stride;  /* rows must not overlap (not checked) */
  long long token_stride;
} fa_cache;

/*
 * fa_cache_plan - block table entries and slots of new tokens, from the
 * requests' lengths.
 *
 * lens        : [B] int32, tokens of each request cached so far.
 * new_lens    : [B] int32, tokens to append to each (>= 0).
 * block_table : [B][table_width] int32, in and out: row b lists the
 *               ceil(lens[b] / block) blocks of request b; the entries of the
 *               blocks that its new tokens open are written behind them. No
 *               other entry is written.
 * free_blocks : [n_free] int32, ids of free blocks; those from index
 *               free_pos[0] on are handed out in order, request by request.
 * free_pos    : [1] int32.
 * slots       : [T] int32, written: the slots of the new tokens, request by
 *               request, and -1 behind the last one (T may be larger than the
 *               sum of new_lens).
 * cu_new      : [B + 1] int32, written: row of each request's first new token,
 *               and the number of new tokens (at most T each).
 * kv_lens     : [B] int32, written: lens + new_lens.
 * free_next   : [1] int32, written: free_pos of the next call.
 * block       : tokens in a block: 16, 32, 64 or 128.
 *
 * A request is refused if its length or number of new tokens is negative, if
 * its table row is too short, if its rows do not all fit into T, or if the
 * free blocks run out (the first request that they do not suffice for and
 * every later one that needs a block). Its slots are -1, its kv_lens is its
 * length (0 for a negative one), and it gets no block; its rows keep their
 * place in cu_new. So kv_lens == lens tells a refusal of a request with new
 * tokens. A block id of the table is taken as it is (a negative one gives
 * slot -1).
 * Every written array must differ from every read one but block_table.
 * Pointers 4-byte aligned; 1 <= B <= 2^20, 0 <= T <= 2^30, table_width >= 1,
 * n_free >= 0. Deterministic; one launch.
 */
fa_status fa_cache_plan(const int32_t* lens, const int32_t* new_lens, int32_t* block_table,
                        int table_width, const int32_t* free_blocks, int n_free,
                        const int32_t* free_pos, int32_t* slots, int T, int32_t* cu_new,
                        int32_t* kv_lens, int32_t* free_next, int B, int block, void* stream);

/*
 * fa_cache_append - K and V of new tokens into the cache, in 8 bits.
 *
 * k, v    : [T][Hkv][d] of `dtype`, read only, 16-byte aligned; strides: host
 *           pointer to two fa_strides, of k and v: n is the token stride and h
 *           the head stride in elements (multiples of 8; b is not used).
 * slots   : [T] int32 (fa_cache_plan's). A token whose slot is not in
 *           [0, num_blocks * block) is skipped. The new tokens of one block
 *           must be consecutive tokens with consecutive slots, as the plan
 *           gives them: a block met twice in one call, or a slot twice, leaves
 *           that block's contents undefined (nothing else).
 * cache   : host pointer to the cache's description, read during the call.
 *
 * Scales: with amax the largest finite |value| of a block and head among the
 * new tokens, the scale becomes the smallest power of two s >= 2^-40 with
 * amax <= 448 s, or the block's present scale (rounded up to a power of two)
 * if that is larger and the block holds older tokens; a block whose row 0 is
 * among the new tokens starts afresh. (A present scale that is not above 0 is
 * taken as none.) Codes are value / s rounded to nearest
 * even; if s grew, the codes of the block's older rows (those before the first
 * new one) are brought to it, code * old / s, rounded again. With powers of
 * two that is exact, and loses bits only where a code becomes subnormal.
 * Infinities and NaN are stored as NaN.
 * T >= 0 (0: nothing is enqueued). Deterministic; one launch.
 */
fa_status fa_cache_append(const void* k, const void* v, const fa_strides* strides,
                          const int32_t* slots, int T, const fa_cache* cache, fa_dtype dtype,
                          void* stream);

/*
 * fa_fwd_cache - attention of each sequence's last tokens over the cache.
 *
 *     O[t,h,:] = sum_j softmax_j(scale * q_t . k_j) v_j,  LSE[t,h] = ln sum_j exp(scale * q_t . k_j)
 *
 * over the keys j < kv_lens[b] of t's sequence b; if causal, query i of the
 * n query tokens of b sees the keys j <= kv_lens[b] - n + i: the queries are
 * the sequence's last tokens. A row that sees no key gets O = 0 and LSE =
 * -inf. Query head h reads K / V head h / (H / Hkv).
 *
 * q, o        : q read, o written (16-byte aligned, `dtype`). With cu_q: rows
 *               [T][H][d], sequence b's queries are rows cu_q[b] ..
 *               cu_q[b + 1] - 1 (clamped to 0 .. T). cu_q NULL: [B][n][H][d]
 *               rows, n = T / B queries for every sequence (T a multiple of
 *               B). strides: host pointer to two fa_strides, of q and o, in
 *               elements, multiples of 8 (b is read only if cu_q is NULL).
 * lse         : float32, written: [T][H] contiguous with cu_q, [B][H][n]
 *               without.
 * cache       : as in fa_cache_append; its k, v and scales are read only.
 * block_table : [B][table_width] int32. Entries out of [0, num_blocks) hide
 *               their keys: they weigh nothing.
 * kv_lens     : [B] int32; taken as within 0 .. table_width * block.
 * B, T, H     : sequences, query rows, query heads (a multiple of Hkv), >= 1
 *               (T >= 0; 0: nothing is enqueued). B <= 2^20, T * H <= 2^31 - 1,
 *               table_width * block <= 2^30.
 * Rows of o and lse that belong to no sequence are left as they are. Keys at
 * and behind kv_lens[b], and those that the causal rule hides, do not reach a
 * row, whatever their codes: NaN neither.
 * workspace   : device scratch of fa_fwd_cache_workspace_size bytes, 16-byte
 *               aligned; overwritten, and not to be used by another call at
 *               the same time. Nothing is kept in it between calls.
 * Scores, softmax sums and O are formed in fp32 from the exact products of
 * 16-bit queries and 8-bit codes. For the product with V, whatever `dtype` is,
 * the weights w_j = exp(score) times V's scale are rounded to fp16's 11 bits: by
 * at most 2^-11 of themselves, or by 2^-33 W where they are below 2^-22 W, W the
 * largest of them in the row. (So a column of O that lives on keys far below the
 * row's largest, or on blocks of a far smaller V scale, is off by up to 2^-33 W
 * sum |code| / sum w.) For FA_DTYPE_FP16 and up to 16 rows to a K / V head they
 * are kept in two such parts: 2^-22 of themselves, or 2^-33 W. With d = 128
 * and 17 to 128 rows to a K / V head (on average over the sequences) query
 * elements below 2^-6 of their row's largest (bf16: 2^-9) may be rounded, by
 * 2^-17 of that largest one at most. Where scale * max |q| of a row is below
 * 2^-64, its scores may be off by up to 2^-48 of the K scale. A query row that
 * holds an infinity or NaN gives NaN if it sees a key. V scales of one sequence
 * may differ by a factor of up to 2^100; the logarithm of one is off by at most
 * 2^-22 of itself (or 2^-22), and the weights of its block in proportion.
 * Up to three launches (a kernel for sequences of up to 16 rows to a K / V
 * head, one for more, and one that joins what they split), by the sizes that
 * the host knows: with cu_q it does not know how the rows are spread. Where all
 * sequences have the same number of query tokens, the call without cu_q spares a
 * launch (16 x 5 tokens: 60 us in place of 70). A batch with cu_q and T <= B is
 * taken for one of single tokens; a long piece in it is computed right, but at a
 * third of its speed. Deterministic: the same call gives the same bits.
 */
fa_status fa_fwd_cache(const void* q, const fa_cache* cache, const int32_t* block_table,
                       int table_width, const int32_t* kv_lens, const int32_t* cu_q, void* o,
                       float* lse, int B, int T, int H, const fa_strides* strides, int causal,
                       float scale, fa_dtype dtype, void* workspace, size_t workspace_size,
                       void* stream);

/*
 * fa_fwd_cache_workspace_size - bytes of the workspace fa_fwd_cache needs for
 * these sizes on the current device. Host only.
 */
fa_status fa_fwd_cache_workspace_size(int B, int T, int H, int Hkv, int d, size_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* FA_SM103_CACHE_H */
