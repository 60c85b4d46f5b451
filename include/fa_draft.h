/*
 * fa_draft.h - C ABI of attention for trees of drafted tokens over the 8-bit
 * block cache (fa_cache.h).
 *
 * A request's drafted tokens form a tree: each follows another one of them, its
 * parent, or the request's context. Their K and V are appended to the cache
 * like any others, behind the context, in an order in which parents come
 * first; what tells the branches apart is which of them a token sees: itself
 * and its ancestors, beside the whole context. That set is a bit mask of
 * 64-bit words: bit c % 64 of word c / 64 is the request's c-th drafted token.
 * One step of a serving loop is
 *
 *     fa_cache_plan      slots of the drafted tokens
 *     fa_cache_tree      their masks and positions, from their parents
 *     fa_cache_append    their K and V
 *     fa_fwd_cache_tree  their attention
 *
 * Conventions are fa_cache.h's.
 */
#ifndef FA_SM103_DRAFT_H
#define FA_SM103_DRAFT_H

#include "fa_cache.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * fa_cache_tree - which drafted tokens each one sees, and its position.
 *
 * parents   : [T] int32: each token's parent among its request's drafted tokens (0 is
 *             the first one). One that is not an earlier token (below 0, or not
 *             below the token's own number) is none: the token follows the context.
 * cu        : [B + 1] int32, rows of each request's tokens (fa_cache_plan's cu_new;
 *             clamped to 0 .. T).
 * lens      : [B] int32, tokens of each request's context (below 0: taken as 0).
 * masks     : [T][words] uint64, written: itself and its ancestors. Tokens from
 *             64 * words on have no bit, and no ancestors: their masks are empty.
 * positions : [T] int32, written: lens plus the number of its ancestors.
 * Rows that belong to no request are left as they are.
 * Pointers 4-byte (masks 8-byte) aligned; 1 <= B <= 2^20, T >= 0 (0: nothing is
 * enqueued), 1 <= words <= 16, T * words <= 2^31 - 1. Deterministic; one launch.
 */
fa_status fa_cache_tree(const int32_t* parents, const int32_t* cu, const int32_t* lens,
                        uint64_t* masks, int32_t* positions, int B, int T, int words, void* stream);

/*
 * fa_fwd_cache_tree - fa_fwd_cache for drafted tokens of a tree.
 *
 * Everything is as there but which keys a row sees: with n the number of a
 * sequence's query tokens, query i sees the keys j < kv_lens[b] - n and those
 * keys kv_lens[b] - n + c, 0 <= c < n, whose bit c is set in the mask of query
 * i; c >= 64 * words is not seen. (A chain's masks give fa_fwd_cache's causal
 * results.) A row that sees no key gets O = 0 and LSE = -inf. Keys that a row
 * does not see do not reach it, whatever their codes.
 *
 * masks : [T][words] uint64, 8-byte aligned: the mask of query row t (without cu_q:
 *         of query i of sequence b in row b * n + i). They need not be those of a
 *         tree: any set is allowed, the token's own bit is like any other.
 * words : 1 .. 16; T * words <= 2^31 - 1.
 * workspace : of fa_fwd_cache_workspace_size bytes, as there.
 *
 * Roundings are fa_fwd_cache's, but for which sequences are taken for large: a call
 * with cu_q and more than 16 rows to a K / V head on average (T * H / Hkv over B, rows
 * of no sequence included) computes all of its sequences as those of more rows,
 * however many rows each has. So with
 * FA_DTYPE_FP16 the weights of a small sequence in such a call are one fp16 value (2^-11
 * of themselves, not 2^-22), and with d = 128 its small query elements may be rounded (by
 * 2^-17 of their row's largest): the last bits of its results depend on the
 * sequences beside it. Launches: one kernel for such a call, and one that joins; otherwise as there.
 */
fa_status fa_fwd_cache_tree(const void* q, const fa_cache* cache, const int32_t* block_table,
                            int table_width, const int32_t* kv_lens, const int32_t* cu_q,
                            const uint64_t* masks, int words, void* o, float* lse, int B, int T,
                            int H, const fa_strides* strides, float scale, fa_dtype dtype,
                            void* workspace, size_t workspace_size, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FA_SM103_DRAFT_H */
