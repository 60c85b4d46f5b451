/*
 * fa_pages.h - C ABI of the 8-bit block cache's upkeep (fa_cache.h): dropping
 * drafted tokens that were not accepted, handing blocks back, sharing them
 * between requests.
 *
 *     fa_cache_keep     the kept ones of a request's last tokens together (each layer's cache)
 *     fa_cache_release  blocks behind a request's new length, to the free list (once)
 *     fa_cache_fork     table rows of requests that go on from others' tokens (once)
 *     fa_cache_copy     contents of the blocks that they do not share (each layer's cache)
 *
 * Blocks that several requests hold are counted in shares [num_blocks]: the
 * number of holders beside the first one. Blocks that fa_cache_plan hands out
 * have one holder, so an array of zeros is where a program starts, and
 * fa_cache_release leaves 0 where it hands a block back.
 *
 * Tokens are appended to a request's last block, if that is not full, and to those
 * behind it, and fa_cache_fork does not share a last block that is not full. So a
 * shared block is not written while requests only grow. A request must not be
 * shortened to a length inside a block that it shares and then grow again: what it
 * appends, and a scale that grows, would change the other holders' tokens, and no
 * call notices. Hence:
 *   - drafted tokens that are not kept are dropped before a request is forked;
 *   - a request that goes back to an earlier token of its own goes on as a fork of
 *     itself: fa_cache_fork with the shorter length (the block that it then ends in is
 *     copied by fa_cache_copy), then fa_cache_release of its whole old row
 *     (new_lens 0).
 *
 * Conventions are fa_cache.h's.
 */
#ifndef FA_SM103_PAGES_H
#define FA_SM103_PAGES_H

#include "fa_cache.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * fa_cache_keep - some of each sequence's last tokens, moved together.
 *
 * block_table : [B][table_width] int32, read only.
 * kv_lens     : [B] int32, tokens of each sequence, the last ones included.
 * cu          : [B + 1] int32: sequence b's last n = cu[b + 1] - cu[b] tokens are at
 *               stake (fa_cache_plan's cu_new).
 * keep        : [B][words] uint64: bit c % 64 of word c / 64 says that the c-th of them
 *               stays (fa_cache_tree's mask of an accepted token, for its path). Bits
 *               from n on say nothing; tokens from 64 * words on do not stay.
 * lens_out    : [B] int32, written: the lengths after. The kept tokens come in their order
 *               behind the kv_lens - n tokens before them; the rows behind lens_out
 *               hold what they happen to hold.
 * A sequence is left alone, with lens_out = kv_lens, unless 0 <= n <= kv_lens <=
 * table_width * block and the table lists existing blocks for its last n tokens.
 * Those blocks must be the sequence's own: no other one's, and none listed twice.
 *
 * Scales: a block into which a token moves takes the largest scale of the blocks that
 * its tokens come from, its own among them if it holds tokens before the last n
 * (or one of them that stays where it is); each rounded up to a power of two, one that
 * is not above 0 counting for nothing (none at all: 2^-40). Codes are brought to
 * it, code * (old / new) in fp32, rounded to nearest even: with powers of two that is
 * exact, but where a code becomes subnormal. Blocks whose tokens all stay where they are
 * are not touched.
 * lens_out must differ from the read arrays. Pointers 4-byte (keep 8-byte)
 * aligned; 1 <= B <= 2^20, 1 <= words <= 16, table_width >= 1, table_width *
 * block <= 2^30. Deterministic; one launch.
 */
fa_status fa_cache_keep(const fa_cache* cache, const int32_t* block_table, int table_width,
                        const int32_t* kv_lens, const int32_t* cu, const uint64_t* keep, int words,
                        int32_t* lens_out, int B, void* stream);

/*
 * fa_cache_release - blocks that requests do not need any more, to the free list.
 *
 * block_table : [B][table_width] int32, read only. Request b gives up the entries from
 *               ceil(new_lens[b] / block) on to ceil(lens[b] / block) - 1; they
 *               stay in the table as they are.
 * lens, new_lens : [B] int32: tokens held, and kept (0: all blocks go back). A request
 *               without 0 <= new_lens <= lens <= table_width * block gives up nothing.
 *               (One that keeps a part of a block that it shares must not grow: see above.)
 * shares      : [num_blocks] int32, in and out, or NULL: blocks have one holder. A block
 *               goes to the free list when its last holder gives it up; before that
 *               its count falls. (Given up more often than it has holders, it goes
 *               there once.)
 * num_blocks  : with shares: entries out of [0, num_blocks) are passed over. Without,
 *               those below 0 are, and num_blocks is not read.
 * free_blocks : [n_free] int32, in and out: the ids go in front of free_pos[0], from
 *               free_pos[0] - 1 downwards, in the order of the requests and of
 *               their entries. Ids that find no place there (more of them than were
 *               handed out) are dropped.
 * free_pos    : [1] int32, in 0 .. n_free; otherwise nothing is done.
 * free_next   : [1] int32, written: free_pos of the next call.
 * Written arrays must differ from each other and from read ones. Pointers 4-byte aligned;
 * 1 <= B <= 2^20, table_width >= 1, B * table_width <= 2^30, n_free >= 0.
 * Deterministic; one launch.
 */
fa_status fa_cache_release(const int32_t* block_table, int table_width, const int32_t* lens,
                           const int32_t* new_lens, int32_t* shares, int num_blocks,
                           int32_t* free_blocks, int n_free, const int32_t* free_pos,
                           int32_t* free_next, int B, int block, void* stream);

/*
 * fa_cache_fork - requests that go on from other requests' tokens.
 *
 * block_table : [B][table_width] int32 and lens [B] int32, the present requests'. (Lengths
 *               may be shorter than what requests hold: the new ones start from those.)
 * src         : [n] int32: new request k starts as a copy of request src[k] (any number
 *               of them from the same one).
 * shares      : [num_blocks] int32, in and out: counts of the full blocks that are now
 *               shared go up. (Entries out of [0, num_blocks) are copied and not counted.)
 * free_blocks, n_free, free_pos : the free list, read only: fa_cache_plan's.
 * new_table   : [n][table_width] int32, written: the source's full blocks, a free block
 *               in place of a last one that is not full, -1 behind them. May be
 *               other rows of block_table's own array, but none that is read.
 * new_lens    : [n] int32, written: the source's length.
 * copies      : [n][3] int32, written, for fa_cache_copy: block to copy from, block to
 *               copy to, rows; -1, -1, 0 where there is nothing to copy.
 * free_next   : [1] int32, written: free_pos of the next call.
 * A new request is refused if src[k] is not in [0, B), the source's length is below 0 or
 * beyond its table row, or the free blocks run out (the first that they do not
 * suffice for and every later one that needs one): it has length 0 and a row of -1.
 * A last block that is not full and that does not exist is copied as an entry, and
 * needs no free one.
 * Written arrays must differ from each other and from read ones (but as said).
 * Pointers 4-byte aligned; 1 <= B, n <= 2^20, table_width >= 1, table_width * block <=
 * 2^30, n_free >= 0, num_blocks >= 1. Deterministic; one launch.
 */
fa_status fa_cache_fork(const int32_t* block_table, int table_width, const int32_t* lens, int B,
                        const int32_t* src, int n, int32_t* shares, int num_blocks,
                        const int32_t* free_blocks, int n_free, const int32_t* free_pos,
                        int32_t* new_table, int32_t* new_lens, int32_t* copies, int32_t* free_next,
                        int block, void* stream);

/*
 * fa_cache_copy - rows of blocks into other blocks, with the blocks' scales.
 *
 * copies : [n][3] int32: from, to, rows. The first `rows` rows (at most a block) of K and
 *          V of all heads, and the scales, of block `from` go to block `to`. Entries with
 *          a block out of [0, num_blocks), from = to or rows <= 0 are passed over.
 * A block must not be copied to twice in one call, nor from and to.
 * 4-byte aligned; 0 <= n <= 2^20 (0: nothing is enqueued). One launch.
 */
fa_status fa_cache_copy(const fa_cache* cache, const int32_t* copies, int n, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FA_SM103_PAGES_H */
