/*
 * fa_paged.h -- attention over a paged key/value cache, the cache's writes
 * and reads, rotary positions, trees of drafted tokens, and eviction (same shared
 * library as fa.h).
 *
 * The serving path: fa_rope() turns the new queries and keys, fa_cache_write()
 * puts the new keys and values into the pages of a cache, fa_fwd_paged()
 * attends from the new queries to everything a sequence has in its pages, and
 * fa_cache_read() copies pages back into packed rows (the layout of fa_fwd()
 * and fa_bwd() with cu_seqlens).  For training, fa_rope() with `inverse` is
 * the gradient of fa_rope().
 *
 * Speculative decoding: the new tokens are a tree of drafts, whose masks and
 * depths fa_tree_mask() makes; fa_fwd_paged_tree() attends with them, and
 * fa_cache_keep() moves the accepted ones together.  Eviction: after an attention
 * call (after a tree's, once the accepted tokens lie together), fa_cache_weights() adds the weights that each key got to its sum,
 * fa_cache_select() chooses by the sums which tokens each head keeps, and
 * fa_cache_keep() moves those together.
 *
 * The rules of fa.h hold (BF16 element types, FP32 LSE, contiguous arrays with
 * D innermost, D 64 or 128, 16-byte aligned device pointers, asynchronous on
 * `stream`, nothing allocated).  In addition:
 *   - Pages.  k_pages and v_pages are [num_pages, Hkv, page_size, D]: a page
 *     holds page_size tokens, head by head, so that one head's rows of a page
 *     are one contiguous block.  page_size is a power of two, 16 to 1024.
 *   - block_table, device int32 [B, max_pages]: entry j of row b is the page
 *     with tokens [j * page_size, (j + 1) * page_size) of sequence b.  Entries
 *     behind a sequence's last page are never read.  Sequences may share pages
 *     that are only read.  max_pages * page_size <= 2^30.
 *   - seq_lens, device int32 [B]: how many tokens sequence b has in the cache,
 *     the new ones of this call among them; 0 <= seq_lens[b] <=
 *     max_pages * page_size.
 *   - New tokens.  cu_seqlens == NULL (dense): every sequence has Sn of them,
 *     arrays are [B, Sn, H, D].  Otherwise (packed): arrays are [Sn, H, D],
 *     sequence b owns rows [cu_seqlens[b], cu_seqlens[b + 1]); cu_seqlens is a
 *     device int32 [B + 1] of non-decreasing offsets, cu_seqlens[0] = 0 and
 *     cu_seqlens[B] <= Sn.  Rows from cu_seqlens[B] on are not written, and what
 *     they hold has no effect (kernels may load it).  At most 1024 sequences.
 *   - The n new tokens of a sequence are its last ones: token i of them is at
 *     position seq_lens[b] - n + i.  A token whose position is negative (a
 *     padded entry of a batch: seq_lens[b] < n) is not written to the cache
 *     and, as a query under the causal mask, sees no key.
 *   - Cache types.  Without scales the pages are BF16.  With k_scale and
 *     v_scale, uint8 [num_pages, Hkv, page_size], they are FP8 E4M3: a row (one
 *     token of one head) is D codes and one power of two 2^e, e the smallest
 *     exponent in [-110, 119] with amax <= 448 * 2^e (values that are still
 *     larger saturate), stored as the byte e + 127; each code is the row's
 *     value * 2^-e rounded to nearest even.  What a code stands for is exact
 *     in BF16.  A row that holds a NaN or an infinity gets the byte 255 and
 *     zero codes and stands for NaN.  The two NaN codes, 0x7F and 0xFF, and
 *     bytes outside 17 ... 246 and 255 are made by no write and mean nothing.
 *   - Offsets, lengths and page numbers live on the device, so their rules are
 *     checked there.  Offsets or lengths that break them make fa_fwd_paged(),
 *     fa_fwd_paged_tree() and fa_cache_weights() compute nothing, and the others skip
 *     all rows of the sequences they concern; a page number outside [0, num_pages) that is needed reads
 *     as zeros (a token that would be written to it is skipped).  fa_get_device_error()
 *     reports each as FA_ERR_INVALID_ARG.
 */
#ifndef FA_GB300_FA_PAGED_H
#define FA_GB300_FA_PAGED_H

#include "fa.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Rotary positions with one to four axes, on queries and keys in one launch.
 *   q, k         [tokens, Hq, D] and [tokens, Hkv, D], at most 2^31 - 513
 *                tokens; k may be NULL (Hkv is then ignored)
 *   q_out, k_out where the turned rows go; may be q and k themselves, and
 *                must not overlap them in any other way
 *   positions    device int32 [axes, tokens]; any int32 value
 *   sections     host int [axes]: the number of rotary pairs each axis turns,
 *                every one >= 1; their sum R is at most D / 2.  Pairs are
 *                numbered from 0: axis 0 has the first sections[0] of them,
 *                and so on.  The 2 R leading elements of a row are turned, the
 *                others copied.
 *   base         >= 1, finite.  Pair i turns by
 *                positions[axis of i] * base^(-i / R), with `restart`
 *                base^(-j / sections[axis]), j counting from 0 on each axis.
 *   interleaved  0: pair i is elements i and i + R; 1: elements 2 i, 2 i + 1
 *   inverse      1: turns backwards -- the gradient of the call with 0
 * An angle's error is below 2^-25 turns for positions within 2^27 of zero, and
 * below 2^-22 turns at every int32.
 */
FA_API fa_status fa_rope(const void* q, const void* k, void* q_out, void* k_out, int tokens, int Hq, int Hkv, int D,
                         const int* positions, int axes, const int* sections, double base, int restart,
                         int interleaved, int inverse, fa_stream_t stream);

/*
 * Writes the new keys and values k, v ([B, Sn, Hkv, D] or packed) into the
 * pages.  Slots that no new token goes to keep what they hold.  Two tokens of
 * one call that go to the same slot (sequences sharing the page) race.
 */
FA_API fa_status fa_cache_write(const void* k, const void* v, void* k_pages, void* v_pages, void* k_scale,
                                void* v_scale, int B, int Hkv, int Sn, int D, int num_pages, int page_size,
                                int max_pages, const int* block_table, const int* seq_lens, const int* cu_seqlens,
                                fa_stream_t stream);

/*
 * Reads the first cu_seqlens[b + 1] - cu_seqlens[b] tokens of every sequence
 * into packed BF16 rows k, v [total, Hkv, D], sequence b at rows
 * [cu_seqlens[b], cu_seqlens[b + 1]); exact for both cache types.
 */
FA_API fa_status fa_cache_read(const void* k_pages, const void* v_pages, const void* k_scale, const void* v_scale,
                               void* k, void* v, int B, int Hkv, int total, int D, int num_pages, int page_size,
                               int max_pages, const int* block_table, const int* cu_seqlens, fa_stream_t stream);

/*
 * Bytes of device workspace fa_fwd_paged() needs: the partial results of
 * queries whose keys are split over thread blocks.  It depends on these
 * arguments alone, not on the sequences' lengths.  Returns 0 for arguments
 * fa_fwd_paged() would reject.
 */
FA_API size_t fa_fwd_paged_workspace_size(int B, int Hq, int Hkv, int Sn, int D, int packed, int max_q);

/*
 * Attention of new tokens over the cache: O and LSE as fa_fwd() defines them,
 * the keys of sequence b being its seq_lens[b] tokens in the cache (whose new
 * ones fa_cache_write() has put there).
 *   q, o         [B, Sn, Hq, D] or packed [Sn, Hq, D]
 *   lse          FP32 [B, Hq, Sn] or packed [Hq, Sn]
 *   causal       1: new token i of n sees the keys up to its own position
 *                seq_lens[b] - n + i; 0: all of the sequence's keys
 *   max_q        packed: an upper bound of the new tokens of any one sequence
 *                (a larger count is reported as FA_ERR_INVALID_ARG on the
 *                device); dense: ignored
 *   workspace    device, 256-byte aligned, at least
 *                fa_fwd_paged_workspace_size(...) bytes; contents on entry are
 *                ignored and clobbered.  Calls whose work overlaps on the GPU
 *                need one each.
 *   scale        > 0; scale * log2(e) a normal FP32 number
 * o and lse overlap none of the inputs.  Hq is a multiple of Hkv, Hq / Hkv at
 * most 128, Hkv at most 4096.
 * A row that sees no key gets O = 0 and LSE = -inf, always.  Slots behind a sequence's
 * last token may hold anything (NaN and infinities too).  A NaN or an infinity
 * in a key reaches the rows that see it; one in a value may reach any row of
 * the same sequence and key/value head that sees a key.
 * Roundings, besides O's to BF16 (scores, sums and O are FP32):
 *   - BF16 pages: weights to BF16 (2^-8 of each at most); O is divided by the
 *     sum of the weights as rounded.
 *   - E4M3 pages: the products take FP16.  Queries are exact but for elements
 *     below 2^-30 of their row's largest (off by 2^-38 of it at most), and but
 *     for what moves no score by more than 2^-15.  A score may overflow FP32 on
 *     its way, and come out NaN, where `scale` times a query's largest element
 *     is above 2^100.  Codes
 *     are exact where a row's scale is at least 2^-15 of the largest among the
 *     sequence's keys (values); codes of a row further below may be off by
 *     2^-25 of that largest scale.  A weight times its value's scale is off by
 *     2^-11 of itself, or by 2^-31 of the largest weight times the largest
 *     scale.
 * Results are bitwise repeatable.
 */
FA_API fa_status fa_fwd_paged(const void* q, const void* k_pages, const void* v_pages, const void* k_scale,
                              const void* v_scale, void* o, float* lse, int B, int Hq, int Hkv, int Sn, int D,
                              int num_pages, int page_size, int max_pages, int causal, float scale,
                              const int* block_table, const int* seq_lens, const int* cu_seqlens, int max_q,
                              void* workspace, size_t workspace_bytes, fa_stream_t stream);

/* Most drafted tokens of one sequence. */
#define FA_MAX_TREE 1024

/*
 * Masks and depths of trees of drafted tokens (speculative decoding), dense
 * (cu_seqlens == NULL: B trees of Sn tokens) or packed (Sn rows, offsets and
 * max_q as fa_fwd_paged() has them).  At most FA_MAX_TREE tokens a tree.
 *   parents      device int32 [B, Sn] or [Sn]: the number, in its own tree, of
 *                the token that a token follows, or -1 where it follows the last
 *                token of the cache; smaller than its own number.  A parent that
 *                is not is reported on the device, and counts as -1.
 *   mask         device [B, Sn, W] or [Sn, W], W = ceil(max_q / 32) (dense: of
 *                Sn): bit j % 32 of word j / 32 of token i is set where j is i or
 *                an ancestor of i
 *   depth        device int32 [B, Sn] or [Sn]: how many ancestors a token has; its
 *                position is that of the last token of the cache + 1 + depth
 * Rows from cu_seqlens[B] on, and those of a sequence whose offsets break the
 * rules, are not written.
 */
FA_API fa_status fa_tree_mask(const int* parents, unsigned* mask, int* depth, int B, int Sn, const int* cu_seqlens,
                              int max_q, fa_stream_t stream);

/*
 * fa_fwd_paged() where the new tokens of a sequence are a tree of drafts, whose
 * keys and values fa_cache_write() has put behind the sequence's others, in the
 * tokens' order.  New token i of n sees the seq_lens[b] - n keys before the tree,
 * and new token j of the tree where bit j of its mask is set.  Arguments are those
 * of fa_fwd_paged(), but
 *   tree         device, W words for each new token as fa_tree_mask() lays them
 *                out (any bits will do: a row may be empty; bits from n on mean
 *                nothing), in place of the causal mask
 *   max_q        (dense: Sn) at most FA_MAX_TREE
 * A padded token (its position seq_lens[b] - n + i is negative) sees no key.
 */
FA_API fa_status fa_fwd_paged_tree(const void* q, const void* k_pages, const void* v_pages, const void* k_scale,
                                   const void* v_scale, void* o, float* lse, int B, int Hq, int Hkv, int Sn, int D,
                                   int num_pages, int page_size, int max_pages, const unsigned* tree, float scale,
                                   const int* block_table, const int* seq_lens, const int* cu_seqlens, int max_q,
                                   void* workspace, size_t workspace_bytes, fa_stream_t stream);

/*
 * Sums of the attention weights that the keys of the cache get: for every head h of
 * every sequence b that has new tokens, and each of its tokens t,
 *   sums[t] = decay * sums[t] + sum over rows r that see t of exp(scale * q_r k_t - lse_r)
 * where the rows are the new tokens' query heads of the group, a token's slot in `sums`
 * is that of its key, and a new token's sum starts at zero (so does every sum with
 * decay 0, whatever it holds).  Only a call in which a token is new starts its sum; a
 * token without one has the sum that its slot held before.
 *   Not for a tree of drafts as new tokens: this call knows no tree's mask, and with
 * another one the tree's LSE belongs to other keys.  Once fa_cache_keep() has moved the
 * accepted drafts together, what each saw is what the causal mask gives: call this with
 * their rows of the tree's q and LSE, packed, as the new tokens of sequences
 * start[b] + counts[b] long.
 *   q, causal, scale, block_table, seq_lens, cu_seqlens, max_q, and the pages
 *                as fa_fwd_paged() had them
 *   lse          as fa_fwd_paged() wrote it for the same keys; a row with -inf and
 *                finite queries gives no weight
 *   sums         FP32 [num_pages, Hkv, page_size], laid out like the pages' scales;
 *                slots that are no token's stay as they are
 *   scale        > 0, a normal FP32 number
 *   decay        >= 0, finite
 * Weights and sums are FP32.  Over E4M3 pages, with up to 32 rows of a sequence and
 * head, queries are FP16 as fa_fwd_paged() has them; else keys are BF16, exactly (with a
 * scale below 2^-110 some are off, by what moves no score by 2^-100).  A score may
 * overflow on its way where its size is above 2^18 (over BF16 pages: where the product of
 * query and key does), or, over E4M3 pages with up to 32 rows, where `scale` times a query's
 * largest element is above 2^100.  A token in a bad page gets no sum.  What is not
 * finite in a key reaches that key's own sum alone.  Every token's slot is read and
 * written, so the sequences with new tokens must not share pages.  Results are bitwise
 * repeatable.
 */
FA_API fa_status fa_cache_weights(const void* q, const float* lse, const void* k_pages, const void* k_scale,
                                  float* sums, int B, int Hq, int Hkv, int Sn, int D, int num_pages, int page_size,
                                  int max_pages, int causal, float scale, float decay, const int* block_table,
                                  const int* seq_lens, const int* cu_seqlens, int max_q, fa_stream_t stream);

/*
 * Eviction: which tokens each key/value head keeps of a sequence that is over its
 * budget.  Of the seq_lens[b] tokens of sequence b, kept[b] = min(seq_lens[b],
 * keep) stay: the first `first` and the last `recent` ones, and of the others those
 * with the largest sums.  Of equal sums (-0 and 0 are) the lowest token stays first;
 * a NaN counts as larger than every number.
 *   sums         FP32 [num_pages, Hkv, page_size], laid out like the pages' scales
 *   keep         >= 1, first + recent <= keep <= 2^30
 *   index        device int32 [B, Hkv, keep]: the tokens that stay, in ascending
 *                order; -1 behind the kept[b]-th
 *   kept         device int32 [B]
 * The sum of a token in a bad page reads as zero; a sequence whose length breaks the
 * rules keeps no token.
 */
FA_API fa_status fa_cache_select(const float* sums, int* index, int* kept, int B, int Hkv, int num_pages, int page_size,
                                 int max_pages, int keep, int first, int recent, const int* block_table,
                                 const int* seq_lens, fa_stream_t stream);

/*
 * Moves rows of the cache together, in place: for i < counts[b] token index[b][h][i]
 * of sequence b and head h goes to slot start[b] + i, its key, its value, their
 * scales and its sum alike.  Slots that no token goes to keep what they hold.  After
 * an eviction the sequence is counts[b] tokens long; after drafts were accepted (their
 * tokens' numbers in the sequence in `index`, the number of tokens before the tree in
 * `start`) start[b] + counts[b].
 *   index        device int32 [B, heads, most], heads = Hkv, or 1: the same tokens for
 *                all heads.  The first counts[b] of a list are ascending, none twice,
 *                start[b] or more, and within the block table; a list that is not so is
 *                reported, and nothing of it moves.
 *   counts       device int32 [B], 0 ... most
 *   start        device int32 [B], >= 0, or NULL: 0
 *   sums         as fa_cache_select() has them, or NULL
 * A token whose old or new page is bad is not moved.  No page that a row is written
 * to may be in the table twice.
 */
FA_API fa_status fa_cache_keep(void* k_pages, void* v_pages, void* k_scale, void* v_scale, float* sums, int B, int Hkv,
                               int D, int num_pages, int page_size, int max_pages, const int* block_table,
                               const int* index, int heads, int most, const int* counts, const int* start,
                               fa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FA_GB300_FA_PAGED_H */
