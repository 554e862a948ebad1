/*
 * tp_search.h -- C ABI of libring_collectives.so, third part: beam search over
 * a paged key/value cache, and the cache in 4 bits.  One step of a search:
 *
 *   all_gather_gemm          x_shard, Wvocab  -> logits, split over the ranks by columns
 *   beam_select              logits, scores   -> parents, tokens, scores
 *   kv_fork, kv_copy_pages   parents          -> block table, shared lengths; pages copied and freed
 *   kv_plan                  (tp_attention.h)    slots of the new tokens
 *   tp_kv4_write             k, v, slots      -> 4-bit cache rows
 *   tp_attention_decode_kv4  q, cache         -> o
 *
 * kv_fork, kv_compact and kv_copy_pages serve any paged cache, the bf16 one of
 * tp_attention.h too.  Sampling, and other ways to end a request, need no
 * selection: their parents are the rows that go on.
 *
 * Conventions are those of tp_attention.h (error codes, streams, alignment,
 * arrays of P pointers, nothing allocated, no memset recorded, nothing that
 * device memory holds trusted).  In ws, besides:
 *   - kv_fork and kv_compact need their counters in ws zero and leave them
 *     zero; where another call left data there, they stop with RING_EWORKSPACE
 *     in the workspace's error word (ring_last_error) and undefined outputs
 *     (with few rows and pages they use no counters, and do not).  The calls of
 *     this header that leave data record where.
 */
#ifndef TP_SEARCH_H
#define TP_SEARCH_H

#include "tp_attention.h"

#ifdef __cplusplus
extern "C" {
#endif

#define BEAM_SELECT_MAX 64
#define KV_FORK_MAX_ROWS 8192

/*
 * The `keep` best continuations of each of N groups of `beams` rows.  logits[r]
 * (RING_F32 or RING_BF16): N * beams rows, `stride` elements apart, of `width`
 * columns: column c is token r * width + c, and tokens from `vocab` on (a
 * padded vocabulary) take no part, nor do logits that are not finite.  With
 *     lp(row, t) = logit - log sum exp(logits of the row)
 * the candidates of group n are scores[n][w] + lp(n * beams + w, t) over all w
 * and t; with done != NULL, a beam with done[n][w] != 0 has the one candidate
 * (w, end_token) of score scores[n][w] instead.  Written, best first, of equal
 * scores the lowest w, then the largest logit (scores[n][w] may be so large
 * that logits that differ give one score), then the lowest t:
 *   parents       [N][keep] the candidate's row, n * beams + w
 *   tokens        [N][keep] its t
 *   scores_after  [N][keep] its score
 *   done_after    [N][keep] whether it was done or t is end_token (0 or 1)
 * Beams whose score is not finite have no candidates.  Places that no candidate
 * is left for hold parent -1, token -1, score -inf and done 0.
 * Scores are compared in 64 bits, and rounded once to fp32.  log sum exp is a
 * 64-bit sum of fp32 exponentials, 16 at a time added in fp32: some 1e-8 off,
 * up to 2e-7 where one token has most of the weight, whatever the row's width.
 * done and done_after go together; end_token may be -1 (none) without them.
 * beams and keep are 1 .. BEAM_SELECT_MAX; outputs may not overlap inputs (over
 * scores or done: RING_EINVAL).
 */
int beam_select(const void *const *logits, const float *scores, const unsigned char *done, int *parents, int *tokens,
                float *scores_after, unsigned char *done_after, int P, int N, int beams, int keep, int width, int vocab,
                long long stride, int end_token, int dtype, void *ws, size_t ws_bytes, void *stream);
size_t beam_select_workspace_bytes(int P, int N, int beams, int keep, int width);

/*
 * The block table of rows that go on: row i of the new table (B_after rows) is
 * row parents[i] of the old one (B rows of table_stride pages, lengths[b]
 * tokens), with its first keep[i] tokens only where keep != NULL.  A parent
 * outside [0, B) makes an empty row.  Rows may repeat (beams that split), and
 * rows that no parent names end.  Written:
 *   table_after    [B_after][table_stride] pages that hold tokens, then -1
 *   lengths_after  [B_after]
 *   copies         [B_after][2] pages to copy, from and to (kv_copy_pages),
 *                  then -1: a partly filled last page that several new rows
 *                  hold is written by one of them, the first that has it as
 *                  its partly filled last page (none, where a row has it full);
 *                  the others get a page of their own
 *   n_copies       how many
 *   shared         [B_after / group] or NULL: the leading tokens whose pages all
 *                  rows of each `group` rows in turn have in common (a copy
 *                  that no page is left for is in common with none)
 *   used_after, free_pages   the free pages are free_pages[*used .. n_free)
 *                  before and free_pages[*used_after .. n_free) after.  Pages
 *                  of the old table that no new row holds become free.
 *                  Copies take pages that become free first, by number, then
 *                  free_pages[*used] on; what is left of the former goes, by
 *                  number, to the entries right below *used.  Where pages run
 *                  out, the table gets -1 and *used_after exceeds n_free.  A
 *                  *used above n_free (they had run out before, here or in
 *                  kv_plan) counts as n_free.
 * Entries of the table outside [0, pages) are passed on; they are neither
 * copied nor freed.  A page belongs to the table alone: it is in no other
 * table and not among the free ones.  Repeating the call with the same inputs
 * gives the same outputs, free_pages' entries from *used on being read only.
 * None of the outputs may be an input's memory but free_pages, which is both.
 * B, B_after <= KV_FORK_MAX_ROWS, and group divides B_after.  B_after = 0 frees
 * every page.  table_stride * page_size and pages are below 2^31 - 2^20.
 */
int kv_fork(const int *block_table, const int *lengths, const int *parents, const int *keep, int *free_pages,
            const int *used, int *table_after, int *lengths_after, int *copies, int *n_copies, int *shared,
            int *used_after, int B, int B_after, int group, int n_free, int table_stride, int page_size, int pages,
            void *ws, size_t ws_bytes, void *stream);
size_t kv_fork_workspace_bytes(int B_after, int pages);

/*
 * The pages in use moved to the front of the pool, pages first_page ..
 * first_page + n_free - 1: if n of them hold tokens of the B rows, those
 * numbered from first_page + n on take, in order, the free numbers below.
 * Written:
 *   table_after  [B][table_stride] the pages' new numbers, then -1 past each
 *                row's tokens (entries outside the pool are passed on)
 *   copies       [n_free / 2][2] pages to copy, from and to, then -1; n_copies
 *   free_pages   [n_free] first_page, first_page + 1, ...; used_after = n, so
 *                that free_pages[n ..] are the free pages
 * B <= KV_FORK_MAX_ROWS; table_stride * page_size and n_free are below 2^31 -
 * 2^20, first_page + n_free below 2^31.
 */
int kv_compact(const int *block_table, const int *lengths, int *table_after, int *free_pages, int *copies,
               int *n_copies, int *used_after, int B, int n_free, int table_stride, int page_size, int first_page,
               void *ws, size_t ws_bytes, void *stream);
size_t kv_compact_workspace_bytes(int n_free);

/*
 * Page copies[i][0] copied to page copies[i][1] in each of n_caches caches of
 * `pages` pages of page_bytes bytes (a multiple of 16; caches 16-byte aligned),
 * for i < min(*n_copies, capacity).  Copies from or to a page outside [0,
 * pages) are left out.  A page copied to must not be copied from, nor be copied
 * to twice (kv_fork and kv_compact make no such lists).  1 <= n_caches <= 2
 * RING_MAX_RANKS.
 */
int kv_copy_pages(void *const *caches, const int *copies, const int *n_copies, int n_caches, int capacity, int pages,
                  long long page_bytes, void *stream);

/*
 * The 4-bit cache.  cache[r] holds `pages` pages of Hkv heads, a page of one
 * head being one run of kv4_page_bytes(1, D, page_size) bytes:
 *     key codes    page_size rows of D / 2 bytes: value 2 i in the low half of byte i
 *     value codes  likewise
 *     key scales   page_size rows of D / 32 bytes
 *     value scales likewise
 * A code is a sign (8) and a magnitude 0, 0.5, 1, 1.5, 2, 3, 4, 6; a scale
 * byte s means 2^(s - 127) for 32 values in turn, 255 NaN (the microscaling
 * format with e2m1 elements).  A block's scale is the least, from 2^-126 to
 * 2^125, with no magnitude above 7 times it, so that no value is off by more
 * than one scale; values round to the nearest code, halfway to the even one.
 * (What is above 7 * 2^125 is stored as 6 * 2^125, up to two scales off: bf16
 * could not hold 6 times the next scale.)
 * A block that holds a value that is not finite is stored as NaN.
 * page_size is a power of two of at least 16.  Slots are kv_plan's: slot s is
 * row s % page_size of page s / page_size.
 *
 * tp_kv4_write: rows k[r], v[r] (T rows of Hkv heads of D bf16) to cache rows
 * slots[t]; a slot outside the cache writes nothing.  Two tokens of one slot
 * leave a row that is neither's (codes and scales, keys and values may be of
 * different ones, so a value may have any size), and change no other row.
 * tp_kv4_read: the values of cache rows slots[t] to k[r], v[r] (exact in bf16
 * but for values below 2^-133); zeros for a slot outside the cache.  With it,
 * a prompt that continues behind cached tokens runs through tp_attention.
 */
size_t kv4_page_bytes(int Hkv, int D, int page_size);
int tp_kv4_write(const void *const *k, const void *const *v, void *const *cache, const long long *slots, int P, int T,
                 int Hkv, int D, int page_size, int pages, long long k_stride, long long v_stride, void *stream);
int tp_kv4_read(const void *const *cache, const long long *slots, void *const *k, void *const *v, int P, int T, int Hkv,
                int D, int page_size, int pages, long long k_stride, long long v_stride, void *stream);

/*
 * Attention of one query token per row over the 4-bit cache: q[r], o[r]: B rows
 * of Hq heads (bf16); o[r] = softmax(scale q k^T) v over row b's keys j <
 * lengths[b], at page block_table[b * table_stride + j / page_size].  Rows come
 * in groups of `group` in turn (beams of one prompt, tokens of one request, or
 * requests behind one prompt): the first shared[g] keys of all rows of group g
 * are the same ones (kv_fork gives such numbers; NULL: none are), are found
 * through the table row of the group's first row, and are read once for up to
 * 32 (row, head of the group that shares a key head).  shared[g] is clamped to
 * the lengths of the group's rows.
 * Products in bf16 on the matrix cores (4-bit values are exact in bf16) with
 * fp32 sums, statistics in fp32, the softmax weights rounded to bf16 and summed
 * as rounded.
 * Lengths are clamped to [0, table_stride * page_size]; keys whose page lies
 * outside [0, pages) take no part; a row without keys gives o = 0.  Rows of the
 * cache that are no key of a row never reach its result.
 * Where the table's rows hold more than 2048 keys, or keys are shared, the keys
 * are shared out evenly among the compute units whatever the lengths.
 * B <= KV_FORK_MAX_ROWS, group divides B.  The workspace of a batch holds every
 * smaller one with the same other sizes.
 */
int tp_attention_decode_kv4(const void *const *q, const void *const *cache, void *const *o, const int *block_table,
                            const int *lengths, const int *shared, int P, int B, int group, int Hq, int Hkv, int D,
                            int table_stride, int page_size, int pages, long long q_stride, long long o_stride,
                            float scale, void *ws, size_t ws_bytes, void *stream);
size_t tp_attention_decode_kv4_workspace_bytes(int P, int B, int group, int Hq, int Hkv, int D);

#ifdef __cplusplus
}
#endif

#endif /* TP_SEARCH_H */
