/*
 * tp_attention.h -- C ABI of libring_collectives.so, second part: the
 * attention half of a tensor-parallel layer over P virtual ranks.  Rank r
 * holds Hq query heads and Hkv key/value heads of width D of its own (heads
 * split over ranks, as W1's columns are in tp_mlp_layer), so no call here
 * moves data between ranks; one launch works for all of them.  Between the
 * two collective products they make the layer's attention:
 *
 *   all_gather_gemm      x_shard, Wqkv       -> fp32 rows of q | k | v heads
 *   kv_plan              request lengths     -> block table, slots, positions
 *   tp_qk_norm_rope      rows, slots         -> q, k, v in bf16, cache rows
 *   tp_attention         packed prompts      -> o     (and tp_attention_grad)
 *   tp_attention_decode  one token a request -> o
 *   gemm_reduce_scatter  o, Wo               -> out_shard
 *
 * Conventions, beside those of ring_collectives.h (error codes, streams,
 * nothing allocated, printed or thrown, no memset recorded):
 *   - arrays of P pointers are host arrays of device pointers, read during
 *     the call only; single pointers are device pointers to one copy that all
 *     ranks read (lengths, tables, positions).
 *   - bf16 data and fp32 `dtype` data is 16-byte aligned, integers and lse are
 *     aligned as their types are; a row stride counts elements from one token's
 *     row to the next, is a multiple of 8, at least heads * D and below 2^21.
 *     The heads of a row lie D apart, so q, k and v may be slices of one packed
 *     row.  What has no element may have no address.
 *   - D is 64 or 128 and Hkv divides Hq: query head h reads key head
 *     h / (Hq / Hkv).  Others: RING_EUNSUPPORTED.
 *   - outputs must not overlap inputs or each other (not checked; tensors
 *     that interleave in one packed row are fine).
 *   - what lies in device memory cannot be refused by a call.  Lengths,
 *     offsets, pages, slots and positions that lie outside their tables are
 *     never followed: each call says what such an entry gives instead.
 *   - ws: as in ring_collectives.h (256-byte aligned, zeroed once before its
 *     first use, calls that share one are ordered); the calls leave data in
 *     it and record where.
 */
#ifndef TP_ATTENTION_H
#define TP_ATTENTION_H

#include "ring_collectives.h"

#ifdef __cplusplus
extern "C" {
#endif

#define KV_PLAN_MAX_REQUESTS 8192

/*
 * The cache bookkeeping of one step, on the GPU.  Request b holds lengths[b]
 * tokens in the cache and adds new_tokens[b] (negative values count as 0).
 * A cache row is a slot; page p is the page_size slots from p * page_size on
 * (page_size a power of two); block_table[b * table_stride + j] is the page
 * of b's tokens j * page_size and following.
 *
 * Pages a request needs beyond those its lengths[b] tokens fill come from
 * free_pages[0 .. n_free), in request order, from entry *used on.  Written:
 *   block_table    the entries of those pages (others keep their value); an
 *                  entry past the end of free_pages is set to -1
 *   lengths_after  [B] lengths[b] + new_tokens[b]
 *   cu_new         [B + 1] 0 and the running sums of new_tokens
 *   positions      [capacity] prefix_len + lengths[b] + i for new token i of
 *                  b, at cu_new[b] + i; 0 from cu_new[B] on
 *   slots          [capacity] its cache row, -1 where its page is -1 or lies
 *                  past table_stride, and from cu_new[B] on
 *   used_after     *used plus the pages needed: more than n_free tells that
 *                  the pages ran out
 * used_after and lengths_after must not be used's, lengths' or new_tokens'
 * memory (RING_EINVAL): a caller that goes step by step keeps two of each.
 * Tokens past `capacity` are left out.  1 <= B <= KV_PLAN_MAX_REQUESTS, else
 * RING_EUNSUPPORTED.  B = 0 is RING_OK without a launch, and writes nothing:
 * a caller that swaps used and used_after does not swap them then.
 */
int kv_plan(const int *lengths, const int *new_tokens, const int *free_pages, const int *used, int *block_table,
            int *lengths_after, int *cu_new, int *positions, long long *slots, int *used_after, int B, int n_free,
            int table_stride, int page_size, int capacity, int prefix_len, void *stream);

/*
 * Query/key norm and position rotation of T tokens in one pass, with the
 * cache write.  qkv[r]: T rows of (Hq + 2 Hkv) heads of D values, q heads
 * first, then k, then v; RING_F32 or RING_BF16.  For every q and k head row x
 *     y = x / sqrt(mean(x^2) + eps) * gain       (gain_q[r], gain_k[r]: D fp32)
 * and the first rot values of y turn in pairs (i, i + rot / 2) by the angle of
 * the token's position:
 *     (y_i cos - y_{i+rot/2} sin,  y_{i+rot/2} cos + y_i sin),
 * cos = cos_sin[pos][i], sin = cos_sin[pos][rot / 2 + i]; the others pass.
 * All in fp32, rounded once to bf16.  v is rounded and passed.
 *   gain_q, gain_k  NULL: no norm and no gain, rotation only
 *   cos_sin  table_rows rows of rot fp32; pos: T positions.  rot a multiple
 *            of 16, 0 <= rot <= D.  A position outside the table gives NaN in
 *            that token's q and k heads.
 *   q[r]     T rows of Hq heads;  k[r], v[r] (both or neither may be NULL)
 *            T rows of Hkv heads, all with packed rows
 *   k_cache[r], v_cache[r], slots (all or none NULL): token t's k and v heads
 *            also go to cache row slots[t] (cache_rows rows of Hkv heads,
 *            packed); a slot outside [0, cache_rows) writes nothing.  Two
 *            tokens of one slot give either's values.
 */
int tp_qk_norm_rope(const void *const *qkv, const float *const *gain_q, const float *const *gain_k,
                    const float *cos_sin, const int *pos, void *const *q, void *const *k, void *const *v,
                    void *const *k_cache, void *const *v_cache, const long long *slots, int P, int T, int Hq, int Hkv,
                    int D, int rot, long long table_rows, long long cache_rows, long long qkv_stride, float eps,
                    int dtype, void *stream);

/*
 * Its gradient: from dq, dk, dv (bf16, packed rows; the gradients of the
 * rotated q, k and of v) and the call's inputs, dqkv[r] (T rows like qkv, of
 * `dtype`, packed) and the gains' gradients dgain_q[r], dgain_k[r] (D fp32,
 * summed over the rank's tokens and heads in a fixed order).  With NULL gains
 * dgain_q and dgain_k are not written and may be NULL.  A token whose position
 * lies outside the table gives NaN in the q and k heads of dqkv and adds
 * nothing to the gains' gradients.
 */
int tp_qk_norm_rope_grad(const void *const *dq, const void *const *dk, const void *const *dv, const void *const *qkv,
                         const float *const *gain_q, const float *const *gain_k, const float *cos_sin, const int *pos,
                         void *const *dqkv, float *const *dgain_q, float *const *dgain_k, int P, int T, int Hq, int Hkv,
                         int D, int rot, long long table_rows, long long qkv_stride, float eps, int dtype, void *ws,
                         size_t ws_bytes, void *stream);
size_t tp_qk_norm_rope_grad_workspace_bytes(int P, int D);

/*
 * Attention over B packed prompts.  Prompt b's queries are rows cu_q[b] ..
 * cu_q[b + 1] of q[r] (Tq rows, bf16), its keys and values rows cu_k[b] ..
 * cu_k[b + 1] of k[r], v[r] (Tk rows).  With S = scale q k^T over the keys a
 * query sees -- all of its prompt, or with causal != 0 key j for query i
 * when j <= i + (its prompt's keys - its queries), so that the last query sees
 * every key -- o[r] = softmax(S) v (bf16), lse[r][h][t] = log sum exp(S) (Hq x
 * Tq fp32; lse may be NULL).  A query that sees no key gives o = 0 and lse =
 * -inf.  Products in bf16 on the matrix cores with fp32 sums, statistics in
 * fp32, the softmax weights rounded to bf16 for the second product.
 * Offsets are clamped to [0, Tq] and [0, Tk], and one below its prompt's start
 * makes the prompt empty; rows that no prompt covers are not written.
 * scale > 0, and finite times log2(e).  A key or value that is not finite
 * reaches only the queries that see it.
 */
int tp_attention(const void *const *q, const void *const *k, const void *const *v, void *const *o, float *const *lse,
                 const int *cu_q, const int *cu_k, int P, int B, int Tq, int Tk, int Hq, int Hkv, int D,
                 long long q_stride, long long k_stride, long long v_stride, long long o_stride, int causal, float scale,
                 void *stream);

/*
 * Its gradient, from dout[r] (the gradient of o) and tp_attention's inputs
 * and outputs: dq[r] (Tq rows), dk[r], dv[r] (Tk rows), bf16, with fp32 sums
 * in a fixed order (the same bits every time).  P and dS = P (dP - sum(dout
 * o)) are computed again from q, k, v and lse in fp32 and rounded to bf16 for
 * the products that they enter; sum(dout o) is taken in fp32 from o as it was
 * rounded.  A query that sees no key gives dq = 0 and adds nothing; a key that
 * no query sees gives dk = dv = 0.  Inputs that are not finite may make NaN of
 * any gradient of their prompt (of their rank and group of heads), and of no
 * other.
 */
int tp_attention_grad(const void *const *dout, const void *const *q, const void *const *k, const void *const *v,
                      const void *const *o, const float *const *lse, void *const *dq, void *const *dk, void *const *dv,
                      const int *cu_q, const int *cu_k, int P, int B, int Tq, int Tk, int Hq, int Hkv, int D,
                      long long q_stride, long long k_stride, long long v_stride, long long o_stride,
                      long long dout_stride, long long dq_stride, long long dk_stride, long long dv_stride, int causal,
                      float scale, void *ws, size_t ws_bytes, void *stream);
size_t tp_attention_grad_workspace_bytes(int P, int Tq, int Hq);

/*
 * Attention of one query token per request over a paged cache.  q[r], o[r]: B
 * rows of Hq heads (bf16).  k_cache[r], v_cache[r]: pages * page_size packed
 * rows of Hkv heads.  Request b's keys are the prefix's, key j at row
 * prefix_pages[j / page_size] * page_size + j % page_size for j < prefix_len,
 * shared by all requests, and its own, key j at page block_table[b *
 * table_stride + j / page_size] likewise for j < lengths[b] (the new token's
 * row among them, if it is to be seen).  o[r] = softmax(scale q k^T) v over
 * both; the prefix is read once for every 128 rows (request, head of the group
 * that shares a key head).
 * Lengths are clamped to [0, table_stride * page_size]; keys whose page lies
 * outside [0, pages) take no part; a request without keys gives o = 0.  Rows
 * of the cache that are no key of a request never reach its result.
 * pages * page_size and table_stride * page_size stay below 2^31.
 * scale as in tp_attention.  The workspace's size depends on the device's
 * compute units; that of a batch holds every smaller batch with the same other
 * sizes.
 */
int tp_attention_decode(const void *const *q, const void *const *k_cache, const void *const *v_cache, void *const *o,
                        const int *block_table, const int *lengths, const int *prefix_pages, int P, int B, int Hq,
                        int Hkv, int D, int table_stride, int page_size, int pages, int prefix_len, long long q_stride,
                        long long o_stride, float scale, void *ws, size_t ws_bytes, void *stream);
size_t tp_attention_decode_workspace_bytes(int P, int B, int Hq, int Hkv, int D, int table_stride, int page_size,
                                           int prefix_len);

#ifdef __cplusplus
}
#endif

#endif /* TP_ATTENTION_H */
