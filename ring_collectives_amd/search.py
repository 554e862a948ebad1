"""Python entry points of beam search over a paged cache and of the 4-bit
cache, one per C-ABI call of tp_search.h, in the manner of attention.py: lists
of per-rank torch tensors, single tensors that all ranks read, torch's current
HIP stream (or `stream`), ValueError and TypeError for tensors that do not fit,
RingError for what the library refuses, and workspaces made when none is given
and returned for the next call of the same sizes.
"""
from __future__ import annotations

import torch

from . import _native as N
from .attention import _at, _binding, _lead, _new_ws, _scale, _shape


def beam_select(logits, scores, parents, tokens, scores_after, vocab: int, done=None, done_after=None, end_token: int = -1,
                ws=None, stream=None):
    """The best continuations of each group of beams: logits[r] (groups *
    beams, width; fp32 or bf16) are the columns of tokens r * width on, those
    from `vocab` on padding; scores (groups, beams) fp32.  parents, tokens
    (int32) and scores_after (fp32), (groups, places), get the candidates
    scores + log softmax(logits) in order, best first, of equal ones the lowest
    beam, then the largest logit, then the lowest token: parents the rows of
    logits they go on from, -1 where there are none left.  A beam of which done
    (uint8 or bool) is set goes on as end_token with the score it has;
    done_after tells which places are done or end with it.  Logits and scores
    that are not finite take no part."""
    if ws is None:
        s, out = _shape(scores, 2, "scores"), _shape(parents, 2, "parents")
        ws = _new_ws(N.lib().beam_select_workspace_bytes(len(logits), s[0], s[1], out[1], _lead(logits, 2, "logits")[1]),
                     logits[0].device, stream)
    N.check(_binding().beam_select(logits, scores, parents, tokens, scores_after, vocab, done, done_after, end_token, ws,
                                   *_at(stream)), "beam_select")
    return ws


def kv_fork(block_table, lengths, parents, free_pages, used, table_after, lengths_after, copies, n_copies, used_after,
            page_size: int, pages: int, keep=None, shared=None, group: int = 1, ws=None, stream=None):
    """table_after (rows, W) and lengths_after <- the rows parents[i] of
    block_table (B, W), the first keep[i] tokens of them where given; -1 makes
    an empty row.  copies (rows, 2) and n_copies: the pages to copy, for
    kv_copy_pages, so that rows of one parent do not write to the same page.
    Pages that no row holds any more join the free ones: free_pages[used..]
    before, free_pages[used_after..] after.  shared (rows / group): the leading
    tokens that `group` rows in turn have on the same pages, for
    tp_attention_decode_kv4.  All int32."""
    if ws is None:
        ws = _new_ws(N.lib().kv_fork_workspace_bytes(_shape(table_after, 2, "table_after")[0], pages), table_after.device, stream)
    N.check(_binding().kv_fork(block_table, lengths, parents, keep, free_pages, used, table_after, lengths_after, copies, n_copies,
                               shared, used_after, group, page_size, pages, ws, *_at(stream)), "kv_fork")
    return ws


def kv_compact(block_table, lengths, table_after, free_pages, copies, n_copies, used_after, page_size: int, first_page: int = 0,
               ws=None, stream=None):
    """The pages that hold tokens moved to the lowest numbers of the pool,
    first_page .. first_page + len(free_pages): table_after, the copies to make
    (len(free_pages) / 2, 2), and free_pages in order, free from used_after on.
    All int32."""
    if ws is None:
        ws = _new_ws(N.lib().kv_compact_workspace_bytes(_shape(free_pages, 1, "free_pages")[0]), free_pages.device, stream)
    N.check(_binding().kv_compact(block_table, lengths, table_after, free_pages, copies, n_copies, used_after, page_size, first_page,
                                  ws, *_at(stream)), "kv_compact")
    return ws


def kv_copy_pages(caches, copies, n_copies, pages: int, stream=None) -> None:
    """Page copies[i, 0] copied to page copies[i, 1] of each cache, for i <
    n_copies: any contiguous tensors of one size that hold `pages` pages one
    after the other, a multiple of 16 bytes each (bf16 caches of every rank,
    keys and values; 4-bit ones)."""
    N.check(_binding().kv_copy_pages(caches, copies, n_copies, pages, *_at(stream)), "kv_copy_pages")


def kv4_cache(pages: int, Hkv: int, D: int, page_size: int, device="cuda") -> torch.Tensor:
    """One rank's empty 4-bit cache: (pages, Hkv, bytes of a page of one head)."""
    n = N.lib().kv4_page_bytes(1, D, page_size)
    if not n or Hkv < 1 or pages < 0:
        raise ValueError("kv4_cache: %d pages of %d rows of %d heads of %d are not supported" % (pages, page_size, Hkv, D))
    return torch.zeros(pages, Hkv, n, dtype=torch.uint8, device=device)


def tp_kv4_write(k, v, cache, slots, page_size: int, stream=None) -> None:
    """Keys and values k[r], v[r] (T, Hkv, D; bf16) to the cache rows slots[t]
    (T int64, as kv_plan gives them) of the 4-bit caches cache[r] (kv4_cache),
    in blocks of 32 values with a power-of-two scale each.  Slots that are the
    same leave a row that may mix their tokens."""
    N.check(_binding().tp_kv4_write(k, v, cache, slots, page_size, *_at(stream)), "tp_kv4_write")


def tp_kv4_read(cache, slots, k, v, page_size: int, stream=None) -> None:
    """k[r], v[r] (T, Hkv, D; bf16) <- the values of the 4-bit cache's rows
    slots[t]; zeros for a slot outside the cache."""
    N.check(_binding().tp_kv4_read(cache, slots, k, v, page_size, *_at(stream)), "tp_kv4_read")


def tp_attention_decode_kv4(q, cache, o, block_table, lengths, page_size: int, shared=None, group: int = 1, scale=None, ws=None,
                            stream=None):
    """o[r] <- attention of one query token per row, q[r] (B, Hq, D), over the
    first lengths[b] rows of block_table[b] (B, W int32) of the 4-bit cache.
    The first shared[g] of them are the same for `group` rows in turn, and read
    once for up to 32 (row, head of the group that shares a key head).  The
    workspace of a batch holds smaller ones."""
    if ws is None:
        B, Hq, D = _lead(q, 3, "q")
        ws = _new_ws(N.lib().tp_attention_decode_kv4_workspace_bytes(len(q), B, group, Hq, _lead(cache, 3, "cache")[1], D),
                     q[0].device, stream)
    N.check(_binding().tp_attention_decode_kv4(q, cache, o, block_table, lengths, page_size, shared, group, _scale(scale, q), ws,
                                               *_at(stream)), "tp_attention_decode_kv4")
    return ws
