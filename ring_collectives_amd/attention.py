"""Python entry points of the attention half of a tensor-parallel layer, one
per C-ABI call of tp_attention.h.

Each takes lists of per-rank torch tensors and single tensors that all ranks
read, and calls the library on torch's current HIP stream (or `stream`).  The
extension module _binding checks shapes, types and layouts (ValueError,
TypeError) and marshals; the library's own refusals raise RingError.  Nothing
here computes (only kv_plan's outputs for no request at all are filled in
here).  A call's workspace is made when none is given, and returned
for the next one of the same sizes.
"""
from __future__ import annotations

import os

import torch

from . import _native as N
from .collectives import _ordered

_c = None


def _binding():
    global _c
    if _c is None:
        N.lib()
        if not os.path.exists(os.path.join(N.HERE, "_binding.so")):
            raise RuntimeError("_binding.so is not built (expected in %s); run "
                               "`python -m ring_collectives_amd.build`" % N.HERE)
        from . import _binding as c
        _c = c
    return _c


def _at(stream):
    """(stream handle, current device), what every call ends with."""
    dev = torch.cuda.current_device()
    return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(dev), dev


def _shape(t, dims: int, what: str):
    """The shape that a default is computed from; _binding checks the rest."""
    if not isinstance(t, torch.Tensor) or t.dim() != dims:
        raise ValueError("%s must be a tensor of %d dimensions" % (what, dims))
    return t.shape


def _lead(ts, dims: int, what: str):
    if not len(ts):
        raise ValueError("1..%d rank buffers, got 0" % N.MAX_RANKS)
    return _shape(ts[0], dims, what)


def _scale(scale, q) -> float:
    if scale is not None:
        return float(scale)
    D = _lead(q, 3, "q")[2]
    return D ** -0.5 if D else 0.0


def _new_ws(nbytes: int, device, stream) -> torch.Tensor:
    return _ordered(torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device), stream)


def kv_plan(lengths, new_tokens, free_pages, used, block_table, lengths_after, cu_new, positions, slots, used_after,
            page_size: int, prefix_len: int = 0, stream=None) -> None:
    """Block table entries, cache slots and positions of the tokens that a
    batch of requests adds to a paged cache (int32 tensors, slots int64):
    block_table (B, W) gets the pages from free_pages[used..] that the new
    tokens need, positions[cu_new[b] + i] = prefix_len + lengths[b] + i and
    slots[...] that token's cache row.  used_after > len(free_pages): the pages
    ran out, and the tokens without one have slot -1.  Without requests nothing
    is added: used_after = used, cu_new = [0], positions 0 and slots -1."""
    N.check(_binding().kv_plan(lengths, new_tokens, free_pages, used, block_table, lengths_after, cu_new, positions, slots,
                               used_after, page_size, prefix_len, *_at(stream)), "kv_plan")
    if not lengths.numel():          # the library launches nothing and writes nothing then
        with torch.cuda.stream(stream):
            used_after.copy_(used)
            cu_new.zero_()
            positions.zero_()
            slots.fill_(-1)


def tp_qk_norm_rope(qkv, gain_q, gain_k, cos_sin, pos, q, k=None, v=None, k_cache=None, v_cache=None, slots=None,
                    eps: float = 1e-6, stream=None) -> None:
    """q[r], k[r] <- the RMS-normed, rotated query and key heads of the rows
    qkv[r] (T, (Hq + 2 Hkv) D; fp32 or bf16), v[r] <- its value heads, all
    bf16 (T, heads, D).  With k_cache, v_cache (rows, Hkv, D) and slots (T
    int64) the keys and values also go to the cache rows slots[t]; k and v may
    then be left out.  cos_sin: (positions, rot) fp32, cos then sin of the
    angles of pairs (i, i + rot / 2); pos: T int32.  gain_q[r], gain_k[r]: D
    fp32, or None for no norm."""
    N.check(_binding().tp_qk_norm_rope(qkv, gain_q, gain_k, cos_sin, pos, q, k, v, k_cache, v_cache, slots, eps,
                                       *_at(stream)), "tp_qk_norm_rope")


def tp_qk_norm_rope_grad(dq, dk, dv, qkv, gain_q, gain_k, cos_sin, pos, dqkv, dgain_q=None, dgain_k=None,
                         eps: float = 1e-6, ws=None, stream=None):
    """dqkv[r] <- the gradient of tp_qk_norm_rope's rows (their type), and
    dgain_q[r], dgain_k[r] <- the gains', from dq, dk, dv (bf16)."""
    if ws is None:
        ws = _new_ws(N.lib().tp_qk_norm_rope_grad_workspace_bytes(len(dq), _lead(dq, 3, "dq")[2]), dq[0].device, stream)
    N.check(_binding().tp_qk_norm_rope_grad(dq, dk, dv, qkv, gain_q, gain_k, cos_sin, pos, dqkv, dgain_q, dgain_k, eps, ws,
                                            *_at(stream)), "tp_qk_norm_rope_grad")
    return ws


def tp_attention(q, k, v, o, cu_q, cu_k, lse=None, causal: bool = True, scale=None, stream=None) -> None:
    """o[r] <- softmax(scale q[r] k[r]^T) v[r] over packed prompts: prompt b's
    queries are rows cu_q[b]..cu_q[b + 1] of q[r] (Tq, Hq, D), its keys and
    values rows cu_k[b]..cu_k[b + 1] of k[r], v[r] (Tk, Hkv, D); causal aligns
    its last query with its last key.  bf16, fp32 sums; rows may be slices of a
    packed row.  lse[r] (Hq, Tq fp32) <- the rows' log sum exp.  scale: 1 /
    sqrt(D) unless given."""
    N.check(_binding().tp_attention(q, k, v, o, cu_q, cu_k, lse, int(bool(causal)), _scale(scale, q),
                                    *_at(stream)), "tp_attention")


def tp_attention_grad(do, q, k, v, o, lse, dq, dk, dv, cu_q, cu_k, causal: bool = True, scale=None, ws=None, stream=None):
    """dq[r], dk[r], dv[r] <- the gradient of tp_attention for do[r], the
    gradient of o[r], from its inputs and outputs (the same bits every time)."""
    if ws is None:
        Tq, Hq, _ = _lead(q, 3, "q")
        ws = _new_ws(N.lib().tp_attention_grad_workspace_bytes(len(q), Tq, Hq), q[0].device, stream)
    N.check(_binding().tp_attention_grad(q, k, v, o, cu_q, cu_k, lse, do, dq, dk, dv, int(bool(causal)),
                                         _scale(scale, q), ws, *_at(stream)), "tp_attention_grad")
    return ws


def tp_attention_decode(q, k_cache, v_cache, o, block_table, lengths, page_size: int, prefix_pages=None,
                        prefix_len: int = 0, scale=None, ws=None, stream=None):
    """o[r] <- attention of one query token per request, q[r] (B, Hq, D), over
    the paged cache k_cache[r], v_cache[r] (rows, Hkv, D): the first prefix_len
    rows of prefix_pages, shared by all requests and read once for every 128
    (request, head of the group), and the first lengths[b] rows of
    block_table[b] (B, W int32).  The workspace of a batch holds smaller ones."""
    if ws is None:
        B, Hq, D = _lead(q, 3, "q")
        Hkv, W = _lead(k_cache, 3, "k_cache")[1], _shape(block_table, 2, "block_table")[1]
        ws = _new_ws(N.lib().tp_attention_decode_workspace_bytes(len(q), B, Hq, Hkv, D, W, page_size, prefix_len),
                     q[0].device, stream)
    N.check(_binding().tp_attention_decode(q, k_cache, v_cache, o, block_table, lengths, page_size, prefix_pages, prefix_len,
                                           _scale(scale, q), ws, *_at(stream)), "tp_attention_decode")
    return ws
