"""Python entry points of the attention half of a tensor-parallel layer, one
per C-ABI call of tp_attention.h.

Each takes lists of per-rank torch tensors and single tensors that all ranks
read, checks shapes, types and layouts, and calls the library on torch's
current HIP stream (or `stream`).  Nothing here computes.
"""
from __future__ import annotations

import math

import torch

from . import _native as N
from .collectives import _ordered, _stream, _wsarg

_BF = torch.bfloat16


def _rows(ts, what: str, name: str, P: int, shape, dtype=_BF, packed: bool = False):
    """(pointer array, row stride) of P per-rank tensors of one shape: the
    last dimensions dense, the first one (tokens) at a stride of its own, or
    everything dense where `packed` (row stride 0, not used)."""
    if len(ts) != P:
        raise ValueError("%s: %s needs %d rank buffers, got %d" % (what, name, P, len(ts)))
    t0 = ts[0]
    device, stride = t0.device, t0.stride()
    if packed:
        if not t0.is_contiguous():
            raise ValueError("%s: %s must be contiguous" % (what, name))
        row = 0
    else:
        row = 1
        for n, s in zip(reversed(shape[1:]), reversed(stride[1:])):
            if n > 1 and s != row and t0.numel():
                raise ValueError("%s: the heads of a row of %s must be dense" % (what, name))
            row *= n
        if shape[0] > 1 and t0.numel():
            row = stride[0]
    ptrs = (N._vp * P)()
    for i, t in enumerate(ts):
        if t.shape != shape:
            raise ValueError("%s: every rank's %s must be %s, got %s" % (what, name, tuple(shape), tuple(t.shape)))
        if t.dtype != dtype:
            raise TypeError("%s: %s must be %s, got %s" % (what, name, dtype, t.dtype))
        if not t.is_cuda or t.device != device or (t is not t0 and t.stride() != stride):
            raise ValueError("%s: every rank's %s must be on one device, with the same strides" % (what, name))
        ptrs[i] = t.data_ptr()
    return ptrs, row


def _one(t, what: str, name: str, device, dtype=torch.int32, numel=None):
    """Pointer of one contiguous device tensor that all ranks read."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.device != device or not t.is_contiguous():
        raise ValueError("%s: %s must be a contiguous tensor on the ranks' device" % (what, name))
    if t.dtype != dtype:
        raise TypeError("%s: %s must be %s, got %s" % (what, name, dtype, t.dtype))
    if numel is not None and t.numel() != numel:
        raise ValueError("%s: %s needs %d elements, got %d" % (what, name, numel, t.numel()))
    return t.data_ptr()


def _lists(what: str, *lists):
    """Number of ranks of per-rank lists, the first of which must not be empty."""
    if not 1 <= len(lists[0]) <= N.MAX_RANKS:
        raise ValueError("%s: 1..%d rank buffers, got %d" % (what, N.MAX_RANKS, len(lists[0])))
    for ts in lists:
        for t in ts:
            if not isinstance(t, torch.Tensor):
                raise TypeError("%s: rank buffers are torch tensors" % what)
    return len(lists[0])


def _heads(t, what: str, name: str):
    if t.dim() != 3:
        raise ValueError("%s: %s is (tokens, heads, width), got %s" % (what, name, tuple(t.shape)))
    return t.shape


def kv_plan(lengths, new_tokens, free_pages, used, block_table, lengths_after, cu_new, positions, slots, used_after,
            page_size: int, prefix_len: int = 0, stream=None) -> None:
    """Block table entries, cache slots and positions of the tokens that a
    batch of requests adds to a paged cache (int32 tensors, slots int64):
    block_table (B, W) gets the pages from free_pages[used..] that the new
    tokens need, positions[cu_new[b] + i] = prefix_len + lengths[b] + i and
    slots[...] that token's cache row.  used_after > len(free_pages): the pages
    ran out, and the tokens without one have slot -1."""
    what = "kv_plan"
    B, dev = lengths.numel(), lengths.device
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("kv_plan: block_table is (requests, pages), got %s" % (tuple(block_table.shape),))
    if positions.numel() != slots.numel():
        raise ValueError("kv_plan: positions and slots hold one entry per token each")
    N.check(N.lib().kv_plan(
        _one(lengths, what, "lengths", dev), _one(new_tokens, what, "new_tokens", dev, numel=B),
        _one(free_pages, what, "free_pages", dev), _one(used, what, "used", dev, numel=1),
        _one(block_table, what, "block_table", dev), _one(lengths_after, what, "lengths_after", dev, numel=B),
        _one(cu_new, what, "cu_new", dev, numel=B + 1), _one(positions, what, "positions", dev),
        _one(slots, what, "slots", dev, torch.int64), _one(used_after, what, "used_after", dev, numel=1), B,
        free_pages.numel(), block_table.shape[1], page_size, positions.numel(), prefix_len, _stream(stream)), what)


def _qkv(qkv, gain_q, gain_k, cos_sin, pos, Hq: int, D: int, what: str):
    """What the norm-and-rotation calls share: (pointers, sizes) of the
    projected rows, the gains and the angle table."""
    P, dev = _lists(what, qkv), qkv[0].device
    if qkv[0].dim() != 2:
        raise ValueError("%s: qkv is (tokens, (Hq + 2 Hkv) D), got %s" % (what, tuple(qkv[0].shape)))
    T, width = qkv[0].shape
    dt = qkv[0].dtype
    if dt not in (torch.float32, _BF):
        raise TypeError("%s: qkv is float32 or bfloat16, got %s" % (what, dt))
    Hkv = (width // D - Hq) // 2 if D else 0
    if D == 0 or Hkv < 1 or (Hq + 2 * Hkv) * D != width:
        raise ValueError("%s: rows of %d values are not %d query heads and two equal groups of heads of width %d"
                         % (what, width, Hq, D))
    x, stride = _rows(qkv, what, "qkv", P, (T, width), dt)
    if (gain_q is None) != (gain_k is None):
        raise ValueError("%s: both gains or neither" % what)
    gq = gk = None
    if gain_q is not None:
        gq, gk = (_rows(g, what, n, P, (D,), torch.float32, packed=True)[0]
                  for g, n in ((gain_q, "gain_q"), (gain_k, "gain_k")))
    if cos_sin.dim() != 2:
        raise ValueError("%s: cos_sin is (positions, rotated width), got %s" % (what, tuple(cos_sin.shape)))
    cs = _one(cos_sin, what, "cos_sin", dev, torch.float32)
    return P, T, Hkv, x, stride, gq, gk, cs, _one(pos, what, "pos", dev, numel=T), N.RING_F32 if dt == torch.float32 else N.RING_BF16


def tp_qk_norm_rope(qkv, gain_q, gain_k, cos_sin, pos, q, k=None, v=None, k_cache=None, v_cache=None, slots=None,
                    eps: float = 1e-6, stream=None) -> None:
    """q[r], k[r] <- the RMS-normed, rotated query and key heads of the rows
    qkv[r] (T, (Hq + 2 Hkv) D; fp32 or bf16), v[r] <- its value heads, all
    bf16 (T, heads, D).  With k_cache, v_cache (rows, Hkv, D) and slots (T
    int64) the keys and values also go to the cache rows slots[t]; k and v may
    then be left out.  cos_sin: (positions, rot) fp32, cos then sin of the
    angles of pairs (i, i + rot / 2); pos: T int32.  gain_q[r], gain_k[r]: D
    fp32, or None for no norm."""
    what = "tp_qk_norm_rope"
    P = _lists(what, q)
    T, Hq, D = _heads(q[0], what, "q")
    P2, T2, Hkv, x, stride, gq, gk, cs, ps, dt = _qkv(qkv, gain_q, gain_k, cos_sin, pos, Hq, D, what)
    if P2 != P or T2 != T:
        raise ValueError("%s: q and qkv differ in ranks or tokens" % what)
    qp = _rows(q, what, "q", P, (T, Hq, D), packed=True)[0]
    if (k is None) != (v is None) or (k_cache is None) != (v_cache is None) or (k_cache is None) != (slots is None):
        raise ValueError("%s: k and v, and k_cache, v_cache and slots, go together" % what)
    kp = vp = kcp = vcp = sl = None
    rows = 0
    if k is not None:
        kp, vp = (_rows(t, what, n, P, (T, Hkv, D), packed=True)[0] for t, n in ((k, "k"), (v, "v")))
    if k_cache is not None:
        rows = k_cache[0].shape[0]
        kcp, vcp = (_rows(t, what, n, P, (rows, Hkv, D), packed=True)[0]
                    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")))
        sl = _one(slots, what, "slots", q[0].device, torch.int64, T)
    N.check(N.lib().tp_qk_norm_rope(x, gq, gk, cs, ps, qp, kp, vp, kcp, vcp, sl, P, T, Hq, Hkv, D, cos_sin.shape[1],
                                    cos_sin.shape[0], rows, stride, eps, dt, _stream(stream)), what)


def tp_qk_norm_rope_grad(dq, dk, dv, qkv, gain_q, gain_k, cos_sin, pos, dqkv, dgain_q=None, dgain_k=None,
                         eps: float = 1e-6, ws=None, stream=None):
    """dqkv[r] <- the gradient of tp_qk_norm_rope's rows (their type), and
    dgain_q[r], dgain_k[r] <- the gains', from dq, dk, dv (bf16)."""
    what = "tp_qk_norm_rope_grad"
    _lists(what, dq)
    T, Hq, D = _heads(dq[0], what, "dq")
    P, T2, Hkv, x, stride, gq, gk, cs, ps, dt = _qkv(qkv, gain_q, gain_k, cos_sin, pos, Hq, D, what)
    if len(dq) != P or T2 != T:
        raise ValueError("%s: dq and qkv differ in ranks or tokens" % what)
    dqp = _rows(dq, what, "dq", P, (T, Hq, D), packed=True)[0]
    dkp, dvp = (_rows(t, what, n, P, (T, Hkv, D), packed=True)[0] for t, n in ((dk, "dk"), (dv, "dv")))
    dxp = _rows(dqkv, what, "dqkv", P, (T, (Hq + 2 * Hkv) * D), qkv[0].dtype, packed=True)[0]
    dgq = dgk = None
    if gain_q is not None:
        if dgain_q is None or dgain_k is None:
            raise ValueError("%s: the gains' gradients need buffers" % what)
        dgq, dgk = (_rows(t, what, n, P, (D,), torch.float32, packed=True)[0]
                    for t, n in ((dgain_q, "dgain_q"), (dgain_k, "dgain_k")))
    if ws is None:
        nb = int(N.lib().tp_qk_norm_rope_grad_workspace_bytes(P, D))
        ws = _ordered(torch.zeros(max(nb, 256), dtype=torch.uint8, device=dq[0].device), stream)
    N.check(N.lib().tp_qk_norm_rope_grad(dqp, dkp, dvp, x, gq, gk, cs, ps, dxp, dgq, dgk, P, T, Hq, Hkv, D,
                                         cos_sin.shape[1], cos_sin.shape[0], stride, eps, dt, *_wsarg(ws, what),
                                         _stream(stream)), what)
    return ws


def _scale(scale, D: int) -> float:
    return float(scale) if scale is not None else 1.0 / math.sqrt(D) if D else 0.0


def _attn(q, k, v, o, cu_q, cu_k, what):
    """Pointers and sizes of a packed-prompt call."""
    P = _lists(what, q, k, v, o)
    Tq, Hq, D = _heads(q[0], what, "q")
    Tk, Hkv, _ = _heads(k[0], what, "k")
    dev = q[0].device
    qp, qs = _rows(q, what, "q", P, (Tq, Hq, D))
    kp, ks = _rows(k, what, "k", P, (Tk, Hkv, D))
    vp, vs = _rows(v, what, "v", P, (Tk, Hkv, D))
    op, os_ = _rows(o, what, "o", P, (Tq, Hq, D))
    B = cu_q.numel() - 1
    if B < 0:
        raise ValueError("%s: cu_q holds the prompts' offsets, one more than prompts" % what)
    return (qp, kp, vp, op, _one(cu_q, what, "cu_q", dev), _one(cu_k, what, "cu_k", dev, numel=B + 1),
            (P, B, Tq, Tk, Hq, Hkv, D), (qs, ks, vs, os_))


def tp_attention(q, k, v, o, cu_q, cu_k, lse=None, causal: bool = True, scale=None, stream=None) -> None:
    """o[r] <- softmax(scale q[r] k[r]^T) v[r] over packed prompts: prompt b's
    queries are rows cu_q[b]..cu_q[b + 1] of q[r] (Tq, Hq, D), its keys and
    values rows cu_k[b]..cu_k[b + 1] of k[r], v[r] (Tk, Hkv, D); causal aligns
    its last query with its last key.  bf16, fp32 sums; rows may be slices of a
    packed row.  lse[r] (Hq, Tq fp32) <- the rows' log sum exp.  scale: 1 /
    sqrt(D) unless given."""
    what = "tp_attention"
    qp, kp, vp, op, cq, ck, sizes, strides = _attn(q, k, v, o, cu_q, cu_k, what)
    P, _, Tq, _, Hq, _, D = sizes
    lp = None if lse is None else _rows(lse, what, "lse", P, (Hq, Tq), torch.float32, packed=True)[0]
    N.check(N.lib().tp_attention(qp, kp, vp, op, lp, cq, ck, *sizes, *strides, int(bool(causal)),
                                 _scale(scale, D), _stream(stream)), what)


def tp_attention_grad(do, q, k, v, o, lse, dq, dk, dv, cu_q, cu_k, causal: bool = True, scale=None, ws=None, stream=None):
    """dq[r], dk[r], dv[r] <- the gradient of tp_attention for do[r], the
    gradient of o[r], from its inputs and outputs (the same bits every time)."""
    what = "tp_attention_grad"
    qp, kp, vp, op, cq, ck, sizes, strides = _attn(q, k, v, o, cu_q, cu_k, what)
    P, _, Tq, Tk, Hq, Hkv, D = sizes
    _lists(what, q, do, dq, dk, dv, lse)
    gp, gs = _rows(do, what, "do", P, (Tq, Hq, D))
    lp = _rows(lse, what, "lse", P, (Hq, Tq), torch.float32, packed=True)[0]
    dqp, dqs = _rows(dq, what, "dq", P, (Tq, Hq, D))
    dkp, dks = _rows(dk, what, "dk", P, (Tk, Hkv, D))
    dvp, dvs = _rows(dv, what, "dv", P, (Tk, Hkv, D))
    if ws is None:
        nb = int(N.lib().tp_attention_grad_workspace_bytes(P, Tq, Hq))
        ws = _ordered(torch.zeros(max(nb, 256), dtype=torch.uint8, device=q[0].device), stream)
    N.check(N.lib().tp_attention_grad(gp, qp, kp, vp, op, lp, dqp, dkp, dvp, cq, ck, *sizes, *strides, gs, dqs, dks, dvs,
                                      int(bool(causal)), _scale(scale, D), *_wsarg(ws, what), _stream(stream)), what)
    return ws


def tp_attention_decode(q, k_cache, v_cache, o, block_table, lengths, page_size: int, prefix_pages=None,
                        prefix_len: int = 0, scale=None, ws=None, stream=None):
    """o[r] <- attention of one query token per request, q[r] (B, Hq, D), over
    the paged cache k_cache[r], v_cache[r] (rows, Hkv, D): the first prefix_len
    rows of prefix_pages, shared by all requests and read once, and the first
    lengths[b] rows of block_table[b] (B, W int32)."""
    what = "tp_attention_decode"
    P = _lists(what, q, k_cache, v_cache, o)
    B, Hq, D = _heads(q[0], what, "q")
    rows, Hkv, _ = _heads(k_cache[0], what, "k_cache")
    dev = q[0].device
    qp, qs = _rows(q, what, "q", P, (B, Hq, D))
    op, os_ = _rows(o, what, "o", P, (B, Hq, D))
    kp, vp = (_rows(t, what, n, P, (rows, Hkv, D), packed=True)[0] for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")))
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("%s: block_table is (requests, pages), got %s" % (what, tuple(block_table.shape)))
    tab, lens = _one(block_table, what, "block_table", dev), _one(lengths, what, "lengths", dev, numel=B)
    if page_size < 1 or rows % page_size:
        raise ValueError("%s: the cache's %d rows are not whole pages of %d" % (what, rows, page_size))
    pp = None
    if prefix_len:
        if prefix_pages is None or prefix_pages.numel() * page_size < prefix_len:
            raise ValueError("%s: prefix_pages does not hold %d tokens" % (what, prefix_len))
        pp = _one(prefix_pages, what, "prefix_pages", dev)
    W = block_table.shape[1]
    if ws is None:
        nb = int(N.lib().tp_attention_decode_workspace_bytes(P, B, Hq, Hkv, D, W, page_size, prefix_len))
        ws = _ordered(torch.zeros(max(nb, 256), dtype=torch.uint8, device=dev), stream)
    N.check(N.lib().tp_attention_decode(qp, kp, vp, op, tab, lens, pp, P, B, Hq, Hkv, D, W, page_size, rows // page_size,
                                        prefix_len, qs, os_, _scale(scale, D), *_wsarg(ws, what), _stream(stream)), what)
    return ws
