"""Oracle of the attention operators: their definitions in NumPy float64 (and
Python integers), with bounds on how far an fp32/bf16 evaluation may lie from
them.  Test infrastructure only.

U = 2^-24 is fp32's unit roundoff, UB = 2^-8 bf16's (8 significant bits).
The bounds are worst cases, element by element: products of bf16 values are
exact in fp32; a sum of n fp32 terms is off by at most n U sum |terms| in any
order; the hardware's exp2 and log2 are within 4 U relative, an exponent
computed as fma(s, c, -m) within U of its terms.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24
UB = 2.0 ** -8


def kv_plan(lengths, new_tokens, free_pages, used, table, page_size, capacity, prefix_len=0):
    """(table, lengths_after, cu_new, positions, slots, used_after), request by
    request and token by token."""
    table = [list(map(int, row)) for row in table]
    width = len(table[0]) if table else 0
    pos, slots, cu, after = [0] * capacity, [-1] * capacity, [0], []
    at, t = int(used), 0
    for b, (n, add) in enumerate(zip(lengths, new_tokens)):
        n, add = max(0, int(n)), max(0, int(add))
        have = -(-n // page_size)
        for j in range(have, -(-(n + add) // page_size)):
            if j < width:
                table[b][j] = int(free_pages[at]) if 0 <= at < len(free_pages) else -1
            at += 1
        for i in range(add):
            if t < capacity:
                j = (n + i) // page_size
                page = table[b][j] if j < width else -1
                pos[t] = prefix_len + n + i
                slots[t] = page * page_size + (n + i) % page_size if page >= 0 else -1
            t += 1
        cu.append(t)
        after.append(n + add)
    return np.array(table), np.array(after), np.array(cu), np.array(pos), np.array(slots), at


def _turn(y, ang, rot, sign=1.0):
    """Pairs (i, i + rot / 2) of the last axis turned by angles whose cos and
    sin are the halves of ang's; sign -1 turns back."""
    h = rot // 2
    c, s = ang[..., :h], sign * ang[..., h:]
    z = y.copy()
    z[..., :h] = y[..., :h] * c - y[..., h:rot] * s
    z[..., h:rot] = y[..., h:rot] * c + y[..., :h] * s
    return z


def _turn_size(y, ang, rot):
    """Sum of the terms' magnitudes of _turn."""
    h = rot // 2
    y, c, s = np.abs(y), np.abs(ang[..., :h]), np.abs(ang[..., h:])
    z = y.copy()
    z[..., :h] = y[..., :h] * c + y[..., h:rot] * s
    z[..., h:rot] = y[..., h:rot] * c + y[..., :h] * s
    return z


def qk_norm_rope(x, gain, cos_sin, pos, eps):
    """(T, H, D) head rows normed, scaled by gain (or neither for None) and
    turned, and the bound on an fp32 evaluation rounded once to bf16."""
    x = x.astype(np.float64)
    rot = cos_sin.shape[1]
    ang = cos_sin.astype(np.float64)[pos][:, None, :]
    y = x if gain is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * gain.astype(np.float64)
    z = _turn(y, ang, rot)
    # the norm: D + 4 roundings in the mean, half of which reach the root,
    # then root, quotient and two products; the turn: two products and a sum
    return z, (x.shape[-1] + 16) * U * _turn_size(y, ang, rot) + UB * np.abs(z)


def qk_norm_rope_grad(dz, x, gain, cos_sin, pos, eps):
    """(dx, bound, dgain, bound) of qk_norm_rope evaluated in fp32, dx not
    rounded further."""
    x, dz = x.astype(np.float64), dz.astype(np.float64)
    D, rot = x.shape[-1], cos_sin.shape[1]
    ang = cos_sin.astype(np.float64)[pos][:, None, :]
    dy, size = _turn(dz, ang, rot, -1.0), _turn_size(dz, ang, rot)
    if gain is None:
        return dy, 4 * U * size, None, None
    g = gain.astype(np.float64)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * r
    u, su = dy * g, size * np.abs(g)
    dx = r * (u - n * (n * u).mean(-1, keepdims=True))
    bound = (3 * D + 48) * U * r * (su + np.abs(n) * (np.abs(n) * su).mean(-1, keepdims=True))
    dg = (dy * n).sum((0, 1))
    terms = x.shape[0] * x.shape[1]
    return dx, bound, dg, (terms + D + 24) * U * (size * np.abs(n)).sum((0, 1))


def visible(nq, nk, causal):
    """(nq, nk): may query i see key j."""
    if not causal:
        return np.ones((nq, nk), bool)
    return np.arange(nk)[None, :] <= np.arange(nq)[:, None] + (nk - nq)


def attention(q, k, v, see, scale):
    """One head: o, lse and bounds on both for bf16 inputs, fp32 statistics,
    softmax weights and o rounded to bf16.  Masked keys and values take no
    part, whatever they hold."""
    q, k, v = (x.astype(np.float64) for x in (q, k, v))
    k = np.where(see.any(0)[:, None], k, 0)
    v = np.where(see.any(0)[:, None], v, 0)
    s = np.where(see, q @ k.T * scale, -np.inf)
    a = (q.shape[1] + 4) * U * (np.abs(q) @ np.abs(k).T) * scale
    es = np.where(see, a, 0).max(-1, keepdims=True) if see.shape[1] else np.zeros((len(q), 1))
    m = s.max(-1, keepdims=True) if s.shape[1] else np.full((len(q), 1), -np.inf)
    m0 = np.where(np.isfinite(m), m, 0)
    p = np.exp(s - m0)
    l = p.sum(-1, keepdims=True)
    empty = l == 0
    w = p / np.where(empty, 1, l)
    o = w @ v
    with np.errstate(divide="ignore"):
        lse = (m0 + np.log(l))[:, 0]
    top = np.abs(np.where(see, s, 0)).max(-1, keepdims=True) if s.shape[1] else np.zeros((len(q), 1))
    ew = 2 * es + (8 * top + 24) * U                       # of one weight, relative
    eo = (UB + 2 * ew + 2 * s.shape[1] * U) * (w @ np.abs(v)) + UB * np.abs(o)
    el = (ew + s.shape[1] * U)[:, 0] + 8 * U * np.where(empty[:, 0], 0, np.abs(np.where(empty[:, 0], 0, lse)))
    lse = np.where(empty[:, 0], -np.inf, lse)
    return np.where(empty, 0, o), lse, eo, el, w, ew


def attention_grad(do, q, k, v, see, scale):
    """One head: dq, dk, dv and bounds for the same arithmetic, with P and dS
    rounded to bf16 for the second products and delta = sum(do o) taken from
    the o that was rounded to bf16."""
    o, lse, eo, el, w, ew = attention(q, k, v, see, scale)
    do, q, k, v = (x.astype(np.float64) for x in (do, q, k, v))
    D = q.shape[1]
    dp = np.where(see, do @ v.T, 0)
    delta = (do * o).sum(-1, keepdims=True)
    ds = w * (dp - delta)
    edp = (D + 2) * U * (np.abs(do) @ np.abs(v).T)
    edelta = (np.abs(do) * eo).sum(-1, keepdims=True) + (D + 2) * U * (np.abs(do) * np.abs(o)).sum(-1, keepdims=True)
    ew = 2 * ew + 2 * el[:, None]
    eds = w * (edp + edelta) + (UB + ew + 4 * U) * np.abs(ds) + ew * w * (edp + edelta)
    n = max(q.shape[0], k.shape[0]) * U
    dv, dq, dk = w.T @ do, ds @ k * scale, ds.T @ q * scale
    aw, ads = np.abs(w), np.abs(ds) + eds
    edv = ((UB + ew + 2 * n) * aw).T @ np.abs(do) + UB * np.abs(dv)
    edq = ((eds + 2 * n * ads) @ np.abs(k)) * scale + UB * np.abs(dq)
    edk = ((eds + 2 * n * ads).T @ np.abs(q)) * scale + UB * np.abs(dk)
    return (dq, dk, dv), (edq, edk, edv)


def decode(q, k_cache, v_cache, table, length, prefix_pages, prefix_len, page_size, scale):
    """One request and head: o and its bound.  Keys whose page is not in the
    cache take no part."""
    pages = k_cache.shape[0] // page_size
    rows = [(list(prefix_pages), j) for j in range(prefix_len)]
    rows += [(list(table), j) for j in range(max(0, min(int(length), len(table) * page_size)))]
    at = [int(p[j // page_size]) * page_size + j % page_size for p, j in rows if 0 <= p[j // page_size] < pages]
    k, v = k_cache[at], v_cache[at]
    o, _, eo, _, _, _ = attention(q[None, :], k, v, np.ones((1, len(at)), bool), scale)
    return o[0], eo[0]
