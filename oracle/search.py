"""Oracle of the beam search calls and of the 4-bit cache: their definitions in
Python integers and NumPy float64, with bounds on how far the library's
arithmetic may lie from them.  Test infrastructure only."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24
MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


# ---------------------------------------------------------------- choice of continuations
def log_probs(logits):
    """Log softmax of a row over its finite logits, and the bound on a log sum
    exp whose lanes take 16 columns of every 1024 at a time: a term exp(d) is
    off by (3 |d| + 8) U relative (the difference, the exponent's fma and the
    hardware's exponential; exp(0) is 1), and the 16 are added in fp32 in four
    levels of pairs, U each.  All further sums and what scales them are in 64
    bits, off by less than another U."""
    x = np.where(np.isfinite(logits), logits.astype(np.float64), -np.inf)
    m = x.max(initial=-np.inf)
    if m == -np.inf:
        return x, 0.0
    p = np.exp(x - m)
    s = p.sum()
    d = np.where(x > -np.inf, m - x, 0)
    bound = ((p * np.where(d > 0, 3 * d + 8, 0)).sum() / s + 5) * U
    return x - (m + np.log(s)), bound


def select(logits, scores, vocab, keep, done=None, end=-1):
    """logits: (rows, vocab); (parents, tokens, scores, done_after, bound): best
    first, of equal scores the lowest beam, then the largest logit, then the
    lowest token."""
    N, W = scores.shape
    parents, tokens = np.full((N, keep), -1), np.full((N, keep), -1)
    after, done_after = np.full((N, keep), -np.inf), np.zeros((N, keep), bool)
    bound = 0.0
    every = np.full((N, W, vocab), -np.inf)
    for n in range(N):
        for w in range(W):
            if not np.isfinite(scores[n, w]):
                continue
            if done is not None and done[n, w]:
                every[n, w, end] = scores[n, w]
                continue
            lp, b = log_probs(logits[n * W + w, :vocab])
            every[n, w] = float(scores[n, w]) + lp
            bound = max(bound, b)
        flat = every[n].ravel()
        x = logits[n * W : (n + 1) * W, :vocab].astype(np.float64)
        if done is not None:
            x = np.where(done[n][:, None], 0.0, x)
        beam, token = np.divmod(np.arange(W * vocab), vocab)
        order = np.lexsort((token, -x.ravel(), beam, -flat))[:keep]
        for k, at in enumerate(order):
            if flat[at] == -np.inf:
                break
            parents[n, k], tokens[n, k], after[n, k] = n * W + at // vocab, at % vocab, flat[at]
            done_after[n, k] = done is not None and (bool(done[n, at // vocab]) or at % vocab == end)
    return parents, tokens, after, done_after, bound, every


# ---------------------------------------------------------------- pages
def _tokens(n, width, page):
    return max(0, min(int(n), width * page))


def fork(table, lengths, parents, keep, free, used, page, pages, group, width=0):
    """(table_after, lengths_after, copies, n_copies, shared, used_after,
    free_pages); width: of a table without rows."""
    width = len(table[0]) if len(table) else width
    free = [int(x) for x in free]
    used = min(int(used), len(free))                   # more stands for entries that got no page
    before = {int(e) for row, n in zip(table, lengths) for e in row[:-(-_tokens(n, width, page) // page)] if 0 <= e < pages}
    rows, lens = [], []
    for i, p in enumerate(parents):
        n = _tokens(lengths[p], width, page) if 0 <= p < len(table) else 0
        if keep is not None:
            n = max(0, min(n, int(keep[i])))
        lens.append(n)
        rows.append([int(e) for e in table[p][:-(-n // page)]] if n else [])
    held = {e for row in rows for e in row}
    gone = sorted(before - held)
    full = {e for row, n in zip(rows, lens) for e in row[:n // page]}
    copies, writes, own = [], set(full), [list(row) for row in rows]      # own: copies told apart, also where no page is left
    for i, (row, n) in enumerate(zip(rows, lens)):
        if n % page and 0 <= row[-1] < pages:
            if row[-1] in writes:
                k = len(copies)
                at = used + k - len(gone)
                to = gone[k] if k < len(gone) else free[at] if 0 <= at < len(free) else -1
                copies.append((row[-1], to))
                row[-1] = to
                own[i][-1] = "copy %d" % i
            else:
                writes.add(row[-1])
    after = used + len(copies) - len(gone)
    for k, e in enumerate(gone[len(copies):]):
        if 0 <= after + k < len(free):
            free[after + k] = e
    shared = []
    for g in range(len(rows) // group):
        rs, ls = own[g * group:(g + 1) * group], lens[g * group:(g + 1) * group]
        n = min(len(r) for r in rs)
        same = next((j for j in range(n) if any(r[j] != rs[0][j] for r in rs)), None)
        shared.append(min(ls) if same is None else min(min(ls), same * page))
    out = np.full((len(rows), width), -1)
    for i, row in enumerate(rows):
        out[i, :len(row)] = row
    fill = np.full((len(rows), 2), -1)
    if copies:
        fill[:len(copies)] = copies
    return out, np.array(lens, dtype=int), fill, len(copies), np.array(shared, dtype=int), after, np.array(free, dtype=int)


def compact(table, lengths, first, pool, page):
    """(table_after, copies, n_copies, used_after, free_pages)."""
    width = len(table[0]) if len(table) else 0
    rows = [[int(e) for e in row[:-(-_tokens(n, width, page) // page)]] for row, n in zip(table, lengths)]
    live = sorted({e for row in rows for e in row if first <= e < first + pool})
    n, at = len(live), set(live)
    copies = list(zip([e for e in live if e >= first + n], [e for e in range(first, first + n) if e not in at]))
    to = dict(copies)
    out = np.full((len(rows), width), -1)
    for i, row in enumerate(rows):
        out[i, :len(row)] = [to.get(e, e) for e in row]
    fill = np.full((pool // 2, 2), -1)
    if copies:
        fill[:len(copies)] = copies
    return out, fill, len(copies), n, np.arange(first, first + pool)


# ---------------------------------------------------------------- the 4-bit format
def bf16(bits):
    """Values of bf16 bit patterns."""
    return (np.asarray(bits, dtype=np.uint32) << 16).view(np.float32)


def quantise(x):
    """Codes (..., D) and scale bytes (..., D / 32) of rows of finite or other
    bf16 values, by the definition: the least scale with no magnitude above
    seven times it, and the nearest code."""
    with np.errstate(invalid="ignore"):                # (NaN of the signalling kind, on the way to 64 bits)
        b = np.asarray(x, dtype=np.float64).reshape(x.shape[:-1] + (-1, 32))
    bad = ~np.isfinite(b).all(-1)
    a = np.where(bad, 0.0, np.abs(np.where(np.isfinite(b), b, 0)).max(-1))
    scale = np.full(a.shape, 1)
    for s in range(252, 0, -1):                        # the least that does; 252 is the largest there is
        scale = np.where(a <= 7 * 2.0 ** (s - 127), s, scale) if s < 252 else np.full(a.shape, 252)
    y = np.abs(np.where(bad[..., None], 0, np.where(np.isfinite(b), b, 0))) / (2.0 ** (scale.astype(np.float64) - 127))[..., None]
    d = np.abs(y[..., None] - MAGNITUDES)
    even = np.arange(8) % 2 == 0
    code = np.argmin(np.where(even, d, np.nextafter(d, np.inf)), -1)       # halfway: the even one
    code = np.where(y >= 6, 7, code) | (np.signbit(b) << 3)
    return code.reshape(x.shape), np.where(bad, 255, scale)


def values(codes, scales):
    """The values that codes and scale bytes stand for."""
    c = codes.reshape(codes.shape[:-1] + (-1, 32))
    v = MAGNITUDES[c & 7] * np.where(c & 8, -1.0, 1.0) * 2.0 ** (scales.astype(np.float64) - 127)[..., None]
    return np.where((scales == 255)[..., None], np.nan, v).reshape(codes.shape)


def page_of(k, v):
    """The bytes of a page of one head: k, v (page_size, D) bf16 values."""
    out = []
    packed = [quantise(x) for x in (k, v)]
    for codes, _ in packed:
        out.append((codes[..., 0::2] | codes[..., 1::2] << 4).astype(np.uint8).ravel())
    out += [scales.astype(np.uint8).ravel() for _, scales in packed]
    return np.concatenate(out)


def rows_of(page, D):
    """Key and value rows (page_size, D) of the bytes of a page of one head."""
    n = len(page) * 16 // (17 * D)
    codes, scales = page[:n * D].reshape(2, n, D // 2).astype(int), page[n * D:].reshape(2, n, D // 32).astype(int)
    c = np.stack([codes & 15, codes >> 4], -1).reshape(2, n, D)
    return values(c[0], scales[0]), values(c[1], scales[1])
