"""The operators of a beam search over a paged cache, in their plain form and
through the library, over the range of sizes they are used at.

Five operators, the caches and logits spread over P virtual ranks:

  beam     beam_select: the best continuations of every group of beams over
           the vocabulary, whose columns are split over the ranks
  fork     kv_fork, and kv_copy_pages after it: the block table of the chosen
           beams, pages shared, copied and freed
  compact  kv_compact, and kv_copy_pages after it: the pages in use moved to
           the front of the cache
  write    tp_kv4_write, and tp_kv4_read after it: tokens' keys and values to
           the 4-bit cache, and the values that it holds for them
  decode   tp_attention_decode_kv4: one query token per request over the 4-bit
           cache, keys that a group of requests shares read once

`own` chooses the side: False computes with elementary torch operations, in 32
bits or (sums over the vocabulary and the choice between close continuations)
64, True calls the library.
"""
from __future__ import annotations

import math
import random

import torch

own = False


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one sentence, a small vocabulary: what a step costs at least
        dict(name="beam 1 x 4 of 8000", op="beam", N=1, W=4, keep=4, P=4, vocab=8000, f32=True, done=0.0),
        # first step of a batch: every prompt becomes five beams; bf16, odd sizes
        dict(name="beam 37 x 1 to 5 of 50001", op="beam", N=37, W=1, keep=5, P=2, vocab=50001, f32=False, done=0.0),
        # a large batch of beams over a large vocabulary, some of them ended
        dict(name="beam 64 x 8 of 100003", op="beam", N=64, W=8, keep=8, P=8, vocab=100003, f32=True, done=0.1),
        # the beams of a small batch after one step, bf16 cache
        dict(name="fork 8 x 4 of 700", op="fork", N=8, W=4, keep=4, L=700, page=16, P=4, Hkv=2, D=128, kv4=False, cut=False),
        # many beams far into their text, 4-bit cache
        dict(name="fork 128 x 8 of 4000", op="fork", N=128, W=8, keep=8, L=4000, page=16, P=4, Hkv=2, D=128, kv4=True, cut=False),
        # a small cache with holes, bf16
        dict(name="compact 300 pages", op="compact", B=9, L=500, pool=300, page=16, P=2, Hkv=4, D=64, kv4=False),
        # a cache that has shrunk to a third
        dict(name="compact 48000 pages", op="compact", B=200, L=2500, pool=48000, page=32, P=4, Hkv=2, D=128, kv4=True),
        # the tokens of one decode step
        dict(name="write step of 32", op="write", P=4, T=32, Hkv=2, D=128, page=16),
        # a prompt batch, short heads, an odd count
        dict(name="write prompt 16381", op="write", P=4, T=16381, Hkv=4, D=64, page=64),
        # a few short requests
        dict(name="decode 3 of 200", op="decode", P=2, N=3, W=1, L=200, shared=0, Hq=8, Hkv=2, D=64, page=16),
        # beams behind their prompts
        dict(name="decode 24 x 4 of 3000", op="decode", P=4, N=24, W=4, L=3000, shared=2700, Hq=8, Hkv=2, D=128, page=16),
        # few requests with long caches, nothing shared
        dict(name="decode 4 of 120000", op="decode", P=4, N=4, W=1, L=120000, shared=0, Hq=8, Hkv=2, D=128, page=64),
    ]


def _log(rng, lo, hi):
    """A size between lo and hi, spread over its logarithm; off the multiples of 1024 by one."""
    n = max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    return n - 1 if n % 1024 == 0 and n > lo else n


def draw(rng):
    op = rng.choice(["beam", "beam", "fork", "compact", "write", "decode", "decode", "decode"])
    top = max(work(c)["bytes"] for c in listed() if c["op"] == op), max(work(c)["flops"] for c in listed() if c["op"] == op)
    while True:
        P, Hkv, D, page = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 1, 2, 3, 4, 8]), rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
        if op == "beam":
            W = rng.choice([1, 1, 2, 3, 4, 6, 8, 16])
            c = dict(op=op, N=_log(rng, 1, 200), W=W, keep=rng.choice([W, W, 2 * W, 5]), P=P, vocab=_log(rng, 100, 200000),
                     f32=rng.random() < 0.6, done=rng.choice([0.0, 0.0, 0.2]))
        elif op == "fork":
            W = rng.choice([1, 2, 3, 4, 8])
            c = dict(op=op, N=_log(rng, 1, 200), W=W, keep=rng.choice([W, W, W, 2 * W]), L=_log(rng, 1, 5000), page=page, P=P,
                     Hkv=Hkv, D=D, kv4=rng.random() < 0.5, cut=rng.random() < 0.3)
        elif op == "compact":
            B, L = _log(rng, 1, 300), _log(rng, 1, 5000)
            c = dict(op=op, B=B, L=L, pool=int(B * -(-L // page) * rng.uniform(1.1, 4.0)) + 2, page=page, P=P, Hkv=Hkv, D=D,
                     kv4=rng.random() < 0.5)
        elif op == "write":
            c = dict(op=op, P=P, T=_log(rng, 1, 30000), Hkv=Hkv, D=D, page=page)
        else:
            W, L = rng.choice([1, 1, 1, 2, 4, 5, 8, 16]), _log(rng, 1, 100000)
            c = dict(op=op, P=P, N=_log(rng, 1, 100), W=W, L=L, shared=int(L * rng.random()) if W > 1 else 0,
                     Hq=Hkv * rng.choice([1, 2, 3, 4, 5, 8, 16]), Hkv=Hkv, D=D, page=page)
            if c["P"] * c["N"] * W * L * Hkv * D > (1 << 30):
                continue
        if op in ("fork", "compact") and _pool(c) * _page_bytes(c) * P > (8 << 30):
            continue
        w = work(c)
        if w["bytes"] <= top[0] and w["flops"] <= top[1]:
            return c


# ---------------------------------------------------------------- sizes and lengths (the case's own)
def _width(c):
    """Columns of one rank: its share of the vocabulary, padded as the products that make logits need it."""
    return -(-c["vocab"] // (128 * c["P"])) * 128


def _fork_lens(c):
    """Tokens of each group's beams before the step, and those it keeps (all, but for `cut`)."""
    r = random.Random(c["L"] * 131 + c["N"])
    lens = [max(1, min(c["L"], int(c["L"] * r.uniform(0.4, 1.1)))) for _ in range(c["N"])]
    return lens, [n - min(n - 1, r.randrange(0, 9)) if c["cut"] else n for n in lens]


def _compact_lens(c):
    r = random.Random(c["L"] * 137 + c["B"])
    return [int(c["L"] * r.uniform(0.0, 1.0)) for _ in range(c["B"])]


def _decode_lens(c):
    """Each request's tokens, and how many of them its group shares."""
    r = random.Random(c["L"] * 139 + c["N"])
    lens, shared = [], []
    for _ in range(c["N"]):
        n = max(1, min(c["L"], int(c["L"] * r.uniform(0.4, 1.1))))
        shared.append(n * c["shared"] // c["L"] if c["W"] > 1 else 0)
        lens += [n] * c["W"]
    return lens, shared


def _pages(n, page):
    return -(-n // page)


def _pool(c):
    """Pages of the case's cache."""
    if c["op"] == "compact":
        return c["pool"]
    lens, _ = _fork_lens(c)
    return sum(c["W"] * _pages(n, c["page"]) for n in lens) + c["N"] * c["keep"] + 40


def _page_bytes(c):
    """Bytes of one page of one rank, keys and values."""
    values = c["page"] * c["Hkv"] * c["D"]
    return values * 17 // 16 if c["kv4"] else 4 * values


def work(c):
    op = c["op"]
    if op == "beam":
        rows = c["N"] * c["W"]
        live = rows - int(rows * c["done"])
        return dict(bytes=live * c["vocab"] * (4 if c["f32"] else 2) + 4 * rows + 12 * c["N"] * c["keep"], flops=0)
    if op == "fork":
        before, after = _fork_lens(c)
        old, new = (sum(_pages(n, c["page"]) for n in x) for x in (before, after))
        copies = sum((c["keep"] - 1) // 2 for n in after if n % c["page"])       # about every second beam's last page
        return dict(bytes=4 * (c["W"] * old + c["keep"] * new) + 2 * copies * c["P"] * _page_bytes(c), flops=0)
    if op == "compact":
        held = sum(_pages(n, c["page"]) for n in _compact_lens(c))
        moves = held * (c["pool"] - held) // c["pool"]                         # of pages anywhere in the pool
        return dict(bytes=8 * held + 4 * c["pool"] + 2 * moves * c["P"] * _page_bytes(c), flops=0)
    if op == "write":
        n = 2 * c["P"] * c["T"] * c["Hkv"] * c["D"]
        return dict(bytes=4 * n + 2 * (n * 17 // 32) + 16 * c["T"], flops=0)      # in, to the cache; from it, out
    lens, shared = _decode_lens(c)
    keys = sum(shared) + sum(n - shared[b // c["W"]] for b, n in enumerate(lens))
    return dict(bytes=c["P"] * (keys * c["Hkv"] * c["D"] * 17 // 16 + 4 * len(lens) * c["Hq"] * c["D"]) +
                4 * sum(_pages(n, c["page"]) for n in lens), flops=4 * c["P"] * sum(lens) * c["Hq"] * c["D"])


# ---------------------------------------------------------------- the 4-bit cache in elementary operations
# Blocks of 32 values along a head row: 2^e times a sign and one of the eight
# magnitudes, e the least with every value of the block at most 7 times 2^e,
# each value rounded to the nearest (halfway: the even code).  A page of one
# head is one run of bytes: key codes (two a byte, the even value low), value
# codes, key scales (e + 127), value scales.
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _pack(x):
    """Codes (..., D / 2) and scales (..., D / 32) of rows x (..., D)."""
    b = x.float().unflatten(-1, (-1, 32))
    m, e = torch.frexp(b.abs().amax(-1))               # amax = m 2^e, 0.5 <= m < 1; 7 is 0.875 times 8
    e = torch.where(m == 0, -126, (e - 3 + (m > 0.875).int()).clamp(min=-126))
    y = torch.ldexp(b, -e[..., None]).abs()            # exact: powers of two
    code = (y > 0.25).byte()
    for half, up in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (y >= half) if up else (y > half)
    code = (code | (torch.signbit(b).byte() << 3)).flatten(-2)
    return code[..., 0::2] | code[..., 1::2] << 4, (e + 127).to(torch.uint8)


def _unpack(codes, scales):
    """The rows (..., D) that they stand for, fp32."""
    table = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=codes.device)
    x = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1).flatten(-2).unflatten(-1, (-1, 32))
    return torch.ldexp(x, scales.int()[..., None] - 127).flatten(-2)


def _parts(cache, page, D):
    """Views of one rank's cache (pages, Hkv, bytes): key codes, value codes, key scales, value scales, each (pages, Hkv, page, .)."""
    n = page * D // 2
    kc, vc, ks, vs = cache.split([n, n, page * D // 32, page * D // 32], dim=2)
    return tuple(x.unflatten(2, (page, -1)) for x in (kc, vc, ks, vs))


# ---------------------------------------------------------------- inputs
def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _new(*shape, dtype=torch.int32):
    return torch.empty(shape, dtype=dtype, device="cuda")


def _caches(c, pages, g):
    """Caches of P ranks with something in every page: bf16 keys and values, or 4-bit pages."""
    P, H, D, page = c["P"], c["Hkv"], c["D"], c["page"]
    if c["kv4"]:
        return [torch.randint(0, 256, (pages, H, page * D * 17 // 16), generator=g, device="cuda", dtype=torch.uint8) for _ in range(P)]
    return [torch.randn(pages * page, H, D, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2 * P)]


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    bf, op = torch.bfloat16, c["op"]
    s = dict(case=c)

    def normal(*shape, dtype=bf, std=1.0):
        x = torch.empty(shape, dtype=dtype, device="cuda")
        for part in x:                         # rank by rank: little scratch memory
            part.copy_(torch.randn(part.shape, generator=g, device="cuda") * std)
        return x

    if op == "beam":
        N, W, K, P = c["N"], c["W"], c["keep"], c["P"]
        rows = N * W
        x = normal(P, rows, _width(c), dtype=torch.float32 if c["f32"] else bf, std=2.5)
        scores = -torch.rand(N, W, generator=g, device="cuda").cumsum(1) * 3 - 5       # best first
        done = torch.zeros(rows, dtype=torch.bool, device="cuda")
        done[torch.randperm(rows, generator=g, device="cuda")[:int(rows * c["done"])]] = True
        s.update(logits=list(x.unbind(0)), scores=scores, done=done.view(N, W) if c["done"] else None, end=c["vocab"] // 3,
                 parents=_new(N, K), tokens=_new(N, K), after=_new(N, K, dtype=torch.float32),
                 done_after=_new(N, K, dtype=torch.bool) if c["done"] else None)
        return s
    if op == "fork":
        N, W, K, page = c["N"], c["W"], c["keep"], c["page"]
        lens, kept = _fork_lens(c)
        pages, width = _pool(c), _pages(max(lens), page) + 2
        free = torch.randperm(pages, generator=g, device="cuda").int()
        # every group's beams share two thirds of their pages; the rest is their own
        n = torch.tensor([_pages(x, page) for x in lens], device="cuda")
        j = torch.arange(width, device="cuda")
        row = torch.arange(N * W, device="cuda")
        common = (n * 2 // 3)[row // W][:, None]
        first = (row // W * W)[:, None]
        held = j < n[row // W][:, None]
        takes = held & ((j >= common) | (row[:, None] == first))
        at = (takes.flatten().cumsum(0) - 1).view(N * W, width)
        at = torch.where(j < common, at[first[:, 0]], at)
        table = torch.where(held, free[at.clamp(min=0)], -1).int()
        used = takes.sum().int().view(1)
        parents = torch.randint(0, W, (N, K), generator=g, device="cuda").int() + _i32(list(range(0, N * W, W)))[:, None]
        s.update(table=table, lengths=_i32([x for x in lens for _ in range(W)]), parents=parents, free=free, used=used,
                 keep=_i32([x for x in kept for _ in range(K)]) if c["cut"] else None, pages=pages,
                 table_after=_new(N * K, width), lengths_after=_new(N * K), shared=_new(N), copies=_new(N * K, 2), n_copies=_new(1),
                 used_after=_new(1), caches=_caches(c, pages, g))
        return s
    if op == "compact":
        page, pages = c["page"], c["pool"]
        lens = _compact_lens(c)
        n = [_pages(x, page) for x in lens]
        width = max(n) + 1
        pool = torch.randperm(pages, generator=g, device="cuda").int()
        table = torch.full((c["B"], width), -1, dtype=torch.int32, device="cuda")
        held = torch.arange(width, device="cuda") < _i32(n)[:, None]
        table[held] = pool[:sum(n)]
        s.update(table=table, lengths=_i32(lens), free=pool.clone(), pages=pages, table_after=_new(c["B"], width),
                 copies=_new(pages // 2, 2), n_copies=_new(1), used_after=_new(1), caches=_caches(c, pages, g))
        return s
    P, Hkv, D, page = c["P"], c["Hkv"], c["D"], c["page"]
    size = page * D * 17 // 16
    if op == "write":
        T = c["T"]
        pages = _pages(T, page) + 5
        t = torch.arange(T, device="cuda")
        order = torch.randperm(pages, generator=g, device="cuda")
        # heads of different sizes, a few channels far above the others
        std = torch.exp(torch.randn(D, generator=g, device="cuda"))
        s.update(k=list((normal(P, T, Hkv, D) * std.to(bf)).unbind(0)), v=list(normal(P, T, Hkv, D).unbind(0)),
                 slots=order[t // page] * page + t % page, cache=[torch.zeros(pages, Hkv, size, dtype=torch.uint8, device="cuda") for _ in range(P)],
                 k_read=list(_new(P, T, Hkv, D, dtype=bf).unbind(0)), v_read=list(_new(P, T, Hkv, D, dtype=bf).unbind(0)))
        return s
    lens, shared = _decode_lens(c)
    B, W = len(lens), c["W"]
    width = _pages(max(lens), page)
    # groups hold whole shared pages in common, the rest page by page
    n = _i32([_pages(x, page) for x in lens])[:, None]
    whole = _i32([x // page for x in shared]).repeat_interleave(W)[:, None]
    j, row = torch.arange(width, device="cuda"), torch.arange(B, device="cuda")
    first = row // W * W
    takes = (j < n) & ((j >= whole) | (row == first)[:, None])
    at = (takes.flatten().cumsum(0) - 1).view(B, width)
    at = torch.where(j < whole, at[first], at)
    pages = sum(_pages(x, page) for x in lens) - sum((W - 1) * (x // page) for x in shared) + 3
    table = torch.where(j < n, torch.randperm(pages, generator=g, device="cuda").int()[at.clamp(min=0)], 0).int()
    cache = []
    for _ in range(P):
        x = torch.empty(pages, Hkv, size, dtype=torch.uint8, device="cuda")
        kc, vc, ks, vs = _parts(x, page, D)
        step = max(1, (1 << 25) // (Hkv * page * D))
        for p in range(0, pages, step):                # a part of the pages at a time: little scratch memory
            shape = kc[p:p + step].shape[:3] + (D,)
            for codes, scales in ((kc, ks), (vc, vs)):
                a, b = _pack(torch.randn(shape, generator=g, device="cuda").to(bf))
                codes[p:p + step], scales[p:p + step] = a, b
        cache.append(x)
    sharp = torch.linspace(0.5, 2.5, c["Hq"], device="cuda")[:, None]
    s.update(q=list((normal(P, B, c["Hq"], D) * sharp.to(bf)).unbind(0)), cache=cache, table=table, lengths=_i32(lens),
             shared=_i32([x // page * page for x in shared]) if W > 1 else None, o=list(_new(P, B, c["Hq"], D, dtype=bf).unbind(0)))
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    return (_RUN_OWN if own else _RUN_PLAIN)[s["case"]["op"]](s)


# the library ------------------------------------------------------------
def _own_beam(s):
    from ring_collectives_amd import search as S
    s["ws"] = S.beam_select(s["logits"], s["scores"], s["parents"], s["tokens"], s["after"], vocab=s["case"]["vocab"],
                            done=s["done"], done_after=s["done_after"], end_token=s["end"], ws=s.get("ws"))
    return {k: s[k] for k in ("parents", "tokens", "after", "done_after")}


def _own_fork(s):
    from ring_collectives_amd import search as S
    c = s["case"]
    s["ws"] = S.kv_fork(s["table"], s["lengths"], s["parents"], s["free"], s["used"], s["table_after"], s["lengths_after"],
                        s["copies"], s["n_copies"], s["used_after"], page_size=c["page"], pages=s["pages"], keep=s["keep"],
                        shared=s["shared"], group=c["keep"], ws=s.get("ws"))
    S.kv_copy_pages(s["caches"], s["copies"], s["n_copies"], pages=s["pages"])
    return {k: s[k] for k in ("table_after", "lengths_after", "shared", "copies", "n_copies", "used_after", "free", "caches")}


def _own_compact(s):
    from ring_collectives_amd import search as S
    s["ws"] = S.kv_compact(s["table"], s["lengths"], s["table_after"], s["free"], s["copies"], s["n_copies"], s["used_after"],
                           page_size=s["case"]["page"], ws=s.get("ws"))
    S.kv_copy_pages(s["caches"], s["copies"], s["n_copies"], pages=s["pages"])
    return {k: s[k] for k in ("table_after", "copies", "n_copies", "used_after", "free", "caches")}


def _own_write(s):
    from ring_collectives_amd import search as S
    page = s["case"]["page"]
    S.tp_kv4_write(s["k"], s["v"], s["cache"], s["slots"], page_size=page)
    S.tp_kv4_read(s["cache"], s["slots"], s["k_read"], s["v_read"], page_size=page)
    return dict(k=s["k_read"], v=s["v_read"])


def _own_decode(s):
    from ring_collectives_amd import search as S
    c = s["case"]
    s["ws"] = S.tp_attention_decode_kv4(s["q"], s["cache"], s["o"], s["table"], s["lengths"], page_size=c["page"],
                                        shared=s["shared"], group=c["W"], ws=s.get("ws"))
    return s["o"]


# elementary operations --------------------------------------------------
def _plain_beam(s):
    c = s["case"]
    N, W, K, V = c["N"], c["W"], c["keep"], c["vocab"]
    x = torch.cat(s["logits"], 1)[:, :V].double()
    m = x.amax(1, keepdim=True)
    x = x.sub_(m + (x - m).exp_().sum(1, keepdim=True).log_()).view(N, W, V).add_(s["scores"].double()[:, :, None])
    if s["done"] is not None:                          # an ended beam goes on as itself, and nothing else
        x.masked_fill_(s["done"][:, :, None], -math.inf)
        x[:, :, s["end"]] = torch.where(s["done"], s["scores"].double(), x[:, :, s["end"]])
    x = x.view(N, W * V)
    place = torch.arange(W * V, device="cuda")
    picks, best = [], []
    for _ in range(K):                                 # the best of what is left, the first of equals
        top = x.amax(1, keepdim=True)
        at = torch.where(x == top, place, W * V).amin(1, keepdim=True)
        at = torch.where(top > -math.inf, at, -1)
        picks.append(at)
        best.append(top)
        x.scatter_(1, at.clamp(min=0), -math.inf)
    at, best = torch.cat(picks, 1), torch.cat(best, 1)
    w = at // V
    out = dict(parents=torch.where(at >= 0, w + torch.arange(0, N * W, W, device="cuda")[:, None], -1).int(),
               tokens=torch.where(at >= 0, at % V, -1).int(), after=best.float(), done_after=None)
    if s["done"] is not None:
        out["done_after"] = (s["done"].gather(1, w.clamp(min=0)) | (out["tokens"] == s["end"])) & (at >= 0)
    return out


def _plain_copy(caches, copies, pages):
    src, dst = copies[:, 0].long(), copies[:, 1].long()
    for x in caches:
        x = x.view(pages, -1)
        ok = (src >= 0) & (dst >= 0)
        # what is no copy writes a page of the first copy again (page 0 onto itself if there is none)
        a = torch.where(ok, src, torch.where(ok[:1], src[:1], 0))
        b = torch.where(ok, dst, torch.where(ok[:1], dst[:1], 0))
        for i in range(0, a.numel(), 8192):
            x[b[i:i + 8192]] = x[a[i:i + 8192]]


def _plain_fork(s):
    c = s["case"]
    page, M, free = c["page"], s["pages"], s["free"]
    table, lengths, parents = s["table"].long(), s["lengths"].long(), s["parents"].flatten().long()
    width, rows = table.shape[1], parents.numel()
    j, row = torch.arange(width, device="cuda"), torch.arange(rows, device="cuda")
    n = torch.where(parents >= 0, lengths[parents.clamp(min=0)], 0)
    if s["keep"] is not None:
        n = torch.minimum(n, s["keep"].long())
    new = torch.where(j < (-(-n // page))[:, None], table[parents.clamp(min=0)], -1)

    def mark(pages, where):
        out = torch.zeros(M + 1, dtype=torch.bool, device="cuda")
        out[torch.where(where & (pages >= 0) & (pages < M), pages, M)] = True
        return out

    old = mark(table, j < (-(-lengths // page))[:, None])
    full = mark(new, j < (n // page)[:, None])
    at = (n // page).clamp(max=width - 1)              # the partly filled last page of each row
    last = new.gather(1, at[:, None])[:, 0]
    last = torch.where((n % page > 0) & (last >= 0) & (last < M), last, M)
    owner = torch.full((M + 1,), rows, device="cuda").scatter_reduce_(0, last, row, "amin")
    copy = (last < M) & (full[last] | (owner[last] != row))
    freed = (old & ~full & (owner == rows))[:M]
    k, f = copy.cumsum(0) - 1, freed.cumsum(0) - 1
    n_copies, n_freed, used = copy.sum(), freed.sum(), s["used"].long()
    ids = torch.full((M + 1,), -1, device="cuda").scatter_(0, torch.where(freed, f, M), torch.arange(M, device="cuda"))
    entry = used + k - n_freed
    taken = torch.where(entry < free.numel(), free[entry.clamp(0, free.numel() - 1)].long(), -1)
    dst = torch.where(k < n_freed, ids[k.clamp(0, M)], taken)
    new.scatter_(1, at[:, None], torch.where(copy, dst, new.gather(1, at[:, None])[:, 0])[:, None])
    copies = torch.full((rows + 1, 2), -1, device="cuda")
    copies[torch.where(copy, k, rows)] = torch.stack([last, dst], 1)
    back = torch.arange(M, device="cuda")              # freed pages that no copy took, below the first free entry
    to = torch.where((back >= n_copies) & (back < n_freed), used - n_freed + back, free.numel())
    spare = torch.cat([free.long(), free.new_zeros(1).long()])
    spare[to] = ids[:M]
    free.copy_(spare[:-1])
    s["table_after"].copy_(new)
    groups, K = new.view(c["N"], c["keep"], width), c["keep"]
    same = (groups == groups[:, :1]).all(1)
    common = torch.where(same, width, j).amin(1) * page
    out = dict(table_after=s["table_after"], lengths_after=n.int(), shared=torch.minimum(common, n.view(-1, K).amin(1)).int(),
               copies=copies[:rows].int(), n_copies=n_copies.int().view(1), used_after=(used + n_copies - n_freed).int(), free=free,
               caches=s["caches"])
    _plain_copy(s["caches"], out["copies"], M)
    return out


def _plain_compact(s):
    page, M = s["case"]["page"], s["pages"]
    table = s["table"].long()
    held = torch.arange(table.shape[1], device="cuda") < (-(-s["lengths"] // page))[:, None]
    live = torch.zeros(M + 1, dtype=torch.bool, device="cuda")
    live[torch.where(held & (table >= 0) & (table < M), table, M)] = True
    live = live[:M]
    n, at = live.sum(), torch.arange(M, device="cuda")
    move, hole = live & (at >= n), ~live & (at < n)
    k, h = move.cumsum(0) - 1, hole.cumsum(0) - 1
    holes = torch.full((M + 1,), -1, device="cuda").scatter_(0, torch.where(hole, h, M), at)
    to = torch.where(move, holes[k.clamp(min=0)], at)
    copies = torch.full((M // 2 + 1, 2), -1, device="cuda")
    copies[torch.where(move, k, M // 2)] = torch.stack([at, to], 1)
    copies[M // 2] = -1
    table = torch.where(held, torch.where((table >= 0) & (table < M), to[table.clamp(0, M - 1)], table), -1)
    s["free"].copy_(at)
    _plain_copy(s["caches"], copies, M)
    return dict(table_after=table.int(), copies=copies[:M // 2].int(), n_copies=move.sum().int().view(1), used_after=n.int().view(1),
                free=s["free"], caches=s["caches"])


def _plain_write(s):
    c = s["case"]
    page, D = c["page"], c["D"]
    p, i = s["slots"] // page, s["slots"] % page
    out = dict(k=[], v=[])
    for r in range(c["P"]):
        kc, vc, ks, vs = _parts(s["cache"][r], page, D)
        for name, codes, scales in (("k", kc, ks), ("v", vc, vs)):
            a, b = _pack(s[name][r])
            codes[p, :, i], scales[p, :, i] = a, b
            out[name].append(_unpack(codes[p, :, i], scales[p, :, i]).to(torch.bfloat16))
    return out


def _plain_decode(s):
    c = s["case"]
    Hq, Hkv, D, page = c["Hq"], c["Hkv"], c["D"], c["page"]
    G, B = Hq // Hkv, s["table"].shape[0]
    dead = torch.arange(s["table"].shape[1] * page, device="cuda") >= s["lengths"][:, None]      # (B, L)
    out = []
    for r in range(c["P"]):
        o = []
        q = s["q"][r].float().view(B, Hkv, G, D) / math.sqrt(D)
        step = max(1, (1 << 28) // (dead.shape[1] * Hkv * D))          # requests at a time: little scratch memory
        for b in range(0, B, step):
            kc, vc, ks, vs = _parts(s["cache"][r][s["table"][b:b + step].long()].flatten(0, 1), page, D)
            n = q[b:b + step].shape[0]

            def keys(codes, scales):                    # (n width, Hkv, page, .) -> (n, Hkv, L, D)
                return _unpack(codes, scales).view(n, -1, Hkv, page, D).transpose(1, 2).reshape(n, Hkv, -1, D)

            x = (q[b:b + step] @ keys(kc, ks).transpose(-1, -2)).masked_fill_(dead[b:b + step, None, None, :], -math.inf)
            p = x.sub_(x.amax(-1, keepdim=True)).exp_()
            o.append((p / p.sum(-1, keepdim=True)) @ keys(vc, vs))
        out.append(torch.cat(o).to(torch.bfloat16).view(B, Hq, D))
    return out


_RUN_OWN = dict(beam=_own_beam, fork=_own_fork, compact=_own_compact, write=_own_write, decode=_own_decode)
_RUN_PLAIN = dict(beam=_plain_beam, fork=_plain_fork, compact=_plain_compact, write=_plain_write, decode=_plain_decode)


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_beam(c, s):
    N, W, K, V = c["N"], c["W"], c["keep"], c["vocab"]
    parents, tokens, after = [], [], []
    for n in range(N):
        rows = []
        for w in range(W):
            if s["done"] is not None and bool(s["done"][n, w]):
                lp = torch.full((V,), -math.inf, dtype=torch.float64, device="cuda")
                lp[s["end"]] = 0.0
            else:
                lp = torch.log_softmax(torch.cat([x[n * W + w] for x in s["logits"]])[:V].double(), 0)
            rows.append(lp + s["scores"][n, w].double())
        best, at = torch.sort(torch.cat(rows), descending=True, stable=True)
        best, at = best[:K], at[:K]
        short = K - best.numel()                       # fewer continuations than places
        best = torch.cat([best, best.new_full((short,), -math.inf)])
        at = torch.cat([at, at.new_full((short,), -1)])
        at = torch.where(best > -math.inf, at, -1)
        after.append(best)
        parents.append(torch.where(at >= 0, n * W + at // V, -1))
        tokens.append(torch.where(at >= 0, at % V, -1))
    out = dict(parents=torch.stack(parents).int(), tokens=torch.stack(tokens).int(), after=torch.stack(after), done_after=None)
    if s["done"] is not None:
        was = s["done"].flatten()[out["parents"].long().clamp(min=0)]
        out["done_after"] = (out["parents"] >= 0) & (was | (out["tokens"] == s["end"]))
    return out


def _exact_values(x):
    """Every value of rows x replaced by the nearest one that its block can hold."""
    x = x.double()
    b = x.unflatten(-1, (-1, 32))
    a = b.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(torch.where(a > 0, a, 1.0) / 7.0))       # the least e with a <= 7 2^e, up to a rounding
    e = torch.where(a > 7.0 * torch.exp2(e), e + 1, torch.where(a <= 7.0 * torch.exp2(e - 1), e - 1, e))
    unit = torch.exp2(e)
    grid = torch.tensor(MAGNITUDES, dtype=torch.float64, device="cuda")
    y = b.abs() / unit
    up = torch.searchsorted(grid, y.contiguous()).clamp(max=7)
    down = (up - 1).clamp(min=0)
    high, low = grid[up] - y, y - grid[down]
    code = torch.where((high < low) | ((high == low) & (up % 2 == 0)), up, down)
    code = torch.where(y > 6, 7, code)
    return (torch.copysign(grid[code], b) * unit).flatten(-2)


def _exact_copies(caches, copies, pages):
    """The caches (floating ones in 64 bits) after the copies, one after the other."""
    out = []
    for x in caches:
        y = (x.double() if x.is_floating_point() else x.clone()).view(pages, -1)
        for a, b in copies:
            y[b] = y[a]
        out.append(y.view(x.shape))
    return out


def _exact_fork(c, s):
    """Page by page, with counts of who holds what."""
    page = c["page"]
    table, lengths, free, used = s["table"].tolist(), s["lengths"].tolist(), s["free"].tolist(), s["used"].item()
    kept = s["keep"].tolist() if s["keep"] is not None else None
    new, lens, shared, copies = [], [], [], []
    for i, p in enumerate(s["parents"].flatten().tolist()):
        lens.append(min(lengths[p], kept[i]) if kept else lengths[p])
        new.append(table[p][:_pages(lens[i], page)])
    before = {x for row, n in zip(table, lengths) for x in row[:_pages(n, page)]}
    gone = sorted(before - {x for row in new for x in row})
    spare = gone + free[used:]
    written = {x for row, n in zip(new, lens) for x in row[:n // page]}       # pages that are full for some row
    for row, n in zip(new, lens):
        if n % page:
            if row[-1] in written:
                copies.append((row[-1], spare[len(copies)]))
                row[-1] = copies[-1][1]
            else:
                written.add(row[-1])                                    # the first to go on writing in it
    left = gone[len(copies):]
    after = used + len(copies) - len(gone)
    free[after:after + len(left)] = left
    for g in range(c["N"]):
        rows = new[g * c["keep"]:(g + 1) * c["keep"]]
        n = 0
        while all(n < len(row) and row[n] == rows[0][n] for row in rows):
            n += 1
        shared.append(min([n * page] + lens[g * c["keep"]:(g + 1) * c["keep"]]))
    width, fill = s["table"].shape[1], [(-1, -1)] * (len(new) - len(copies))
    return dict(table_after=_i32([row + [-1] * (width - len(row)) for row in new]), lengths_after=_i32(lens), shared=_i32(shared),
                copies=_i32(copies + fill), n_copies=_i32([len(copies)]), used_after=_i32([after]), free=_i32(free),
                caches=_exact_copies(s["caches"], copies, s["pages"]))


def _exact_compact(c, s):
    page, pages = c["page"], c["pool"]
    rows = [row[:_pages(n, page)] for row, n in zip(s["table"].tolist(), s["lengths"].tolist())]
    live = sorted({x for row in rows for x in row})
    n, at = len(live), set(live)
    copies = list(zip([x for x in live if x >= n], [x for x in range(n) if x not in at]))
    to = dict(copies)
    width, fill = s["table"].shape[1], [(-1, -1)] * (pages // 2 - len(copies))
    return dict(table_after=_i32([[to.get(x, x) for x in row] + [-1] * (width - len(row)) for row in rows]),
                copies=_i32(copies + fill), n_copies=_i32([len(copies)]), used_after=_i32([n]), free=_i32(list(range(pages))),
                caches=_exact_copies(s["caches"], copies, pages))


def exact(c, seed):
    op = c["op"]
    s = prepare(c, seed)
    if op == "fork":
        return _exact_fork(c, s)
    if op == "compact":
        return _exact_compact(c, s)
    if op == "beam":
        return _exact_beam(c, s)
    if op == "write":
        return dict(k=[_exact_values(x) for x in s["k"]], v=[_exact_values(x) for x in s["v"]])
    P, Hq, Hkv, D, page = c["P"], c["Hq"], c["Hkv"], c["D"], c["page"]
    G = Hq // Hkv
    lens, _ = _decode_lens(c)
    pair = torch.tensor([[m * f for m in MAGNITUDES] for f in (1, -1)], dtype=torch.float64, device="cuda").flatten()
    byte = torch.arange(256, device="cuda")
    pair = torch.stack([pair[byte % 16], pair[byte // 16]], 1)        # the two values of a byte
    out = []
    for r in range(P):
        o = torch.empty(len(lens), Hq, D, dtype=torch.float64, device="cuda")
        flat = s["cache"][r]
        for b, n in enumerate(lens):
            j = torch.arange(n, device="cuda")
            at, i = s["table"][b].long()[j // page], j % page
            for h in range(Hkv):
                rows = []
                for which in (0, 1):                   # keys, values
                    codes = which * page * D // 2 + i[:, None] * (D // 2) + torch.arange(D // 2, device="cuda")
                    scale = page * D + which * page * D // 32 + i[:, None] * (D // 32) + torch.arange(D // 32, device="cuda")
                    x = pair[flat[at[:, None], h, codes].long()].view(n, D // 32, 32)
                    rows.append((x * torch.exp2(flat[at[:, None], h, scale].double() - 127)[:, :, None]).view(n, D))
                q = s["q"][r][b, h * G:(h + 1) * G].double()
                o[b, h * G:(h + 1) * G] = torch.softmax(q @ rows[0].t() * D ** -0.5, -1) @ rows[1]
        out.append(o)
    return out
