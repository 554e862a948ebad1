"""The attention operators of the tensor-parallel layer, in their plain form
and through the library, over the range of sizes they are used at.

Five operators, each over P virtual ranks (a rank holds its own heads):

  plan    kv_plan: the block table, cache slots and positions of the tokens
          that a batch of requests adds to a paged key/value cache
  rope    tp_qk_norm_rope: RMS norm of every query and key head, the position
          rotation and the cache write, from one projected row per token
  ropeg   tp_qk_norm_rope_grad: its gradient
  attn    tp_attention, and with "train" tp_attention_grad after it: attention
          over packed prompts of different lengths with grouped heads
  decode  tp_attention_decode: one query token per request over the paged
          cache, with a prefix that all requests share

`own` chooses the side: False computes with elementary torch operations in
32 bits, True calls the library.
"""
from __future__ import annotations

import math
import random

import torch

own = False

EPS = 1e-6


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step of a small batch: every request adds one token
        dict(name="plan step of 24", op="plan", B=24, T=24, page=16, past=700),
        # admission of many prompts at once, continuing requests among them
        dict(name="plan prompts of 1500", op="plan", B=1500, T=200001, page=64, past=900),
        # the new tokens of one decode step, written to the cache (fp32 product
        # of the fused all-gather + GEMM)
        dict(name="rope step of 32", op="rope", P=4, T=32, Hq=8, Hkv=2, D=128, rot=128, f32=True,
             cache=True, keep=False, page=16),
        # a whole prompt batch, to the cache and to the prompt attention
        dict(name="rope prompt 8192", op="rope", P=4, T=8192, Hq=8, Hkv=2, D=128, rot=128, f32=True,
             cache=True, keep=True, page=64),
        # a training batch with short heads, part of each head rotated, odd count
        dict(name="rope grad 4097", op="ropeg", P=4, T=4097, Hq=8, Hkv=8, D=64, rot=32, f32=False),
        # a handful of short prompts of odd lengths
        dict(name="prompts 5 of 400", op="attn", P=2, B=5, T=403, past=0, Hq=4, Hkv=2, D=64,
             causal=True, train=False, packed=False),
        # a batch of ordinary prompts, packed
        dict(name="prompts 12 of 8192", op="attn", P=4, B=12, T=8192, past=0, Hq=8, Hkv=2, D=128,
             causal=True, train=False, packed=False),
        # one long prompt
        dict(name="prompt of 16384", op="attn", P=4, B=1, T=16384, past=0, Hq=4, Hkv=1, D=128,
             causal=True, train=False, packed=False),
        # training on packed samples of different lengths, short heads
        dict(name="train 9 of 2999", op="attn", P=4, B=9, T=2999, past=0, Hq=4, Hkv=4, D=64,
             causal=True, train=True, packed=True),
        # training on one long sample
        dict(name="train 1 of 8192", op="attn", P=4, B=1, T=8192, past=0, Hq=8, Hkv=2, D=128,
             causal=True, train=True, packed=False),
        # few requests with long caches, nothing shared
        dict(name="decode 4 of 60000", op="decode", P=4, B=4, L=60000, prefix=0, Hq=8, Hkv=2, D=128, page=16),
        # a batch of requests behind one long system prompt
        dict(name="decode 64 on 8192", op="decode", P=4, B=64, L=700, prefix=8192, Hq=8, Hkv=2, D=128, page=64),
    ]


def _log(rng, lo, hi):
    """A size between lo and hi, spread over its logarithm; off the multiples of 1024 by one."""
    n = max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    return n - 1 if n % 1024 == 0 and n > lo else n


def draw(rng):
    op = rng.choice(["plan", "rope", "ropeg", "attn", "attn", "train", "decode", "decode"])
    top = {}
    for c in listed():
        w = work(c)
        k = "train" if c.get("train") else c["op"]
        for f in ("bytes", "flops"):
            top[k, f] = max(top.get((k, f), 0), w[f])
    while True:
        P = rng.choice([1, 2, 3, 4, 8])
        Hkv = rng.choice([1, 1, 2, 3, 4, 8])
        D = rng.choice([64, 128])
        heads = dict(P=P, Hq=Hkv * rng.choice([1, 2, 3, 4, 5, 8]), Hkv=Hkv, D=D)
        if op == "plan":
            B = _log(rng, 1, 3000)
            c = dict(op=op, B=B, T=B if rng.random() < 0.4 else _log(rng, B, 200000),
                     page=rng.choice([8, 16, 32, 64, 128]), past=_log(rng, 1, 1000))
        elif op in ("rope", "ropeg"):
            c = dict(op=op, T=_log(rng, 1, 12000), rot=rng.choice([D, D, D // 2, D // 4]),
                     f32=rng.random() < 0.5, **heads)
            if op == "rope":
                c.update(cache=rng.random() < 0.6, page=rng.choice([8, 16, 64]))
                c["keep"] = not c["cache"] or rng.random() < 0.5
        elif op in ("attn", "train"):
            B = _log(rng, 1, 40)
            c = dict(op="attn", B=B, T=_log(rng, max(4, B), 16384), past=rng.choice([0, 0, 0, 5, 300]),
                     causal=rng.random() < 0.85, train=op == "train", packed=rng.random() < 0.5, **heads)
            lq, lk = _lens(c)
            if c["P"] * c["Hq"] * B * max(lq) * max(lk) > (1 << 32):
                continue                       # the plain form pads every prompt to the longest
        else:
            c = dict(op=op, B=_log(rng, 1, 200), L=_log(rng, 1, 60000),
                     prefix=0 if rng.random() < 0.5 else _log(rng, 16, 16384),
                     page=rng.choice([8, 16, 32, 64, 128]), **heads)
            if c["P"] * c["B"] * c["L"] * c["Hkv"] * c["D"] > (1 << 29):
                continue
        w, k = work(c), "train" if c.get("train") else c["op"]
        if w["bytes"] <= top[k, "bytes"] and w["flops"] <= top[k, "flops"]:
            return c


# ---------------------------------------------------------------- lengths (the case's own)
def _split(total, parts, rng):
    """`parts` uneven lengths, at least 1 each, that add up to `total`."""
    w = [rng.uniform(0.15, 1.85) for _ in range(parts)]
    n = [1 + int((total - parts) * x / sum(w)) for x in w]
    n[rng.randrange(parts)] += total - sum(n)
    return n


def _lens(c):
    """Query and key lengths of the packed prompts."""
    lq = _split(c["T"], c["B"], random.Random(c["T"] * 131 + c["B"]))
    return lq, [n + c["past"] for n in lq]


def _plan_lens(c):
    """Cached and new tokens of each request."""
    r = random.Random(c["T"] * 137 + c["B"])
    return [r.randrange(0, 2 * c["past"]) for _ in range(c["B"])], _split(c["T"], c["B"], r)


def _decode_lens(c):
    r = random.Random(c["L"] * 139 + c["B"])
    return [max(1, min(c["L"], int(c["L"] * r.uniform(0.3, 1.1)))) for _ in range(c["B"])]


def _pairs(c):
    """(query, key) pairs that attend, of one head."""
    lq, lk = _lens(c)
    if not c["causal"]:
        return sum(a * b for a, b in zip(lq, lk))
    return sum(a * (b - a) + a * (a + 1) // 2 for a, b in zip(lq, lk))


def work(c):
    op = c["op"]
    if op == "plan":
        cached, new = _plan_lens(c)
        pages = sum(-(-(a + b) // c["page"]) - -(-a // c["page"]) for a, b in zip(cached, new))
        return dict(bytes=16 * c["B"] + 8 * pages + 12 * c["T"], flops=0)
    if op in ("rope", "ropeg"):
        n, m = c["P"] * c["T"] * (c["Hq"] + 2 * c["Hkv"]) * c["D"], c["P"] * c["T"] * 2 * c["Hkv"] * c["D"]
        x = 4 if c["f32"] else 2
        tab = c["T"] * (4 * c["rot"] + 4)
        if op == "ropeg":                      # the projected q and k heads, the three gradients in; one gradient out
            return dict(bytes=(n - m // 2) * x + 2 * n + n * x + tab, flops=12 * n)
        out = n - m + (m if c["keep"] else 0) + (m if c["cache"] else 0)
        return dict(bytes=n * x + 2 * out + tab, flops=6 * n)
    if op == "attn":
        lk = sum(_lens(c)[1])
        q, kv = c["P"] * c["T"] * c["Hq"] * c["D"], c["P"] * lk * c["Hkv"] * c["D"]
        pairs = _pairs(c) * c["P"] * c["Hq"]
        b, f = 2 * (2 * q + 2 * kv) + 4 * c["P"] * c["T"] * c["Hq"], 4 * c["D"] * pairs
        if c["train"]:
            b, f = b + 2 * (4 * q + 4 * kv), f + 10 * c["D"] * pairs
        return dict(bytes=b, flops=f)
    keys = sum(_decode_lens(c)) + c["prefix"]
    seen = sum(_decode_lens(c)) + c["B"] * c["prefix"]
    return dict(bytes=4 * c["P"] * keys * c["Hkv"] * c["D"] + 4 * c["P"] * c["B"] * c["Hq"] * c["D"],
                flops=4 * c["P"] * seen * c["Hq"] * c["D"])


# ---------------------------------------------------------------- inputs
def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cu(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return _i32(out)


def _table(rows, rot):
    """cos and sin of position times frequency, base 10000: (rows, rot)."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * f[None, :]
    return torch.cat([a.cos(), a.sin()], dim=1).float()


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    bf = torch.bfloat16

    def normal(*shape, dtype=bf, std=1.0):
        x = torch.empty(shape, dtype=dtype, device="cuda")
        for part in x:                         # rank by rank: little scratch memory
            part.copy_(torch.randn(part.shape, generator=g, device="cuda") * std)
        return x

    s, op = dict(case=c), c["op"]
    if op == "plan":
        cached, new = _plan_lens(c)
        B, page = c["B"], c["page"]
        held = sum(-(-a // page) for a in cached)
        need = sum(-(-(a + b) // page) for a, b in zip(cached, new)) - held
        width = max(-(-(a + b) // page) for a, b in zip(cached, new)) + 2
        pool = torch.randperm(held + need + 50, generator=g, device="cuda").int()
        table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        at = torch.arange(width, device="cuda")[None, :] < _i32([-(-a // page) for a in cached])[:, None]
        table[at] = pool[:held]
        cap = c["T"] + 7                       # a step's buffers are a little larger than the step
        s.update(lengths=_i32(cached), new=_i32(new), free=pool[held:].contiguous(), used=_i32([0]), table=table,
                 after=_i32([0] * B), cu=_i32([0] * (B + 1)), positions=_i32([0] * cap),
                 slots=torch.zeros(cap, dtype=torch.int64, device="cuda"), used_after=_i32([0]), prefix=0)
        return s
    P, Hq, Hkv, D = c["P"], c["Hq"], c["Hkv"], c["D"]
    if op in ("rope", "ropeg"):
        T, rot = c["T"], c["rot"]
        dt = torch.float32 if c["f32"] else bf
        rows = T + 1000
        # positions of several prompts: runs that start anywhere
        first = torch.randint(0, 900, (1 + T // 200,), generator=g, device="cuda")
        t = torch.arange(T, device="cuda")
        s.update(qkv=normal(P, T, (Hq + 2 * Hkv) * D, dtype=dt), gq=1 + normal(P, D, dtype=torch.float32, std=0.2),
                 gk=1 + normal(P, D, dtype=torch.float32, std=0.2), table=_table(rows, rot),
                 pos=(first[t // 200] + t % 200).int())
        if op == "ropeg":
            s.update(dq=normal(P, T, Hq, D), dk=normal(P, T, Hkv, D), dv=normal(P, T, Hkv, D),
                     dqkv=torch.empty_like(s["qkv"]), dgq=torch.empty(P, D, device="cuda"), dgk=torch.empty(P, D, device="cuda"))
        else:
            s["q"] = torch.empty(P, T, Hq, D, dtype=bf, device="cuda")
            s["k"] = s["v"] = s["kc"] = s["vc"] = s["slots"] = None
            if c["keep"]:
                s.update(k=torch.empty(P, T, Hkv, D, dtype=bf, device="cuda"), v=torch.empty(P, T, Hkv, D, dtype=bf, device="cuda"))
            if c["cache"]:
                n = (T + 8 * c["page"]) // c["page"] * c["page"]
                pages = torch.randperm(n // c["page"], generator=g, device="cuda")
                s["slots"] = pages[t // c["page"]] * c["page"] + t % c["page"]
                s.update(kc=normal(P, n, Hkv, D), vc=normal(P, n, Hkv, D))
    elif op == "attn":
        lq, lk = _lens(c)
        T, Tk = sum(lq), sum(lk)
        # heads from flat to sharp
        sharp = torch.linspace(0.5, 2.5, Hq, device="cuda")[:, None]
        if c["packed"] and c["past"] == 0:     # slices of one row per token
            x = normal(P, T, Hq + 2 * Hkv, D)
            x[:, :, :Hq] *= sharp
            s.update(q=x[:, :, :Hq], k=x[:, :, Hq:Hq + Hkv], v=x[:, :, Hq + Hkv:])
        else:
            s.update(q=normal(P, T, Hq, D), k=normal(P, Tk, Hkv, D), v=normal(P, Tk, Hkv, D))
            s["q"] *= sharp
        s.update(cuq=_cu(lq), cuk=_cu(lk), o=torch.empty(P, T, Hq, D, dtype=bf, device="cuda"),
                 lse=torch.empty(P, Hq, T, device="cuda"), lmax=(max(lq), max(lk)))
        if c["train"]:
            s.update(do=normal(P, T, Hq, D), dq=torch.empty(P, T, Hq, D, dtype=bf, device="cuda"),
                     dk=torch.empty(P, Tk, Hkv, D, dtype=bf, device="cuda"), dv=torch.empty(P, Tk, Hkv, D, dtype=bf, device="cuda"))
    else:
        lens, page = _decode_lens(c), c["page"]
        B, width = c["B"], -(-max(_decode_lens(c)) // page)
        shared = -(-c["prefix"] // page)
        n = sum(-(-a // page) for a in lens) + shared + 3
        pool = torch.randperm(n, generator=g, device="cuda").int()
        table = torch.zeros((B, width), dtype=torch.int32, device="cuda")
        at = torch.arange(width, device="cuda")[None, :] < _i32([-(-a // page) for a in lens])[:, None]
        table[at] = pool[shared:shared + int(at.sum())]
        sharp = torch.linspace(0.5, 2.5, Hq, device="cuda")[:, None]
        s.update(q=normal(P, B, Hq, D) * sharp.to(bf), kc=normal(P, n * page, Hkv, D), vc=normal(P, n * page, Hkv, D),
                 table=table, lengths=_i32(lens), pages=pool[:shared].contiguous() if shared else None, lmax=max(lens),
                 o=torch.empty(P, B, Hq, D, dtype=bf, device="cuda"))
    for k in list(s):                          # each rank's buffers
        if k not in ("case", "table", "pos", "slots", "cuq", "cuk", "lengths", "pages") and isinstance(s[k], torch.Tensor):
            s[k + "_r"] = list(s[k].unbind(0))
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    return (_RUN_OWN if own else _RUN_PLAIN)[s["case"]["op"]](s)


# the library ------------------------------------------------------------
def _own_plan(s):
    from ring_collectives_amd import attention as A
    A.kv_plan(s["lengths"], s["new"], s["free"], s["used"], s["table"], s["after"], s["cu"], s["positions"], s["slots"],
              s["used_after"], page_size=s["case"]["page"], prefix_len=s["prefix"])
    return {k: s[k] for k in ("table", "after", "cu", "positions", "slots", "used_after")}


def _own_rope(s):
    from ring_collectives_amd import attention as A
    A.tp_qk_norm_rope(s["qkv_r"], s["gq_r"], s["gk_r"], s["table"], s["pos"], s["q_r"], s.get("k_r"), s.get("v_r"),
                      s.get("kc_r"), s.get("vc_r"), s["slots"], eps=EPS)
    return {k: s[k] for k in ("q", "k", "v", "kc", "vc")}


def _own_ropeg(s):
    from ring_collectives_amd import attention as A
    s["ws"] = A.tp_qk_norm_rope_grad(s["dq_r"], s["dk_r"], s["dv_r"], s["qkv_r"], s["gq_r"], s["gk_r"], s["table"], s["pos"],
                                     s["dqkv_r"], s["dgq_r"], s["dgk_r"], eps=EPS, ws=s.get("ws"))
    return {k: s[k] for k in ("dqkv", "dgq", "dgk")}


def _own_attn(s):
    from ring_collectives_amd import attention as A
    c = s["case"]
    A.tp_attention(s["q_r"], s["k_r"], s["v_r"], s["o_r"], s["cuq"], s["cuk"], lse=s["lse_r"], causal=c["causal"])
    if not c["train"]:
        return {k: s[k] for k in ("o", "lse")}
    s["ws"] = A.tp_attention_grad(s["do_r"], s["q_r"], s["k_r"], s["v_r"], s["o_r"], s["lse_r"], s["dq_r"], s["dk_r"],
                                  s["dv_r"], s["cuq"], s["cuk"], causal=c["causal"], ws=s.get("ws"))
    return {k: s[k] for k in ("o", "lse", "dq", "dk", "dv")}


def _own_decode(s):
    from ring_collectives_amd import attention as A
    c = s["case"]
    s["ws"] = A.tp_attention_decode(s["q_r"], s["kc_r"], s["vc_r"], s["o_r"], s["table"], s["lengths"], page_size=c["page"],
                                    prefix_pages=s["pages"], prefix_len=c["prefix"], ws=s.get("ws"))
    return s["o"]


# elementary operations in 32 bits ---------------------------------------
def _plain_plan(s):
    page, before, table = s["case"]["page"], s["lengths"].long(), s["table"]
    after = before + s["new"]
    have, want = (before + page - 1) // page, (after + page - 1) // page
    need = (want - have).cumsum(0)
    cu = torch.cat([need.new_zeros(1), s["new"].long().cumsum(0)])
    j = torch.arange(table.shape[1], device="cuda")[None, :]
    src = s["used"].long() + (need - (want - have))[:, None] + j - have[:, None]
    n = s["free"].numel()
    page_at = torch.where(src < n, s["free"][src.clamp(0, n - 1)], -1)
    table.copy_(torch.where((j >= have[:, None]) & (j < want[:, None]), page_at, table))
    t = torch.arange(s["slots"].numel(), device="cuda")
    b = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=before.numel() - 1)
    live = t < cu[-1]
    at = before[b] + t - cu[b]
    p = table[b, (at // page).clamp(max=table.shape[1] - 1)].long()
    slots = torch.where(live & (p >= 0), p * page + at % page, -1)
    positions = torch.where(live, at + s["prefix"], 0)
    return dict(table=table, after=after.int(), cu=cu.int(), positions=positions.int(), slots=slots,
                used_after=(s["used"] + need[-1]).int())


def _angles(s):
    cs = s["table"][s["pos"].long()][None, :, None, :]
    h = cs.shape[-1] // 2
    return cs[..., :h], cs[..., h:]


def _turn(y, cos, sin):
    """The rotation of the first 2h values of every head, pair (i, i + h)."""
    h = cos.shape[-1]
    a, b = y[..., :h], y[..., h:2 * h]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, y[..., 2 * h:]], dim=-1)


def _heads(s):
    c = s["case"]
    x = s["qkv"].view(c["P"], c["T"], c["Hq"] + 2 * c["Hkv"], c["D"])
    return x[:, :, :c["Hq"]], x[:, :, c["Hq"]:c["Hq"] + c["Hkv"]], x[:, :, c["Hq"] + c["Hkv"]:]


def _plain_rope(s):
    bf = torch.bfloat16
    q, k, v = _heads(s)
    cos, sin = _angles(s)

    def norm_turn(x, g):
        x = x.float()
        return _turn(x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * g[:, None, None, :], cos, sin).to(bf)

    k, v = norm_turn(k, s["gk"]), v.to(bf)
    if s["kc"] is not None:
        s["kc"][:, s["slots"]] = k
        s["vc"][:, s["slots"]] = v
    keep = s["case"]["keep"]
    return dict(q=norm_turn(q, s["gq"]), k=k if keep else None, v=v if keep else None, kc=s["kc"], vc=s["vc"])


def _plain_ropeg(s):
    q, k, _ = _heads(s)
    cos, sin = _angles(s)

    def back(x, g, dy):
        x, dz, g = x.float(), _turn(dy.float(), cos, -sin), g[:, None, None, :]
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        n, u = x * r, dz * g
        return r * (u - n * (n * u).mean(-1, keepdim=True)), (dz * n).sum((1, 2))

    dq, dgq = back(q, s["gq"], s["dq"])
    dk, dgk = back(k, s["gk"], s["dk"])
    d = torch.cat([dq, dk, s["dv"].float()], dim=2).view(s["qkv"].shape).to(s["qkv"].dtype)
    return dict(dqkv=d, dgq=dgq, dgk=dgk)


def _plain_attn(s):
    c = s["case"]
    P, B, Hq, Hkv, D = c["P"], c["B"], c["Hq"], c["Hkv"], c["D"]
    G, bf, scale = Hq // Hkv, torch.bfloat16, 1.0 / math.sqrt(D)
    Lq, Lk = s["lmax"]
    cuq, cuk = s["cuq"].long(), s["cuk"].long()
    nq, nk = cuq.diff(), cuk.diff()
    iq, ik = torch.arange(Lq, device="cuda"), torch.arange(Lk, device="cuda")
    okq, okk = iq[None, :] < nq[:, None], ik[None, :] < nk[:, None]
    atq = (cuq[:-1, None] + iq).clamp(max=s["q"].shape[1] - 1)
    atk = (cuk[:-1, None] + ik).clamp(max=s["k"].shape[1] - 1)

    def rows(x, at, ok, groups):               # (P, T, H, D) -> (P, Hkv, B, groups L, D), zeros past the end
        x = (x[:, at].float() * ok[None, :, :, None, None]).view(P, B, at.shape[1], Hkv, groups, D)
        return x.permute(0, 3, 1, 4, 2, 5).reshape(P, Hkv, B, groups * at.shape[1], D)

    def places(cu, n, L):                      # where each packed row stands among the padded ones
        t = torch.arange(n, device="cuda")
        b = torch.searchsorted(cu, t, right=True) - 1
        return b * L + t - cu[b]

    def packed(x, at, L, groups):              # the way back
        x = x.view(P, Hkv, B, groups, L, D).permute(0, 2, 4, 1, 3, 5)
        return x.reshape(P, B * L, Hkv * groups, D)[:, at]

    placeq, placek = places(cuq, s["q"].shape[1], Lq), places(cuk, s["k"].shape[1], Lk)

    q, k, v = rows(s["q"], atq, okq, G), rows(s["k"], atk, okk, 1), rows(s["v"], atk, okk, 1)
    sees = okk[:, None, :].expand(B, Lq, Lk)
    if c["causal"]:
        sees = sees & (ik[None, None, :] - iq[None, :, None] <= (nk - nq)[:, None, None])
    sees = sees[:, None].expand(B, G, Lq, Lk).reshape(B, G * Lq, Lk)
    x = (q * scale) @ k.transpose(-1, -2)
    x = x.masked_fill_(~sees, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = x.sub_(torch.where(m > -math.inf, m, 0)).exp_()
    l = p.sum(-1, keepdim=True)
    p = p.div_(torch.where(l > 0, l, 1))
    o = p @ v
    lse = (m + l.log()).view(P, Hkv, B, G, Lq).permute(0, 1, 3, 2, 4).reshape(P, Hq, B * Lq)[:, :, placeq]
    out = dict(o=packed(o, placeq, Lq, G).to(bf), lse=lse)
    if c["train"]:
        do = rows(s["do"], atq, okq, G)
        dv = p.transpose(-1, -2) @ do
        ds = (do @ v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
        out.update(dq=packed(ds @ k, placeq, Lq, G).to(bf), dk=packed(ds.transpose(-1, -2) @ q, placek, Lk, 1).to(bf),
                   dv=packed(dv, placek, Lk, 1).to(bf))
    return out


def _plain_decode(s):
    c = s["case"]
    P, B, Hq, Hkv, D, page = c["P"], c["B"], c["Hq"], c["Hkv"], c["D"], c["page"]
    G = Hq // Hkv
    q = s["q"].float().view(P, B, Hkv, G, D) / math.sqrt(D)
    j = torch.arange(s["lmax"], device="cuda")
    at = s["table"][:, j // page].long() * page + j % page
    k, v = (s[n][:, at].float().permute(0, 1, 3, 2, 4) for n in ("kc", "vc"))       # (P, B, Hkv, L, D)
    x = (q @ k.transpose(-1, -2)).masked_fill_(j[None, None, None, None, :] >= s["lengths"][None, :, None, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    if c["prefix"]:
        i = torch.arange(c["prefix"], device="cuda")
        at = s["pages"][i // page].long() * page + i % page
        kp, vp = (s[n][:, at].float().permute(0, 2, 1, 3) for n in ("kc", "vc"))    # (P, Hkv, Lp, D)
        y = (q.transpose(1, 2).reshape(P, Hkv, B * G, D) @ kp.transpose(-1, -2))
        y = y.view(P, Hkv, B, G, -1).transpose(1, 2)
        m = torch.maximum(m, y.amax(-1, keepdim=True))
    p = x.sub_(m).exp_()
    o, l = p @ v, p.sum(-1, keepdim=True)
    if c["prefix"]:
        r = (y - m).exp_()
        l = l + r.sum(-1, keepdim=True)
        o = o + (r.transpose(1, 2).reshape(P, Hkv, B * G, -1) @ vp).view(P, Hkv, B, G, D).transpose(1, 2)
    return (o / l).to(torch.bfloat16).view(P, B, Hq, D)


_RUN_OWN = dict(plan=_own_plan, rope=_own_rope, ropeg=_own_ropeg, attn=_own_attn, decode=_own_decode)
_RUN_PLAIN = dict(plan=_plain_plan, rope=_plain_rope, ropeg=_plain_ropeg, attn=_plain_attn, decode=_plain_decode)


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_norm_turn(x, gain, angle_table, pos, eps):
    """One head row after the other as complex numbers: normalise, scale, multiply by e^(i angle)."""
    x = x * gain * (x.square().sum(-1, keepdim=True) / x.shape[-1] + eps) ** -0.5
    h = angle_table.shape[1] // 2
    cs = angle_table.double()[pos.long()][:, None, :]
    z = torch.complex(x[..., :h], x[..., h:2 * h]) * torch.complex(cs[..., :h], cs[..., h:])
    return torch.cat([z.real, z.imag, x[..., 2 * h:]], dim=-1)


def exact(c, seed):
    s = prepare(c, seed)
    op = c["op"]
    if op == "plan":
        return None                            # whole numbers
    P, Hq, Hkv, D = c["P"], c["Hq"], c["Hkv"], c["D"]
    G = Hq // Hkv
    if op == "rope":
        out = dict(q=[], k=[], v=[])
        for r in range(P):
            x = s["qkv"][r].double().view(c["T"], -1, D)
            out["q"].append(_exact_norm_turn(x[:, :Hq], s["gq"][r].double(), s["table"], s["pos"], EPS))
            out["k"].append(_exact_norm_turn(x[:, Hq:Hq + Hkv], s["gk"][r].double(), s["table"], s["pos"], EPS))
            out["v"].append(x[:, Hq + Hkv:])
        out = {n: torch.stack(t) for n, t in out.items()}
        kc = vc = None
        if c["cache"]:
            kc, vc = s["kc"].double(), s["vc"].double()
            kc.index_copy_(1, s["slots"], out["k"])
            vc.index_copy_(1, s["slots"], out["v"])
        return dict(q=out["q"], k=out["k"] if c["keep"] else None, v=out["v"] if c["keep"] else None, kc=kc, vc=vc)
    if op == "ropeg":
        d, gq, gk = [], [], []
        for r in range(P):
            x = s["qkv"][r].double().requires_grad_()
            a, b = s["gq"][r].double().requires_grad_(), s["gk"][r].double().requires_grad_()
            h = x.view(c["T"], -1, D)
            y = torch.cat([_exact_norm_turn(h[:, :Hq], a, s["table"], s["pos"], EPS),
                           _exact_norm_turn(h[:, Hq:Hq + Hkv], b, s["table"], s["pos"], EPS), h[:, Hq + Hkv:]], dim=1)
            dy = torch.cat([s["dq"][r], s["dk"][r], s["dv"][r]], dim=1).double()
            gx, ga, gb = torch.autograd.grad(y, (x, a, b), dy)
            d.append(gx)
            gq.append(ga)
            gk.append(gb)
        return dict(dqkv=torch.stack(d), dgq=torch.stack(gq), dgk=torch.stack(gk))
    if op == "attn":
        lq, lk = _lens(c)
        out = dict(o=torch.zeros(P, sum(lq), Hq, D, dtype=torch.float64, device="cuda"),
                   lse=torch.zeros(P, Hq, sum(lq), dtype=torch.float64, device="cuda"))
        if c["train"]:
            out.update(dq=torch.zeros_like(out["o"]), dk=torch.zeros(P, sum(lk), Hkv, D, dtype=torch.float64, device="cuda"),
                       dv=torch.zeros(P, sum(lk), Hkv, D, dtype=torch.float64, device="cuda"))
        for r in range(P):
            q0 = k0 = 0
            for a, b in zip(lq, lk):
                qs, ks = slice(q0, q0 + a), slice(k0, k0 + b)
                q0, k0 = q0 + a, k0 + b
                hide = None
                if c["causal"]:
                    hide = torch.ones(a, b, dtype=torch.bool, device="cuda").triu(b - a + 1)
                for h in range(Hkv):
                    kk, vv = s["k"][r, ks, h].double(), s["v"][r, ks, h].double()
                    for i in range(h * G, h * G + G):
                        qq = s["q"][r, qs, i].double()
                        x = qq @ kk.t() * D ** -0.5
                        if hide is not None:
                            x.masked_fill_(hide, -math.inf)
                        lse = torch.logsumexp(x, dim=-1)
                        p = (x - lse[:, None]).exp()
                        out["lse"][r, i, qs] = lse
                        o = p @ vv
                        out["o"][r, qs, i] = o
                        if c["train"]:
                            do = s["do"][r, qs, i].double()
                            dp = do @ vv.t()
                            ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * D ** -0.5
                            out["dq"][r, qs, i] = ds @ kk
                            out["dk"][r, ks, h] += ds.t() @ qq
                            out["dv"][r, ks, h] += p.t() @ do
        return out
    page = c["page"]
    o = torch.empty(P, c["B"], Hq, D, dtype=torch.float64, device="cuda")
    j = torch.arange(max(c["prefix"], c["L"]), device="cuda")
    for b, n in enumerate(_decode_lens(c)):
        at = s["table"][b, j[:n] // page].long() * page + j[:n] % page
        if c["prefix"]:
            i = j[:c["prefix"]]
            at = torch.cat([s["pages"][i // page].long() * page + i % page, at])
        k, v = (s[n_][:, at].double().transpose(1, 2) for n_ in ("kc", "vc"))
        q = s["q"][:, b].double().view(P, Hkv, G, D)
        o[:, b] = (torch.softmax(q @ k.transpose(-1, -2) * D ** -0.5, dim=-1) @ v).reshape(P, Hq, D)
    return o
