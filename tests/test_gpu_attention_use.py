"""GPU tests of how the attention calls are used: what the Python entry points
refuse, streams and graph capture, caches and rows past 4 GiB, and the layer
of examples/attention_layer.py end to end."""
import math
import os
import sys

import numpy as np
import pytest
import torch

from oracle import attention as oa
from ring_collectives_amd import _native as N
from ring_collectives_amd import attention as A
from ring_collectives_amd import collectives as rc

from _gpu_helpers import note
from test_gpu_attention import (BF, attn_inputs, check_attention, check_decode, check_grad, cu, decode_inputs, f64, i32, poisoned,
                                rope_inputs, within)

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    N.lib()
    yield


# ---------------------------------------------------------------- refusals
def test_prompt_refusals():
    q, k, v = attn_inputs(2, [8], [8], 4, 2, 64, seed=1)
    o, c = [poisoned((8, 4, 64)) for _ in range(2)], cu([8])

    def bad(exc, match, **kw):
        d = dict(q=q, k=k, v=v, o=o, cu_q=c, cu_k=c)
        d.update(kw)
        with pytest.raises(exc, match=match):
            A.tp_attention(**d)

    bad(ValueError, "rank buffers", k=k[:1])
    bad(ValueError, "must be", v=[v[0], v[1][:4]])
    bad(ValueError, "must be", o=[o[0], o[1][:, :2]])
    bad(TypeError, "BFloat16", q=[t.float() for t in q])
    bad(TypeError, "Int", cu_q=c.long())
    bad(ValueError, "current device", k=[k[0], k[1].cpu()])
    bad(ValueError, "current device", cu_k=c.cpu())
    bad(ValueError, "elements", cu_k=i32([0, 4, 8]))
    bad(ValueError, "offsets", cu_q=i32([]))
    bad(ValueError, "dense", q=[t.transpose(0, 1).contiguous().transpose(0, 1) for t in q])
    bad(ValueError, "same strides", k=[k[0], torch.empty(8, 3, 64, dtype=BF, device="cuda")[:, :2]])
    bad(ValueError, "be", lse=[torch.empty(8, 4, device="cuda")] * 2)
    bad(N.RingError, "failed", q=[t[:, :3] for t in q], o=[t[:, :3] for t in o])   # 3 heads on 2
    bad(N.RingError, "failed", scale=-1.0)
    x = torch.empty(8 * 2 * 64 + 1, dtype=BF, device="cuda")
    bad(N.RingError, "failed", k=[x[1:].view(8, 2, 64)] * 2)                # not 16-byte aligned
    with pytest.raises(ValueError, match="workspace"):
        A.tp_attention_grad(o, q, k, v, o, [torch.empty(4, 8, device="cuda")] * 2, o, k, v, c, c, ws=torch.zeros(9999))
    with pytest.raises(N.RingError):
        A.tp_attention_grad(o, q, k, v, o, [torch.empty(4, 8, device="cuda")] * 2, o, k, v, c, c,
                            ws=torch.zeros(300, dtype=torch.uint8, device="cuda"))


def test_rope_and_plan_refusals():
    x, gq, gk, cs, pos = rope_inputs(1, 4, 2, 1, 64, 64, BF, seed=2)
    q, k = [poisoned((4, 2, 64))], [poisoned((4, 1, 64))]
    for kw, exc in ((dict(qkv=[x[0].half()]), TypeError), (dict(qkv=[x[0][:, :-64]]), ValueError), (dict(k=k), ValueError),
                    (dict(gain_k=None), ValueError), (dict(pos=pos[:3]), ValueError), (dict(pos=pos.long()), TypeError),
                    (dict(cos_sin=cs.double()), TypeError), (dict(cos_sin=cs[:, 0]), ValueError),
                    (dict(k_cache=k), ValueError), (dict(q=[q[0][:, :1]]), ValueError), (dict(eps=-1.0), N.RingError),
                    (dict(cos_sin=torch.zeros(9, 24, device="cuda")), N.RingError),
                    (dict(gain_q=[gq[0][:32]], gain_k=[gk[0][:32]]), ValueError)):
        d = dict(qkv=x, gain_q=gq, gain_k=gk, cos_sin=cs, pos=pos, q=q)
        d.update(kw)
        with pytest.raises(exc):
            A.tp_qk_norm_rope(**d)
    with pytest.raises(ValueError, match="buffers"):
        A.tp_qk_norm_rope_grad(q, k, k, x, gq, gk, cs, pos, [torch.empty_like(x[0])])
    a = dict(lengths=i32([1, 2]), new_tokens=i32([1, 1]), free_pages=i32([0, 1]), used=i32([0]), block_table=i32([[0], [1]]),
             lengths_after=i32([0, 0]), cu_new=i32([0, 0, 0]), positions=i32([0, 0]),
             slots=torch.zeros(2, dtype=torch.int64, device="cuda"), used_after=i32([0]), page_size=16)
    A.kv_plan(**a)
    for kw, exc in ((dict(new_tokens=i32([1])), ValueError), (dict(cu_new=i32([0, 0])), ValueError),
                    (dict(slots=i32([0, 0])), TypeError), (dict(positions=i32([0])), ValueError),
                    (dict(block_table=i32([0, 1])), ValueError), (dict(page_size=10), N.RingError),
                    (dict(used_after=a["used"]), N.RingError), (dict(lengths_after=a["lengths"]), N.RingError)):
        with pytest.raises(exc):
            A.kv_plan(**{**a, **kw})


def test_decode_refusals():
    q, kc, vc, table, ln, pp = decode_inputs(1, [20, 5], 17, 2, 1, 64, 16, seed=3)
    o = [poisoned((2, 2, 64))]
    for kw, exc in ((dict(page_size=15), ValueError), (dict(page_size=0), ValueError), (dict(lengths=ln[:1]), ValueError),
                    (dict(block_table=table[0]), ValueError), (dict(prefix_len=40), ValueError), (dict(prefix_pages=None), ValueError),
                    (dict(v_cache=[vc[0][:16]]), ValueError), (dict(scale=0.0), N.RingError),
                    (dict(ws=torch.zeros(256, dtype=torch.uint8, device="cuda")), N.RingError)):
        d = dict(q=q, k_cache=kc, v_cache=vc, o=o, block_table=table, lengths=ln, page_size=16, prefix_pages=pp, prefix_len=17)
        d.update(kw)
        with pytest.raises(exc):
            A.tp_attention_decode(**d)


# ---------------------------------------------------------------- streams, graphs
def test_calls_on_a_side_stream():
    """Workspaces that a call makes itself are ready on the call's stream, and
    kept while its kernels there run."""
    lq = [200, 33]
    q, k, v = attn_inputs(2, lq, lq, 4, 2, 64, seed=5)
    s = torch.cuda.Stream()
    o, lse = [poisoned((233, 4, 64)) for _ in range(2)], [poisoned((4, 233), torch.float32) for _ in range(2)]
    do = [torch.randn(233, 4, 64, device="cuda").to(BF) for _ in range(2)]
    d = [[poisoned(tuple(t.shape)) for t in x] for x in (q, k, v)]
    c = cu(lq)
    s.wait_stream(torch.cuda.current_stream())
    A.tp_attention(q, k, v, o, c, c, lse=lse, stream=s)
    A.tp_attention_grad(do, q, k, v, o, lse, *d, c, c, stream=s)
    junk = [torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]     # takes freed blocks
    s.synchronize()
    check_attention(q, k, v, o, lse, lq, lq, True, 1 / 8)
    check_grad(do, q, k, v, *d, lq, lq, True, 1 / 8)
    assert len(junk) == 8


def test_decode_step_captured_in_a_graph():
    """A whole decode step - plan, norm and rotation to the cache, attention -
    captured once and replayed on changing lengths and rows: every replay's
    output and cache equal those of the same calls made one by one."""
    P, B, Hq, Hkv, D, page = 2, 5, 4, 2, 64, 16
    g = torch.Generator(device="cuda").manual_seed(6)
    pages = 400
    lens = [0, 31, 500, 64, 1]
    free = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.full((B, 40), -1, dtype=torch.int32, device="cuda")
    have = [-(-n // page) for n in lens]
    at = 0
    for b, n in enumerate(have):
        table[b, :n] = free[at:at + n]
        at += n
    new, used = torch.ones(B, dtype=torch.int32, device="cuda"), i32([at])
    kc, vc = ([torch.randn(pages * page, Hkv, D, generator=g, device="cuda").to(BF) for _ in range(P)] for _ in range(2))
    _, gq, gk, cs, _ = rope_inputs(P, 1, Hq, Hkv, D, D, BF, seed=7, rows=600)
    x = [torch.randn(B, (Hq + 2 * Hkv) * D, generator=g, device="cuda") for _ in range(P)]
    lengths = i32(lens)
    bufs = dict(after=i32([0] * B), cu=i32([0] * (B + 1)), pos=i32([0] * B), slots=torch.zeros(B, dtype=torch.int64, device="cuda"),
                ua=i32([0]))
    q, o = ([poisoned((B, Hq, D)) for _ in range(P)] for _ in range(2))
    ws = torch.zeros(1 << 23, dtype=torch.uint8, device="cuda")

    def step(lengths, used, table, kc, vc, q, o, bufs, ws):
        A.kv_plan(lengths, new, free, used, table, bufs["after"], bufs["cu"], bufs["pos"], bufs["slots"], bufs["ua"], page_size=page)
        A.tp_qk_norm_rope(x, gq, gk, cs, bufs["pos"], q, None, None, kc, vc, bufs["slots"])
        A.tp_attention_decode(q, kc, vc, o, table, bufs["after"], page_size=page, ws=ws)

    twin = dict(lengths=lengths.clone(), used=used.clone(), table=table.clone(), kc=[t.clone() for t in kc], vc=[t.clone() for t in vc],
                q=[torch.empty_like(t) for t in q], o=[torch.empty_like(t) for t in o], bufs={n: t.clone() for n, t in bufs.items()},
                ws=torch.zeros_like(ws))
    args = (lengths, used, table, kc, vc, q, o, bufs, ws)
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        A._binding()
    with torch.cuda.graph(graph):
        step(*args)
    for i in range(20):
        for t in x:
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        graph.replay()
        step(**twin)
        torch.cuda.synchronize()
        for a, b in zip(o + kc + vc + [table, bufs["after"], bufs["slots"]],
                        twin["o"] + twin["kc"] + twin["vc"] + [twin["table"], twin["bufs"]["after"], twin["bufs"]["slots"]]):
            assert torch.equal(a, b), i
        for d in (dict(lengths=lengths, used=used, bufs=bufs), twin):
            d["lengths"].copy_(d["bufs"]["after"])
            d["used"].copy_(d["bufs"]["ua"])
    assert lengths.tolist() == [n + 20 for n in lens]
    # the last step against the oracle (lengths count the token that it added)
    check_decode([q[0]], [kc[0]], [vc[0]], [o[0]], table, lengths.tolist(), None, 0, page, D ** -0.5)


def test_prompt_and_gradient_captured_in_a_graph():
    lq = [90, 40]
    q, k, v = attn_inputs(1, lq, lq, 2, 1, 128, seed=8)
    do = [torch.randn(130, 2, 128, device="cuda").to(BF)]
    o, lse = [poisoned((130, 2, 128))], [poisoned((2, 130), torch.float32)]
    d = [[poisoned(tuple(t[0].shape))] for t in (q, k, v)]
    c, ws = cu(lq), torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")

    def step():
        A.tp_attention(q, k, v, o, c, c, lse=lse)
        A.tp_attention_grad(do, q, k, v, o, lse, *d, c, c, ws=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(5):
        for t in q + k + v + do:
            t.copy_(torch.randn(t.shape, device="cuda"))
        graph.replay()
        got = [t.clone() for t in o + lse + d[0] + d[1] + d[2]]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, o + lse + d[0] + d[1] + d[2])), i
    check_grad(do, q, k, v, *d, lq, lq, True, 128 ** -0.5)


# ---------------------------------------------------------------- past 4 GiB
def test_decode_cache_past_4_gib():
    """Pages whose rows lie past 2^32 bytes, of a cache of 8.6 GB a tensor."""
    note("decode: 8.6 GB caches")
    Hkv, D, page = 8, 128, 64
    rows = 1 << 22
    kc, vc = ([torch.empty(rows, Hkv, D, dtype=BF, device="cuda")] for _ in range(2))
    pages = rows // page
    lens = [300, 100]
    table = i32([[pages - 1, 5, pages // 2, pages // 2 + 1, 7], [pages - 2, pages // 4 + 3, -1, -1, -1]])
    pp = i32([pages - 5, 1])
    for t in kc + vc:
        for p in table.flatten().tolist() + pp.tolist():
            if p >= 0:
                t[p * page:(p + 1) * page] = torch.randn(page, Hkv, D, device="cuda").to(BF)
    q, o = [torch.randn(2, 8, D, device="cuda").to(BF)], [poisoned((2, 8, D))]
    A.tp_attention_decode(q, kc, vc, o, table, i32(lens), page_size=page, prefix_pages=pp, prefix_len=70)
    # the oracle on a small cache of the pages used
    small = [p for p in table.flatten().tolist() + pp.tolist() if p >= 0]
    where = {p: i for i, p in enumerate(small)}
    pick = lambda t: torch.cat([t[p * page:(p + 1) * page] for p in small])       # noqa: E731
    tab = torch.tensor([[where.get(p, -1) for p in r] for r in table.tolist()])
    check_decode(q, [pick(kc[0])], [pick(vc[0])], o, tab, lens, torch.tensor([where[p] for p in pp.tolist()]), 70, page, D ** -0.5)
    # and the write side: slots past 2^31 elements and 2^32 bytes
    x, gq, gk, cs, pos = rope_inputs(1, 4, 8, 8, D, D, BF, seed=9)
    slots = torch.tensor([rows - 1, 3, rows // 2 + 1, rows], device="cuda")
    k, v, qq = ([poisoned((4, 8, D))] for _ in range(3))
    A.tp_qk_norm_rope(x, gq, gk, cs, pos, qq, k, v, kc, vc, slots)
    torch.cuda.synchronize()
    for i in range(3):
        assert torch.equal(kc[0][slots[i]], k[0][i]) and torch.equal(vc[0][slots[i]], v[0][i])


def test_prompt_rows_past_4_gib():
    """Prompts at the end of tensors whose rows span 4.6 GB."""
    note("attention: rows past 4 GiB")
    T, W = 1100000, 2048                                     # rows of 16 heads of 128, 2 of them used
    lens = [1, 130, 70]
    first = T - sum(lens)
    big = [torch.empty(T, W, dtype=BF, device="cuda") for _ in range(4)]
    for t in big:
        t[first:] = torch.randn(sum(lens), W, device="cuda").to(BF)
    view = lambda t, h0, n: t.view(T, 16, 128)[:, h0:h0 + n]              # noqa: E731
    q, k, v, do = [view(big[0], 14, 2)], [view(big[1], 15, 1)], [view(big[2], 0, 1)], [view(big[3], 3, 2)]
    o = [torch.zeros(T, W, dtype=BF, device="cuda").view(T, 16, 128)[:, 5:7]]
    lse = [torch.zeros(2, T, device="cuda")]
    c = i32([first + n for n in [0] + list(np.cumsum(lens))])
    A.tp_attention(q, k, v, o, c, c, lse=lse)
    part = slice(first, T)
    cut = lambda x: [t[part].clone() for t in x]                          # noqa: E731
    check_attention(cut(q), cut(k), cut(v), cut(o), [lse[0][:, part]], lens, lens, True, 128 ** -0.5)
    dq, dk, dv = [view(torch.zeros_like(big[0]), 1, 2)], [view(torch.zeros_like(big[0]), 9, 1)], [view(torch.zeros_like(big[0]), 2, 1)]
    A.tp_attention_grad(do, q, k, v, o, lse, dq, dk, dv, c, c)
    check_grad(cut(do), cut(q), cut(k), cut(v), cut(dq), cut(dk), cut(dv), lens, lens, True, 128 ** -0.5)
    assert not dq[0][:first].any() and not dk[0][:first].any()            # rows of no prompt are not written


# ---------------------------------------------------------------- the layer
def _layer():
    import attention_layer
    return attention_layer


def test_layer_prompts_then_steps():
    """The example layer: its decode steps give what its prompt pass gives for
    the same tokens in one prompt, and that is the plain layer's output."""
    ex = _layer()
    lens, more = [300, 17, 511, 196], 3
    g = torch.Generator(device="cuda").manual_seed(3)
    one, two = ex.AttentionLayer(seed=4), ex.AttentionLayer(seed=4)
    rows = [torch.randn(n + more, one.model, generator=g, device="cuda").to(BF) for n in lens]
    one.requests(4, 600)
    n1 = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out1 = torch.cat(one.prompts(list(torch.cat([r[:n] for r, n in zip(rows, lens)]).chunk(4)), n1))
    steps = [one.step(torch.stack([r[n + i] for r, n in zip(rows, lens)]))[0].clone() for i in range(more)]
    assert one.lengths.tolist() == [n + more for n in lens]

    # plain: fp32 everywhere, prompts of lens + more
    P, Hq, Hkv, D = one.P, one.Hq, one.Hkv, one.D

    def plain(x):
        out = 0
        T = x.shape[0]
        cs = one.cos_sin[:T, None]
        for r in range(P):
            h = (x.float() @ one.wqkv[r].float()).view(T, Hq + 2 * Hkv, D)
            def nr(y, gain):
                y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * gain
                a, b = y[..., :D // 2], y[..., D // 2:]
                return torch.cat([a * cs[..., :D // 2] - b * cs[..., D // 2:], b * cs[..., :D // 2] + a * cs[..., D // 2:]], -1)
            q, k, v = nr(h[:, :Hq], one.gain_q[r]), nr(h[:, Hq:Hq + Hkv], one.gain_k[r]), h[:, Hq + Hkv:]
            mask = torch.ones(T, T, dtype=torch.bool, device="cuda").triu(1)
            o = []
            for i in range(Hq):
                s = (q[:, i] @ k[:, i * Hkv // Hq].T * D ** -0.5).masked_fill(mask, -math.inf)
                o.append(s.softmax(-1) @ v[:, i * Hkv // Hq])
            out = out + torch.stack(o, 1).view(T, -1) @ one.wo[r].float()
        return out

    at = 0
    for b, n in enumerate(lens):
        want = plain(rows[b])
        # bf16 roundings of q, k, v, P, o and of the step's projections: about
        # 2^-8 of the output's size each, with random signs
        size = want.square().mean().sqrt()
        assert (out1[at:at + n] - want[:n]).square().mean().sqrt() < 0.02 * size
        for i in range(more):
            assert (steps[i][b] - want[n + i]).square().mean().sqrt() < 0.04 * size
        at += n


def test_layer_training_step():
    """The example's training step against autograd of the plain layer."""
    ex = _layer()
    layer = ex.AttentionLayer(P=2, Hq=4, Hkv=2, D=64, model=256, seed=5)
    g = torch.Generator(device="cuda").manual_seed(6)
    T, lens = 300, [180, 120]
    qkv = [torch.randn(T, 8 * 64, generator=g, device="cuda") for _ in range(2)]
    do = [torch.randn(T, 4, 64, generator=g, device="cuda").to(BF) for _ in range(2)]
    pos = torch.cat([torch.arange(n) for n in lens]).int().cuda()
    o, d, gq, gk = layer.train(qkv, pos, cu(lens), do)
    a, b = (t[0].cpu().double().requires_grad_() for t in (layer.gain_q, layer.gain_k))
    cs = layer.cos_sin.cpu().double()[pos.cpu().long()][:, None]
    total, xs = 0, []
    for r in range(2):
        x = qkv[r].cpu().double().requires_grad_()
        xs.append(x)
        h = x.view(T, 8, 64)

        def nr(y, gain):
            y = y / ((y * y).mean(-1, keepdim=True) + 1e-6).sqrt() * gain
            u, w = y[..., :32], y[..., 32:]
            return torch.cat([u * cs[..., :32] - w * cs[..., 32:], w * cs[..., :32] + u * cs[..., 32:]], -1)

        q, k, v = nr(h[:, :4], a), nr(h[:, 4:6], b), h[:, 6:]
        at = 0
        for n in lens:
            p = slice(at, at + n)
            at += n
            mask = torch.ones(n, n, dtype=torch.bool).triu(1)
            for i in range(4):
                s = (q[p, i] @ k[p, i // 2].T / 8).masked_fill(mask, -math.inf)
                total = total + ((s.softmax(-1) @ v[p, i // 2]) * do[r][p, i].cpu().double()).sum()
    want = torch.autograd.grad(total, xs + [a, b])
    # bf16 q, k, v, o, P, dS and gradients of them: some 2^-8 each, random signs
    for got, w in zip(d + [gq, gk], want):
        assert (got.cpu().double() - w).norm() < 0.02 * w.norm()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [[50, 45, 70], [300, 45, 1000]])
def test_gradient_of_other_prompts_keeps_clear_of_a_prompt_of_nan(D, lens):
    """Inputs that are not finite stay within their prompt, and within their
    group of heads, going back."""
    n = sum(lens)
    q, k, v = attn_inputs(1, lens, lens, 4, 2, D, seed=D + n)
    do = [torch.randn(n, 4, D, device="cuda").to(BF)]
    c, mid = cu(lens), slice(lens[0], lens[0] + lens[1])

    def grads():
        o, lse = [poisoned((n, 4, D))], [poisoned((4, n), torch.float32)]
        A.tp_attention(q, k, v, o, c, c, lse=lse)
        d = [[poisoned(tuple(t[0].shape))] for t in (q, k, v)]
        A.tp_attention_grad(do, q, k, v, o, lse, *d, c, c)
        torch.cuda.synchronize()
        return [t[0] for t in d]

    want = grads()
    v[0][mid, 1] = float("inf")                              # key head 1: query heads 2, 3
    k[0][mid.start + 3, 1, 0] = float("nan")
    q[0][mid.stop - 1, 3, 1] = float("nan")
    for got, w in zip(grads(), want):
        h = got.shape[1] // 2
        rest = torch.ones(n, dtype=torch.bool, device="cuda")
        rest[mid] = False
        assert torch.equal(got[rest], w[rest]) and torch.equal(got[:, :h], w[:, :h])
        assert torch.isfinite(w).all()
