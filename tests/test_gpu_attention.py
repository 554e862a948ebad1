"""GPU tests of the attention operators against the float64 oracle, at the
sizes, layouts and masks where they can go wrong.  Tolerances are the oracle's
element-by-element worst-case bounds; whole numbers are compared exactly."""
import math

import numpy as np
import pytest
import torch

from oracle import attention as oa
from ring_collectives_amd import _native as N
from ring_collectives_amd import attention as A
from ring_collectives_amd import collectives as rc

from _gpu_helpers import note

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    N.lib()
    yield


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def f64(t):
    return t.detach().double().cpu().numpy()


def within(got, want, bound, what):
    """Every element within its bound; NaN and infinities in the same places."""
    got = f64(got) if isinstance(got, torch.Tensor) else got
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)]), what
    d = np.abs(got[fine] - want[fine])
    over = d > bound[fine] + 1e-30
    assert not over.any(), "%s: %d of %d elements outside, worst %.3g of its bound" % (
        what, over.sum(), d.size, (d / np.maximum(bound[fine], 1e-30)).max())


def poisoned(shape, dtype=BF):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


# ---------------------------------------------------------------- kv_plan
def run_plan(lengths, new, free, used, table, page, cap, prefix):
    B = len(lengths)
    tab = i32(table).reshape(B, -1)
    after, cu, ua = i32([-7] * B), i32([-7] * (B + 1)), i32([-7])
    pos, slots = i32([-7] * cap), torch.full((cap,), -7, dtype=torch.int64, device="cuda")
    A.kv_plan(i32(lengths), i32(new), i32(free), i32([used]), tab, after, cu, pos, slots, ua, page_size=page,
              prefix_len=prefix)
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in (tab, after, cu, pos, slots, ua)]


@pytest.mark.parametrize("B,page,longest,spare,used,prefix", [
    (1, 16, 1, 3, 0, 0), (1, 1, 40, 3, 0, 5), (3, 8, 30, 1, 2, 0), (64, 16, 90, 0, 0, 0), (65, 32, 200, 9, 4, 1000),
    (257, 16, 50, 9, 4, 0), (1000, 64, 300, 3, 0, 7), (8192, 128, 40, 50, 11, 0)])
@pytest.mark.parametrize("short", [False, True])
def test_plan(B, page, longest, spare, used, prefix, short):
    note("kv_plan B=%d page=%d short=%s" % (B, page, short))
    rng = np.random.default_rng(B * 7 + page)
    lengths = rng.integers(0, longest + 1, B) * (rng.random(B) < 0.8)
    new = rng.integers(0, longest + 1, B) * (rng.random(B) < 0.7)
    if B == 3:
        lengths[0], new[1] = -4, -1                      # negative: none
    n0, n1 = np.maximum(lengths, 0), np.maximum(new, 0)
    need = int((-(-(n0 + n1) // page) + (-n0 // page)).sum())
    width = int((-(-(n0 + n1) // page)).max()) + 1
    if short:
        width = max(1, width - 2)                        # tokens past the table
    free = rng.permutation(used + need + spare + 5)[:max(0, used + need + (spare if not short else -3))]
    table = rng.integers(-1, 5000, (B, width))
    cap = int(n1.sum()) + (3 if not short else -min(2, int(n1.sum())))
    want = oa.kv_plan(lengths, new, free, used, table, page, cap, prefix)
    got = run_plan(lengths.tolist(), new.tolist(), free.tolist(), used, table.tolist(), page, cap, prefix)
    for g, w, name in zip(got, want, ("table", "after", "cu", "positions", "slots", "used")):
        assert np.array_equal(g.reshape(-1), np.asarray(w).reshape(-1)), name


def test_plan_of_large_page_numbers():
    """Slots past 2^31."""
    lengths, new, free = [63, 0], [2, 1], [2000000000, 70000001]
    want = oa.kv_plan(lengths, new, free, 0, [[5, -1], [-1, -1]], 64, 4)
    got = run_plan(lengths, new, free, 0, [[5, -1], [-1, -1]], 64, 4, 0)
    for g, w in zip(got, want):
        assert np.array_equal(g.reshape(-1), np.asarray(w).reshape(-1))
    assert got[4].max() > 2 ** 31


# ---------------------------------------------------------------- norm and rotation
def rope_inputs(P, T, Hq, Hkv, D, rot, dtype, seed, rows=50, pad=0):
    g = torch.Generator().manual_seed(seed)
    W = (Hq + 2 * Hkv) * D
    x = torch.randn(P, T, W + pad, generator=g) * torch.exp(2 * torch.randn(P, T, 1, generator=g))
    x = x.to(dtype).cuda()
    ang = torch.randn(rows, rot // 2, generator=g) * 3
    return ([x[r, :, :W] for r in range(P)], [(1 + 0.3 * torch.randn(D, generator=g)).cuda() for _ in range(P)],
            [(1 + 0.3 * torch.randn(D, generator=g)).cuda() for _ in range(P)],
            torch.cat([ang.cos(), ang.sin()], 1).contiguous().cuda(), torch.randint(0, rows, (T,), generator=g).int().cuda())


ROPE = [(1, 1, 1, 1, 64, 64), (2, 5, 3, 1, 64, 32), (3, 33, 8, 2, 128, 128), (2, 7, 5, 5, 128, 96), (1, 130, 4, 4, 128, 16),
        (1, 3, 2, 1, 64, 0), (4, 2, 12, 3, 64, 48)]


@pytest.mark.parametrize("P,T,Hq,Hkv,D,rot", ROPE)
@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("norm", [True, False])
def test_qk_norm_rope(P, T, Hq, Hkv, D, rot, dtype, norm):
    note("qk_norm_rope P=%d T=%d %s norm=%s" % (P, T, dtype, norm))
    x, gq, gk, cs, pos = rope_inputs(P, T, Hq, Hkv, D, rot, dtype, seed=T + D, pad=8 if T == 33 else 0)
    rows = T + 9
    g = torch.Generator().manual_seed(5)
    slots = torch.randperm(rows, generator=g)[:T].cuda()
    q = [poisoned((T, Hq, D)) for _ in range(P)]
    k, v = ([poisoned((T, Hkv, D)) for _ in range(P)] for _ in range(2))
    kc, vc = ([torch.full((rows, Hkv, D), 7.0, dtype=BF, device="cuda") for _ in range(P)] for _ in range(2))
    if T > 4:
        slots[1], slots[3] = -1, rows                   # not written
    A.tp_qk_norm_rope(x, gq if norm else None, gk if norm else None, cs, pos, q, k, v, kc, vc, slots, eps=1e-5)
    torch.cuda.synchronize()
    cs_, pos_, sl = cs.cpu().numpy(), pos.cpu().numpy(), slots.cpu().numpy()
    ok = (sl >= 0) & (sl < rows)
    for r in range(P):
        h = f64(x[r]).reshape(T, -1, D)
        for got, part, gain, cache in ((q[r], h[:, :Hq], gq[r], None), (k[r], h[:, Hq:Hq + Hkv], gk[r], kc[r])):
            want, bound = oa.qk_norm_rope(part, f64(gain) if norm else None, cs_, pos_, 1e-5)
            within(got, want, bound, "heads")
            if cache is not None:
                keep = np.full((rows, Hkv, D), 7.0)
                keep[sl[ok]] = f64(got)[ok]
                assert np.array_equal(f64(cache), keep)
        want_v = x[r].reshape(T, -1, D)[:, Hq + Hkv:].to(BF)
        assert torch.equal(v[r], want_v)
        keep = torch.full((rows, Hkv, D), 7.0, dtype=BF, device="cuda")
        keep[slots[torch.from_numpy(ok).cuda()]] = want_v[torch.from_numpy(ok).cuda()]
        assert torch.equal(vc[r], keep)


def test_qk_norm_rope_positions_outside_the_table_give_nan():
    x, gq, gk, cs, pos = rope_inputs(1, 4, 2, 1, 64, 64, BF, seed=1, rows=10)
    pos[1], pos[2] = 10, -1
    q, k, v = [poisoned((4, 2, 64))], [poisoned((4, 1, 64))], [poisoned((4, 1, 64))]
    A.tp_qk_norm_rope(x, gq, gk, cs, pos, q, k, v)
    bad = torch.tensor([False, True, True, False], device="cuda")
    for t in (q[0], k[0]):
        assert torch.equal(t.isnan().flatten(1).all(1), bad) and torch.equal(t.isnan().flatten(1).any(1), bad)
    assert not v[0].isnan().any()


@pytest.mark.parametrize("P,T,Hq,Hkv,D,rot", ROPE + [(2, 2100, 2, 1, 64, 64)])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("norm", [True, False])
def test_qk_norm_rope_grad(P, T, Hq, Hkv, D, rot, dtype, norm):
    note("qk_norm_rope_grad P=%d T=%d %s norm=%s" % (P, T, dtype, norm))
    x, gq, gk, cs, pos = rope_inputs(P, T, Hq, Hkv, D, rot, dtype, seed=T + D + 1, pad=8 if T == 33 else 0)
    g = torch.Generator().manual_seed(6)
    dq, dk, dv = ([torch.randn(T, h, D, generator=g).to(BF).cuda() for _ in range(P)] for h in (Hq, Hkv, Hkv))
    dx = [poisoned((T, (Hq + 2 * Hkv) * D), dtype) for _ in range(P)]
    dgq, dgk = ([poisoned((D,), torch.float32) for _ in range(P)] for _ in range(2))
    if norm:
        ws = A.tp_qk_norm_rope_grad(dq, dk, dv, x, gq, gk, cs, pos, dx, dgq, dgk, eps=1e-5)
        first = [t.clone() for t in dgq + dgk]
        A.tp_qk_norm_rope_grad(dq, dk, dv, x, gq, gk, cs, pos, dx, dgq, dgk, eps=1e-5, ws=ws)
        assert all(torch.equal(a, b) for a, b in zip(first, dgq + dgk))      # a fixed order of sums
    else:
        A.tp_qk_norm_rope_grad(dq, dk, dv, x, None, None, cs, pos, dx, eps=1e-5)
    torch.cuda.synchronize()
    cs_, pos_ = cs.cpu().numpy(), pos.cpu().numpy()
    for r in range(P):
        h, d = f64(x[r]).reshape(T, -1, D), f64(dx[r]).reshape(T, -1, D)
        for got, part, dz, gain, dg in ((d[:, :Hq], h[:, :Hq], dq[r], gq[r], dgq[r]),
                                        (d[:, Hq:Hq + Hkv], h[:, Hq:Hq + Hkv], dk[r], gk[r], dgk[r])):
            want, bound, wg, bg = oa.qk_norm_rope_grad(f64(dz), part, f64(gain) if norm else None, cs_, pos_, 1e-5)
            within(got, want, bound + (oa.UB * np.abs(want) if dtype == BF else 0), "dx")
            if norm:
                within(dg, wg, bg, "dgain")
        assert np.array_equal(d[:, Hq + Hkv:], f64(dv[r]))


# ---------------------------------------------------------------- packed prompts
def cu(lens):
    return i32([0] + list(np.cumsum(lens)))


def attn_inputs(P, lq, lk, Hq, Hkv, D, seed, layout="dense"):
    g = torch.Generator().manual_seed(seed)
    Tq, Tk = sum(lq), sum(lk)
    rnd = lambda *s: torch.randn(*s, generator=g).to(BF).cuda()      # noqa: E731
    if layout == "packed":                               # slices of one row per token
        assert Tq == Tk
        x = [rnd(Tq, Hq + 2 * Hkv, D) for _ in range(P)]
        return [t[:, :Hq] for t in x], [t[:, Hq:Hq + Hkv] for t in x], [t[:, Hq + Hkv:] for t in x]
    return [rnd(Tq, Hq, D) for _ in range(P)], [rnd(Tk, Hkv, D) for _ in range(P)], [rnd(Tk, Hkv, D) for _ in range(P)]


def check_attention(q, k, v, o, lse, lq, lk, causal, scale, ranks=None):
    Hq, Hkv = q[0].shape[1], k[0].shape[1]
    G = Hq // Hkv
    for r in ranks or range(len(q)):
        qr, kr, vr, orr, lr = f64(q[r]), f64(k[r]), f64(v[r]), f64(o[r]), f64(lse[r])
        a = b = 0
        for nq, nk in zip(lq, lk):
            see = oa.visible(nq, nk, causal)
            for h in range(Hq):
                wo, wl, eo, el, _, _ = oa.attention(qr[a:a + nq, h], kr[b:b + nk, h // G], vr[b:b + nk, h // G], see, scale)
                within(orr[a:a + nq, h], wo, eo, "o, prompt of %d, head %d" % (nq, h))
                within(lr[h, a:a + nq], wl, el, "lse, prompt of %d, head %d" % (nq, h))
            a, b = a + nq, b + nk


# (query lengths, key lengths or None for the same)
MANY = [150, 61, 200] * 14                               # enough workgroups for every compute unit
LENS = [([1], None), (MANY, None), ([31], None), ([32], None), ([33], None), ([64], None), ([65], None), ([127], None), ([129], None),
        ([300], None), ([0], None), ([5, 0, 1, 64, 0, 130, 2], None), ([1] * 70, None), ([3, 2] * 65, None),
        ([1, 1, 7], [300, 1, 129]),                      # fewer queries than keys: a prompt's last part
        ([70, 9, 4], [5, 0, 4])]                         # more queries than keys: causal rows that see none


@pytest.mark.parametrize("lq,lk", LENS)
@pytest.mark.parametrize("Hq,Hkv,D", [(1, 1, 64), (3, 1, 128), (4, 2, 64), (8, 1, 128), (10, 2, 128)])
@pytest.mark.parametrize("causal", [True, False])
def test_attention(lq, lk, Hq, Hkv, D, causal):
    note("attention lq=%s lk=%s Hq=%d Hkv=%d D=%d causal=%s" % (lq[:8], lk, Hq, Hkv, D, causal))
    lk = lk or lq
    P = 2
    q, k, v = attn_inputs(P, lq, lk, Hq, Hkv, D, seed=sum(lq) + D, layout="packed" if lk is lq and Hq == 4 else "dense")
    o, lse = [poisoned((sum(lq), Hq, D)) for _ in range(P)], [poisoned((Hq, sum(lq)), torch.float32) for _ in range(P)]
    A.tp_attention(q, k, v, o, cu(lq), cu(lk), lse=lse, causal=causal)
    torch.cuda.synchronize()
    check_attention(q, k, v, o, lse, lq, lk, causal, 1 / math.sqrt(D), ranks=None if sum(lq) < 100 else [1])


@pytest.mark.parametrize("scale", [0.01, 3.0])
def test_attention_scales_and_large_scores(scale):
    """Scores far apart: the running maximum moves by more than the exponent
    range and most weights vanish."""
    lq, Hq, Hkv, D = [200, 77], 2, 1, 128
    q, k, v = attn_inputs(1, lq, lq, Hq, Hkv, D, seed=3)
    for i in range(0, 277, 13):
        k[0][i] *= 1 + i / 20
    o, lse = [poisoned((277, Hq, D))], [poisoned((Hq, 277), torch.float32)]
    A.tp_attention(q, k, v, o, cu(lq), cu(lq), lse=lse, scale=scale)
    torch.cuda.synchronize()
    check_attention(q, k, v, o, lse, lq, lq, True, scale)


def test_attention_many_ranks_and_no_lse():
    lq, Hq, Hkv, D, P = [40, 3], 2, 2, 64, 5
    q, k, v = attn_inputs(P, lq, lq, Hq, Hkv, D, seed=4)
    o, o2 = ([poisoned((43, Hq, D)) for _ in range(P)] for _ in range(2))
    lse = [poisoned((Hq, 43), torch.float32) for _ in range(P)]
    A.tp_attention(q, k, v, o, cu(lq), cu(lq), lse=lse)
    A.tp_attention(q, k, v, o2, cu(lq), cu(lq))
    torch.cuda.synchronize()
    check_attention(q, k, v, o, lse, lq, lq, True, 1 / 8)
    assert all(torch.equal(a, b) for a, b in zip(o, o2))


def test_attention_rows_of_other_prompts_take_no_part():
    """Infinities and NaN in the keys and values of neighbouring prompts, and
    past the last prompt's end, leave a prompt's rows alone."""
    lq, Hq, Hkv, D = [50, 45, 70], 4, 2, 128
    q, k, v = attn_inputs(1, [170], [170], Hq, Hkv, D, seed=8)
    for t in (k[0], v[0]):
        t[:50], t[95:120], t[165:] = float("nan"), float("inf"), float("nan")
    o, lse = [poisoned((170, Hq, D))], [poisoned((Hq, 170), torch.float32)]
    A.tp_attention(q, k, v, o, cu(lq), cu(lq), lse=lse)
    torch.cuda.synchronize()
    mid = slice(50, 95)
    check_attention([q[0][mid]], [k[0][mid]], [v[0][mid]], [o[0][mid]], [lse[0][:, mid]], [45], [45], True, 1 / math.sqrt(D))
    assert o[0][:50].isnan().all()                       # a prompt of NaN is NaN


@pytest.mark.parametrize("at,bad", [(70, float("nan")), (40, float("inf")), (199, float("-inf")), (0, float("nan"))])
@pytest.mark.parametrize("Hq,Hkv,D", [(1, 1, 64), (4, 1, 128)])
def test_attention_keys_and_values_that_a_causal_query_does_not_see(at, bad, Hq, Hkv, D):
    """A key and value that are not finite reach only the queries from their
    own place on; the others, of the same tiles too, are as without them."""
    lq = [200]
    q, k, v = attn_inputs(1, lq, lq, Hq, Hkv, D, seed=at)
    o, lse = ([poisoned((200, Hq, D))], [poisoned((Hq, 200), torch.float32)])
    v[0][at, 0, 5] = bad
    A.tp_attention(q, k, v, o, cu(lq), cu(lq), lse=lse)
    torch.cuda.synchronize()
    if at:
        part = slice(0, at)
        check_attention([q[0][part]], [k[0][part]], [v[0][part]], [o[0][part]], [lse[0][:, part]], [at], [at], True, D ** -0.5)
    assert not o[0][at:, :, 5].isfinite().any() and o[0][at:, :, 6].isfinite().all()
    k[0][at, 0, 3] = float("nan")
    A.tp_attention(q, k, v, o, cu(lq), cu(lq), lse=lse)
    torch.cuda.synchronize()
    if at:
        check_attention([q[0][part]], [k[0][part]], [v[0][part]], [o[0][part]], [lse[0][:, part]], [at], [at], True, D ** -0.5)
    assert o[0][at:].isnan().all()


def test_attention_offsets_outside_the_tensors_are_not_followed():
    q, k, v = attn_inputs(1, [60], [60], 2, 1, 64, seed=9)
    o, lse = [torch.zeros(60, 2, 64, dtype=BF, device="cuda")], [torch.zeros(2, 60, device="cuda")]
    A.tp_attention(q, k, v, o, i32([-5, 20, 10, 1000]), i32([0, 20, 1 << 30, 60]), lse=lse)
    torch.cuda.synchronize()
    check_attention([q[0][:20]], [k[0][:20]], [v[0][:20]], [o[0][:20]], [lse[0][:, :20]], [20], [20], True, 1 / 8)


def check_grad(do, q, k, v, dq, dk, dv, lq, lk, causal, scale, ranks=None):
    Hq, Hkv = q[0].shape[1], k[0].shape[1]
    G = Hq // Hkv
    for r in ranks or range(len(q)):
        t = [f64(x[r]) for x in (do, q, k, v, dq, dk, dv)]
        a = b = 0
        for nq, nk in zip(lq, lk):
            see = oa.visible(nq, nk, causal)
            A_, B_ = slice(a, a + nq), slice(b, b + nk)
            for h in range(Hkv):
                wk = wv = ek = ev = 0
                for i in range(h * G, h * G + G):
                    (wq, k1, v1), (eq, k2, v2) = oa.attention_grad(t[0][A_, i], t[1][A_, i], t[2][B_, h], t[3][B_, h], see, scale)
                    within(t[4][A_, i], wq, eq, "dq, prompt of %d, head %d" % (nq, i))
                    wk, wv, ek, ev = wk + k1, wv + v1, ek + k2, ev + v2
                within(t[5][B_, h], wk, ek, "dk, prompt of %d, head %d" % (nq, h))
                within(t[6][B_, h], wv, ev, "dv, prompt of %d, head %d" % (nq, h))
            a, b = a + nq, b + nk


@pytest.mark.parametrize("lq,lk", LENS)
@pytest.mark.parametrize("Hq,Hkv,D", [(1, 1, 64), (3, 1, 128), (4, 2, 64), (10, 2, 128)])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_grad(lq, lk, Hq, Hkv, D, causal):
    note("attention_grad lq=%s lk=%s Hq=%d Hkv=%d D=%d causal=%s" % (lq[:8], lk, Hq, Hkv, D, causal))
    lk = lk or lq
    P, Tq, Tk = 2, sum(lq), sum(lk)
    packed = lk is lq and Hq == 4
    q, k, v = attn_inputs(P, lq, lk, Hq, Hkv, D, seed=Tq + D, layout="packed" if packed else "dense")
    g = torch.Generator().manual_seed(11)
    do = [torch.randn(Tq, Hq, D, generator=g).to(BF).cuda() for _ in range(P)]
    o, lse = [poisoned((Tq, Hq, D)) for _ in range(P)], [poisoned((Hq, Tq), torch.float32) for _ in range(P)]
    A.tp_attention(q, k, v, o, cu(lq), cu(lk), lse=lse, causal=causal)
    if packed:                                           # slices of one packed row, as the inputs
        x = [poisoned((Tq, Hq + 2 * Hkv, D)) for _ in range(P)]
        dq, dk, dv = [t[:, :Hq] for t in x], [t[:, Hq:Hq + Hkv] for t in x], [t[:, Hq + Hkv:] for t in x]
    else:
        dq, (dk, dv) = [poisoned((Tq, Hq, D)) for _ in range(P)], [[poisoned((Tk, Hkv, D)) for _ in range(P)] for _ in range(2)]
    ws = A.tp_attention_grad(do, q, k, v, o, lse, dq, dk, dv, cu(lq), cu(lk), causal=causal)
    first = [t.clone() for t in dq + dk + dv]
    A.tp_attention_grad(do, q, k, v, o, lse, dq, dk, dv, cu(lq), cu(lk), causal=causal, ws=ws)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, dq + dk + dv))
    check_grad(do, q, k, v, dq, dk, dv, lq, lk, causal, 1 / math.sqrt(D), ranks=None if Tq < 100 else [1])


def test_attention_grad_against_differences():
    """The gradient along a direction of each input is the change of sum(o do)
    when the input moves along it, taken from the kernel's own forward pass at
    steps large enough for bf16.  The step's second-order part cancels in the
    two-sided difference; what is left of the tolerance is o's bf16 rounding,
    2^-9 |o do| a term with random signs, over the step."""
    lq, Hq, Hkv, D = [150, 90], 4, 2, 64
    q, k, v = attn_inputs(1, lq, lq, Hq, Hkv, D, seed=21)
    g = torch.Generator().manual_seed(22)
    do = [torch.randn(240, Hq, D, generator=g).to(BF).cuda()]
    o, lse = [poisoned((240, Hq, D))], [poisoned((Hq, 240), torch.float32)]
    A.tp_attention(q, k, v, o, cu(lq), cu(lq), lse=lse)
    d = [[torch.empty_like(t[0])] for t in (q, k, v)]
    A.tp_attention_grad(do, q, k, v, o, lse, *d, cu(lq), cu(lq))
    step = 2.0 ** -4
    for i in range(3):
        # a direction along the gradient's signs: moves of one step, kept
        # exact by rounding both sides to bf16 and taking the move that is left
        x = [q, k, v]
        up, down = ((x[i][0].float() + s * d[i][0].float().sign()).to(BF) for s in (step, -step))
        sums = []
        for t in (up, down):
            y = list(x)
            y[i] = [t]
            A.tp_attention(*y, o, cu(lq), cu(lq))
            sums.append((o[0].double() * do[0].double()).sum())
        want = (d[i][0].double() * (up.double() - down.double())).sum()
        got = sums[0] - sums[1]
        noise = 2.0 ** -9 * 8 * (o[0].double() * do[0].double()).norm()
        # third-order part: up to step^2 of the whole for directions of unit size per element
        assert abs(float(got - want)) <= float(noise) + 0.1 * abs(float(want)), (i, float(got), float(want), float(noise))


# ---------------------------------------------------------------- decode
def decode_inputs(P, lens, prefix, Hq, Hkv, D, page, seed, spare=3):
    g = torch.Generator().manual_seed(seed)
    B, per = len(lens), [-(-max(0, n) // page) for n in lens]
    shared = -(-prefix // page)
    pages = sum(per) + shared + spare
    pool = torch.randperm(pages, generator=g).int()
    width = max(per + [1])
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = shared
    for b, n in enumerate(per):
        table[b, :n] = pool[at:at + n]
        at += n
    rnd = lambda *s: torch.randn(*s, generator=g).to(BF).cuda()      # noqa: E731
    kc, vc = ([rnd(pages * page, Hkv, D) for _ in range(P)] for _ in range(2))
    q = [rnd(B, Hq, D) for _ in range(P)]
    # rows that no key fills must not matter
    used = torch.zeros(pages * page, dtype=torch.bool)
    for p, n in [(pool[:shared], prefix)] + [(table[b, :per[b]], lens[b]) for b in range(B)]:
        for j in range(max(0, n)):
            used[int(p[j // page]) * page + j % page] = True
    for t in kc + vc:
        t[~used.cuda()] = float("nan")
    return q, kc, vc, table.cuda(), i32(list(lens)), pool[:shared].cuda() if shared else None


def check_decode(q, kc, vc, o, table, lens, pp, prefix, page, scale):
    tab, pre = table.cpu().numpy(), [] if pp is None else pp.cpu().numpy()
    for r in range(len(q)):
        qr, kr, vr, orr = f64(q[r]), f64(kc[r]), f64(vc[r]), f64(o[r])
        G = qr.shape[1] // kr.shape[1]
        for b in range(qr.shape[0]):
            for h in range(qr.shape[1]):
                w, e = oa.decode(qr[b, h], kr[:, h // G], vr[:, h // G], tab[b], lens[b], pre, prefix, page, scale)
                within(orr[b, h], w, e, "request %d, head %d" % (b, h))


@pytest.mark.parametrize("lens,prefix", [
    ([1], 0), ([31, 32, 33], 0), ([0, 5, -3, 64], 0), ([65, 1, 200], 17), ([0], 64), ([0, 3], 1), ([700, 20], 0),
    ([2100], 0), ([40, 41] * 20, 300), ([5000], 0), ([7], 2000)])
@pytest.mark.parametrize("Hq,Hkv,D,page", [(1, 1, 64, 16), (4, 2, 128, 16), (8, 1, 64, 64), (3, 3, 128, 1), (34, 1, 64, 8)])
def test_decode(lens, prefix, Hq, Hkv, D, page):
    note("decode lens=%s prefix=%d Hq=%d Hkv=%d D=%d page=%d" % (lens[:6], prefix, Hq, Hkv, D, page))
    P = 2
    q, kc, vc, table, ln, pp = decode_inputs(P, lens, prefix, Hq, Hkv, D, page, seed=len(lens) + prefix)
    o = [poisoned((len(lens), Hq, D)) for _ in range(P)]
    ws = A.tp_attention_decode(q, kc, vc, o, table, ln, page_size=page, prefix_pages=pp, prefix_len=prefix)
    first = [t.clone() for t in o]
    A.tp_attention_decode(q, kc, vc, o, table, ln, page_size=page, prefix_pages=pp, prefix_len=prefix, ws=ws)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, o))
    check_decode(q, kc, vc, o, table, lens, pp, prefix, page, 1 / math.sqrt(D))


def test_decode_pages_outside_the_cache_take_no_part():
    lens, page = [100, 70, 40], 16
    q, kc, vc, table, ln, pp = decode_inputs(1, lens, 50, 2, 1, 64, page, seed=77)
    table[0, 2], table[0, 5], table[1, 0], pp[1] = -1, 1 << 30, kc[0].shape[0] // page, -9
    table[2, :] = -1
    o = [poisoned((3, 2, 64))]
    A.tp_attention_decode(q, kc, vc, o, table, ln, page_size=page, prefix_pages=pp, prefix_len=50)
    torch.cuda.synchronize()
    check_decode(q, kc, vc, o, table, lens, pp, 50, page, 1 / 8)


def test_decode_lengths_past_the_table_are_clamped():
    q, kc, vc, table, ln, _ = decode_inputs(1, [64, 32], 0, 2, 1, 64, 16, seed=78)
    o = [poisoned((2, 2, 64))]
    A.tp_attention_decode(q, kc, vc, o, table[:, :2].contiguous(), i32([1000, 1 << 30]), page_size=16)
    torch.cuda.synchronize()
    check_decode(q, kc, vc, o, table[:, :2], [32, 32], None, 0, 16, 1 / 8)
