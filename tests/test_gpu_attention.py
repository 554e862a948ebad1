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
LENS = [([1], None), ([31], None), ([32], None), ([33], None), ([64], None), ([65], None), ([127], None), ([129], None),
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


def test_attention_offsets_outside_the_tensors_are_not_followed():
    q, k, v = attn_inputs(1, [60], [60], 2, 1, 64, seed=9)
    o, lse = [torch.zeros(60, 2, 64, dtype=BF, device="cuda")], [torch.zeros(2, 60, device="cuda")]
    A.tp_attention(q, k, v, o, i32([-5, 20, 10, 1000]), i32([0, 20, 1 << 30, 60]), lse=lse)
    torch.cuda.synchronize()
    check_attention([q[0][:20]], [k[0][:20]], [v[0][:20]], [o[0][:20]], [lse[0][:, :20]], [20], [20], True, 1 / 8)
