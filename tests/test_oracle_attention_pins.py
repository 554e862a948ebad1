"""Pins of the attention oracle that need no GPU: its gradients against
differences of its own forward formulas in float64, its attention against
another way of writing the sum, its cache plan against a token-by-token model,
and its bounds against plausible slips."""
import numpy as np
import pytest

from oracle import attention as oa


def rng(seed):
    return np.random.default_rng(seed)


@pytest.mark.parametrize("nq,nk,causal", [(5, 5, True), (3, 7, True), (4, 4, False), (7, 3, True), (1, 1, True), (2, 0, True)])
def test_attention_is_the_weighted_mean_of_the_values_seen(nq, nk, causal):
    r = rng(1)
    q, k, v = r.normal(size=(nq, 8)), r.normal(size=(nk, 8)), r.normal(size=(nk, 8))
    o, lse = oa.attention(q, k, v, oa.visible(nq, nk, causal), 0.3)[:2]
    for i in range(nq):
        top = np.zeros(8)
        tot = 0.0
        for j in range(nk):
            if causal and j > i + (nk - nq):
                continue
            w = np.exp(0.3 * float(q[i] @ k[j]))
            top, tot = top + w * v[j], tot + w
        if tot == 0:
            assert not o[i].any() and lse[i] == -np.inf
        else:
            assert np.allclose(o[i], top / tot, rtol=1e-12) and np.isclose(lse[i], np.log(tot), rtol=1e-12)


@pytest.mark.parametrize("nq,nk,causal", [(4, 4, True), (2, 6, True), (6, 3, True), (3, 5, False)])
def test_attention_gradient_against_differences(nq, nk, causal):
    r = rng(2)
    q, k, v, do = (r.normal(size=(n, 6)) for n in (nq, nk, nk, nq))
    see = oa.visible(nq, nk, causal)
    grads = oa.attention_grad(do, q, k, v, see, 0.4)[0]
    x = [q, k, v]
    h = 1e-6
    for a, g in enumerate(grads):
        for i in np.ndindex(x[a].shape):
            f = []
            for s in (h, -h):
                y = [t.copy() for t in x]
                y[a][i] += s
                f.append((oa.attention(*y, see, 0.4)[0] * do).sum())
            assert abs((f[0] - f[1]) / (2 * h) - g[i]) < 1e-7


@pytest.mark.parametrize("D,rot", [(8, 8), (8, 4), (16, 0)])
@pytest.mark.parametrize("norm", [True, False])
def test_norm_and_rotation_gradient_against_differences(D, rot, norm):
    r = rng(3)
    x, dz, gain = r.normal(size=(3, 2, D)), r.normal(size=(3, 2, D)), 1 + 0.3 * r.normal(size=D)
    ang = r.normal(size=(5, rot // 2))
    cs, pos = np.concatenate([np.cos(ang), np.sin(ang)], 1), np.array([4, 0, 2])
    f = lambda x, g: (oa.qk_norm_rope(x, g if norm else None, cs, pos, 1e-3)[0] * dz).sum()      # noqa: E731
    dx, _, dg, _ = oa.qk_norm_rope_grad(dz, x, gain if norm else None, cs, pos, 1e-3)
    h = 1e-6
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = h
        assert abs((f(x + e, gain) - f(x - e, gain)) / (2 * h) - dx[i]) < 1e-7
    if norm:
        for i in range(D):
            e = np.zeros(D)
            e[i] = h
            assert abs((f(x, gain + e) - f(x, gain - e)) / (2 * h) - dg[i]) < 1e-7


def test_rotation_turns_pairs_and_keeps_lengths():
    r = rng(4)
    x, ang = r.normal(size=(2, 1, 8)), r.normal(size=(3, 2))
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    z = oa.qk_norm_rope(x, None, cs, np.array([1, 2]), 0.0)[0]
    for t, p in enumerate((1, 2)):
        for i in range(2):
            w = complex(x[t, 0, i], x[t, 0, i + 2]) * np.exp(1j * ang[p, i])
            assert np.allclose([z[t, 0, i], z[t, 0, i + 2]], [w.real, w.imag])
        assert np.array_equal(z[t, 0, 4:], x[t, 0, 4:])


def test_plan_small_example():
    # pages of 4: request 0 holds 3 tokens (page 7) and adds 2, request 1 adds
    # none, request 2 starts with 5; free pages from entry 1 on
    table, after, cu, pos, slots, used = oa.kv_plan([3, 6, 0], [2, 0, 5], [9, 2, 5, 1], 1, [[7, -1], [3, 4], [-1, -1]], 4, 9,
                                                    prefix_len=100)
    assert table.tolist() == [[7, 2], [3, 4], [5, 1]] and after.tolist() == [5, 6, 5] and cu.tolist() == [0, 2, 2, 7]
    assert pos.tolist() == [103, 104, 100, 101, 102, 103, 104, 0, 0]
    assert slots.tolist() == [31, 8, 20, 21, 22, 23, 4, -1, -1] and used == 4


def test_plan_gives_every_token_a_row_of_its_own():
    r = rng(5)
    lens, new = r.integers(0, 40, 30), r.integers(0, 20, 30)
    have, want = -(-lens // 8), -(-(lens + new) // 8)
    pool = r.permutation(int(want.sum()))
    table = np.full((30, want.max()), -1)
    at = 0
    for b in range(30):
        table[b, :have[b]] = pool[at:at + have[b]]
        at += have[b]
    out = oa.kv_plan(lens, new, pool[at:], 0, table, 8, int(new.sum()))
    rows = list(out[4])
    for b in range(30):
        rows += [int(out[0][b, j // 8]) * 8 + j % 8 for j in range(lens[b])]
    assert min(rows) >= 0 and len(set(rows)) == len(rows) == int((lens + new).sum())
    assert out[5] == len(pool) - at


@pytest.mark.parametrize("slip", ["scale", "mask", "neighbour", "no max", "value"])
def test_attention_bounds_reject_slips(slip):
    r = rng(6)
    q, k, v = (r.normal(size=(40, 64)).astype(np.float32).astype(np.float64) for _ in range(3))
    see = oa.visible(40, 40, True)
    o, lse, eo, el, _, _ = oa.attention(q, k, v, see, 0.125)
    if slip == "scale":
        got = oa.attention(q, k, v, see, 0.13)[0]
    elif slip == "mask":
        got = oa.attention(q, k, v, np.tril(np.ones((40, 40), bool), -1), 0.125)[0]
    elif slip == "neighbour":
        got = np.roll(o, 1, 0)
    elif slip == "no max":
        s = np.where(see, q @ k.T * 0.125, 0.0)          # masked scores of 0 instead of none
        got = (np.exp(s) @ v) / np.exp(s).sum(-1, keepdims=True)
    else:
        w = v.copy()
        w[3] += 0.5
        got = oa.attention(q, k, w, see, 0.125)[0]
    assert (np.abs(got - o) > eo).any()
