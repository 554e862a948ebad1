"""GPU tests of long prompts in many workgroups, which take the kernels that
the longest calls take (one share of waves a workgroup, 128 keys a workgroup
for dK and dV), and of calls of 16 and 64 ranks."""
import pytest
import torch

from oracle import attention as oa
from ring_collectives_amd import _native as N
from ring_collectives_amd import attention as A

from _gpu_helpers import note
from test_gpu_attention import (BF, attn_inputs, check_attention, check_decode, check_grad, cu, decode_inputs, f64, poisoned,
                                rope_inputs, within)
from test_gpu_attention_shares import run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    N.lib()
    yield


def groups(total, per, prompts, units):
    """Workgroups of 128 rows that a call makes (an upper bound, as it is launched)."""
    return (total * per // 128 + prompts) * units


@pytest.mark.parametrize("P,Hq,Hkv,D", [(8, 8, 8, 64), (3, 8, 8, 128), (4, 8, 4, 128)])
@pytest.mark.parametrize("lq,lk", [([1100, 1333], None), ([900, 1100], [1400, 1333])])
@pytest.mark.parametrize("causal", [True, False])
def test_long_prompts_in_many_workgroups(P, Hq, Hkv, D, lq, lk, causal):
    note("attention P=%d Hq=%d Hkv=%d D=%d lq=%s lk=%s causal=%s" % (P, Hq, Hkv, D, lq, lk, causal))
    lk = lk or lq
    Tq, Tk, B, units = sum(lq), sum(lk), len(lq), P * Hkv
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    # neither the forward pass nor dQ in shares, nor dK and dV in workgroups of 32 keys
    assert groups(Tq, Hq // Hkv, B, units) > (4 * cus if D == 64 else 1.5 * cus)
    assert groups(Tk, 1, B, units) > cus + units
    q, k, v = attn_inputs(P, lq, lk, Hq, Hkv, D, seed=Tq + D)
    g = torch.Generator().manual_seed(31)
    do = [torch.randn(Tq, Hq, D, generator=g).to(BF).cuda() for _ in range(P)]
    o, lse = [poisoned((Tq, Hq, D)) for _ in range(P)], [poisoned((Hq, Tq), torch.float32) for _ in range(P)]
    d = [[poisoned(tuple(t.shape)) for t in x] for x in (q, k, v)]
    A.tp_attention(q, k, v, o, cu(lq), cu(lk), lse=lse, causal=causal)
    A.tp_attention_grad(do, q, k, v, o, lse, *d, cu(lq), cu(lk), causal=causal)
    torch.cuda.synchronize()
    G = Hq // Hkv
    for r, h in ((0, Hkv - 1), (P - 1, 0)):                  # one key head each of the first and the last rank
        key = lambda x: [x[r][:, h:h + 1]]                                # noqa: E731
        query = lambda x: [x[r][:, h * G:h * G + G]]                      # noqa: E731
        check_attention(query(q), key(k), key(v), query(o), [lse[r][h * G:h * G + G]], lq, lk, causal, D ** -0.5)
        check_grad(query(do), query(q), key(k), key(v), query(d[0]), key(d[1]), key(d[2]), lq, lk, causal, D ** -0.5)
    assert all(bool(t.isfinite().all()) for x in (o, lse, *d) for t in x)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_gradient_in_two_shares_with_a_full_last_tile(causal, D):
    """831 keys: thirteen tiles, the last of 63, so that leaving any out shows."""
    run(2, [831], [831], 2, 1, D, causal, seed=831, train=True)


@pytest.mark.parametrize("P", [16, 64])
@pytest.mark.parametrize("D", [64, 128])
def test_many_ranks(P, D):
    """Every rank's own buffers, in each of the calls."""
    note("attention calls of %d ranks, D=%d" % (P, D))
    Hq, Hkv, lens = 2, 1, [37, 5]
    T = sum(lens)
    some = sorted({0, 1, P // 2 + 3, P - 1})
    x, gq, gk, cs, pos = rope_inputs(P, T, Hq, Hkv, D, D, torch.float32, seed=P + D)
    q, k, v = ([poisoned((T, h, D)) for _ in range(P)] for h in (Hq, Hkv, Hkv))
    A.tp_qk_norm_rope(x, gq, gk, cs, pos, q, k, v, eps=1e-5)
    do = [torch.randn(T, Hq, D, device="cuda").to(BF) for _ in range(P)]
    o, lse = [poisoned((T, Hq, D)) for _ in range(P)], [poisoned((Hq, T), torch.float32) for _ in range(P)]
    dq, dk, dv = ([poisoned(tuple(t.shape)) for t in y] for y in (q, k, v))
    A.tp_attention(q, k, v, o, cu(lens), cu(lens), lse=lse)
    A.tp_attention_grad(do, q, k, v, o, lse, dq, dk, dv, cu(lens), cu(lens))
    dx = [poisoned(tuple(t.shape), torch.float32) for t in x]
    dgq, dgk = ([poisoned((D,), torch.float32) for _ in range(P)] for _ in range(2))
    A.tp_qk_norm_rope_grad(dq, dk, dv, x, gq, gk, cs, pos, dx, dgq, dgk, eps=1e-5)
    torch.cuda.synchronize()
    cs_, pos_ = cs.cpu().numpy(), pos.cpu().numpy()
    for r in some:
        h, d = f64(x[r]).reshape(T, -1, D), f64(dx[r]).reshape(T, -1, D)
        for got, part, gain, dz, dpart, dg in ((q[r], h[:, :Hq], gq[r], dq[r], d[:, :Hq], dgq[r]),
                                               (k[r], h[:, Hq:Hq + Hkv], gk[r], dk[r], d[:, Hq:Hq + Hkv], dgk[r])):
            within(got, *oa.qk_norm_rope(part, f64(gain), cs_, pos_, 1e-5), "heads of rank %d" % r)
            want, bound, wg, bg = oa.qk_norm_rope_grad(f64(dz), part, f64(gain), cs_, pos_, 1e-5)
            within(dpart, want, bound, "dx of rank %d" % r)
            within(dg, wg, bg, "dgain of rank %d" % r)
        assert torch.equal(v[r], x[r].view(T, -1, D)[:, Hq + Hkv:].to(BF))
    check_attention(q, k, v, o, lse, lens, lens, True, D ** -0.5, ranks=some)
    check_grad(do, q, k, v, dq, dk, dv, lens, lens, True, D ** -0.5, ranks=some)
    # decode, behind a prefix and without one
    for prefix in (0, 20):
        q1, kc, vc, table, ln, pp = decode_inputs(P, [33, 0, 70], prefix, Hq, Hkv, D, 16, seed=P)
        o1 = [poisoned((3, Hq, D)) for _ in range(P)]
        A.tp_attention_decode(q1, kc, vc, o1, table, ln, page_size=16, prefix_pages=pp, prefix_len=prefix)
        torch.cuda.synchronize()
        pick = lambda y: [y[r] for r in some]                             # noqa: E731
        check_decode(pick(q1), pick(kc), pick(vc), pick(o1), table, [33, 0, 70], pp, prefix, 16, D ** -0.5)
