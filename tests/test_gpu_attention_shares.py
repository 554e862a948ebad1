"""GPU tests of long prompts in few workgroups, whose keys go to two or four
shares of waves that are joined at the end."""
import numpy as np
import pytest
import torch

from ring_collectives_amd import _native as N
from ring_collectives_amd import attention as A

from test_gpu_attention import BF, attn_inputs, check_attention, check_grad, cu, poisoned

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    N.lib()
    yield


def run(P, lq, lk, Hq, Hkv, D, causal, seed, train=False):
    Tq = sum(lq)
    q, k, v = attn_inputs(P, lq, lk, Hq, Hkv, D, seed=seed)
    o, lse = [poisoned((Tq, Hq, D)) for _ in range(P)], [poisoned((Hq, Tq), torch.float32) for _ in range(P)]
    A.tp_attention(q, k, v, o, cu(lq), cu(lk), lse=lse, causal=causal)
    check_attention(q, k, v, o, lse, lq, lk, causal, D ** -0.5)
    if train:
        do = [torch.randn(Tq, Hq, D, device="cuda").to(BF) for _ in range(P)]
        d = [[poisoned(tuple(t.shape)) for t in x] for x in (q, k, v)]
        A.tp_attention_grad(do, q, k, v, o, lse, *d, cu(lq), cu(lk), causal=causal)
        check_grad(do, q, k, v, *d, lq, lk, causal, D ** -0.5)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("P,lq,lk,Hq,Hkv,D", [
    (1, [257], [257], 2, 1, 64),             # two shares, five tiles: the second share's last is missing
    (2, [300, 1, 211], [300, 600, 211], 4, 2, 64),
    (1, [700, 40], [600, 1], 2, 2, 64),      # rows that see no key; a prompt of one tile, the other shares idle
    (1, [1, 2, 3], [900, 0, 1000], 3, 1, 64),
    (1, [600], [600], 2, 1, 128),
    (2, [70, 513], [900, 700], 2, 2, 128),
    (1, [1200, 30], [1000, 64], 2, 1, 128),
])
def test_two_shares(P, lq, lk, Hq, Hkv, D, causal):
    run(P, lq, lk, Hq, Hkv, D, causal, seed=sum(lq) + D)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lq,lk", [([33], [2049]), ([2100], [2100]), ([200, 5], [70, 4200])])
def test_four_shares(lq, lk, causal):
    run(1, lq, lk, 2, 1, 64, causal, seed=sum(lq))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lq,lk", [([769], [769]), ([300, 700], [1500, 900])])
def test_gradient_in_two_shares(lq, lk, causal, D):
    run(2, lq, lk, 2, 1, D, causal, seed=sum(lk), train=True)


@pytest.mark.parametrize("D,n", [(64, 300), (64, 2200), (128, 700)])
def test_values_not_finite_past_the_mask(D, n):
    """A value or a key that is not finite reaches only the queries that see
    it, whichever share it falls to."""
    q, k, v = attn_inputs(1, [n], [n], 2, 1, D, seed=n)
    o, want = [poisoned((n, 2, D))], [poisoned((n, 2, D))]
    A.tp_attention(q, k, v, want, cu([n]), cu([n]))
    for at in (n - 1, n - 70, n - 140):
        for t, x in ((v, float("inf")), (v, float("nan")), (k, float("nan"))):
            keep = t[0][at].clone()
            t[0][at] = x
            A.tp_attention(q, k, v, o, cu([n]), cu([n]))
            t[0][at] = keep
            torch.cuda.synchronize()
            # rows made again key by key differ by their roundings alone
            assert torch.allclose(o[0][:at].float(), want[0][:at].float(), rtol=2.0 ** -6, atol=2.0 ** -6)
            assert not torch.isfinite(o[0][at:].float()).all(dim=-1).any()
    assert np.isfinite(want[0].float().cpu().numpy()).all()
