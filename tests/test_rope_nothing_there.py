"""Norm and rotation where a tensor has no element, and so no address: no
tokens for the cache, a cache without rows, a table without positions."""
import pytest
import torch

from ring_collectives_amd import _native as N
from ring_collectives_amd import attention as A

BF = torch.bfloat16


def test_no_tokens_for_the_cache():
    """The slots of no token may be a null pointer; those of some may not."""
    def call(T, slots=None, cache=True):
        p = [N.ptr_array([(i + 1) << 28, ((i + 1) << 28) + 0x1000000])[0] for i in range(4)]
        kc = (p[2], p[3]) if cache else (None, None)
        return N.lib().tp_qk_norm_rope(p[0], None, None, 0x20000, 0x30000, p[1], None, None, *kc, slots, 2, T, 4, 2, 64, 64,
                                       100, 50, 512, 1e-6, N.RING_BF16, None)

    assert call(0) == N.RING_OK == call(0, slots=0x40000)
    assert call(3) == N.RING_EINVAL
    assert call(3, slots=0x40000, cache=False) == N.RING_EINVAL
    assert call(0, slots=0x40004) == N.RING_EINVAL               # not aligned


def inputs(T, rows, P=2, Hq=4, Hkv=2, D=64):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    x = [torch.randn(T, (Hq + 2 * Hkv) * D, device="cuda").to(BF) for _ in range(P)]
    gain = [torch.ones(D, device="cuda") for _ in range(P)]
    e = lambda n: [torch.full((T, n, D), 5.0, dtype=BF, device="cuda") for _ in range(P)]      # noqa: E731
    return x, gain, torch.ones(rows, D, device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda"), e(Hq), e(Hkv), e(Hkv)


@pytest.mark.gpu
@pytest.mark.parametrize("keep", [False, True])
def test_no_tokens(keep):
    x, gain, cs, pos, q, k, v = inputs(0, 10)
    cache = [[torch.full((32, 2, 64), 5.0, dtype=BF, device="cuda") for _ in range(2)] for _ in range(2)]
    slots = torch.empty(0, dtype=torch.int64, device="cuda")
    A.tp_qk_norm_rope(x, gain, gain, cs, pos, q, k if keep else None, v if keep else None, *cache, slots)
    torch.cuda.synchronize()
    assert all(bool((t == 5).all()) for t in cache[0] + cache[1])


@pytest.mark.gpu
@pytest.mark.parametrize("keep", [False, True])
def test_a_cache_without_rows_takes_nothing(keep):
    T = 7
    x, gain, cs, pos, q, k, v = inputs(T, 10)
    _, _, _, _, q2, k2, v2 = inputs(T, 10)
    cache = [[torch.empty(0, 2, 64, dtype=BF, device="cuda") for _ in range(2)] for _ in range(2)]
    A.tp_qk_norm_rope(x, gain, gain, cs, pos, q, k if keep else None, v if keep else None, *cache,
                      torch.arange(-2, T - 2, device="cuda"))
    A.tp_qk_norm_rope(x, gain, gain, cs, pos, q2, k2, v2)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(q + (k + v if keep else []), q2 + (k2 + v2 if keep else [])))


@pytest.mark.gpu
def test_a_table_without_positions_has_none():
    """Every position lies outside it."""
    T = 7
    x, gain, cs, pos, q, k, v = inputs(T, 0)
    A.tp_qk_norm_rope(x, gain, gain, cs, pos, q, k, v)
    d = [torch.zeros_like(t) for t in x]
    dg = [[torch.full((64,), 5.0, device="cuda") for _ in range(2)] for _ in range(2)]
    do = [[torch.ones_like(t) for t in u] for u in (q, k, v)]
    A.tp_qk_norm_rope_grad(*do, x, gain, gain, cs, pos, d, *dg)
    torch.cuda.synchronize()
    for r in range(2):
        assert q[r].isnan().all() and k[r].isnan().all()
        assert torch.equal(v[r], x[r].view(T, 8, 64)[:, 6:])
        h = d[r].view(T, 8, 64)
        assert h[:, :6].isnan().all() and torch.equal(h[:, 6:], do[2][r])
        assert not dg[0][r].any() and not dg[1][r].any()
