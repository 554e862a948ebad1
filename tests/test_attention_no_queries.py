"""Gradient calls without a query: every key's gradient is zero, also where
the query tensors, having no element, have no address."""
import pytest
import torch

from ring_collectives_amd import _native as N
from ring_collectives_amd import attention as A


def test_null_query_pointers_pass_the_host_checks():
    """A call that has keys alone gets as far as the workspace check."""
    def ptrs(base):
        return N.ptr_array([base + r * 0x1000000 if base else 0 for r in range(2)])[0]

    def call(Tq, empty, Tk=10, full=0x10000000):
        q, kv = ptrs(empty), ptrs(full)
        s = [256, 128, 128, 256, 256, 256, 128, 128]
        return N.lib().tp_attention_grad(q, q, kv, kv, q, q, q, kv, kv, 0x1000, 0x2000, 2, 3, Tq, Tk, 4, 2, 64, *s, 1, 0.1,
                                         None, 0, None)

    assert call(0, 0) == N.RING_EWORKSPACE
    assert call(0, 0x20000000) == N.RING_EWORKSPACE
    assert call(1, 0) == N.RING_EINVAL                       # a query without an address
    assert call(0, 0, full=0) == N.RING_EINVAL               # keys without one
    assert call(0, 0, Tk=0, full=0) == N.RING_OK             # nothing to do


@pytest.mark.gpu
@pytest.mark.parametrize("P,Hq,Hkv,D", [(2, 4, 2, 64), (1, 2, 1, 128), (8, 8, 8, 64), (8, 8, 8, 128)])
@pytest.mark.parametrize("lk", [[5], [0, 70, 3], [130, 1, 300]])
@pytest.mark.parametrize("causal", [True, False])
def test_keys_without_queries_have_zero_gradients(P, Hq, Hkv, D, lk, causal):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    BF, Tk = torch.bfloat16, sum(lk)
    e = lambda *s: [torch.empty(*s, dtype=BF, device="cuda") for _ in range(P)]            # noqa: E731
    q, do, o, dq = (e(0, Hq, D) for _ in range(4))
    k, v = ([torch.randn(Tk, Hkv, D, device="cuda").to(BF) for _ in range(P)] for _ in range(2))
    dk, dv = ([torch.full((Tk, Hkv, D), float("nan"), dtype=BF, device="cuda") for _ in range(P)] for _ in range(2))
    lse = [torch.empty(Hq, 0, device="cuda") for _ in range(P)]
    cu_q = torch.zeros(len(lk) + 1, dtype=torch.int32, device="cuda")
    cu_k = torch.tensor([0] + lk, device="cuda").cumsum(0).int()
    A.tp_attention(q, k, v, o, cu_q, cu_k, lse=lse, causal=causal)
    A.tp_attention_grad(do, q, k, v, o, lse, dq, dk, dv, cu_q, cu_k, causal=causal)
    torch.cuda.synchronize()
    for t in dk + dv:
        assert torch.equal(t, torch.zeros_like(t))


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_queries_without_keys(D, causal):
    """The other way round: o = 0, lse = -inf, dq = 0."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    BF, Tq = torch.bfloat16, 140
    q, do = (([torch.randn(Tq, 4, D, device="cuda").to(BF)]) for _ in range(2))
    o, dq = ([torch.full((Tq, 4, D), float("nan"), dtype=BF, device="cuda")] for _ in range(2))
    k, v, dk, dv = ([torch.empty(0, 2, D, dtype=BF, device="cuda")] for _ in range(4))
    lse = [torch.full((4, Tq), float("nan"), device="cuda")]
    cu_q, cu_k = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 133, Tq], [0, 0, 0]))
    A.tp_attention(q, k, v, o, cu_q, cu_k, lse=lse, causal=causal)
    A.tp_attention_grad(do, q, k, v, o, lse, dq, dk, dv, cu_q, cu_k, causal=causal)
    torch.cuda.synchronize()
    assert torch.equal(o[0], torch.zeros_like(o[0])) and torch.equal(dq[0], torch.zeros_like(dq[0]))
    assert torch.equal(lse[0], torch.full_like(lse[0], -float("inf")))
