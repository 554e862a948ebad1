"""GPU tests of kv_plan for a step without requests: a caller that goes on
from the call's outputs, two of each in turn, goes on from the same cache."""
import os
import sys

import pytest
import torch

from ring_collectives_amd import _native as N
from ring_collectives_amd import attention as A

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    N.lib()
    yield


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("capacity", [0, 5])
@pytest.mark.parametrize("side", [False, True])
def test_outputs(capacity, side):
    none = i32([])
    cu, pos, after, used_after = i32([-7]), i32([-7] * capacity), i32([]), i32([-7])
    slots = torch.full((capacity,), -7, dtype=torch.int64, device="cuda")
    s = torch.cuda.Stream() if side else None
    if side:
        s.wait_stream(torch.cuda.current_stream())
    A.kv_plan(none, none, i32([3, 1, 2]), i32([2]), torch.empty(0, 4, dtype=torch.int32, device="cuda"), after, cu, pos, slots,
              used_after, page_size=16, prefix_len=9, stream=s)
    torch.cuda.synchronize()
    assert used_after.tolist() == [2] and cu.tolist() == [0]
    assert pos.tolist() == [0] * capacity and slots.tolist() == [-1] * capacity


def test_outputs_are_checked_as_ever():
    none, table = i32([]), torch.empty(0, 4, dtype=torch.int32, device="cuda")
    ok = dict(lengths=none, new_tokens=none, free_pages=i32([1]), used=i32([0]), block_table=table, lengths_after=i32([]),
              cu_new=i32([0]), positions=none, slots=torch.empty(0, dtype=torch.int64, device="cuda"), used_after=i32([0]),
              page_size=16)
    for kw, exc in ((dict(cu_new=i32([0, 0])), ValueError), (dict(used_after=i32([])), ValueError),
                    (dict(used_after=i32([0]).long()), TypeError), (dict(page_size=3), N.RingError)):
        with pytest.raises(exc):
            A.kv_plan(**{**ok, **kw})


def test_layer_goes_on_after_a_plan_without_requests():
    import attention_layer
    layer = attention_layer.AttentionLayer(P=2, Hq=2, Hkv=1, D=64, model=256, pages=16, seed=1)
    BF = torch.bfloat16
    layer.requests(3, 64)
    for _ in range(2):
        layer.step(torch.randn(3, 256, device="cuda").to(BF))
    used = layer.used.item()
    assert used == 3
    layer.requests(0, 64)
    junk = [torch.full((n,), 1 << 20, dtype=torch.int32, device="cuda") for n in (1, 1, 2, 2, 3, 3)]
    del junk                                             # what new buffers hold
    cu, pos, slots = layer.plan(i32([]), 0)
    assert cu.tolist() == [0] and pos.numel() == 0 == slots.numel() and layer.used.item() == used
    layer.requests(2, 64)
    layer.step(torch.randn(2, 256, device="cuda").to(BF))
    assert layer.used.item() == used + 2
    assert layer.table[:, 0].tolist() == layer.free[used:used + 2].tolist()
