"""The workspace of a decode call, returned for the next one, holds that one
too where its batch has become smaller (the keys of fewer requests are cut into
more parts)."""
import pytest
import torch

from ring_collectives_amd import _native as N
from ring_collectives_amd import attention as A


@pytest.mark.parametrize("P,Hq,Hkv,D,W,page,prefix", [
    (4, 8, 2, 128, 256, 16, 0), (4, 8, 2, 128, 16, 64, 8192), (1, 1, 1, 64, 4096, 16, 0), (2, 34, 1, 64, 900, 8, 300),
    (8, 40, 8, 128, 64, 128, 100000), (1, 6, 3, 64, 2, 16, 20000), (64, 64, 64, 64, 1000, 1, 5000), (1, 300, 1, 64, 100, 128, 4000)])
def test_size_never_falls_as_the_batch_grows(P, Hq, Hkv, D, W, page, prefix):
    f = lambda B: N.lib().tp_attention_decode_workspace_bytes(P, B, Hq, Hkv, D, W, page, prefix)      # noqa: E731
    sizes = [f(B) for B in list(range(0, 700)) + [1000, 1001, 4095, 20000, 33000, 100000]]
    assert sizes == sorted(sizes) and sizes[0] > 0


@pytest.mark.gpu
@pytest.mark.parametrize("prefix", [0, 700])
def test_a_batch_that_shrinks(prefix):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from test_gpu_attention import check_decode, decode_inputs, poisoned
    Hq, Hkv, D, page, P = 8, 2, 64, 16, 4
    lens = [600 - 7 * b for b in range(64)]
    q, kc, vc, table, ln, pp = decode_inputs(P, lens, prefix, Hq, Hkv, D, page, seed=prefix)
    ws = None
    for B in (64, 33, 4, 1):
        cut = lambda x: [t[:B].contiguous() for t in x]                    # noqa: E731
        o = [poisoned((B, Hq, D)) for _ in range(P)]
        ws = A.tp_attention_decode(cut(q), kc, vc, o, table[:B].contiguous(), ln[:B].contiguous(), page_size=page, prefix_pages=pp,
                                   prefix_len=prefix, ws=ws)
        torch.cuda.synchronize()
        if B < 5:
            check_decode(cut(q)[-1:], kc[-1:], vc[-1:], o[-1:], table, lens, pp, prefix, page, D ** -0.5)
        else:
            assert all(bool(t.isfinite().all()) for t in o)
