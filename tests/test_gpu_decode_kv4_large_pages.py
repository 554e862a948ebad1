"""tp_attention_decode_kv4 where a page of all heads holds more than 4 GiB."""
import numpy as np
import pytest
import torch

from oracle import attention as oa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hkv,D,page", [(490, 128, 65536), (970, 64, 65536), (15500, 128, 2048)])
def test_decode_of_pages_past_4_gib(Hkv, D, page):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from _gpu_helpers import note
    from ring_collectives_amd import search as S
    from test_gpu_attention import BF, f64, i32, poisoned, within
    note("decode_kv4 Hkv=%d D=%d page=%d" % (Hkv, D, page))
    cache = [S.kv4_cache(2, Hkv, D, page)]
    assert cache[0].stride(0) > 1 << 32
    g = torch.Generator().manual_seed(D)
    k, v = (torch.randn(6, Hkv, D, generator=g).to(BF).cuda() for _ in range(2))
    # the first rows of page 1 are the first request's, the last of page 0 the end of the second's
    lengths = [4, page]
    slots = torch.tensor([page, page + 1, page + 2, page + 3, page - 2, page - 1], device="cuda")
    S.tp_kv4_write([k], [v], cache, slots, page_size=page)
    kr, vr = torch.empty_like(k), torch.empty_like(v)
    S.tp_kv4_read(cache, slots, [kr], [vr], page_size=page)
    assert torch.isfinite(kr).all() and kr.any(2).all()
    q = torch.randn(2, Hkv, D, generator=g).to(BF).cuda()
    o = [poisoned((2, Hkv, D))]
    S.tp_attention_decode_kv4([q], cache, o, i32([[1], [0]]), i32(lengths), page_size=page)
    for h in (0, 1, Hkv // 2, Hkv - 2, Hkv - 1):
        for b, (n, at) in enumerate(((4, slice(0, 4)), (page, slice(4, 6)))):
            keys, values = np.zeros((n, D)), np.zeros((n, D))
            keys[-(at.stop - at.start):], values[-(at.stop - at.start):] = f64(kr[at, h]), f64(vr[at, h])
            want, _, bound, _, _, _ = oa.attention(f64(q[b, h:h + 1]), keys, values, np.ones((1, n), bool), D ** -0.5)
            # the sum is of the rounded weights: UB |o| more, as in test_gpu_search.py
            within(o[0][b, h:h + 1], want, bound + oa.UB * np.abs(want), "row %d head %d" % (b, h))
