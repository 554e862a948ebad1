"""tp_kv4_write with slots that several tokens name: every other row is as it
would be, and every byte of the row itself is one of the tokens' (which, is not
said: codes and scales, keys and values may be of different ones)."""
import numpy as np
import pytest
import torch

from oracle import search as osr

pytestmark = pytest.mark.gpu


def row_bytes(cache, slot, D, page):
    """The bytes of a cache row: (Hkv, D + D / 16), from a (pages, Hkv, bytes) array."""
    p, i, n = slot // page, slot % page, page * D // 2
    parts = [cache[p, :, kv * n + i * D // 2:kv * n + (i + 1) * D // 2] for kv in (0, 1)]
    parts += [cache[p, :, 2 * n + kv * n // 16 + i * D // 32:2 * n + kv * n // 16 + (i + 1) * D // 32] for kv in (0, 1)]
    return np.concatenate(parts, 1)


@pytest.mark.parametrize("T,Hkv,D", [(40, 2, 64), (700, 3, 128)])
@pytest.mark.parametrize("order", ["same tile", "far apart", "every token"])
def test_repeated_slots(T, Hkv, D, order):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from _gpu_helpers import note
    from ring_collectives_amd import search as S
    note("kv4 write of repeated slots T=%d D=%d %s" % (T, D, order))
    page, pages = 16, 64
    g = torch.Generator().manual_seed(T)
    k, v = (torch.randn(T, Hkv, D, generator=g) * torch.exp2(torch.randint(-9, 9, (T, 1, 1), generator=g)) for _ in range(2))
    k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    slots = torch.randperm(page * pages - 1, generator=g)[:T]
    if order == "same tile":
        slots[3] = slots[9]
        same = [3, 9]
    elif order == "far apart":
        slots[T - 1] = slots[T // 2] = slots[0]
        same = [0, T // 2, T - 1]
    else:
        slots[:] = page * pages - 1                        # a row that padding goes to
        same = list(range(T))
    cache = S.kv4_cache(pages, Hkv, D, page)
    for _ in range(3):
        S.tp_kv4_write([k.cuda()], [v.cuda()], [cache], slots.cuda(), page_size=page)
    got = cache.cpu().numpy()
    at = slots.tolist()
    if len(same) < 9:                                      # each token's row, from a page of it alone
        def page_row(t, h):
            x = [y[t:t + 1, h].float().numpy().repeat(page, 0) for y in (k, v)]
            return row_bytes(osr.page_of(*x)[None, None], 0, D, page)[0]
        rows = np.stack([[page_row(t, h) for h in range(Hkv)] for t in same])
        assert (rows == row_bytes(got, at[same[0]], D, page)).any(0).all()
    alone = S.kv4_cache(pages, Hkv, D, page)
    others = [t for t in range(T) if t not in set(same)]
    if others:
        S.tp_kv4_write([k[others].cuda()], [v[others].cuda()], [alone], slots[others].cuda(), page_size=page)
    want = alone.cpu().numpy()
    for slot in range(page * pages):
        if slot != at[same[0]]:
            assert np.array_equal(row_bytes(got, slot, D, page), row_bytes(want, slot, D, page)), slot
