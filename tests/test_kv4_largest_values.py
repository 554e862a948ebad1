"""The 4-bit format at bf16's largest values: scales end at 2^125, as 6 * 2^126
is past bf16, so that what is above 7 * 2^125 is stored as 6 * 2^125."""
import numpy as np
import pytest
import torch

from oracle import search as osr

BITS = np.arange(0x7D00, 0x7F80)                           # 2^123 and up


def test_oracle():
    x = np.zeros((len(BITS), 64))
    x[:, 3] = osr.bf16(BITS)
    codes, scales = osr.quantise(x)
    got, scale = osr.values(codes, scales)[:, 3], 2.0 ** (scales[:, 0] - 127.0)
    assert np.isfinite(got).all() and (got <= 6 * 2.0 ** 125).all()
    inside = x[:, 3] <= 7 * 2.0 ** 125
    assert (np.abs(got - x[:, 3])[inside] <= scale[inside]).all()
    assert not inside.all() and (got[~inside] == 6 * 2.0 ** 125).all()
    assert (np.abs(got - x[:, 3]) < 2 * scale).all()


@pytest.mark.gpu
def test_write_and_read():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from ring_collectives_amd import search as S
    T = len(BITS)
    x = torch.zeros(T, 1, 64, dtype=torch.bfloat16)
    x[:, 0, 3] = torch.from_numpy(osr.bf16(BITS)).to(torch.bfloat16)
    cache, k, v = S.kv4_cache(T // 64, 1, 64, 64), torch.empty_like(x).cuda(), torch.empty_like(x).cuda()
    S.tp_kv4_write([x.cuda()], [-x.cuda()], [cache], torch.arange(T, device="cuda"), page_size=64)
    S.tp_kv4_read([cache], torch.arange(T, device="cuda"), [k], [v], page_size=64)
    want = osr.values(*osr.quantise(x.double().numpy()))
    assert np.array_equal(k.double().cpu().numpy(), want) and torch.equal(k, -v)
