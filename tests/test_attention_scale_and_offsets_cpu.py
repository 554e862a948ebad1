"""Host-side checks of the attention calls' scale and offsets (fake pointers;
nothing is launched where they are refused)."""
import pytest

from ring_collectives_amd import _native as N

L = N.lib()


def ptrs(i):
    return N.ptr_array([(i + 1) << 28, ((i + 1) << 28) + 0x1000000])[0]


def fwd(scale=0.1, cq=0x1000, ck=0x2000):
    return L.tp_attention(*[ptrs(i) for i in range(4)], None, cq, ck, 2, 3, 10, 10, 4, 2, 64, 256, 128, 128, 256, 1, scale, None)


def grad(scale=0.1, cq=0x1000, ck=0x2000):
    return L.tp_attention_grad(*[ptrs(i) for i in range(9)], cq, ck, 2, 3, 10, 10, 4, 2, 64, 256, 128, 128, 256, 256, 256, 128, 128,
                               1, scale, 0x100000, 1 << 40, None)


def decode(scale=0.1):
    return L.tp_attention_decode(*[ptrs(i) for i in range(4)], 0x1000, 0x2000, 0x3000, 2, 3, 4, 2, 64, 4, 16, 20, 0, 256, 256, scale,
                                 0x100000, 1 << 40, None)


@pytest.mark.parametrize("call", [fwd, grad, decode])
@pytest.mark.parametrize("scale", [3.0e38, 2.4e38, 1e300])
def test_a_scale_that_is_infinite_in_base_2_is_refused(call, scale):
    """The kernels multiply by scale log2(e): an infinite one would make NaN
    of scores of zero, whose weights are plain."""
    assert call(scale=scale) == N.RING_EINVAL


@pytest.mark.parametrize("call", [fwd, grad])
@pytest.mark.parametrize("kw", [dict(cq=0x1002), dict(ck=0x2001), dict(cq=0x1003, ck=0x2003)])
def test_offsets_off_their_alignment_are_refused(call, kw):
    assert call(**kw) == N.RING_EINVAL
