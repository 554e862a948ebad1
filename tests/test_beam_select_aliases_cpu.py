"""beam_select refuses outputs that lie in its inputs (other groups would still
read what one has written), before the device is touched; so do kv_fork and
kv_compact."""
import pytest

from ring_collectives_amd import _native as N
from test_search_abi_cpu import beam, compact, fork

# three groups of four beams into four places: scores are 48 bytes from 0x1000, done 12 from 0x5000


@pytest.mark.parametrize("kw", [
    dict(after=0x1000), dict(parents=0x1000), dict(tokens=0x102C), dict(after=0xFD4), dict(done=0x5000, done_after=0x5000, end=3),
    dict(done=0x5000, done_after=0x500B, end=3), dict(done=0x5000, done_after=0x4FF5, end=3), dict(done=0x5000, done_after=0x6000, end=3, tokens=0x4FD4),
    dict(done=0x5000, done_after=0x1010, end=3)])
def test_select_outputs_in_inputs(kw):
    assert beam(**kw) == N.RING_EINVAL


@pytest.mark.parametrize("kw", [
    dict(after=0x1030), dict(tokens=0xFD0), dict(done=0x5000, done_after=0x500C, end=3), dict(done=0x5000, done_after=0x4FF4, end=3)])
def test_select_outputs_next_to_inputs(kw):
    """Not refused: the workspace is, after them."""
    assert beam(ws=(None, 0), **kw) == N.RING_EWORKSPACE


def test_fork_and_compact():
    assert fork(used2=0x5000) == fork(lens2=0x2000) == fork(table2=0x1000) == compact(table2=0x1000) == N.RING_EINVAL
