"""tp_attention_decode_kv4 gives the same bits every time where keys are shared
by whole tiles, one row tile (group * heads up to 16) and two, and in workspaces
that held other calls."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group,G,D", [(4, 4, 128), (8, 4, 128), (5, 7, 64)])
def test_same_bits(group, G, D):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from _gpu_helpers import note
    from ring_collectives_amd import search as S
    from test_gpu_attention import i32, poisoned
    from test_gpu_search import check_decode_kv4, decode_state
    note("decode_kv4 repeated, groups of %d, %d heads, D=%d" % (group, G, D))
    groups, Hkv, page = 5, 2, 16
    lead = [3000, 192, 700, 64, 2100][:groups]             # keys that a group's rows have in common
    lengths = [lead[b // group] + 37 * (b % group) + b % 3 for b in range(groups * group)]
    B = len(lengths)
    q, cache, table = decode_state(2, B, G * Hkv, Hkv, D, page, lengths, 16 + group)
    for b in range(B):
        n = lead[b // group] // page
        table[b][:n] = table[b // group * group][:n]
    shared = [n // page * page for n in lead]
    assert all(n >= 64 for n in shared)                    # whole tiles of 32
    check_decode_kv4(q, cache, table, lengths, page, shared=shared, group=group)
    args = (i32(table), i32(lengths))
    first, ws = None, None
    for turn in range(6):
        o = [poisoned((B, G * Hkv, D)) for _ in range(2)]
        ws = S.tp_attention_decode_kv4(q, cache, o, *args, page_size=page, shared=i32(shared), group=group, ws=ws)
        bits = torch.stack(o).view(torch.int16)
        first = bits if first is None else first
        assert torch.equal(bits, first), turn
        # another call in between, of fewer rows and none shared
        S.tp_attention_decode_kv4([t[:group].contiguous() for t in q], cache, [t[:group].contiguous() for t in o], args[0][:group].contiguous(),
                                  args[1][:group].contiguous(), page_size=page, group=group, ws=ws)
