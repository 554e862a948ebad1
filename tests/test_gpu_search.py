"""GPU tests of the beam search calls and of the 4-bit cache against the oracle,
at the sizes, layouts and masks where they can go wrong.  Whole numbers, pages
and stored codes are compared exactly, computed numbers within the oracle's
element-by-element worst-case bounds."""
import math

import numpy as np
import pytest
import torch

from oracle import attention as oa
from oracle import search as osr
from ring_collectives_amd import _native as N
from ring_collectives_amd import search as S

from _gpu_helpers import note
from test_gpu_attention import BF, f64, i32, poisoned, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    N.lib()
    yield


# ---------------------------------------------------------------- beam_select
def split(x, P, width, dtype, pad=0):
    """(rows, vocab) logits as P ranks' columns, padded with what must not be chosen."""
    rows, vocab = x.shape
    full = torch.full((rows, P * width), 50.0)
    full[:, :vocab] = x
    out = []
    for r in range(P):
        t = torch.full((rows, width + pad), 60.0, dtype=dtype)
        t[:, :width] = full[:, r * width:(r + 1) * width]
        out.append(t.cuda()[:, :width])
    return out


def run_select(logits, scores, vocab, keep, done=None, end=-1, flag=torch.bool):
    n = scores.shape[0]
    parents, tokens = i32([[-7] * keep] * n), i32([[-7] * keep] * n)
    after = torch.full((n, keep), float("nan"), device="cuda")
    d = None if done is None else torch.from_numpy(done).to(flag).cuda()
    da = None if done is None else torch.full((n, keep), 1, dtype=torch.uint8, device="cuda").view(flag)
    S.beam_select(logits, torch.from_numpy(scores).float().cuda(), parents, tokens, after, vocab=vocab, done=d, done_after=da, end_token=end)
    torch.cuda.synchronize()
    return parents.cpu().numpy(), tokens.cpu().numpy(), after.cpu().numpy(), None if da is None else da.cpu().numpy().astype(bool)


def check_select(x, scores, P, width, keep, dtype, done=None, end=-1, pad=0, flag=torch.bool):
    """x: (rows, vocab) fp32 tensor."""
    vocab = x.shape[1]
    x = x.to(dtype).float()
    scores = scores.astype(np.float32)
    parents, tokens, after, da = run_select(split(x, P, width, dtype, pad), scores, vocab, keep, done, end, flag)
    ep, et, ea, ed, bound, every = osr.select(x.numpy(), scores, vocab, keep, done, end)
    W = scores.shape[1]
    assert np.array_equal(parents >= 0, ep >= 0) and np.array_equal(tokens >= 0, ep >= 0)
    got = np.where(parents >= 0, np.take_along_axis(every.reshape(len(scores), -1),
                                                    np.where(parents >= 0, parents % W * vocab + tokens, 0), 1), -np.inf)
    fine = ep >= 0
    assert (parents[fine] // W == ep[fine] // W).all()
    # what was chosen scores as much as what the oracle chose, and is the same where that tells
    assert (np.abs(got[fine] - ea[fine]) <= 2 * bound).all(), np.abs(got[fine] - ea[fine]).max()
    other = (parents != ep) | (tokens != et)
    assert other.sum() <= 0.01 * other.size, "%d of %d differ" % (other.sum(), other.size)
    for n in range(len(scores)):
        pairs = [(p, t) for p, t in zip(parents[n], tokens[n]) if p >= 0]
        assert len(set(pairs)) == len(pairs)
    size = np.abs(np.where(np.isfinite(scores), scores, 0)).max() + np.abs(np.where(fine, ea, 0)).max()
    assert (np.abs(after[fine] - got[fine]) <= bound + 4 * osr.U * size).all(), np.abs(after[fine] - got[fine]).max()
    assert (after[~fine] == -np.inf).all()
    if done is not None:
        want = np.zeros_like(da)
        for n, k in np.argwhere(fine):
            want[n, k] = done[n, parents[n, k] % W] or tokens[n, k] == end
        assert np.array_equal(da, want)
    return parents, tokens, after


def beam_inputs(n, W, vocab, seed, std=2.5):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(n * W, vocab, generator=g) * std, -np.random.default_rng(seed).random((n, W)).cumsum(1) * 3


@pytest.mark.parametrize("P,n,W,keep,width,vocab", [
    (1, 1, 1, 1, 8, 5), (1, 1, 1, 1, 1, 1), (2, 3, 2, 4, 128, 201), (1, 2, 1, 5, 128, 3), (2, 1, 3, 64, 16, 20), (4, 2, 4, 4, 2048, 8000),
    (3, 5, 3, 6, 16672, 50001), (2, 2, 64, 64, 136, 271), (64, 2, 2, 3, 128, 8191), (1, 1, 16, 16, 33333, 33333), (4, 3, 1, 9, 256, 300),
    (8, 40, 8, 8, 1152, 9001), (1, 1, 1, 1, 1024, 1024), (1, 2, 2, 7, 1025, 1025), (2, 300, 5, 5, 104, 207)])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_select(P, n, W, keep, width, vocab, dtype):
    note("beam_select P=%d groups=%d beams=%d keep=%d vocab=%d %s" % (P, n, W, keep, vocab, dtype))
    x, s = beam_inputs(n, W, vocab, P * 131 + vocab)
    check_select(x, s, P, width, keep, dtype, pad=(-width) % 8)


@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("flag", [torch.bool, torch.uint8])
def test_select_with_ended_beams(dtype, flag):
    x, s = beam_inputs(7, 4, 3001, 5)
    done = np.random.default_rng(5).random((7, 4)) < 0.4
    done[0], done[1] = True, False
    x[::3, 17] += 20                                        # beams that end now
    check_select(x, s, 2, 1504, 6, dtype, done, 17, flag=flag)


@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_select_of_what_is_not_finite(dtype):
    x, s = beam_inputs(6, 3, 2500, 11)
    x[0] = -math.inf                                        # a row that its mask leaves nothing of
    x[1, ::2] = -math.inf
    x[2, 7] = math.inf
    x[4, 100:2400] = math.nan
    x[6:9] = -math.inf                                      # a whole group
    x[9] = torch.finfo(dtype).min                           # the type's lowest value, everywhere
    x[10, 5:] = torch.finfo(dtype).min
    x[12, 1:] = -math.inf                                   # one token left
    s[4, 0], s[4, 2], s[5] = -np.inf, np.nan, -np.inf
    check_select(x, s, 2, 1256, 5, dtype)


def test_select_takes_the_lowest_of_equals():
    """Equal logits in a row, equal rows, and everything equal."""
    note("beam_select ties")
    for vocab, P, width in ((5000, 1, 5000), (5000, 3, 1680), (40, 1, 40)):
        x = torch.zeros(3, vocab)
        parents, tokens, _, _ = run_select(split(x, P, width, torch.float32), np.zeros((1, 3)), vocab, 7)
        assert parents.tolist() == [[0] * 7] and tokens.tolist() == [list(range(7))]
    g = torch.Generator().manual_seed(3)
    x = torch.randint(0, 8, (1, 20000), generator=g).float()
    best = torch.nonzero(x[0] == 7)[:9, 0].tolist()
    _, tokens, _, _ = run_select(split(x, 2, 10000, BF), np.zeros((1, 1)), 20000, 9)
    assert tokens.tolist() == [best]
    x = torch.randn(1, 3000, generator=g).repeat(4, 1)     # four equal beams: the best token of each in turn
    parents, tokens, _, _ = run_select(split(x, 2, 1504, torch.float32), np.zeros((1, 4)), 3000, 8)
    top = x[0].argsort(descending=True)[:2].tolist()
    assert parents.tolist() == [[0, 1, 2, 3] * 2] and tokens.tolist() == [[top[0]] * 4 + [top[1]] * 4]


@pytest.mark.parametrize("W,P,keep", [(2, 1, 7), (2, 3, 7), (33, 4, 5), (64, 2, 64)])
@pytest.mark.parametrize("score,std", [(-1e25, 1.0), (0.0, 1e-25)])
def test_select_orders_by_logits_where_scores_are_equal(score, std, W, P, keep):
    """Logits that differ, and scores that do not in 64 bits: next to a large
    score, and next to the logarithm of the number of tokens."""
    note("beam_select equal scores W=%d P=%d %g" % (W, P, score))
    x = torch.randn(W, 5001, generator=torch.Generator().manual_seed(W)) * std
    s, done = np.full((1, W), score, np.float32), np.zeros((1, W), bool)
    done[0, 0] = True
    parents, tokens, _, _ = run_select(split(x, P, -(-5001 // P // 8) * 8, torch.float32), s, 5001, keep, done, 3)
    ep, et = osr.select(x.numpy(), s, 5001, keep, done, 3)[:2]
    assert et[0, 1:].tolist() == x[1].argsort(descending=True)[:keep - 1].tolist()
    assert parents.tolist() == ep.tolist() and tokens.tolist() == et.tolist()


@pytest.mark.parametrize("base", [-1e4, 0.0, 3e4])
def test_select_at_any_level(base):
    """Logits far from zero, ascending (every step raises the maximum) and descending."""
    x = torch.linspace(base, base + 60, 9000).repeat(2, 1)
    x[1] = x[1].flip(0)
    check_select(x, np.array([[-1.0, -1.5]]), 1, 9000, 8, torch.float32)


def test_select_finds_the_last_odd_column():
    x = torch.zeros(1, 3333)
    x[0, 3332] = 9.0
    _, tokens, _, _ = run_select([torch.cat([x, torch.full((1, 3), 60.0)], 1).to(BF).cuda()[:, :3333]], np.zeros((1, 1)), 3333, 2)
    assert tokens.tolist() == [[3332, 0]]


# ---------------------------------------------------------------- kv_fork
def run_fork(table, lengths, parents, keep, free, used, page, pages, group, repeat=1, ws=None, shared=True):
    width = len(table[0]) if len(table) else 3
    tab, rows = i32(table).reshape(len(table), width), len(parents)
    fp, out, lens = i32(list(free)), i32([[-7] * width] * rows).reshape(rows, width), i32([-7] * rows)
    copies, n, used2 = i32([[-7, -7]] * rows).reshape(rows, 2), i32([-7]), i32([-7])
    sh = i32([-7] * (rows // group)) if shared else None
    for _ in range(repeat):
        ws = S.kv_fork(tab, i32(list(lengths)), i32(list(parents)), fp, i32([used]), out, lens, copies, n, used2, page_size=page, pages=pages,
                       keep=None if keep is None else i32(list(keep)), shared=sh, group=group, ws=ws)
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in (out, lens, copies, n, sh if shared else lens, used2, fp)], ws


def check_fork(table, lengths, parents, keep, free, used, page, pages, group, **kw):
    want = osr.fork(table, lengths, parents, keep, free, used, page, pages, group, 3)
    got, ws = run_fork(table, lengths, parents, keep, free, used, page, pages, group, **kw)
    for g, w, name in zip(got, want, ("table", "lengths", "copies", "n_copies", "shared", "used", "free")):
        if name == "shared" and not kw.get("shared", True):
            continue
        assert np.array_equal(g.reshape(-1), np.asarray(w).reshape(-1)), name
    if pages <= 8192:                                          # and as with more pages than one workgroup's LDS holds
        check_fork(table, lengths, parents, keep, free, used, page, pages + 8193, group, **{**kw, "ws": None})
    return got, ws


def fork_state(B, page, longest, width, spare, seed, common=0.6, group=1):
    """A table of B rows, `group` of which share their first pages, its free list and use."""
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, longest + 1, B)
    lens = np.minimum(lens, width * page)
    need = -(-lens // page)
    ids = rng.permutation(int(need.sum()) + spare)
    table, used = np.full((B, width), -1), 0
    for b in range(B):
        first = b // group * group
        k = int(min(need[b], need[first]) * common) if b != first else 0
        table[b, :k] = table[first, :k]
        table[b, k:need[b]] = ids[used:used + need[b] - k]
        used += need[b] - k
    return table.tolist(), lens.tolist(), ids.tolist(), int(used), len(ids)


@pytest.mark.parametrize("B,B2,group,page,longest,width", [
    (1, 1, 1, 16, 5, 1), (4, 4, 4, 16, 100, 8), (4, 8, 2, 16, 100, 7), (6, 3, 3, 1, 9, 12), (33, 40, 5, 8, 600, 76), (64, 64, 8, 16, 1500, 130),
    (100, 1000, 4, 4, 70, 20), (1030, 1030, 5, 16, 300, 19), (2048, 1025, 1, 32, 400, 13), (8192, 8192, 8, 16, 60, 5), (3, 8192, 1, 16, 500, 40),
    # rows of several waves' pieces
    (3, 6, 2, 1, 5000, 5003), (1, 4, 4, 16, 40000, 2501), (6, 4, 4, 2, 2050, 1025), (20, 30, 3, 1, 2049, 2048)])
@pytest.mark.parametrize("cut", [False, True])
def test_fork(B, B2, group, page, longest, width, cut):
    note("kv_fork B=%d to %d group=%d page=%d cut=%s" % (B, B2, group, page, cut))
    rng = np.random.default_rng(B * 7 + B2)
    table, lens, free, used, pages = fork_state(B, page, longest, width, B2 + 9, B + 5, group=group if B % group == 0 else 1)
    parents = rng.integers(0, B, B2)
    if B2 >= 8:
        parents[::7] = -1
        parents[5] = B + 3
    keep = rng.integers(0, longest + 1, B2).tolist() if cut else None
    got, ws = check_fork(table, lens, parents.tolist(), keep, free, used, page, pages, group)
    check_fork(table, lens, parents.tolist(), keep, free, used, page, pages, group, repeat=2, ws=ws)
    # the same beams go on: nothing to do
    same = check_fork(table, lens, list(range(B)), None, free, used, page, pages, 1, ws=None)[0]
    assert same[3][0] == 0 and same[5][0] == used


def test_fork_frees_and_takes_what_is_freed():
    """Rows that end pay for the copies of those that split, and the rest goes back."""
    table, lens, free, used, pages = fork_state(40, 16, 300, 20, 5, 1)
    for parents in ([0] * 40, [39, 39, 39], [7], [-1] * 4, []):
        check_fork(table, lens, parents, None, free, used, 16, pages, 1)
    check_fork([], [], [], None, free, 3, 16, pages, 1)
    check_fork([], [], [0, 1], None, free, 3, 16, pages, 2)


def test_fork_of_every_row_from_one_and_back_to_one():
    table = [[4, 2, 7]]
    got, _ = check_fork(table, [39], [0] * 65, None, list(range(8, 100)), 0, 16, 100, 65)
    assert got[3][0] == 64 and got[4].tolist() == [32]
    check_fork(got[0].tolist(), got[1].tolist(), [64], None, got[6].tolist(), int(got[5][0]), 16, 100, 1)


def test_fork_when_pages_run_out():
    got, _ = check_fork([[0, 1], [2, 3]], [20, 25], [0, 0, 0, 0, 1], None, [9, 9, 9, 9, 5], 4, 16, 10, 1)
    assert got[5][0] == 7 and got[0][2].tolist() == [0, -1]
    check_fork([[0, 1], [2, 3]], [20, 25], [0, 0, 0], None, [], 0, 16, 10, 1)


def test_fork_of_one_row_into_a_group_when_pages_run_out():
    """Copies that get no page are not in common, though the table holds -1 for each."""
    for spare in (0, 1, 2):
        got, _ = check_fork([[0, 1]], [20], [0] * 8, None, [1, 0] + [2, 3][:spare], 2, 16, 2 + spare, 4)
        assert got[4].tolist() == [16, 16] and got[5][0] == 9


def test_fork_passes_on_what_is_no_page():
    check_fork([[-1, 5, 900], [3, -4, 2]], [40, 40], [0, 0, 1, 1], None, list(range(6, 20)), 0, 16, 20, 2)
    check_fork([[5, 6, 7]], [-3], [0], None, [1, 2], 0, 16, 10, 1)
    check_fork([[5, 6, 7]], [1000], [0, 0], [1000, -5], [1, 2], 0, 16, 10, 2)


def test_fork_cut_into_pages_that_others_have_full():
    check_fork([[0, 1, 2], [0, 1, 3]], [48, 48], [0, 1, 0, 1, 0], [48, 20, 20, 33, 25], [5, 6, 7, 8, 9], 0, 16, 10, 1)
    check_fork([[0, 1, 2]], [48], [0, 0, 0], [20, 21, 22], [5, 6, 7, 8, 9], 0, 16, 10, 3)


def test_fork_without_shared_lengths():
    table, lens, free, used, pages = fork_state(12, 16, 200, 14, 30, 3, group=4)
    check_fork(table, lens, [0, 0, 1, 2, 5, 5, 5, 4, 8, 9, 9, 9], None, free, used, 16, pages, 4, shared=False)


def test_fork_of_many_pages():
    """More pages than a bit set's words for one pass of a workgroup."""
    table, lens, free, used, _ = fork_state(50, 16, 4000, 251, 100, 9, group=5)
    rng = np.random.default_rng(2)
    spread = rng.permutation(1 << 20)[:len(free)]
    table = [[int(spread[e]) if e >= 0 else -1 for e in row] for row in table]
    check_fork(table, lens, rng.integers(0, 50, 50).tolist(), None, spread.tolist(), used, 16, 1 << 20, 5)


def test_fork_refuses_a_workspace_with_data_in_it():
    """Counters would lie in what decoding left: an error, not a wrong table."""
    table, lens, free, used, pages = fork_state(8, 16, 200, 14, 30, 3)
    q, cache = [torch.ones(2, 4, 64, dtype=BF, device="cuda")], [S.kv4_cache(9, 2, 64, 16)]
    pages_of = i32([[0, 1] + [-1] * 200, [2, 3] + [-1] * 200])
    ws = S.tp_attention_decode_kv4(q, cache, [torch.empty_like(q[0])], pages_of, i32([30, 20]), page_size=16)
    run_fork(table, lens, [0] * 8, None, free, used, 16, pages + 9000, 1, ws=ws)
    from ring_collectives_amd import collectives as rc
    assert rc.last_error(ws)[0] == N.RING_EWORKSPACE
    ws.zero_()
    check_fork(table, lens, [0] * 8, None, free, used, 16, pages + 9000, 1, ws=ws)


# ---------------------------------------------------------------- kv_compact
def check_compact(table, lengths, first, pool, page, ws=None):
    width = len(table[0]) if len(table) else 2
    tab = i32(table).reshape(len(table), width)
    out, fp = i32([[-7] * width] * len(table)).reshape(len(table), width), i32([-7] * pool)
    copies, n, used = i32([[-7, -7]] * (pool // 2)).reshape(pool // 2, 2), i32([-7]), i32([-7])
    ws = S.kv_compact(tab, i32(list(lengths)), out, fp, copies, n, used, page_size=page, first_page=first, ws=ws)
    torch.cuda.synchronize()
    want = osr.compact(table, lengths, first, pool, page)
    for g, w, name in zip((out, copies, n, used, fp), want, ("table", "copies", "n_copies", "used", "free")):
        assert np.array_equal(g.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1)), name
    if pool <= 8192:                                           # and as with more pages than one workgroup's LDS holds
        check_compact(table, lengths, first, pool + 8193, page)
    return ws


@pytest.mark.parametrize("B,page,longest,width,spare,first", [
    (1, 16, 10, 1, 0, 0), (1, 16, 10, 1, 1, 5), (3, 16, 100, 8, 20, 0), (40, 8, 300, 40, 500, 3), (200, 32, 2500, 80, 9000, 0),
    (1500, 16, 90, 7, 0, 1), (8192, 1, 6, 6, 100, 0), (20, 16, 900, 60, 200000, 77),
    (2, 1, 5000, 5003, 20, 3), (1, 16, 50000, 3126, 9000, 0), (9, 2, 2050, 1025, 300, 0)])
def test_compact(B, page, longest, width, spare, first):
    note("kv_compact B=%d page=%d spare=%d" % (B, page, spare))
    table, lens, _, _, pool = fork_state(B, page, longest, width, spare, B + 1, group=3)
    table = [[e + first if e >= 0 else -1 for e in row] for row in table]
    ws = check_compact(table, lens, first, pool, page)
    check_compact(table, lens, first, pool, page, ws=ws)


def test_compact_of_nothing_of_everything_and_of_others_pages():
    check_compact([[3, 4]], [0], 0, 9, 16)
    check_compact([], [], 2, 9, 16)
    check_compact([[0, 0]], [30], 0, 0, 16)
    check_compact([[6, 5], [4, 3]], [32, 32], 3, 4, 16)
    check_compact([[0, 11, 7], [2, 50, -9]], [48, 48], 3, 9, 16)         # pages outside the pool stay
    check_compact([[31], [63], [64], [95]], [1, 1, 1, 1], 0, 96, 16)
    check_compact([[8, 9]], [-5], 0, 12, 16)


# ---------------------------------------------------------------- kv_copy_pages
@pytest.mark.parametrize("dtype,shape,pages", [(BF, (16, 2, 128), 40), (BF, (64, 3, 64), 17), (torch.uint8, (2, 16 * 136), 300),
                                               (torch.uint8, (1, 16), 9), (torch.float32, (5000, 4), 12), (torch.uint8, (3, 64 * 68), 50)])
@pytest.mark.parametrize("caches", [1, 2, 7])
def test_copy_pages(dtype, shape, pages, caches):
    note("kv_copy_pages %s x %d of %s, %d caches" % (shape, pages, dtype, caches))
    rng = np.random.default_rng(pages)
    order = rng.permutation(pages)
    n = pages // 2
    copies = np.stack([order[:n], order[n:2 * n]], 1)
    copies = np.concatenate([copies, [[0, 1], [-1, -1]]])                   # beyond n_copies: not made
    x = [torch.randint(0, 100, (pages, *shape), device="cuda").to(dtype) for _ in range(caches)]
    want = [t.clone() for t in x]
    for t in want:
        t[copies[:n, 1]] = t[copies[:n, 0]]
    S.kv_copy_pages([t.view(pages * shape[0], *shape[1:]) if dtype == BF else t for t in x], i32(copies.tolist()), i32([n]), pages=pages)
    torch.cuda.synchronize()
    for t, w in zip(x, want):
        assert torch.equal(t, w)


def test_copy_pages_leaves_out_what_is_no_copy():
    x = torch.arange(10 * 64, dtype=torch.int32, device="cuda").view(10, 64)
    want = x.clone()
    want[4] = want[2]
    S.kv_copy_pages([x], i32([[-1, 3], [2, 4], [3, -1], [10, 5], [6, 10], [7, 7], [5, 2000000000]]), i32([100]), pages=10)
    torch.cuda.synchronize()
    assert torch.equal(x, want)
    S.kv_copy_pages([x], i32([[1, 3]]), i32([-4]), pages=10)
    S.kv_copy_pages([x], i32([[1, 3]]), i32([0]), pages=10)
    S.kv_copy_pages([x], torch.empty((0, 2), dtype=torch.int32, device="cuda"), i32([3]), pages=10)
    torch.cuda.synchronize()
    assert torch.equal(x, want)


def test_copy_pages_past_4_gib():
    """Byte offsets past 2^32, one page beyond 2^31."""
    note("kv_copy_pages past 4 GiB")
    x = torch.zeros(5, 1 << 30, dtype=torch.uint8, device="cuda")
    x[4, -64:] = 9
    x[4, :64] = 7
    S.kv_copy_pages([x], i32([[4, 1]]), i32([1]), pages=5)
    torch.cuda.synchronize()
    assert (x[1, -64:] == 9).all() and (x[1, :64] == 7).all() and not x[1, 64:-64].any() and not x[0].any() and not x[2].any()


# ---------------------------------------------------------------- the 4-bit cache
def pattern(T, Hkv, D, seed):
    """bf16 rows over the type's whole range, zeros and what is not finite among them."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, Hkv, D)) * np.exp(rng.standard_normal((T, Hkv, 1)) * 3)
    x = torch.from_numpy(x).to(BF)
    b = x.view(torch.int16).numpy().view(np.uint16).copy()
    blocks = b.reshape(-1, 32)
    blocks[0] = 0
    if len(blocks) > 12:
        blocks[1], blocks[2, 5], blocks[3, 31], blocks[4, 0] = 0x8000, 0x7F80, 0xFFC1, 0xFF80
        blocks[5] = rng.integers(0, 0x7F, 32)                      # subnormal
        blocks[6] = rng.integers(0x7F00, 0x7F80, 32)               # the largest
        blocks[7], blocks[8] = 0x0001, 0x7F7F
        blocks[9] = rng.integers(0, 0x7F80, 32)                    # any finite bits
        blocks[10] = rng.integers(0x8000, 0xFF80, 32)
        blocks[11] = np.arange(32) * 8 + 0x3F00                    # on and around the halves
    return b.reshape(T, Hkv, D)


def to_dev(bits):
    return torch.from_numpy(bits.view(np.int16).copy()).cuda().view(BF)


@pytest.mark.parametrize("P,T,Hkv,D,page,pages,gap", [(1, 1, 1, 64, 16, 1, 0), (2, 37, 2, 128, 16, 7, 0), (1, 100, 3, 64, 32, 5, 8), (3, 15, 8, 128, 64, 1, 64),
                                                      (1, 1000, 1, 128, 1024, 2, 0), (2, 513, 4, 64, 16, 40, 16)])
def test_kv4_write_and_read(P, T, Hkv, D, page, pages, gap):
    note("kv4 write P=%d T=%d Hkv=%d D=%d page=%d" % (P, T, Hkv, D, page))
    rng = np.random.default_rng(T + D)
    slots = rng.permutation(page * pages)[:T]
    T = len(slots)
    if T > 5:
        slots[3], slots[5] = -1, page * pages                    # of no page
    ks, vs, caches, start = [], [], [], []
    for r in range(P):
        start.append(rng.integers(0, 256, (pages, Hkv, page * D * 17 // 16), dtype=np.uint8))
        caches.append(torch.from_numpy(start[r].copy()).cuda())
        ks.append(pattern(T, Hkv, D, 10 * r + T))
        vs.append(pattern(T, Hkv, D, 10 * r + T + 1))

    def rows(bits):                                              # slices of wider rows
        t = torch.zeros(T, Hkv * D + gap, dtype=BF, device="cuda")
        t[:, :Hkv * D] = to_dev(bits).view(T, -1)
        return t[:, :Hkv * D].view(T, Hkv, D) if not gap else t[:, :Hkv * D].unflatten(1, (Hkv, D))

    kd, vd = [rows(b) for b in ks], [rows(b) for b in vs]
    sl = torch.from_numpy(slots).long().cuda()
    S.tp_kv4_write(kd, vd, caches, sl, page_size=page)
    kr, vr = ([torch.full((T, Hkv, D), 3.0, dtype=BF, device="cuda") for _ in range(P)] for _ in range(2))
    S.tp_kv4_read(caches, sl, kr, vr, page_size=page)
    torch.cuda.synchronize()
    live = (slots >= 0) & (slots < page * pages)
    for r in range(P):
        want, values = start[r].copy(), []
        n = page * D // 2
        for which, bits in enumerate((ks[r], vs[r])):
            codes, scales = osr.quantise(osr.bf16(bits))
            values.append(np.where(live[:, None, None], osr.values(codes, scales), 0))
            nan = np.repeat(scales == 255, 16, -1)               # codes of a block that holds NaN may be any
            packed = (codes[..., 0::2] | codes[..., 1::2] << 4).astype(np.uint8)
            c = want[:, :, which * n:(which + 1) * n].reshape(pages, Hkv, page, D // 2)
            s = want[:, :, 2 * n + which * n // 16:2 * n + (which + 1) * n // 16].reshape(pages, Hkv, page, D // 32)
            got = caches[r].cpu().numpy()[:, :, which * n:(which + 1) * n].reshape(c.shape)
            for t in np.flatnonzero(live):
                p, i = slots[t] // page, slots[t] % page
                c[p, :, i] = np.where(nan[t], got[p, :, i], packed[t])
                s[p, :, i] = scales[t]
            want[:, :, which * n:(which + 1) * n] = c.reshape(pages, Hkv, n)
            want[:, :, 2 * n + which * n // 16:2 * n + (which + 1) * n // 16] = s.reshape(pages, Hkv, n // 16)
        assert np.array_equal(caches[r].cpu().numpy(), want)
        for got, w in zip((kr[r], vr[r]), values):
            assert np.array_equal(f64(got), w, equal_nan=True)


def test_kv4_every_value_and_scale():
    """Every bf16 number alone in its block, with and without a larger one beside it."""
    bits = np.zeros((65536 // 2, 1, 64), dtype=np.uint16)
    every = np.arange(65536, dtype=np.uint16).reshape(-1, 2)
    bits[:, 0, 3], bits[:, 0, 40] = every[:, 0], every[:, 1]
    beside = bits.copy()
    top = np.minimum((every & 0x7F80) + 0x0123, 0x7F7F)
    beside[:, 0, 9], beside[:, 0, 50] = top[:, 0], top[:, 1]
    cache = [S.kv4_cache(len(bits) // 64, 1, 64, 64)]
    sl = torch.arange(len(bits), device="cuda")
    kr, vr = ([torch.empty(len(bits), 1, 64, dtype=BF, device="cuda")] for _ in range(2))
    S.tp_kv4_write([to_dev(bits)], [to_dev(beside)], cache, sl, page_size=64)
    S.tp_kv4_read(cache, sl, kr, vr, page_size=64)
    for got, b in zip((kr, vr), (bits, beside)):
        assert np.array_equal(f64(got[0]), osr.values(*osr.quantise(osr.bf16(b))), equal_nan=True)


def test_kv4_empty_calls():
    cache, e = [S.kv4_cache(0, 2, 64, 16)], [torch.empty(0, 2, 64, dtype=BF, device="cuda")]
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    S.tp_kv4_write(e, e, cache, none, page_size=16)
    x = [torch.ones(3, 2, 64, dtype=BF, device="cuda")]
    S.tp_kv4_write(x, x, cache, torch.zeros(3, dtype=torch.int64, device="cuda"), page_size=16)
    S.tp_kv4_read(cache, torch.zeros(3, dtype=torch.int64, device="cuda"), x, x, page_size=16)
    assert not x[0].any()


# ---------------------------------------------------------------- decoding
def random_cache(P, pages, Hkv, D, page, seed):
    """Caches whose codes are any and whose scales are around one."""
    g = torch.Generator().manual_seed(seed)
    n = page * D
    out = []
    for _ in range(P):
        codes = torch.randint(0, 256, (pages, Hkv, n), generator=g, dtype=torch.uint8)
        scales = torch.randint(123, 128, (pages, Hkv, n // 16), generator=g, dtype=torch.uint8)
        out.append(torch.cat([codes, scales], 2).cuda())
    return out


def check_decode_kv4(q, cache, table, lengths, page, shared=None, group=1, scale=None, ws=None, o=None, wide=False):
    """Runs the call and holds every row to the oracle's bound; wide: with a
    table of more than 2048 keys a row, whose keys are shared out."""
    P, (B, Hq, D) = len(q), q[0].shape
    if wide:
        table = [list(row) + [-1] * (2048 // page + 1) for row in table]
    pages, Hkv = cache[0].shape[:2]
    o = o or [poisoned((B, Hq, D)) for _ in range(P)]
    ws = S.tp_attention_decode_kv4(q, cache, o, i32(table).reshape(B, -1), i32(lengths), page_size=page,
                                   shared=None if shared is None else i32(shared), group=group, scale=scale, ws=ws)
    torch.cuda.synchronize()
    width = len(table[0])
    G = Hq // Hkv
    for r in range(P):
        raw = cache[r].cpu().numpy()
        rows = {}
        for b in range(B):
            n = max(0, min(lengths[b], width * page))
            lead = 0
            if shared is not None and group > 1:
                g0 = b // group * group
                lead = max(0, min([shared[b // group], width * page] + [max(0, min(lengths[x], width * page)) for x in range(g0, g0 + group)]))
                lead = lead // 32 * 32                             # what is left of it, rows find through their own entries
            at = [table[b // group * group if j < lead else b][j // page] for j in range(n)]
            for h in range(Hkv):
                ks, vs = [], []
                for j, p in enumerate(at):
                    if 0 <= p < pages:
                        if (p, h) not in rows:
                            rows[p, h] = osr.rows_of(raw[p, h], D)
                        ks.append(rows[p, h][0][j % page])
                        vs.append(rows[p, h][1][j % page])
                k, v = np.array(ks).reshape(-1, D), np.array(vs).reshape(-1, D)
                qq = f64(q[r][b, h * G:(h + 1) * G])
                want, _, bound, _, _, _ = oa.attention(qq, k, v, np.ones((G, len(k)), bool), scale or D ** -0.5)
                # the oracle's sum is of weights w as they are; the call's is of the
                # rounded w (1 + d), |d| <= UB, so that o is off by sum w d (v - o)
                # instead of sum w d v: UB |o| more at most, as the w add up to 1
                bound = bound + oa.UB * np.abs(want)
                within(o[r][b, h * G:(h + 1) * G], want, bound, "rank %d row %d head %d" % (r, b, h))
    return ws


def decode_state(P, B, Hq, Hkv, D, page, lengths, seed, sharp=1.0):
    need = [-(-n // page) for n in lengths]
    width = max(need + [1])
    rng = np.random.default_rng(seed)
    ids = rng.permutation(sum(need) + 3)
    table, at = [], 0
    for n in need:
        table.append(ids[at:at + n].tolist() + [-1] * (width - n))
        at += n
    g = torch.Generator().manual_seed(seed)
    q = [(torch.randn(B, Hq, D, generator=g) * sharp).to(BF).cuda() for _ in range(P)]
    return q, random_cache(P, len(ids), Hkv, D, page, seed), table


DECODE = [(1, [1], 1, 1, 64, 16), (1, [16], 4, 1, 128, 16), (2, [5, 0, 33], 8, 2, 64, 16), (1, [31, 32, 33, 63, 64, 65], 6, 2, 128, 32),
          (3, [700, 3, 129], 5, 1, 128, 64), (1, [2000], 2, 2, 128, 16), (2, [300] * 9, 16, 1, 64, 128), (1, [90, 200], 40, 2, 128, 16),
          (1, [4100, 1, 77], 8, 1, 128, 16), (4, [100, 50], 8, 8, 64, 16), (16, [40, 41], 2, 1, 128, 32), (1, [500, 260], 34, 1, 64, 16)]


@pytest.mark.parametrize("P,lengths,Hq,Hkv,D,page", DECODE)
@pytest.mark.parametrize("wide", [False, True])
def test_decode_kv4(P, lengths, Hq, Hkv, D, page, wide):
    note("decode_kv4 P=%d lengths=%s heads=%d/%d D=%d page=%d wide=%s" % (P, lengths[:6], Hq, Hkv, D, page, wide))
    q, cache, table = decode_state(P, len(lengths), Hq, Hkv, D, page, lengths, len(lengths) * 7 + D)
    check_decode_kv4(q, cache, table, lengths, page, wide=wide)


@pytest.mark.parametrize("group,G,D,page,shared,own", [
    (2, 1, 64, 16, 40, 30), (4, 4, 128, 16, 300, 50), (4, 2, 64, 32, 31, 40), (3, 5, 128, 64, 64, 1), (8, 8, 128, 16, 100, 20),
    (5, 3, 64, 16, 33, 0), (16, 4, 64, 16, 128, 17), (20, 7, 128, 32, 200, 9), (2, 20, 128, 16, 90, 33), (1, 4, 128, 16, 60, 10)])
def test_decode_kv4_of_groups(group, G, D, page, shared, own):
    note("decode_kv4 groups of %d, %d heads, D=%d page=%d shared=%d" % (group, G, D, page, shared))
    groups, Hkv = 3, 2
    B = groups * group
    rng = np.random.default_rng(group * 11 + D)
    lead = [shared, 0 if shared > 50 else shared, shared + 7]
    lengths = [lead[b // group] + int(rng.integers(0, own + 1)) for b in range(B)]
    q, cache, table = decode_state(2, B, G * Hkv, Hkv, D, page, lengths, group + D)
    # whole shared pages, and the page that holds the last shared keys (copies of it, in earnest: here the same one)
    for b in range(B):
        first = b // group * group
        n = -(-lead[b // group] // page)
        table[b][:n] = table[first][:n]
    sh = [n // page * page for n in lead]
    ws = check_decode_kv4(q, cache, table, lengths, page, shared=sh, group=group)
    check_decode_kv4(q, cache, table, lengths, page, shared=lead, group=group, ws=ws)
    check_decode_kv4(q, cache, table, lengths, page, group=group, ws=ws)
    check_decode_kv4(q, cache, table, lengths, page, shared=sh, group=group, ws=ws, wide=True)


def test_decode_kv4_of_shared_lengths_past_the_rows():
    """shared[g] beyond a row's keys, below zero, and rows without keys."""
    lengths = [100, 40, 70, 0, 64, 64, 200, 200]
    q, cache, table = decode_state(1, 8, 4, 1, 128, 16, lengths, 5)
    for b in range(8):
        n = -(-lengths[b] // 16)
        first = b // 2 * 2
        k = min(n, -(-lengths[first] // 16))
        table[b][:k] = table[first][:k]
    check_decode_kv4(q, cache, table, lengths, 16, shared=[1000, -5, 64, 200], group=2)


def test_decode_kv4_of_several_tokens_of_a_request():
    """Four tokens in turn: a group whose rows see one key more each."""
    n = 333
    q, cache, table = decode_state(1, 4, 8, 2, 64, 16, [n] * 4, 8)
    table = [table[0]] * 4
    lengths = [n - 3, n - 2, n - 1, n]
    check_decode_kv4(q, cache, table, lengths, 16, shared=[n - 3], group=4)


def test_decode_kv4_of_pages_that_are_none():
    lengths = [100, 70, 50, 20]
    q, cache, table = decode_state(1, 4, 4, 2, 128, 16, lengths, 9)
    table[0][1], table[0][4], table[1][0], table[3] = -1, 5000, 1 << 30, [-1] * len(table[3])
    for wide in (False, True):
        check_decode_kv4(q, cache, table, lengths, 16, wide=wide)
        check_decode_kv4(q, cache, table, lengths, 16, shared=[64, 0], group=2, wide=wide)
        check_decode_kv4(q, cache, table, [1 << 30, -4, 50, 20], 16, wide=wide)          # lengths past the table


def test_decode_kv4_without_a_cache():
    q = [torch.ones(2, 4, 64, dtype=BF, device="cuda")]
    o = [poisoned((2, 4, 64))]
    S.tp_attention_decode_kv4(q, [S.kv4_cache(0, 2, 64, 16)], o, i32([[0], [1]]), i32([5, 9]), page_size=16)
    assert not o[0].any()
    o = [poisoned((2, 4, 64))]
    S.tp_attention_decode_kv4(q, [S.kv4_cache(3, 2, 64, 16)], o, i32([[], []]).reshape(2, 0), i32([5, 9]), page_size=16)
    assert not o[0].any()


def test_decode_kv4_sees_no_row_that_is_no_key():
    """NaN scales in every cache row that is no key of a row, in its own pages too."""
    lengths = [45, 10, 64, 33]
    q, cache, table = decode_state(1, 4, 4, 1, 128, 16, lengths, 12)
    n = 16 * 128
    used = {(table[b][j // 16], j % 16) for b in range(4) for j in range(lengths[b])}
    scales = cache[0][:, :, n:].view(cache[0].shape[0], 1, 2, 16, 4)
    for p in range(cache[0].shape[0]):
        for i in range(16):
            if (p, i) not in used:
                scales[p, :, :, i] = 255
    check_decode_kv4(q, cache, table, lengths, 16)
    check_decode_kv4(q, cache, table, lengths, 16, wide=True)
    check_decode_kv4(q, cache, table, lengths, 16, shared=[0, 32], group=2)


def test_decode_kv4_of_keys_and_values_that_are_nan():
    """They reach the rows that see them, and no other."""
    lengths = [40, 40, 40]
    q, cache, table = decode_state(1, 3, 2, 1, 64, 16, lengths, 13)
    n = 16 * 64
    scales = cache[0][:, :, n:].view(cache[0].shape[0], 1, 2, 16, 2)
    scales[table[0][1], 0, 0, 3, 0] = 255                     # a key of row 0
    scales[table[1][2], 0, 1, 5, 1] = 255                     # a value of row 1: its second block
    for pad in (0, 200):
        o = [poisoned((3, 2, 64))]
        S.tp_attention_decode_kv4(q, cache, o, i32([row + [-1] * pad for row in table]), i32(lengths), page_size=16)
        x = f64(o[0])
        assert np.isnan(x[0]).all() and np.isnan(x[1, :, 32:]).all() and np.isfinite(x[1, :, :32]).all() and np.isfinite(x[2]).all()


@pytest.mark.parametrize("sharp", [0.0, 30.0])
def test_decode_kv4_of_flat_and_sharp_rows(sharp):
    lengths = [600, 1000]
    q, cache, table = decode_state(1, 2, 4, 1, 128, 16, lengths, 14, sharp)
    check_decode_kv4(q, cache, table, lengths, 16)
    check_decode_kv4(q, cache, table, lengths, 16, wide=True)


def test_decode_kv4_of_slices_of_wider_rows():
    lengths = [50, 80, 20]
    q, cache, table = decode_state(2, 3, 4, 2, 64, 16, lengths, 15)
    wide = [torch.full((3, 10, 64), 7.0, dtype=BF, device="cuda") for _ in range(2)]
    for w, t in zip(wide, q):
        w[:, 2:6] = t
    o = [torch.full((3, 12, 64), 5.0, dtype=BF, device="cuda") for _ in range(2)]
    check_decode_kv4([w[:, 2:6] for w in wide], cache, table, lengths, 16, o=[t[:, 4:8] for t in o])
    for t in o:
        assert (t[:, :4] == 5).all() and (t[:, 8:] == 5).all()


def test_decode_kv4_gives_the_same_bits_every_time():
    lengths = [3000, 10, 700, 701] * 5
    q, cache, table = decode_state(2, 20, 8, 2, 128, 16, lengths, 16)
    for b in range(20):
        table[b][:12] = table[b // 4 * 4][:12] if lengths[b] >= 192 and lengths[b // 4 * 4] >= 192 else table[b][:12]
    args = (i32(table), i32(lengths))
    first, ws = None, None
    for _ in range(5):
        o = [poisoned((20, 8, 128)) for _ in range(2)]
        ws = S.tp_attention_decode_kv4(q, cache, o, *args, page_size=16, shared=i32([10] * 5), group=4, ws=ws)
        bits = torch.stack(o).view(torch.int16)
        first = bits if first is None else first
        assert torch.equal(bits, first)


def test_decode_kv4_past_4_gib():
    """A cache whose pages lie past 2^32 bytes."""
    note("decode_kv4 past 4 GiB")
    pages, page, D = 40000, 1024, 128                         # 139264 bytes a page and head: 5.2 GiB
    cache = [torch.zeros(pages, 1, page * 136, dtype=torch.uint8, device="cuda")]
    small = random_cache(1, 3, 1, D, page, 17)
    where = [39999, 2, 31000]
    for i, p in enumerate(where):
        cache[0][p] = small[0][i]
    q = [torch.randn(1, 4, D, generator=torch.Generator().manual_seed(17)).to(BF).cuda()]
    outs = []
    for c, t in ((cache, where), (small, [0, 1, 2])):
        o = [poisoned((1, 4, D))]
        S.tp_attention_decode_kv4(q, c, o, i32([t]), i32([2500]), page_size=page)
        outs.append(o[0])
    assert torch.equal(outs[0], outs[1])
    slots = torch.tensor([39999 * 1024 + 5, 31000 * 1024 + 1023], device="cuda")
    x = torch.randn(2, 1, D, generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    k, v = torch.empty_like(x), torch.empty_like(x)
    S.tp_kv4_write([x], [-x], cache, slots, page_size=page)
    S.tp_kv4_read(cache, slots, [k], [v], page_size=page)
    assert torch.equal(k, -v) and np.array_equal(f64(k), osr.values(*osr.quantise(f64(x))))
