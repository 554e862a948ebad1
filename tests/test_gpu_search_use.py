"""GPU tests of how the beam search calls are used: what the Python entry
points refuse, streams and graph capture, a step's calls together, workspaces
of batches that shrink, and the search of examples/beam_search.py."""
import os
import sys

import numpy as np
import pytest
import torch

from oracle import search as osr
from ring_collectives_amd import _native as N
from ring_collectives_amd import attention as A
from ring_collectives_amd import collectives as rc
from ring_collectives_amd import search as S

from _gpu_helpers import note
from test_gpu_attention import BF, f64, i32, poisoned
from test_gpu_search import check_decode_kv4, check_select, decode_state, fork_state, random_cache

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    N.lib()
    yield


# ---------------------------------------------------------------- refusals
def refuses(call, base):
    def bad(exc, match, **kw):
        with pytest.raises(exc, match=match):
            call(**{**base, **kw})
    return bad


def test_select_refusals():
    x = [torch.zeros(6, 128, device="cuda") for _ in range(2)]
    p, f = i32([[0] * 4] * 2), torch.zeros(2, 3, device="cuda")
    d, da = torch.zeros(2, 3, dtype=torch.bool, device="cuda"), torch.zeros(2, 4, dtype=torch.bool, device="cuda")
    bad = refuses(S.beam_select, dict(logits=x, scores=f, parents=p, tokens=p.clone(), scores_after=torch.zeros(2, 4, device="cuda"), vocab=200))
    bad(ValueError, "rank buffers", logits=[])
    bad(ValueError, "must be", logits=[x[0], x[1][:, :64]])
    bad(TypeError, "float32 or bfloat16", logits=[t.double() for t in x])
    bad(ValueError, "rows of logits", scores=torch.zeros(2, 2, device="cuda"))
    bad(ValueError, "parents", parents=i32([[0] * 4] * 3))
    bad(ValueError, "tokens", tokens=i32([[0] * 3] * 2))
    bad(TypeError, "Float", scores=f.double())
    bad(TypeError, "Int", parents=p.long())
    bad(ValueError, "scores_after", scores_after=torch.zeros(2, 5, device="cuda"))
    bad(ValueError, "go together", done=d, end_token=3)
    bad(TypeError, "Byte", done=d.int(), done_after=da, end_token=3)
    bad(ValueError, "done_after", done=d, done_after=d, end_token=3)
    bad(N.RingError, "failed", done=d, done_after=da)                  # no end token
    bad(N.RingError, "failed", vocab=257)
    bad(N.RingError, "failed", vocab=0)
    bad(N.RingError, "failed", logits=[torch.zeros(6, 129, device="cuda")[:, :128] for _ in range(2)])       # rows 129 apart
    bad(ValueError, "current device", scores=f.cpu())
    bad(ValueError, "workspace", ws=torch.zeros(4096, dtype=torch.uint8))
    bad(N.RingError, "workspace", ws=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    bad(ValueError, "at least one beam", logits=[t[:0] for t in x], scores=f[:, :0])


def test_fork_refusals():
    base = dict(block_table=i32([[0, 1], [2, 3]]), lengths=i32([5, 6]), parents=i32([[0, 1]]), free_pages=i32([4, 5]), used=i32([0]),
                table_after=i32([[0, 0]] * 2), lengths_after=i32([0, 0]), copies=i32([[0, 0]] * 2), n_copies=i32([0]), used_after=i32([0]),
                page_size=16, pages=6, shared=i32([0]), group=2)
    S.kv_fork(**base)
    bad = refuses(S.kv_fork, base)
    bad(ValueError, "table_after", table_after=i32([[0, 0, 0]] * 2))
    bad(ValueError, "elements", parents=i32([0, 1, 0]))
    bad(ValueError, "elements", keep=i32([0]))
    bad(ValueError, "elements", lengths_after=i32([0]))
    bad(ValueError, "copies", copies=i32([[0, 0]]))
    bad(ValueError, "elements", shared=i32([0, 0]))
    bad(ValueError, "groups of", group=3)
    bad(ValueError, "groups of", group=0)
    bad(TypeError, "Int", free_pages=i32([4, 5]).long())
    bad(ValueError, "contiguous", block_table=i32([[0, 1, 2], [3, 4, 5]])[:, :2])
    bad(N.RingError, "failed", page_size=24)
    bad(N.RingError, "failed", pages=-1, ws=torch.zeros(4096, dtype=torch.uint8, device="cuda"))
    bad(N.RingError, "failed", used_after=base["used"])
    bad(N.RingError, "failed", lengths_after=base["lengths"])
    bad(N.RingError, "failed", table_after=base["block_table"])
    bad(N.RingError, "workspace", ws=torch.zeros(256, dtype=torch.uint8, device="cuda"))


def test_compact_and_copy_refusals():
    base = dict(block_table=i32([[0, 1], [2, 3]]), lengths=i32([5, 6]), table_after=i32([[0, 0]] * 2), free_pages=i32([0] * 6),
                copies=i32([[0, 0]] * 3), n_copies=i32([0]), used_after=i32([0]), page_size=16)
    S.kv_compact(**base)
    bad = refuses(S.kv_compact, base)
    bad(ValueError, "table_after", table_after=i32([[0, 0]]))
    bad(ValueError, "copies", copies=i32([[0, 0]] * 2))
    bad(ValueError, "elements", lengths=i32([5]))
    bad(N.RingError, "failed", table_after=base["block_table"])
    bad(N.RingError, "failed", first_page=-1)
    x = [torch.zeros(6, 64, device="cuda"), torch.zeros(6, 64, device="cuda")]
    bad = refuses(S.kv_copy_pages, dict(caches=x, copies=i32([[0, 1]]), n_copies=i32([1]), pages=6))
    bad(ValueError, "caches", caches=[])
    bad(ValueError, "caches", caches=x * 65)
    bad(ValueError, "same size", caches=[x[0], x[1][:3]])
    bad(ValueError, "pages", pages=5)
    bad(ValueError, "pages", pages=-6)
    bad(ValueError, "contiguous", caches=[x[0].t()])
    bad(ValueError, "copies", copies=i32([0, 1]))
    bad(ValueError, "copies", copies=i32([[0, 1, 2]]))
    bad(N.RingError, "failed", caches=[torch.zeros(6, 2, device="cuda")])       # 8 bytes a page


def test_kv4_refusals():
    k = [torch.zeros(3, 2, 64, dtype=BF, device="cuda")]
    cache, slots = [S.kv4_cache(4, 2, 64, 16)], torch.zeros(3, dtype=torch.int64, device="cuda")
    for call in (S.tp_kv4_write, S.tp_kv4_read):
        bad = refuses(call, dict(k=k, v=k, cache=cache, slots=slots, page_size=16))
        bad(TypeError, "BFloat16", k=[k[0].float()])
        bad(ValueError, "must be", v=[k[0][:2]])
        bad(ValueError, "heads", cache=[S.kv4_cache(4, 3, 64, 16)])
        bad(ValueError, "bytes a head", cache=[S.kv4_cache(4, 2, 64, 32)])
        bad(ValueError, "bytes a head", page_size=32)
        bad(TypeError, "Byte", cache=[cache[0].view(torch.int8)])
        bad(TypeError, "Long", slots=slots.int())
        bad(ValueError, "elements", slots=slots[:2])
        bad(N.RingError, "failed", page_size=8, cache=[cache[0][:, :, :8 * 68].contiguous()])
        bad(N.RingError, "failed", k=[torch.zeros(3, 2, 96, dtype=BF, device="cuda")], v=[torch.zeros(3, 2, 96, dtype=BF, device="cuda")])
    q = [torch.zeros(4, 4, 64, dtype=BF, device="cuda")]
    bad = refuses(S.tp_attention_decode_kv4, dict(q=q, cache=cache, o=[torch.zeros_like(q[0])], block_table=i32([[0]] * 4), lengths=i32([1] * 4),
                                                  page_size=16))
    bad(ValueError, "bytes a head", page_size=32)
    bad(ValueError, "block_table", block_table=i32([[0]] * 3))
    bad(ValueError, "elements", lengths=i32([1]))
    bad(ValueError, "elements", shared=i32([1]), group=2)
    bad(ValueError, "groups of", group=3)
    bad(ValueError, "rank buffers", cache=cache * 2)
    bad(ValueError, "must be", o=[q[0][:, :2]])
    bad(N.RingError, "failed", scale=0.0)
    bad(N.RingError, "failed", q=[t[:, :3] for t in q], o=[torch.zeros(4, 3, 64, dtype=BF, device="cuda")])
    bad(N.RingError, "workspace", ws=torch.zeros(128, dtype=torch.uint8, device="cuda"))


# ---------------------------------------------------------------- a step's calls together
class Step:
    """Fixed buffers of one step of a search over a 4-bit cache: choose, fork,
    copy, plan, write, decode, and the state back to where it was read."""

    def __init__(self, seed, n=5, W=3, P=2, Hq=4, Hkv=2, D=64, page=16, vocab=700, width=384):
        self.n, self.W, self.P, self.page, self.vocab = n, W, P, page, vocab
        rows = n * W
        table, lens, free, used, pages = fork_state(rows, page, 200, 16, 60, seed, group=W)
        table = [row if ln else [-1] * 16 for row, ln in zip(table, lens)]
        self.pages = pages
        self.table, self.lengths, self.free, self.used = i32(table), i32(lens), i32(free), i32([used])
        self.cache = random_cache(P, pages, Hkv, D, page, seed)
        e = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt, device="cuda")          # noqa: E731
        self.logits = [e(rows, width, dt=torch.float32) for _ in range(P)]
        self.q, self.k, self.v = ([e(rows, h, D, dt=BF) for _ in range(P)] for h in (Hq, Hkv, Hkv))
        self.o = [e(rows, Hq, D, dt=BF) for _ in range(P)]
        self.scores, self.done = e(n, W, dt=torch.float32), e(n, W, dt=torch.bool)
        self.parents, self.tokens, self.after, self.done_after = e(n, W), e(n, W), e(n, W, dt=torch.float32), e(n, W, dt=torch.bool)
        self.table2, self.lengths2, self.copies, self.n_copies, self.shared, self.used2 = e(rows, 16), e(rows), e(rows, 2), e(1), e(n), e(1)
        self.lengths3, self.cu, self.pos, self.slots, self.used3 = e(rows), e(rows + 1), e(rows), e(rows, dt=torch.int64), e(1)
        self.one = torch.ones(rows, dtype=torch.int32, device="cuda")
        self.ws = [None, None, None]

    def feed(self, seed):
        g = torch.Generator().manual_seed(seed)
        for t in self.logits + self.q + self.k + self.v:
            t.copy_(torch.randn(t.shape, generator=g))

    def run(self):
        self.ws[0] = S.beam_select(self.logits, self.scores, self.parents, self.tokens, self.after, vocab=self.vocab, done=self.done,
                                   done_after=self.done_after, end_token=11, ws=self.ws[0])
        self.ws[1] = S.kv_fork(self.table, self.lengths, self.parents, self.free, self.used, self.table2, self.lengths2, self.copies,
                               self.n_copies, self.used2, page_size=self.page, pages=self.pages, shared=self.shared, group=self.W, ws=self.ws[1])
        S.kv_copy_pages(self.cache, self.copies, self.n_copies, pages=self.pages)
        A.kv_plan(self.lengths2, self.one, self.free, self.used2, self.table2, self.lengths3, self.cu, self.pos, self.slots, self.used3,
                  page_size=self.page)
        S.tp_kv4_write(self.k, self.v, self.cache, self.slots, page_size=self.page)
        self.ws[2] = S.tp_attention_decode_kv4(self.q, self.cache, self.o, self.table2, self.lengths3, page_size=self.page, shared=self.shared,
                                               group=self.W, ws=self.ws[2])
        self.scores.copy_(self.after)
        self.done.copy_(self.done_after)
        self.table.copy_(self.table2)
        self.lengths.copy_(self.lengths3)
        self.used.copy_(self.used3)

    def state(self):
        ts = [self.parents, self.tokens, self.after, self.done_after, self.table, self.lengths, self.copies, self.n_copies, self.shared,
              self.used, self.slots, self.free[int(self.used):].sort().values] + self.cache + self.o
        return [t.clone().view(torch.int16) if t.dtype == BF else t.clone() for t in ts]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def check_step(s, before_table, before_lengths, before_used, before_free):
    """What the step did against the oracle, from the state before it."""
    want = osr.fork(before_table, before_lengths, s.parents.flatten().tolist(), None, before_free, before_used, s.page, s.pages, s.W)
    assert np.array_equal(s.copies.cpu().numpy(), want[2]) and s.n_copies.item() == want[3]
    assert np.array_equal(s.shared.cpu().numpy(), want[4]) and s.used2.item() == want[5]
    assert np.array_equal(s.lengths2.cpu().numpy(), want[1])
    assert s.used3.item() <= s.free.numel()
    # every page in use once among the rows' own, none of them free
    held = {e for row, n in zip(s.table.tolist(), s.lengths.tolist()) for e in row[:-(-n // s.page)]}
    assert not held & set(s.free[s.used.item():].tolist())
    check_decode_kv4(s.q, s.cache, s.table.tolist(), s.lengths.tolist(), s.page, shared=s.shared.tolist(), group=s.W)


def test_steps_of_a_search():
    s = Step(1)
    for i in range(6):
        s.feed(100 + i)
        before = s.table.tolist(), s.lengths.tolist(), s.used.item(), s.free.tolist()
        s.run()
        torch.cuda.synchronize()
        check_step(s, *before)
    for ws in s.ws:
        assert rc.last_error(ws)[0] == 0


def test_step_captured_in_a_graph():
    """Replays with the program's own work between them give the eager step's bits."""
    note("beam search step in a graph")
    eager, other = Step(2), Step(2)
    eager.feed(0)
    other.feed(0)
    eager.run()
    other.run()                                            # workspaces are there before the capture
    torch.cuda.synchronize()
    assert same(eager.state(), other.state())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        other.run()
    for i in range(5):
        eager.feed(i + 1)
        eager.run()
        other.feed(i + 1)
        graph.replay()
        torch.cuda.synchronize()
        assert same(eager.state(), other.state()), i
        torch.randn(1000, device="cuda").sort()            # the program's own
    assert all(rc.last_error(ws)[0] == 0 for ws in other.ws)


def test_compaction_captured_in_a_graph():
    table, lens, free, used, pages = fork_state(9, 16, 200, 14, 90, 4, group=3)
    tab, ln, fp = i32(table), i32(lens), i32(free)
    out, copies, n, u = torch.empty_like(tab), i32([[0, 0]] * (pages // 2)), i32([0]), i32([0])
    cache = random_cache(1, pages, 2, 64, 16, 3)
    ws = S.kv_compact(tab, ln, out, fp, copies, n, u, page_size=16)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        S.kv_compact(tab, ln, out, fp, copies, n, u, page_size=16, ws=ws)
        S.kv_copy_pages(cache, copies, n, pages=pages)
    rng = np.random.default_rng(1)
    for i in range(4):
        ln.copy_(i32(np.minimum(lens, rng.integers(0, 200, 9)).tolist()))
        was = cache[0].clone()
        graph.replay()
        torch.cuda.synchronize()
        want = osr.compact(table, ln.tolist(), 0, pages, 16)
        for g, w in zip((out, copies, n, u, fp), want):
            assert np.array_equal(g.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1))
        for a, b in copies[:n.item()].tolist():
            assert torch.equal(cache[0][b], was[a])
        torch.cuda.synchronize()


def test_step_on_a_side_stream():
    here, there = Step(3), Step(3)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    for i in range(3):
        here.feed(i)
        here.run()
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            there.feed(i)
            there.run()
    stream.synchronize()
    assert same(here.state(), there.state())


def test_stream_argument():
    """stream= runs there, behind what that stream has, with a workspace of its own."""
    q, cache, table = decode_state(1, 3, 4, 2, 64, 16, [300, 900, 5], 5)
    o1, o2 = [poisoned((3, 4, 64))], [poisoned((3, 4, 64))]
    S.tp_attention_decode_kv4(q, cache, o1, i32(table), i32([300, 900, 5]), page_size=16)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    args = i32(table), i32([300, 900, 5])
    torch.cuda.synchronize()
    S.tp_attention_decode_kv4(q, cache, o2, *args, page_size=16, stream=stream)
    stream.synchronize()
    assert torch.equal(o1[0].view(torch.int16), o2[0].view(torch.int16))
    x = torch.randn(6, 512, device="cuda")
    sc, p, t, a = torch.zeros(2, 3, device="cuda"), i32([[0] * 3] * 2), i32([[0] * 3] * 2), torch.zeros(2, 3, device="cuda")
    p2, t2, a2 = torch.empty_like(p), torch.empty_like(t), torch.empty_like(a)
    S.beam_select([x], sc, p, t, a, vocab=500)
    torch.cuda.synchronize()
    S.beam_select([x], sc, p2, t2, a2, vocab=500, stream=stream)
    stream.synchronize()
    assert torch.equal(p, p2) and torch.equal(t, t2) and torch.equal(a, a2)


def test_two_searches_at_once_on_two_streams():
    """Each with workspaces of its own."""
    alone = [Step(6), Step(7)]
    for s in alone:
        for i in range(4):
            s.feed(i)
            s.run()
    torch.cuda.synchronize()
    both, streams = [Step(6), Step(7)], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for i in range(4):
        for s, stream in zip(both, streams):
            with torch.cuda.stream(stream):
                s.feed(i)
                s.run()
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        assert same(a.state(), b.state())


# ---------------------------------------------------------------- workspaces
def test_decode_workspace_of_smaller_batches():
    """One made for a batch serves every smaller one, with and without shared keys."""
    ws = None
    for B in (24, 16, 8, 4):
        lengths = [700 + 3 * b for b in range(B)]
        q, cache, table = decode_state(1, B, 4, 2, 64, 16, lengths, B)
        ws = check_decode_kv4(q, cache, table, lengths, 16, group=4, ws=ws)
        check_decode_kv4(q, cache, table, lengths, 16, shared=[0] * (B // 4), group=4, ws=ws)


def test_large_batches():
    """As many rows as the calls take."""
    note("decode_kv4 of 8192 rows")
    B, page, D = 8192, 16, 64
    q = [torch.randn(B, 1, D, device="cuda").to(BF)]
    cache = random_cache(1, 100, 1, D, page, 3)
    table, lens = torch.randint(0, 100, (B, 40), device="cuda").int(), torch.randint(0, 641, (B,), device="cuda").int()
    shared = torch.randint(0, 641, (B // 8,), device="cuda").int()
    table = table.view(-1, 8, 40)[:, :1].expand(-1, 8, -1).reshape(B, 40).contiguous()       # groups on the same pages
    o1, o2 = [poisoned((B, 1, D))], [poisoned((B, 1, D))]
    S.tp_attention_decode_kv4(q, cache, o1, torch.cat([table, table.new_full((B, 100), -1)], 1), lens, page_size=page)
    S.tp_attention_decode_kv4(q, cache, o2, table, lens, page_size=page, shared=shared, group=8)
    some = torch.arange(0, B, 997, device="cuda")
    check_decode_kv4([q[0][some]], cache, table[some].tolist(), lens[some].tolist(), page)
    a, b = o1[0].float(), o2[0].float()
    assert torch.isfinite(a).all() and torch.isfinite(b).all()
    # both are within 2^-8 of their value and 2 2^-8 of the weighted values' sizes (at most 6 here) of the same numbers
    assert (a - b).abs().max() <= 2 * 3 * 6 * 2 ** -8


def test_select_of_many_groups():
    g = torch.Generator().manual_seed(9)
    x = torch.randn(6000, 97, generator=g)
    check_select(x, -np.random.default_rng(9).random((3000, 2)), 1, 104, 2, torch.float32)


# ---------------------------------------------------------------- the search
def test_example_search_runs():
    import beam_search as ex
    s = ex.search()
    seqs, scores = s.results()
    torch.cuda.synchronize()
    assert all(len(q) == 13 for g in seqs for q in g) and all(0 <= t < s.vocab for g in seqs for q in g for t in q)
    assert all(a >= b for g in scores for a, b in zip(g, g[1:]))
    assert all(len({tuple(q) for q in g}) == len(g) for g in seqs)
    # pages: those of the rows, and no others, are in use
    held = {e for row, n in zip(s.table.tolist(), s.lengths.tolist()) for e in row[:-(-n // s.page)]}
    assert len(held) == s.used.item() and not held & set(s.free[s.used.item():].tolist())
    assert all(rc.last_error(ws)[0] == 0 for ws in s.ws.values())
    # prompts of 40, 17 and 90 tokens: their whole pages are shared at least
    assert all(a >= n // 16 * 16 for a, n in zip(s.shared.tolist(), (40, 17, 90)))


def test_example_search_with_compaction_is_the_same():
    """Where pages lie changes nothing, to the bit."""
    import beam_search as ex
    a, b = ex.search().results(), ex.search(compact_every=2).results()
    assert a == b


def test_example_scores_are_the_sequences_log_probabilities():
    """Each beam's score from its tokens alone: the plain layer in fp32 over the
    4-bit values of its keys and values."""
    import beam_search as ex
    s = ex.search(lens=(40,), steps=5)
    seqs, scores = s.results()
    g = torch.Generator(device="cuda").manual_seed(1)
    prompt = torch.randint(0, s.vocab, (40,), generator=g, device="cuda").tolist()
    for seq, score in zip(seqs[0], scores[0]):
        toks, total, kv = prompt + seq, 0.0, []
        x = s.embed[torch.tensor(toks, device="cuda")]
        pos = torch.arange(len(toks), device="cuda").int()
        q, k, v = s.project(x, pos)
        for r in range(s.P):
            kv.append([torch.from_numpy(osr.values(*osr.quantise(f64(t)))).float().cuda() for t in (k[r], v[r])])
        ended = False
        for t in range(39, len(toks) - 1):
            # the prompt's own attention has its keys in bf16
            exact = t == 39
            out = x[t].float()
            for r in range(s.P):
                kk, vv = (k[r].float(), v[r].float()) if exact else kv[r]
                o = []
                for h in range(s.Hq):
                    p = (kk[:t + 1, h * s.Hkv // s.Hq] @ q[r][t, h].float() * s.D ** -0.5).softmax(0)
                    o.append(p @ vv[:t + 1, h * s.Hkv // s.Hq])
                out = out + torch.cat(o) @ s.wo[r].float()
            lp = torch.cat([out @ w.float() for w in s.wvocab])[:s.vocab].log_softmax(0)
            if not ended:
                total += lp[toks[t + 1]].item()
            ended = ended or toks[t + 1] == s.end
        # a step rounds o and the softmax weights to bf16: o is off by two halves
        # of 2^-8 in size, a logit (standard deviation 2 for a hidden vector of
        # size 1 a value) by 2 2^-8 with random signs; four times that for each
        # of six steps, twice for the sum of a logit and its log sum exp
        assert abs(total - score) < 6 * 2 * 4 * 2 * 2 ** -8, (total, score)
