"""beam_select's log sum exp over wide rows: its error does not grow with the
number of columns a lane goes through, whatever order the logits come in."""
import numpy as np
import pytest
import torch

from oracle import search as osr


def rows(vocab, seed):
    """Rows on which a running fp32 sum goes wrong by many roundings."""
    rng = np.random.default_rng(seed)
    peaked = rng.standard_normal((4, vocab))
    peaked[np.arange(4), [vocab // 500, vocab // 3, 0, vocab - 1]] = [16.5, 18.0, 20.0, 17.0]       # a model that is sure
    equal = np.full(vocab, -16.0)
    equal[5] = 0.0
    return np.stack([*peaked, equal, np.linspace(0, 1, vocab), np.linspace(1, 0, vocab), rng.standard_normal(vocab) * 2.5]).astype(np.float32)


def test_bound_does_not_grow_with_the_columns():
    x = np.zeros(1 << 18, np.float32)
    assert osr.log_probs(x)[1] == osr.log_probs(x[:512])[1]
    for row in rows(200000, 1):
        assert osr.log_probs(row)[1] < 2e-6


@pytest.mark.gpu
@pytest.mark.parametrize("vocab,P,groups,beams", [
    (100003, 1, 512, 8), (200000, 1, 64, 64), (200000, 8, 64, 8),       # a part of a row of one rank, or one
    (200000, 1, 8, 1), (150001, 4, 8, 2), (1000, 1, 8, 1)])             # as many parts as there are
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_log_sum_exp(vocab, P, groups, beams, dtype):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from _gpu_helpers import note
    from ring_collectives_amd import search as S
    note("beam_select sums vocab=%d P=%d groups=%d beams=%d %s" % (vocab, P, groups, beams, dtype))
    x = torch.from_numpy(rows(vocab, vocab)).to(dtype)
    width = -(-vocab // (8 * P)) * 8
    n = groups * beams
    at = torch.arange(8) * (n // 8)                        # the rows that have a score; the others are not read
    logits = [torch.empty(n, width, dtype=dtype, device="cuda") for _ in range(P)]
    for r, t in enumerate(logits):
        part = x[:, r * width:(r + 1) * width]
        t[at.cuda(), :part.shape[1]] = part.cuda()
    want, bound = zip(*(osr.log_probs(row) for row in x.float().numpy()))
    best = np.array([w.max() for w in want])
    # scores that all but cancel the best log probability, so that fp32 shows what is left
    scores = torch.full((n,), -float("inf"))
    scores[at] = torch.from_numpy(-best).float()
    parents, tokens = (torch.zeros(groups, 8, dtype=torch.int32, device="cuda") for _ in range(2))
    after = torch.zeros(groups, 8, device="cuda")
    S.beam_select(logits, scores.view(groups, beams).cuda(), parents, tokens, after, vocab=vocab)
    parents, after = parents.flatten().tolist(), after.flatten().tolist()
    for i, row in enumerate(at.tolist()):
        got = max(a for p, a in zip(parents, after) if p == row)
        exact = float(scores[row]) + best[i]               # at most half a step of fp32 of |best|
        assert abs(got - exact) <= bound[i] + osr.U * abs(exact), (i, got - exact, bound[i])
