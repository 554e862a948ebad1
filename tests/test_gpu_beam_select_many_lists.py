"""beam_select where a group's lists are joined by 5 to 16 waves and then by
one: wide vocabularies of few rows, and many ranks."""
import numpy as np
import pytest
import torch

from oracle import search as osr

pytestmark = pytest.mark.gpu

# ranks, groups, beams, places, columns of a rank, tokens; lists of a group
CASES = [(64, 2, 5, 5, 128, 8101, 320), (64, 1, 8, 12, 128, 8190, 512), (64, 2, 12, 8, 128, 8100, 768), (60, 1, 16, 6, 136, 8130, 960),
         (64, 1, 16, 6, 128, 8191, 1024), (63, 1, 16, 1, 128, 8000, 1008), (13, 3, 32, 14, 72, 930, 416)]


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


@pytest.mark.parametrize("P,n,W,keep,width,vocab,lists", CASES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("ended", [False, True])
def test_many_lists(P, n, W, keep, width, vocab, lists, dtype, ended):
    from _gpu_helpers import note
    from test_gpu_search import beam_inputs, check_select
    note("beam_select of %d lists, keep=%d %s ended=%s" % (lists, keep, dtype, ended))
    assert W * P == lists and 4 * 64 < lists <= 1024 and lists * keep <= 6144        # the two-turn join's range
    x, s = beam_inputs(n, W, vocab, lists + keep)
    if not ended:
        check_select(x, s, P, width, keep, dtype)
        return
    done = np.random.default_rng(lists).random((n, W)) < 0.3
    x[1::4, 17] += 20                                      # beams that end now
    x[2] = -np.inf                                         # and one without candidates
    s[0, W - 1] = -np.inf
    check_select(x, s, P, width, keep, dtype, done, 17)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_wide_vocabulary_of_few_rows(dtype):
    """16 beams into 16 of 200000 tokens: some 22 parts a row."""
    from test_gpu_search import beam_inputs, check_select
    x, s = beam_inputs(1, 16, 200000, 16)
    check_select(x, s, 1, 200000, 16, dtype)


@pytest.mark.parametrize("P,n,W,keep,width,vocab,lists", CASES)
@pytest.mark.parametrize("score", [0.0, -1e25])            # -1e25: every logit gives one score
def test_equals_in_the_order_of_beams_and_tokens(P, n, W, keep, width, vocab, lists, score):
    """Equal beams, an ended one among them: each candidate of the first, then of the next."""
    from test_gpu_search import run_select, split
    g = torch.Generator().manual_seed(lists)
    row = torch.randint(-8, 0, (vocab,), generator=g).float()
    row[torch.randperm(vocab, generator=g)[:3]] = 1.0      # three equal ones above the rest, of other ranks mostly
    x = row.repeat(n * W, 1)
    done = np.zeros((n, W), bool)
    done[:, 1] = True
    s = np.full((n, W), score, np.float32)
    parents, tokens, _, _ = run_select(split(x, P, width, torch.bfloat16), s, vocab, keep, done, 3)
    ep, et = osr.select(x.numpy(), s, vocab, keep, done, 3)[:2]
    assert parents.tolist() == ep.tolist() and tokens.tolist() == et.tolist()
