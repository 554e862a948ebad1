"""Pins of the beam search oracle: hand-made cases, and properties that hold
whatever the code does."""
import numpy as np
import pytest

from oracle import search as osr


def test_select_by_hand():
    x = np.log(np.array([[0.5, 0.25, 0.25], [0.9, 0.05, 0.05]]))
    s = np.log(np.array([[0.5, 0.4]]))
    parents, tokens, after, _, bound, _ = osr.select(x, s, 3, 4)
    assert parents.tolist() == [[1, 0, 0, 0]] and tokens.tolist() == [[0, 0, 1, 2]]
    assert np.allclose(np.exp(after), [[0.36, 0.25, 0.125, 0.125]])
    assert 0 < bound < 1e-5


def test_select_done_and_missing():
    x = np.array([[0.0, -np.inf], [5.0, np.nan]])
    parents, tokens, after, done, _, _ = osr.select(x, np.array([[-1.0, -0.5]]), 2, 4, np.array([[False, True]]), 1)
    assert parents.tolist() == [[1, 0, -1, -1]] and tokens.tolist() == [[1, 0, -1, -1]]
    assert after.tolist() == [[-0.5, -1.0, -np.inf, -np.inf]] and done.tolist() == [[True, False, False, False]]


def test_fork_by_hand():
    """Rows of 10, 8 and 6 tokens in pages of 4; the first becomes two, the second goes on, the third ends."""
    table = [[0, 1, 2], [3, 4, -1], [5, 6, -1]]
    out, lens, copies, n, shared, used, free = osr.fork(table, [10, 8, 6], [0, 0, 1], None, [9, 9, 9, 9, 9, 9, 9, 7, 8], 7, 4, 9, 1)
    assert lens.tolist() == [10, 10, 8] and n == 1 and copies.tolist() == [[2, 5], [-1, -1], [-1, -1]]
    assert out.tolist() == [[0, 1, 2], [0, 1, 5], [3, 4, -1]]
    assert used == 6 and free.tolist() == [9, 9, 9, 9, 9, 9, 6, 7, 8] and shared.tolist() == [10, 10, 8]


def test_fork_shares_whole_pages():
    out, lens, _, n, shared, _, _ = osr.fork([[0, 1, 2]], [10], [0, 0], None, [3, 4], 0, 4, 5, 2)
    assert out.tolist() == [[0, 1, 2], [0, 1, 3]] and n == 1 and shared.tolist() == [8]
    out, _, _, n, shared, _, _ = osr.fork([[0, 1, 2]], [8], [0, 0], None, [3, 4], 0, 4, 5, 2)
    assert n == 0 and shared.tolist() == [8]


def test_fork_cut_into_a_page_that_another_row_has_full():
    out, _, copies, n, _, _, _ = osr.fork([[0, 1]], [8], [0, 0], [6, 8], [5], 0, 4, 6, 1)
    assert n == 1 and copies[0].tolist() == [1, 5] and out.tolist() == [[0, 5], [0, 1]]


def test_compact_by_hand():
    out, copies, n, used, free = osr.compact([[7, 2], [9, -1]], [8, 3], 1, 9, 4)
    assert used == 3 and n == 2 and copies.tolist() == [[7, 1], [9, 3], [-1, -1], [-1, -1]]
    assert out.tolist() == [[1, 2], [3, -1]] and free.tolist() == list(range(1, 10))


def test_format_by_hand():
    x = np.zeros((1, 32))
    x[0, :10] = [7.0, -6.0, 5.0, 5.5, 0.25, 0.75, 1.25, 2.5, 3.5, -0.1]
    codes, scales = osr.quantise(x)
    assert scales.tolist() == [[127]]
    assert codes[0, :10].tolist() == [7, 15, 6, 7, 0, 2, 2, 4, 6, 8]
    assert osr.quantise(x * 1.0001)[1].tolist() == [[128]]
    y = osr.values(codes, scales)
    assert y[0, :4].tolist() == [6, -6, 4, 6]


@pytest.mark.parametrize("scale", [1e-30, 1e-3, 1.0, 1e20])
def test_no_value_is_off_by_more_than_a_scale(scale):
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((200, 64)) * np.exp(rng.standard_normal((200, 1)) * 2) * scale)
    codes, scales = osr.quantise(x)
    unit = 2.0 ** (scales - 127.0)
    off = np.abs(osr.values(codes, scales) - x).reshape(200, 2, 32)
    assert (off <= unit[..., None]).all()
    assert (np.abs(x).reshape(200, 2, 32).max(-1) > 3.5 * unit).all()      # the next scale down would not do


def test_format_of_what_is_not_finite():
    x = np.zeros((1, 64))
    x[0, 3] = np.inf
    codes, scales = osr.quantise(x)
    assert scales.tolist() == [[255, 1]] and np.isnan(osr.values(codes, scales)[0, :32]).all()
    assert (osr.values(codes, scales)[0, 32:] == 0).all()
    k = np.arange(64.0).reshape(1, 64).repeat(16, 0)
    a, b = osr.rows_of(osr.page_of(k, -k), 64)
    assert (a == -b).all() and a[5, 0] == 0 and abs(a[0, 63] - 63) <= 16
