"""kv_fork once pages have run out: kv_plan and kv_fork then leave *used above
the number of free-list entries, the excess standing for table entries of -1,
which no page comes back for.  Whatever rows go on or end afterwards, every
page of the pool is held by a row or on the free list, once."""
import numpy as np
import pytest
import torch

from oracle import search as osr


def whole(table, lengths, free, used, page, pool):
    """Every page of the pool is a row's or free, and no page both."""
    held = {int(e) for row, n in zip(table, lengths) for e in row[:-(-int(n) // page)] if e >= 0}
    left = [int(e) for e in free[min(int(used), len(free)):]]
    assert sorted(list(held) + left) == sorted(pool), (held, left)


# (parents of each step in turn), from two rows of 20 and 25 tokens and one free page
RUNS = [([0, 0, 0, 0, 1], []), ([0, 0, 0, 0, 1], [4, 0]), ([0, 0, 0, 0, 1], [0, 1, 2, 3, 4], []), ([0] * 9, [8], [0, 0], []),
        ([0, 0, 1, 1, 1], [0], [0], [0, 0, 0], [])]
POOL = [0, 1, 2, 3, 5]


def run_all(steps, fork):
    table, lengths, free, used = [[0, 1], [2, 3]], [20, 25], list(POOL), 4
    short = False
    for parents in steps:
        table, lengths, _, _, _, used, free = fork(table, lengths, parents, free, used)
        used = int(used)
        short = short or used > len(POOL)
        whole(table, lengths, free, used, 16, POOL)
    assert short
    if not len(steps[-1]):
        assert used == 0 and sorted(free) == POOL


@pytest.mark.parametrize("steps", RUNS)
def test_oracle_loses_no_page(steps):
    run_all(steps, lambda table, lengths, parents, free, used: osr.fork(table, lengths, parents, None, free, used, 16, 10, 1, 2))


@pytest.mark.gpu
@pytest.mark.parametrize("pages", [10, 9000])              # one workgroup with its sets in LDS, and many
@pytest.mark.parametrize("steps", RUNS)
def test_no_page_is_lost(steps, pages):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from test_gpu_search import check_fork

    def fork(table, lengths, parents, free, used):
        got, _ = check_fork(list(map(list, table)), list(map(int, lengths)), parents, None, list(map(int, free)), used, 16, pages, 1)
        table, lengths, copies, n, _, used, free = got
        return table.reshape(-1, 2), lengths, copies, n, None, used.item(), free

    run_all(steps, fork)


@pytest.mark.gpu
@pytest.mark.parametrize("pages", [6, 9000])
def test_no_page_is_lost_where_planning_ran_out(pages):
    """kv_plan asks for three pages of which there is one; then one of the rows ends, then the other."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from ring_collectives_amd import attention as A
    from test_gpu_attention import i32
    from test_gpu_search import check_fork
    table, lengths, free, used = i32([[0, 1, -1, -1], [2, 3, -1, -1]]), i32([20, 25]), i32(POOL), i32([4])
    after, cu, pos = i32([0, 0]), i32([0, 0, 0]), i32([0] * 60)
    slots, used_after = torch.zeros(60, dtype=torch.int64, device="cuda"), i32([0])
    A.kv_plan(lengths, i32([30, 29]), free, used, table, after, cu, pos, slots, used_after, page_size=16)
    assert used_after.item() > len(POOL)
    whole(table.tolist(), after.tolist(), free.tolist(), used_after.item(), 16, POOL)
    got, _ = check_fork(table.tolist(), after.tolist(), [1], None, free.tolist(), used_after.item(), 16, pages, 1)
    table, lengths, _, _, _, used, free = got
    whole(table.reshape(1, 4), lengths, free, used.item(), 16, POOL)
    got, _ = check_fork(table.reshape(1, 4).tolist(), lengths.tolist(), [], None, free.tolist(), used.item(), 16, pages, 1)
    assert got[5].item() == 0 and sorted(got[6].tolist()) == POOL
