"""kda_cache_fork of rows whose length ends inside a page that is not there."""
import pytest
import torch

import kimi_delta_attention_rule_gb300 as kda
from tests.test_cache_pages import Model, ints

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("tail", [-1, 40, 10**9])
def test_a_bad_last_page_is_flagged_and_skipped(tail):
    """Rows 0 and 2 are sound, row 1's last page is not in the pool: its forks take no
    page, keep an empty row and have nothing to copy; the others are as without them."""
    m = Model(40, 8, 4, 16)
    m.alloc([40, 20, 33])
    m.lens = [40, 20, 33, 0, 0, 0, 0, 0]
    m.table[1][1] = tail
    m.refs[3 + 1] = 0  # (the page that the entry named)
    table, lens, refs = m.device()
    ws = kda.cache_workspace(refs, 8)
    got = kda.kda_cache_fork(table, lens, refs, ints([0, 1, 2, 1]), ints([3, 4, 5, 6]), 16, workspace=ws)
    assert kda.kda_workspace_status(ws) == kda.KDA_ERR_DEVICE
    pairs = m.fork([0, -1, 2, -1], [3, 4, 5, 6])
    assert got.tolist() == pairs
    m.agrees(table, lens, refs)


def test_a_length_that_ends_with_a_page_reads_no_further_entry():
    m = Model(10, 3, 2, 16)
    m.alloc([32, 16])
    m.lens = [32, 16, 0]  # row 0's pages end with its table
    table, lens, refs = m.device()
    ws = kda.cache_workspace(refs, 3)
    assert kda.kda_cache_fork(table, lens, refs, ints([0]), ints([2]), 16, workspace=ws).tolist() == [[-1, -1]]
    assert kda.kda_workspace_status(ws) == kda.KDA_OK
    m.fork([0], [2])
    m.agrees(table, lens, refs)


def test_many_forks_with_bad_last_pages():
    """More forks than a block has threads: 1,500, of which every seventh's source is bad."""
    n, page = 1500, 16
    m = Model(4 * n, 2 * n, 2, page)
    m.alloc([20] * n)
    m.lens = [20] * n + [0] * n
    for r in range(0, n, 7):
        m.refs[m.table[r][1]] = 0
        m.table[r][1] = -1
    table, lens, refs = m.device()
    ws = kda.cache_workspace(refs, 2 * n)
    got = kda.kda_cache_fork(table, lens, refs, ints(list(range(n))), ints(list(range(n, 2 * n))), page, workspace=ws)
    assert kda.kda_workspace_status(ws) == kda.KDA_ERR_DEVICE
    pairs = m.fork([-1 if r % 7 == 0 else r for r in range(n)], list(range(n, 2 * n)))
    assert got.tolist() == pairs
    m.agrees(table, lens, refs)
