"""Slot maps of requests whose lengths add up to more than 2^31 - 1 (shared pages): the new tokens' rows are right."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from mla_speculative_decode_tree_gb300 import binding as B  # noqa: E402
from test_slots_gpu import run  # noqa: E402


@pytest.mark.parametrize("page", [4, 5])
def test_new_tokens_behind_sums_that_stopped(page):
    P, T = np.array([2 ** 30, 2 ** 30, 6, 9]), np.array([0, 0, 3, 4])
    table = np.full((4, 4), -1)
    table[2, :2], table[3, :3] = [7, 3], [8, 1, 2]
    free = [5, 6, 9]
    got, status = run(P, T, page, table, free, 100, kv_cap=50)
    assert status & B.MLA_VERIFY_DEV_CAPACITY
    pages = {2: [7, 3], 3: [8, 1, 2][:-(-9 // page)]}
    taken = 0
    rows = []
    for b in (2, 3):
        need = -(-(int(P[b]) + int(T[b])) // page)
        fresh = need - len(pages[b])
        pages[b] += free[taken:taken + fresh]
        taken += fresh
        rows += [pages[b][pos // page] * page + pos % page for pos in range(P[b], P[b] + T[b])]
        assert got["block_table"][b, :need].tolist() == pages[b]
    assert got["out_cache_loc"].tolist() == rows
    assert got["pages_used"][0] == taken
    assert got["qo_indptr"].tolist() == [0, 0, 0, 3, 7]
