"""Free lists as mla_verify_list_free_pages writes them, -1 behind the pages, given whole and running out: the same as the
list cut off where its pages end."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from mla_speculative_decode_tree_gb300 import binding as B  # noqa: E402
from oracle import step as S  # noqa: E402
from test_slots_gpu import expect, run, tables  # noqa: E402
from test_step_gpu import fork_case, run_fork  # noqa: E402


def forks_with_tails(n, page, seed):
    """n forks of sources whose last pages are in part, and one free page more than they take."""
    for k in range(1000):
        pool, src, dst, table, lens, refs = fork_case(np.random.default_rng([seed, k]), 4, n, page, 2, False, 100, spare=1)
        if (lens[src] % page != 0).all():
            return pool, src, dst, table, lens, refs
    raise AssertionError("no such case")


@pytest.mark.parametrize("n,page", [(1, 2), (6, 8), (33, 5), (300, 16)])
@pytest.mark.parametrize("pages", ["none", "one", "half", "one less", "all", "one more"])
def test_forks_on_a_list_that_runs_out(n, page, pages):
    pool, src, dst, table, lens, refs = forks_with_tails(n, page, n)
    have = {"none": 0, "one": 1, "half": n // 2, "one less": n - 1, "all": n, "one more": n + 1}[pages]
    free, count = S.free_list(refs)
    refs[free[have:count]] = 1  # (somebody holds the others)
    free, count = S.free_list(refs)
    assert count == have and free.size == refs.size > count
    whole, cut = (run_fork(pool, src, dst, page, table, lens, refs, f, False) for f in (free, free[:count]))
    ref = S.fork(pool, src, dst, page, table, lens, refs, free)
    for w, c, r in zip(whole, cut, ref):
        assert np.array_equal(w, r) and np.array_equal(c, r)
    assert whole[4] == min(n, have) == (whole[3][free[:count]] == 1).sum()  # every page that it names is held now
    assert whole[5] == (B.MLA_VERIFY_DEV_NO_PAGE if have < n else 0)


def test_entries_that_are_passed_over_stay_free():
    """Fork 2 is left out (its destination is fork 1's) and fork 3 is from nowhere: four entries of the list are gone through,
    and its third page stays free."""
    pool, src, dst, table, lens, refs = forks_with_tails(5, 8, 0)
    free, count = S.free_list(refs)
    dst[2], src[3] = dst[1], -1
    got = run_fork(pool, src, dst, 8, table, lens, refs, free, False)
    for g, r in zip(got, S.fork(pool, src, dst, 8, table, lens, refs, free)):
        assert np.array_equal(g, r)
    assert got[4] == 4 and got[5] == B.MLA_VERIFY_DEV_BAD_ROW
    assert got[3][free[:4]].tolist() == [1, 1, 0, 1]


@pytest.mark.parametrize("n,page", [(3, 4), (70, 2), (600, 16)])
@pytest.mark.parametrize("pages", ["none", "one", "half", "one less", "all", "one more"])
def test_slot_maps_on_a_list_that_runs_out(n, page, pages):
    rng = np.random.default_rng(n)
    P, T = rng.integers(0, 5 * page, n), rng.integers(0, 3 * page, n)
    T[0] = 2 * page
    table, free, rows = tables(P, T, page, n, spare=1)
    want = free.size - 1
    have = {"none": 0, "one": 1, "half": want // 2, "one less": want - 1, "all": want, "one more": want + 1}[pages]
    padded = np.concatenate([free[:have], np.full(want + 9 - have, -1)])
    bits = B.MLA_VERIFY_DEV_NO_PAGE if have < want else 0
    whole, status = run(P, T, page, table, padded, rows)
    expect(whole, status, P, T, page, table, padded, rows, bits)
    assert whole["pages_used"][0] == min(want, have)
    cut, status = run(P, T, page, table, free[:have], rows)
    assert status == bits
    for k, x in whole.items():
        assert np.array_equal(x, cut[k]), k
