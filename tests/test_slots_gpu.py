"""Block tables and slot maps built on the GPU, against the request-by-request oracle (exact)."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from mla_speculative_decode_tree_gb300 import binding as B  # noqa: E402
from oracle import kv4  # noqa: E402


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def run(P, T, page, table, free, pool_rows, kv_cap=None, loc_cap=None, q_len=1, uniform=False, kv4_plan=False):
    n = len(P)
    plan = B.mla_verify_plan(n, 1, q_len, max(q_len, 1), pool_rows, 1, flags=B.MLA_VERIFY_KV4 if kv4_plan else 0)
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    Tn = [q_len] * n if uniform else T
    K, N = int(np.maximum(P, 0).sum()), int(np.maximum(Tn, 0).sum())
    out = dict(block_table=i32(table), pages_used=i32([-9]), kv_indptr=i32(np.full(n + 1, -9)),
               kv_indices=i32(np.full((K if kv_cap is None else kv_cap) + 3, -9)), qo_indptr=i32(np.full(n + 1, -9)),
               out_cache_loc=i32(np.full((N if loc_cap is None else loc_cap) + 3, -9)))
    kv, loc = (out[k][:-3] for k in ("kv_indices", "out_cache_loc"))
    B.mla_verify_build_slots(plan, i32(P), None if uniform else i32(T), n, page, out["block_table"], i32(free),
                             out["pages_used"], out["kv_indptr"], kv, out["qo_indptr"], loc, ws)
    status = B.mla_verify_read_status(plan, ws)
    got = {k: x.cpu().numpy() for k, x in out.items()}
    assert (got["kv_indices"][-3:] == -9).all() and (got["out_cache_loc"][-3:] == -9).all()
    got["kv_indices"], got["out_cache_loc"] = got["kv_indices"][:-3], got["out_cache_loc"][:-3]
    return got, status


def tables(P, T, page, seed, spare=2):
    rng = np.random.default_rng(seed)
    P, T = np.maximum(P, 0), np.maximum(T, 0)
    have, want = -(-P // page), -(-(P + T) // page)
    n_pages = int(want.sum()) + spare
    order = rng.permutation(n_pages)
    table = np.full((len(P), max(1, int(want.max()) + 1)), -1)
    k = 0
    for b, h in enumerate(have):
        table[b, :h] = order[k:k + h]
        k += int(h)
    return table, order[k:], n_pages * page


def expect(got, status, P, T, page, table, free, pool_rows, bits=0):
    ref, no_page, bad = kv4.build_slots(P, T, page, table, free, pool_rows)
    for k, x in ref.items():
        assert np.array_equal(got[k].reshape(-1), np.asarray(x, np.int64).reshape(-1)), k
    assert status == bits
    assert bool(bits & B.MLA_VERIFY_DEV_NO_PAGE) == no_page and bool(bits & B.MLA_VERIFY_DEV_BAD_ROW) == bad


@pytest.mark.parametrize("n,hi,t_hi,page", [
    (1, 1, 1, 1), (1, 0, 9, 1), (3, 40, 16, 1), (16, 3000, 16, 1), (5, 100, 40, 5), (33, 700, 9, 16), (7, 900, 3, 7),
    (256, 200, 4, 64), (257, 90, 2, 3), (1000, 30, 2, 1), (4096, 9, 2, 2), (2, 70000, 20000, 256)])
@pytest.mark.parametrize("seed", [0, 1])
def test_random_lengths(n, hi, t_hi, page, seed):
    rng = np.random.default_rng(seed + 10 * n)
    P, T = rng.integers(0, hi + 1, n), rng.integers(0, t_hi + 1, n)
    P[rng.random(n) < 0.1] = 0
    table, free, rows = tables(P, T, page, seed)
    got, status = run(P, T, page, table, free, rows, kv4_plan=bool(seed))
    expect(got, status, P, T, page, table, free, rows)


def test_uniform_drafts_from_the_plan():
    P = np.array([5, 0, 17])
    table, free, rows = tables(P, np.full(3, 9), 4, 0)
    got, status = run(P, None, 4, table, free, rows, q_len=9, uniform=True)
    expect(got, status, P, [9] * 3, 4, table, free, rows)


def test_all_requests_empty():
    got, status = run(np.zeros(4, int), np.zeros(4, int), 8, np.full((4, 2), -1), [], 64)
    assert status == 0 and got["pages_used"][0] == 0 and not got["kv_indptr"].any() and not got["qo_indptr"].any()


def test_negative_lengths_count_as_zero():
    P, T = np.array([-5, 6, 3]), np.array([2, -1, 4])
    table, free, rows = tables(P, T, 2, 0)
    got, status = run(P, T, 2, table, free, rows)
    expect(got, status, P, T, 2, table, free, rows)


def test_free_pages_used_up():
    P, T = np.array([4, 7, 0]), np.array([9, 2, 5])
    table, free, rows = tables(P, T, 4, 0)
    got, status = run(P, T, 4, table, free[:2], rows)
    expect(got, status, P, T, 4, table, free[:2], rows, B.MLA_VERIFY_DEV_NO_PAGE)
    got, status = run(P, T, 4, table, [], rows)
    expect(got, status, P, T, 4, table, [], rows, B.MLA_VERIFY_DEV_NO_PAGE)


def test_too_few_table_columns():
    P, T = np.array([9, 3]), np.array([8, 1])
    table, free, rows = tables(P, T, 4, 0)
    got, status = run(P, T, 4, table[:, :3], free, rows)
    expect(got, status, P, T, 4, table[:, :3], free, rows, B.MLA_VERIFY_DEV_NO_PAGE)


def test_pages_outside_the_pool():
    P, T = np.array([9, 3]), np.array([2, 2])
    table, free, rows = tables(P, T, 4, 0)
    table[0, 1] = rows // 4          # past the pool's end
    table[1, 0] = -3
    got, status = run(P, T, 4, table, free, rows)
    expect(got, status, P, T, 4, table, free, rows, B.MLA_VERIFY_DEV_BAD_ROW)
    table[0, 1] = 2 ** 31 - 1        # a row id past 32 bits
    got, status = run(P, T, 4, table, free, rows)
    expect(got, status, P, T, 4, table, free, rows, B.MLA_VERIFY_DEV_BAD_ROW)


@pytest.mark.parametrize("kv_cap,loc_cap", [(10, None), (None, 3), (0, 0)])
def test_short_arrays(kv_cap, loc_cap):
    P, T = np.array([9, 8]), np.array([4, 5])
    table, free, rows = tables(P, T, 4, 0)
    got, status = run(P, T, 4, table, free, rows, kv_cap, loc_cap)
    ref, _, _ = kv4.build_slots(P, T, 4, table, free, rows)
    assert status == B.MLA_VERIFY_DEV_CAPACITY
    for k in ("kv_indices", "out_cache_loc"):
        assert got[k].tolist() == ref[k][:got[k].size]
    assert got["kv_indptr"].tolist() == ref["kv_indptr"]


def test_sums_stop_at_the_largest_int32():
    big = 2 ** 30
    got, status = run(np.array([big, big, big, 5]), np.array([0, 0, 0, 0]), big, np.zeros((4, 2), int), [], 2 ** 31 - 1,
                      kv_cap=100)
    assert status & B.MLA_VERIFY_DEV_CAPACITY
    assert got["kv_indptr"].tolist() == [0, big, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1]
    assert got["kv_indices"].tolist() == list(range(100))


def test_a_second_build_on_the_same_arrays_changes_nothing():
    P, T = np.array([5, 0, 300]), np.array([4, 2, 3])
    table, free, rows = tables(P, T, 16, 3)
    got, _ = run(P, T, 16, table, free, rows)
    again, status = run(P, T, 16, got["block_table"], free, rows)
    assert status == 0
    for k, x in got.items():
        assert np.array_equal(x, again[k]), k
