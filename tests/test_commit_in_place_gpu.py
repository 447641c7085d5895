"""Commits that write the new lengths over the old ones, of paths that take more pages than a warp has lanes."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from mla_speculative_decode_tree_gb300 import binding as B  # noqa: E402
from oracle import step as S  # noqa: E402


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def case(rng, batch, layers, page, kv4):
    """Requests of up to 9 tokens with 64 nodes each and paths of 33 to 64 of them."""
    P, q_len = rng.integers(0, 10, batch), 64
    want = -(-(P + q_len) // page)
    cols, pages = int(want.max()) + 70, int(want.sum()) + 3  # (columns behind a request's pages: any page's number)
    table = rng.integers(0, pages, (batch, cols))
    order, refs, k = rng.permutation(pages), np.zeros(pages, np.int64), 0
    loc, acc, num = [], np.full((batch, q_len), -1), np.zeros(batch, np.int64)
    for b in range(batch):
        table[b, :want[b]] = order[k:k + want[b]]
        k += int(want[b])
        refs[table[b, :-(-P[b] // page)]] = 1
        pos = P[b] + np.arange(q_len)
        loc += (table[b, pos // page] * page + pos % page).tolist()
        num[b] = (33, 64, 48, 63)[b % 4]
        acc[b, :num[b]] = np.sort(rng.choice(q_len, num[b], replace=False))
    shape = (layers, pages * page, 384 if kv4 else 576)
    pool = rng.integers(0, 256, shape).astype(np.uint8) if kv4 else rng.integers(-2 ** 15, 2 ** 15, shape).astype(np.int16)
    return P, np.arange(batch + 1) * q_len, np.array(loc), acc, num, table, refs, pool


def test_the_cases_tell_the_old_length_from_the_new_one():
    """Entries from the 33rd on found from the new length, as by a warp that reads it too late: other counts."""
    P, _, _, _, num, table, refs, _ = case(np.random.default_rng(0), 40, 1, 1, True)
    right, late = refs.copy(), refs.copy()
    for b in range(40):
        right[table[b, P[b]:P[b] + num[b]]] = 1
        late[table[b, P[b]:P[b] + 32]] = 1
        late[table[b, P[b] + num[b] + 32:P[b] + 2 * num[b]]] = 1
    assert (right != late).sum() > 100


@pytest.mark.gpu
@pytest.mark.parametrize("kv4", [False, True], ids=["bf16", "kv4"])
@pytest.mark.parametrize("batch,layers,page", [(1, 1, 1), (40, 2, 1), (40, 5, 1), (7, 9, 1), (300, 3, 1), (12, 4, 2)])
def test_in_place(kv4, batch, layers, page):
    rng = np.random.default_rng([batch, layers])
    P, qo, loc, acc, num, table, refs, pool = case(rng, batch, layers, page, kv4)
    ref = S.commit(pool, qo, loc, acc, num, batch, P, page, table, refs)
    assert not ref[3] and np.array_equal(ref[1], P + num)
    plan = B.mla_verify_plan(batch, 1, 64, 64, pool.shape[1], 1, flags=B.MLA_VERIFY_KV4 if kv4 else 0)
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    src, d_loc, d_acc, d_num, d_table = torch.from_numpy(pool).cuda(), i32(loc), i32(acc), i32(num), i32(table)
    for _ in range(8):
        dev, lens, r = src.clone(), i32(P), i32(refs)
        B.mla_verify_commit_drafts(plan, dev if kv4 else dev.view(torch.bfloat16), None, d_loc, d_acc, d_num, batch, lens, lens,
                                   page, d_table, r, ws)
        assert B.mla_verify_read_status(plan, ws) == 0
        assert np.array_equal(r.cpu().numpy(), ref[2]) and np.array_equal(lens.cpu().numpy(), ref[1])
        assert np.array_equal(dev.cpu().numpy(), ref[0])
