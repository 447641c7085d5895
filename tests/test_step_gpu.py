"""Draft verification, commits, free lists, forks and releases on the GPU against the whole-number oracles (exact)."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from mla_speculative_decode_tree_gb300 import binding as B  # noqa: E402
from oracle import step as S  # noqa: E402


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def plan_ws(batch=1, q_len=1, rows=1, flags=0):
    plan = B.mla_verify_plan(batch, 1, q_len, max(q_len, 1), rows, 1, flags=flags)
    return plan, torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")


# ---- verification -------------------------------------------------------------

def probabilities(rng, n, vocab, kind="soft"):
    z = rng.standard_normal((n, vocab)) * (2.5 if kind == "soft" else 0.0 if kind == "flat" else 12.0)
    p = np.exp(z - z.max(1, keepdims=True))
    return (p / p.sum(1, keepdims=True)).astype(np.float32)


def trees(rng, counts):
    return np.concatenate([[-1] + [int(rng.integers(0, i)) for i in range(1, t)] if t else [] for t in counts]
                          + [[]]).astype(np.int64)


class Drafts:
    def __init__(self, counts, vocab, drawn, seed=0, q_len=None, near=0.7, kind="soft"):
        rng = np.random.default_rng(seed)
        self.counts, self.vocab, self.q_len = counts, vocab, q_len or max(max(counts), 1)
        n = sum(counts)
        self.rows = max(n, 1)
        self.qo = np.concatenate([[0], np.cumsum(counts)])
        self.target = probabilities(rng, self.rows, vocab, kind)
        d = np.log(np.maximum(self.target, 1e-30)) + near * rng.standard_normal(self.target.shape)
        d = np.exp(d - d.max(1, keepdims=True))
        self.draft = (d / d.sum(1, keepdims=True)).astype(np.float32) if drawn else None
        self.parents = trees(rng, counts)
        self.tokens = np.zeros(self.rows, np.int64)
        for b, t in enumerate(counts):
            for i in range(1, t):
                row = self.qo[b] + self.parents[self.qo[b] + i]
                p = (self.draft if drawn else self.target)[row].astype(np.float64)
                self.tokens[self.qo[b] + i] = rng.choice(vocab, p=p / p.sum())
        self.u = rng.integers(0, 1 << 24, self.rows).astype(np.float32) / np.float32(1 << 24)
        self.u_next = rng.integers(0, 1 << 24, len(counts)).astype(np.float32) / np.float32(1 << 24)

    def run(self, target=None, draft=None, uniform=False):
        batch = len(self.counts)
        plan, ws = plan_ws(batch, self.q_len)
        out = [torch.full(s, -9, dtype=torch.int32, device="cuda") for s in ((batch, self.q_len), (batch,), (batch,))]
        t = torch.from_numpy(self.target).cuda() if target is None else target
        d = (None if self.draft is None else torch.from_numpy(self.draft).cuda()) if draft is None else draft
        B.mla_verify_accept_drafts(plan, t, d, i32(self.tokens), i32(self.parents if self.parents.size else [-1]),
                                   None if uniform else i32(self.qo), torch.from_numpy(self.u).cuda(),
                                   torch.from_numpy(self.u_next).cuda(), batch, *out, ws)
        torch.cuda.synchronize()
        assert B.mla_verify_read_status(plan, ws) == 0
        return [x.cpu().numpy() for x in out]

    def oracle(self):
        return S.accept(self.target, self.draft, self.tokens, self.parents, self.qo, self.u, self.u_next, len(self.counts),
                        self.q_len)

    def check(self, **kw):
        got, ref = self.run(**kw), self.oracle()
        for g, r in zip(got, ref):
            assert np.array_equal(g, r), (g, r)
        return got


@pytest.mark.parametrize("drawn", [True, False], ids=["drawn", "proposed"])
@pytest.mark.parametrize("vocab", [1, 2, 3, 5, 127, 1000, 4099, 33001])
def test_vocabularies(drawn, vocab):
    Drafts([4, 1, 7, 0, 3], vocab, drawn, seed=vocab).check()


@pytest.mark.parametrize("drawn", [True, False], ids=["drawn", "proposed"])
@pytest.mark.parametrize("seed", range(10))
def test_random_trees(drawn, seed):
    rng = np.random.default_rng([seed, 3])
    counts = [int(rng.integers(0, 2 + 6 * (seed % 3))) for _ in range(int(rng.integers(1, 20)))] + [2]
    Drafts(counts, int(rng.integers(2, 700)), drawn, seed=seed, near=float(rng.choice([0.0, 0.7, 3.0])),
           kind=str(rng.choice(["soft", "flat", "sharp"]))).check()


@pytest.mark.parametrize("drawn", [True, False], ids=["drawn", "proposed"])
def test_many_children_of_one_node(drawn):
    """The root proposes 63 tokens, some of them twice; nearly all are rejected."""
    d = Drafts([64, 64], 50, drawn, seed=1, near=4.0)
    d.parents = np.concatenate([[-1] + [0] * 63] * 2)
    d.tokens = np.random.default_rng(2).integers(0, 50, 128)
    d.u[:] = np.float32(1 - 2.0 ** -24)
    d.check()
    d.u[:] = 0
    d.check()


def test_links_and_tokens_that_lead_nowhere():
    d = Drafts([8, 8], 40, False, seed=3)
    d.parents[1:8] = [-1, 2, 7, 1, -5, 100, 0]  # roots, loops, children of what is not reached
    d.tokens[9:16] = [-1, 40, 2 ** 31 - 1, 5, 6, -2 ** 31, 7]
    d.check()


def test_odd_strides_and_one_row_more():
    """Rows inside a wider tensor, target and draft at different offsets from a 16-byte boundary."""
    d = Drafts([5, 6], 1001, True, seed=4)
    t = torch.zeros((11, 1013), device="cuda")
    q = torch.zeros((11, 1031), device="cuda")
    t[:, 1:1002], q[:, 3:1004] = torch.from_numpy(d.target).cuda(), torch.from_numpy(d.draft).cuda()
    d.check(target=t[:, 1:1002], draft=q[:, 3:1004])


def test_uniform_counts_without_qo_indptr():
    Drafts([6, 6, 6], 300, True, seed=5).check(uniform=True)


def test_values_outside_the_ranges():
    """NaN, negative and large probabilities and random numbers count as the nearest that exist."""
    d = Drafts([5, 5, 3], 64, True, seed=6)
    d.target[0, :3], d.target[3, 5], d.draft[1, 7], d.draft[6, :4] = [np.nan, -1, 3], 2.5, np.inf, np.nan
    d.u[:6] = [np.nan, -1, 1, 7, 0.5, np.inf]
    d.u_next[:] = [1.0, -3.0, np.nan]
    d.check()


def test_rows_of_zeros_have_no_next_token():
    d = Drafts([2, 1], 30, False, seed=7)
    d.target[:] = 0
    assert d.check()[2].tolist() == [-1, -1]


def test_a_large_vocabulary_and_tokens_at_its_ends():
    """One hot rows at the first and the last token, then a soft one of 262,147."""
    d = Drafts([3, 3], 262147, False, seed=8)
    got = d.check()
    d.target[:] = 0
    d.target[:3, 0], d.target[3:, -1] = 1, 1
    d.tokens[:] = [0, 0, 1, 0, 262146, 5]
    got = d.check()
    assert got[2].tolist() == [0, 262146]


@pytest.mark.parametrize("drawn", [True, False], ids=["drawn", "proposed"])
@pytest.mark.parametrize("vocab", [150001, 262147])
def test_many_rejections_in_a_large_vocabulary(drawn, vocab):
    """Ten children of one node: a target that is nearly flat with a draft that is not (nearly all entries have p > q, more
    than are kept), and a draft close to the target."""
    d = Drafts([11, 11], vocab, drawn, seed=9, near=0.3)
    d.parents = np.concatenate([[-1] + [0] * 10] * 2)
    d.target[0] = probabilities(np.random.default_rng(1), 1, vocab, "flat")
    if drawn:
        d.draft[0] = probabilities(np.random.default_rng(2), 1, vocab, "sharp")
        d.tokens[1:11] = np.argsort(d.draft[0])[-10:]
    d.u[:] = np.float32(1 - 2.0 ** -24)
    d.check()


def test_weights_at_their_boundaries():
    """Values around 2^-15, 2^-19 and 2^-39, halves of a weight's step, 1 and what is below the smallest normal float."""
    base = [2.0 ** -15, 2.0 ** -16, 2.0 ** -19, 2.0 ** -38, 2.0 ** -39, 3 * 2.0 ** -39, 5 * 2.0 ** -39, 2.0 ** -40, 1e-40, 0.0,
            0.25, 0.5, 1.0, 2.0 ** -14, 1 / 3, (2 ** 23 - 0.5) * 2.0 ** -38, (2 ** 22 + 0.5) * 2.0 ** -38]
    f = np.array(base, np.float32)
    f = np.unique(np.concatenate([f, np.nextafter(f, np.float32(2)), np.nextafter(f, np.float32(0))]))
    for seed in range(8):
        rng = np.random.default_rng(seed)
        d = Drafts([5, 4, 6], 2 * f.size, True, seed=seed)
        d.parents = np.concatenate([[-1] + [0] * 4, [-1] + [0] * 3, [-1] + [0] * 5])
        d.target[:], d.draft[:] = rng.choice(f, d.target.shape), rng.choice(f, d.target.shape)
        d.u[:] = np.float32(1 - 2.0 ** -24)
        d.check()


def test_distribution_of_the_first_new_token():
    """20,000 requests of one root and two drawn children: counts of the token behind the root within five standard
    deviations of the target's."""
    rng = np.random.default_rng(9)
    n, V = 1000, 6
    p, q = probabilities(rng, 1, V)[0], probabilities(rng, 1, V)[0]
    seen = np.zeros(V)
    plan, ws = plan_ws(n, 3)
    t = torch.from_numpy(np.tile(p, (3 * n, 1))).cuda()
    dq = torch.from_numpy(np.tile(q, (3 * n, 1))).cuda()
    for _ in range(20):
        tokens = rng.choice(V, 3 * n, p=q.astype(np.float64) / q.astype(np.float64).sum())
        out = [torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((n, 3), (n,), (n,))]
        B.mla_verify_accept_drafts(plan, t, dq, i32(tokens), i32(np.tile([-1, 0, 0], n)), None,
                                   torch.rand(3 * n, device="cuda"), torch.rand(n, device="cuda"), n, *out, ws)
        acc, num, nxt = (x.cpu().numpy() for x in out)
        first = np.where(num > 1, tokens.reshape(n, 3)[np.arange(n), acc[:, 1]], nxt)
        seen += np.bincount(first, minlength=V)
    total = seen.sum()
    assert np.all(np.abs(seen - total * p) <= 5 * np.sqrt(total * p * (1 - p)) + 1)


def test_on_another_stream():
    """Every call on a stream that is not the current one, after work that it has to wait for."""
    d = Drafts([5, 4], 1000, True, seed=12)
    plan, ws = plan_ws(2, 5)
    st = torch.cuda.Stream()
    src, draft = torch.from_numpy(d.target).cuda(), torch.from_numpy(d.draft).cuda()
    out = [torch.full(s, -9, dtype=torch.int32, device="cuda") for s in ((2, 5), (2,), (2,))]
    tok, par, qo, u, un = i32(d.tokens), i32(d.parents), i32(d.qo), torch.from_numpy(d.u).cuda(), torch.from_numpy(d.u_next).cuda()
    target, refs, free, count = torch.zeros_like(src), i32(np.ones(5000)), i32(np.zeros(5000)), i32([0])
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(2_000_000)
        target.copy_(src)
        refs[::3] = 0
    B.mla_verify_accept_drafts(plan, target, draft, tok, par, qo, u, un, 2, *out, ws, stream=st)
    B.mla_verify_list_free_pages(plan, refs, free, count, stream=st)
    st.synchronize()
    for g, r in zip(out, d.oracle()):
        assert np.array_equal(g.cpu().numpy(), r)
    assert int(count) == 1667 and free[:3].tolist() == [0, 3, 6]


def test_accept_replays_with_new_contents():
    d = [Drafts([4, 0, 6], 500, True, seed=s) for s in (10, 11)]
    d[1].counts, big = [4, 0, 6], d[0]
    plan, ws = plan_ws(3, 6)
    t, q = torch.from_numpy(big.target).cuda(), torch.from_numpy(big.draft).cuda()
    tok, par, qo = i32(big.tokens), i32(big.parents), i32(big.qo)
    u, un = torch.from_numpy(big.u).cuda(), torch.from_numpy(big.u_next).cuda()
    out = [torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((3, 6), (3,), (3,))]
    args = (plan, t, q, tok, par, qo, u, un, 3, *out, ws)
    B.mla_verify_accept_drafts(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.mla_verify_accept_drafts(*args)
    for x in d[::-1]:
        for dst, src in ((t, x.target), (q, x.draft), (u, x.u), (un, x.u_next)):
            dst.copy_(torch.from_numpy(src))
        tok.copy_(i32(x.tokens))
        par.copy_(i32(x.parents))
        graph.replay()
        torch.cuda.synchronize()
        for g, r in zip(out, x.oracle()):
            assert np.array_equal(g.cpu().numpy(), r)


# ---- commit -----------------------------------------------------------------

def commit_case(rng, batch, q_len, page, layers, kv4, max_len):
    P, T = rng.integers(0, max_len, batch), rng.integers(0, q_len + 1, batch)
    have, want = -(-P // page), -(-(P + T) // page)
    cols, n_pages = int(want.max()) + 2, int(want.sum()) + 3
    order, table = rng.permutation(n_pages), np.full((batch, cols), -1)
    loc, refs, k, qo = [], np.zeros(n_pages, np.int64), 0, np.concatenate([[0], np.cumsum(T)])
    acc, num = np.full((batch, q_len), -1), np.zeros(batch, np.int64)
    for b in range(batch):
        table[b, :want[b]] = order[k:k + want[b]]
        k += int(want[b])
        refs[table[b, :have[b]]] = 1
        pos = P[b] + np.arange(T[b])
        loc += (table[b, pos // page] * page + pos % page).tolist()
        if T[b]:
            path = np.sort(rng.choice(T[b], int(rng.integers(1, T[b] + 1)), replace=False))
            acc[b, :path.size], num[b] = path, path.size
    rows = n_pages * page
    pool = (rng.integers(0, 256, (layers, rows, 384)).astype(np.uint8) if kv4 else
            rng.integers(-2 ** 15, 2 ** 15, (layers, rows, 576)).astype(np.int16))
    return P, T, qo, np.array(loc + [0] * (batch * q_len - len(loc))), acc, num, table, refs, pool


def run_commit(P, qo, loc, acc, num, table, refs, pool, page, kv4, q_len, in_place=False, pages=True, uniform=False):
    plan, ws = plan_ws(len(P), q_len, pool.shape[1], B.MLA_VERIFY_KV4 if kv4 else 0)
    dev = torch.from_numpy(pool).cuda()
    view = dev if kv4 else dev.view(torch.bfloat16)
    lens, r = i32(P), i32(refs)
    new = lens if in_place else i32(np.full(len(P), -9))
    B.mla_verify_commit_drafts(plan, view, None if uniform else i32(qo), i32(loc), i32(acc), i32(num), len(P), lens, new, page,
                               i32(table) if pages else None, r if pages else None, ws)
    status = B.mla_verify_read_status(plan, ws)
    return dev.cpu().numpy(), new.cpu().numpy(), r.cpu().numpy(), status


@pytest.mark.parametrize("kv4", [False, True], ids=["bf16", "kv4"])
@pytest.mark.parametrize("batch,q_len,page,layers", [(1, 1, 1, 1), (3, 5, 1, 2), (7, 16, 16, 5), (40, 64, 5, 3), (2, 33, 64, 9),
                                                     (300, 4, 16, 1)])
def test_commit(kv4, batch, q_len, page, layers):
    rng = np.random.default_rng([batch, page])
    P, T, qo, loc, acc, num, table, refs, pool = commit_case(rng, batch, q_len, page, layers, kv4, 200)
    ref = S.commit(pool, qo, loc, acc, num, batch, P, page, table, refs)
    got = run_commit(P, qo, loc, acc, num, table, refs, pool, page, kv4, q_len, in_place=batch % 2 == 1)
    assert np.array_equal(got[0], ref[0]) and np.array_equal(got[1], ref[1]) and np.array_equal(got[2], ref[2])
    assert got[3] == 0 and not ref[3]
    got = run_commit(P, qo, loc, acc, num, table, refs, pool, page, kv4, q_len, pages=False)
    assert np.array_equal(got[0], ref[0]) and np.array_equal(got[2], refs)


def test_commit_of_paths_and_rows_that_are_wrong():
    rng = np.random.default_rng(5)
    P, T, qo, loc, acc, num, table, refs, pool = commit_case(rng, 6, 8, 4, 2, False, 50)
    T[:], qo = 8, np.arange(7) * 8
    loc = rng.permutation(pool.shape[1])[:48]
    acc[:] = np.arange(8)
    num[:] = [9, -1, 8, 3, 5, 4]
    acc[2] = [0, 2, 2, 3, 4, 5, 6, 7]      # not ascending
    acc[3] = [1, 5, 8, -1, -1, -1, -1, -1]  # outside the tree
    acc[4] = [-1, 1, 2, 3, 4, 5, 6, 7]
    acc[5] = [1, 3, 5, 7, -1, -1, -1, -1]
    loc[40 + 3], loc[40 + 1] = -1, pool.shape[1]
    table[5, :] = -7
    ref = S.commit(pool, qo, loc, acc, num, 6, P, 4, table, refs)
    got = run_commit(P, qo, loc, acc, num, table, refs, pool, 4, False, 8)
    assert ref[3] and got[3] == B.MLA_VERIFY_DEV_BAD_ROW
    for g, r in zip(got[:3], ref[:3]):
        assert np.array_equal(g, r)


# ---- pages ------------------------------------------------------------------

@pytest.mark.parametrize("n", [1, 2, 31, 33, 127, 1000, 8191, 8192, 8193, 40001, 1_000_003, 5_000_001])
@pytest.mark.parametrize("share", [0.0, 0.03, 0.5, 1.0])
def test_free_list(n, share):
    rng = np.random.default_rng(n)
    refs = np.where(rng.random(n) < share, 0, rng.integers(-2, 4, n))
    plan, _ = plan_ws()
    free, count = i32(np.full(n + 1, -9)), i32([-9])
    B.mla_verify_list_free_pages(plan, i32(refs), free[:n], count)
    where = np.flatnonzero(refs == 0)
    got = free.cpu().numpy()
    assert int(count) == where.size and got[n] == -9
    assert np.array_equal(got[:where.size], where) and (got[where.size:n] == -1).all()


def test_free_list_of_an_odd_address_and_of_nothing():
    refs = i32([5, 0, 1, 0, 0, 2, 0, 7])
    plan, _ = plan_ws()
    free, count = i32([-9] * 7), i32([-9])
    B.mla_verify_list_free_pages(plan, refs[1:], free, count)
    assert free.tolist() == [0, 2, 3, 5, -1, -1, -1] and int(count) == 4
    B.mla_verify_list_free_pages(plan, refs[:0], free, count)
    assert int(count) == 0


def fork_case(rng, sources, n, page, layers, kv4, max_len, spare=8):
    P = rng.integers(0, max_len, sources)
    held = -(-P // page)
    requests, cols, n_pages = sources + n + 2, int(held.max()) + 1, int(held.sum()) + n + spare
    order, table = rng.permutation(n_pages), rng.integers(-5, n_pages, (requests, cols))
    lens, refs, k = np.zeros(requests, np.int64), np.zeros(n_pages, np.int64), 0
    place = rng.permutation(requests)
    for i in range(sources):
        table[place[i], :held[i]] = order[k:k + held[i]]
        refs[order[k:k + held[i]]] = 1
        lens[place[i]] = P[i]
        k += int(held[i])
    pool = (rng.integers(0, 256, (layers, n_pages * page, 384)).astype(np.uint8) if kv4 else
            rng.integers(-2 ** 15, 2 ** 15, (layers, n_pages * page, 576)).astype(np.int16))
    return pool, place[rng.integers(0, sources, n)], place[sources:sources + n], table, lens, refs


def run_fork(pool, src, dst, page, table, lens, refs, free, kv4):
    plan, ws = plan_ws(1, 1, pool.shape[1], B.MLA_VERIFY_KV4 if kv4 else 0)
    dev = torch.from_numpy(pool).cuda()
    t, l, r, used = i32(table), i32(lens), i32(refs), i32([-9])
    B.mla_verify_fork(plan, dev if kv4 else dev.view(torch.bfloat16), i32(src), i32(dst), page, t, l, r, i32(free), used, ws)
    return (dev.cpu().numpy(), t.cpu().numpy(), l.cpu().numpy(), r.cpu().numpy(), int(used), B.mla_verify_read_status(plan, ws))


@pytest.mark.parametrize("kv4", [False, True], ids=["bf16", "kv4"])
@pytest.mark.parametrize("sources,n,page,layers,max_len", [(1, 1, 1, 1, 9), (1, 4, 16, 2, 200), (5, 30, 5, 3, 60), (3, 9, 64, 5, 4000),
                                                           (2, 3, 256, 2, 700), (4, 300, 2, 1, 30)])
def test_fork_and_release(kv4, sources, n, page, layers, max_len):
    rng = np.random.default_rng([n, page])
    pool, src, dst, table, lens, refs = fork_case(rng, sources, n, page, layers, kv4, max_len)
    free, count = S.free_list(refs)
    ref = S.fork(pool, src, dst, page, table, lens, refs, free)
    got = run_fork(pool, src, dst, page, table, lens, refs, free, kv4)
    for g, r in zip(got, ref):
        assert np.array_equal(g, r)
    assert got[5] == 0
    which = rng.permutation(np.concatenate([dst, dst[:2]]))
    lens2, refs2, st = S.release(which, page, got[1], got[2], got[3])
    plan, ws = plan_ws()
    l, r = i32(got[2]), i32(got[3])
    B.mla_verify_release(plan, i32(which), page, i32(got[1]), l, r, ws)
    assert np.array_equal(l.cpu().numpy(), lens2) and np.array_equal(r.cpu().numpy(), refs2)
    assert B.mla_verify_read_status(plan, ws) == st == 0
    assert np.array_equal(refs2, refs) or (lens[dst] > 0).any()


def test_fork_without_pages_and_with_wrong_requests():
    rng = np.random.default_rng(3)
    pool, src, dst, table, lens, refs = fork_case(rng, 3, 6, 8, 2, False, 100, spare=0)
    lens[src] = lens[src] // 8 * 8 + 3  # (every last page is in part)
    table[src, :] = np.where(table[src, :] < 0, 0, table[src, :])
    free, _ = S.free_list(refs)
    ref = S.fork(pool, src, dst, 8, table, lens, refs, free[:2])
    got = run_fork(pool, src, dst, 8, table, lens, refs, free[:2], False)
    assert got[5] == ref[5] == B.MLA_VERIFY_DEV_NO_PAGE
    for g, r in zip(got, ref):
        assert np.array_equal(g, r)
    src2, dst2 = src.copy(), dst.copy()
    src2[0], dst2[1], dst2[3] = -1, 10 ** 6, dst2[2]  # not there; not there; the same request twice
    dst2[4] = src2[5]                                  # a source of the same call
    ref = S.fork(pool, src2, dst2, 8, table, lens, refs, free)
    got = run_fork(pool, src2, dst2, 8, table, lens, refs, free, False)
    assert got[5] == ref[5] == B.MLA_VERIFY_DEV_BAD_ROW
    for g, r in zip(got, ref):
        assert np.array_equal(g, r)


def test_release_of_what_is_not_held():
    table, lens, refs = np.array([[0, 1, 9], [2, -1, 3], [4, 4, 4]]), np.array([5, 6, 0]), np.array([1, 0, 2, 1, 5])
    which = np.array([0, 3, 1, 0, -1, 2])
    lens2, refs2, st = S.release(which, 2, table, lens, refs)
    plan, ws = plan_ws()
    l, r = i32(lens), i32(refs)
    B.mla_verify_release(plan, i32(which), 2, i32(table), l, r, ws)
    assert np.array_equal(l.cpu().numpy(), lens2) and np.array_equal(r.cpu().numpy(), refs2)
    assert B.mla_verify_read_status(plan, ws) == st == B.MLA_VERIFY_DEV_BAD_ROW


def test_page_calls_replay_in_a_graph():
    """Free list, fork, release captured together: each replay does the same again."""
    rng = np.random.default_rng(4)
    pool, src, dst, table, lens, refs = fork_case(rng, 2, 5, 16, 2, False, 300)
    plan, ws = plan_ws(1, 1, pool.shape[1])
    dev, t, l, r = torch.from_numpy(pool).cuda(), i32(table), i32(lens), i32(refs)
    free, count, used, s, d = i32(np.zeros(refs.size)), i32([0]), i32([0]), i32(src), i32(dst)

    def calls():
        B.mla_verify_list_free_pages(plan, r, free, count)
        B.mla_verify_fork(plan, dev.view(torch.bfloat16), s, d, 16, t, l, r, free, used, ws)
        B.mla_verify_release(plan, d, 16, t, l, r, ws)

    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    ref = S.fork(pool, src, dst, 16, table, lens, refs, S.free_list(refs)[0])
    assert np.array_equal(dev.cpu().numpy(), ref[0]) and np.array_equal(t.cpu().numpy(), ref[1])
    assert np.array_equal(r.cpu().numpy(), refs) and np.array_equal(l.cpu().numpy(), lens) and int(used) == ref[4]
    assert B.mla_verify_read_status(plan, ws) == 0
