"""Attention over shared prefixes on the GPU against the definition in 64 bits, both kernels."""

import time

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from mla_speculative_decode_tree_gb300 import binding as B  # noqa: E402
from parity_util import bf16_to_f64, compare  # noqa: E402
from shared_util import SCALE, Case, i32  # noqa: E402

SIMT = B.MLA_VERIFY_FORCE_SIMT
SHAPES = [
    # heads, groups [(S, [(P, T), ...]), ...]
    (1, [(1, [(0, 1)])]),                              # one shared key and the draft itself
    (1, [(0, [(0, 1)])]),                              # nothing but the draft
    (16, [(64, [(0, 1)])]),                            # one whole tile
    (16, [(65, [(0, 2), (63, 1)])]),                   # a key into the second tile; own keys that fill one
    (8, [(31, [(1, 1)] * 3)]),                         # all of a tile's first half
    (8, [(33, [(31, 1), (32, 1), (33, 1)])]),          # around the half that each CTA takes
    (64, [(127, [(5, 2), (0, 3)]), (0, [(300, 9)])]),  # a group without a prefix
    (13, [(700, [(40, 3), (0, 0), (333, 5)]), (12, []), (9, [(7, 1)])]),  # no tokens, no requests
    (128, [(500, [(20, 3)] * 2)]),                     # 384 rows and more
    (5, [(1000, [(130, 7)] * 9)]),                     # row groups that end inside a request
    (8, [(3000, [(1 + 37 * i % 200, 1) for i in range(64)])]),  # decode
    (32, [(900 * g, [(11 * g, g % 4)] * 3) for g in range(8)]),  # several prompts
    (3, [(100, [(700, 64)])]),                         # the longest draft tree
    (64, [(9000, [(64, 1)] * 4)]),                     # many tiles, the rings wrap
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "h%d_%d" % (s[0], len(s[1])))
@pytest.mark.parametrize("flags", [0, SIMT], ids=["tc", "simt"])
def test_shapes(shape, flags):
    Case(shape[1], shape[0], seed=shape[0]).check(flags, str(shape))


@pytest.mark.parametrize("seed", range(24))
def test_random_shapes(seed):
    rng = np.random.default_rng([seed, 17])
    groups = []
    for _ in range(int(rng.integers(1, 7))):
        s = int(rng.integers(0, 2 ** int(rng.integers(1, 12))))
        groups.append((s, [(int(rng.integers(0, 2 ** int(rng.integers(1, 9)))), int(rng.integers(0, 6)))
                           for _ in range(int(rng.integers(0, 8)))]))
    groups.append((int(rng.integers(0, 300)), [(3, 2)]))
    Case(groups, int(rng.choice([1, 2, 7, 16, 40, 64])), seed=seed).check(0, "seed %d" % seed)


def test_uniform_counts_without_qo_indptr():
    Case([(200, [(9, 4)] * 3), (50, [(0, 4)])], 16, uniform=4).check(0)
    Case([(200, [(9, 4)] * 3), (50, [(0, 4)])], 16, uniform=4).check(SIMT)


def test_a_larger_plan_serves_a_smaller_batch():
    Case([(300, [(20, 2)] * 3)], 16, seed=2).check(0, max_batch=50, q_len=9)


def test_same_as_the_unshared_call():
    """The rows and the visibility of run_varlen: its result within both calls' roundings."""
    c = Case([(600, [(40, 3), (0, 2)]), (77, [(130, 4)])], 32, seed=4)
    o, lse, status = c.run()
    rows, masks, indptr, b = [], [], [0], 0
    for g in range(2):
        sh = c.shared_indices[int(c.shared_indptr[g]):int(c.shared_indptr[g + 1])]
        for b in range(int(c.group_indptr[g]), int(c.group_indptr[g + 1])):
            rows += [sh, c.kv_indices[int(c.kv_indptr[b]):int(c.kv_indptr[b + 1])]]
            indptr.append(indptr[-1] + c.S[g] + c.P[b])
            masks.append(np.concatenate([np.ones((c.T[b], c.S[g]), bool), c.masks[b]], 1).reshape(-1))
    plan = B.mla_verify_plan(3, 32, c.q_len, 800, c.pool.shape[0], 4)
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    o2, lse2 = c.outputs()
    start = np.concatenate([[0], np.cumsum([m.size for m in masks])])[:-1]
    mask = torch.from_numpy(np.packbits(np.concatenate(masks), bitorder="little")).cuda()
    B.mla_verify_run_varlen(plan, c.q_nope, c.q_rope, c.pool, i32(indptr), torch.cat(rows), c.d_qo, c.loc, mask, i32(start), 3,
                            c.scale, 4, ws, o2, lse2)
    n = int(c.qo_indptr[-1])
    assert status == 0 and float((lse - lse2[:n]).abs().max()) <= 2e-3
    compare(bf16_to_f64(o).reshape(-1, 512), lse.cpu().numpy().reshape(-1), *(x.cpu().numpy().reshape(-1, *s) for x, s in
                                                                             zip(c.exact(), ((512,), ()))))


@pytest.mark.parametrize("flags", [0, SIMT], ids=["tc", "simt"])
def test_masks_that_leave_nothing(flags):
    """A token that sees no own key still sees the prefix; without a prefix its row is 0 and -inf."""
    c = Case([(90, [(100, 4)]), (0, [(80, 3), (0, 2)])], 8, seed=5)
    c.masks[0][1] = False
    c.masks[0][0, :64] = False
    c.masks[1][2] = False
    c.masks[2][:] = False
    c.check(flags)


@pytest.mark.parametrize("q_scale", [0.0, 1e-30, 6.0, 40.0])
@pytest.mark.parametrize("sign", [1.0, -1.0, 0.0])
def test_score_ranges(q_scale, sign):
    """Flat softmax to one key that takes all; scales below and at zero.  Scores reach 40 * 24 * 5 * 0.072 = 346; the
    products' fp32 sums and the base-2 scale are off by a few 2^-24 of the terms' size: 346 * 16 * 2^-24 = 3.3e-4."""
    Case([(700, [(40, 2)] * 3)], 16, seed=6, q_scale=q_scale, scale=sign * SCALE).check(0, lse_slack=3.3e-4)


@pytest.mark.parametrize("step", [0.05, 1.0, 20.0, -20.0])
def test_climbing_scores(step):
    """Every tile raises the maximum (or none does): references move while O stands, jumps far above any headroom."""
    c = Case([(1500, [(200, 2), (10, 3)])], 16, seed=7)
    c.q_rope[..., 0] = 14.0
    j = torch.arange(1500, device="cuda", dtype=torch.float32)
    c.pool[c.shared_indices.long(), 512] = (step * j / 16).to(torch.bfloat16)
    # Scores up to 14 * 20 * 94 * 0.072 = 1900.  The 576 channels are added up in 36 steps of 16, and a step may cut the
    # running fp32 sum off below its last bit, 2^-23 of it: 36 * 2^-23 * 1900 = 8.2e-3, whichever channels come first.
    c.check(0, lse_slack=8.2e-3)


def test_one_half_far_above_the_other():
    """Each CTA of a pair has half of a tile's keys: references 100s apart, in both directions, and one half unseen."""
    c = Case([(256, [(128, 2)])], 16, seed=8)
    c.q_rope[..., 0] = 14.0
    col = torch.zeros(256, device="cuda")
    col[:32], col[96:128], col[130:140] = 150.0, -150.0, 300.0
    c.pool[c.shared_indices.long(), 512] = col.to(torch.bfloat16)
    c.masks[0][0, 0:32] = False
    c.masks[0][1, 32:128] = False
    c.check(0, lse_slack=1e-3)


def test_one_visible_key_gives_its_row():
    c = Case([(0, [(300, 3)])], 8, seed=9)
    for i, j in enumerate((0, 47, 299)):
        c.masks[0][i] = False
        c.masks[0][i, j] = True
    o, _, _ = c.run()
    rows = c.kv_indices[torch.tensor([0, 47, 299], device="cuda")].long()
    assert torch.equal(o, c.pool[rows, None, :512].expand(3, 8, 512))


@pytest.mark.parametrize("flags", [0, SIMT], ids=["tc", "simt"])
def test_rows_outside_the_pool_are_left_out_and_reported(flags):
    c = Case([(200, [(70, 2), (5, 1)])], 16, seed=10)
    c.shared_indices[3], c.shared_indices[100], c.kv_indices[69], c.loc[1] = -1, c.pool.shape[0], -2, 2 ** 31 - 1
    o, lse, status = c.run(flags)
    assert status == B.MLA_VERIFY_DEV_BAD_ROW
    c.match(o, lse)


def test_a_query_that_is_not_finite_leaves_other_rows_alone():
    c = Case([(300, [(20, 2)] * 2)], 16, seed=11)
    good, lse, _ = c.run()
    c.q_nope[1, 3, 5] = float("nan")
    c.q_rope[2, 0, 7] = float("inf")
    o, lse2, _ = c.run()
    assert bool(o[1, 3].isnan().all()) and bool(lse2[1, 3].isnan())
    keep = torch.ones(4, 16, dtype=torch.bool, device="cuda")
    keep[1, 3] = keep[2, 0] = False
    assert torch.equal(o[keep], good[keep]) and torch.equal(lse2[keep], lse[keep])


def test_repeated_calls_give_the_same_bits():
    c = Case([(3000, [(50, 2)] * 20), (100, [(1, 1)])], 16, seed=12)
    first = c.run()
    for _ in range(5):
        again = c.run()
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])


def test_row_groups_of_one_tile():
    """Many own parts of one tile (and a few of more) in a row: what a row group leaves is read before the next one's."""
    c = Case([(70, [(1 + 7 * i % 60 if i % 9 else 150, 2) for i in range(500)])], 64, seed=18)
    c.q_rope[..., 0] = 14.0
    c.pool[c.kv_indices.long(), 512] = (torch.arange(len(c.kv_indices), device="cuda") % 40).to(torch.bfloat16)
    first = c.run()
    assert first[2] == 0
    # A weight in bf16 is off by at most 2^-8 of itself, in O's sum and its divisor alike: |dO| <= 2^-8 sum p |v - O|
    # <= 2^-8 (max|v| + |O|), and as much as 2^-8 |O| more for O's own rounding.  32 million values: no mean hides it.
    o, lse = c.exact()
    v = float(c.pool[:, :512].abs().max())
    assert bool(((first[0].double() - o).abs() <= 2.0 ** -8 * (v + 2 * o.abs())).all())
    assert float((first[1].double() - lse).abs().max()) <= 1e-3
    for _ in range(20):
        again = c.run()
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])


def test_offsets_past_32_bits():
    """A pool of 4.4 GB whose last rows are used."""
    rows = 3_800_000
    c = Case([(130, [(40, 2)])], 16, pool_rows=rows, seed=13)
    c.shared_indices[:] = torch.arange(rows - 130, rows, device="cuda", dtype=torch.int32)
    c.check(0)
    del c
    torch.cuda.empty_cache()


def test_a_captured_call_follows_lengths_and_contents():
    a = Case([(900, [(50, 2)] * 6)], 16, seed=14).device()
    b = Case([(20, [(300, 1), (0, 3)]), (400, [(7, 2), (8, 0), (9, 3), (10, 1)])], 16, seed=15).device()
    big = a if a.pool.shape[0] > b.pool.shape[0] else b
    rows = big.pool.shape[0]
    plan = B.mla_verify_plan(6, 16, 3, 400, rows, 0, flags=B.MLA_VERIFY_SHARED)
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")

    def buf(n, dtype=torch.int32):
        return torch.zeros(n, dtype=dtype, device="cuda")

    s = dict(group=buf(3), shared=buf(3), si=buf(2000), kv=buf(7), ki=buf(2000), qo=buf(7), loc=buf(18), mask=buf(4000, torch.uint8),
             mp=buf(6), pool=torch.zeros((rows, 576), dtype=torch.bfloat16, device="cuda"),
             qn=torch.zeros((18, 16, 512), dtype=torch.bfloat16, device="cuda"),
             qr=torch.zeros((18, 16, 64), dtype=torch.bfloat16, device="cuda"))
    o, lse = torch.zeros((18, 16, 512), dtype=torch.bfloat16, device="cuda"), torch.zeros((18, 16), device="cuda")

    def load(c):
        pad = np.concatenate([c.group_indptr, [c.batch]])[:3], np.concatenate([c.shared_indptr, [c.shared_indptr[-1]]])[:3]
        s["group"].copy_(i32(pad[0]))
        s["shared"].copy_(i32(pad[1]))
        for name, x in (("si", c.shared_indices), ("kv", c.d_kv), ("ki", c.kv_indices), ("qo", c.d_qo), ("loc", c.loc),
                        ("mask", c.mask), ("mp", c.mask_indptr), ("pool", c.pool), ("qn", c.q_nope), ("qr", c.q_rope)):
            s[name][:x.shape[0]].copy_(x)

    def call():
        B.mla_verify_run_shared(plan, s["qn"], s["qr"], s["pool"], s["group"], s["shared"], s["si"], s["kv"], s["ki"], s["qo"],
                                s["loc"], s["mask"], s["mp"], 6, 2, SCALE, ws, o, lse)

    load(a)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for c in (b, a, b):
        load(c)
        graph.replay()
        torch.cuda.synchronize()
        n = int(c.qo_indptr[-1])
        c.match(o[:n], lse[:n])
    assert B.mla_verify_read_status(plan, ws) == 0


def test_two_graphs_that_share_a_workspace():
    """Replayed in turn on one stream: neither call leaves anything that the other one trips over."""
    cases = [Case([(700, [(50, 2)] * 5), (0, [(9, 1)])], 16, seed=40).device(),
             Case([(130, [(300, 3), (4, 1)])], 64, seed=41).device()]
    plans = [c.plan() for c in cases]
    ws = torch.zeros(max(p.workspace_bytes for p in plans), dtype=torch.uint8, device="cuda")
    outs = [c.outputs() for c in cases]
    graphs = []
    for c, p, out in zip(cases, plans, outs):
        c.call(p, ws, *out)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            c.call(p, ws, *out)
    for out in outs:
        out[0].fill_(7), out[1].fill_(7)
    for k in (0, 1, 1, 0, 1, 0):
        graphs[k].replay()
    torch.cuda.synchronize()
    for c, out in zip(cases, outs):
        n = int(c.qo_indptr[-1])
        c.match(out[0][:n], out[1][:n])
    assert B.mla_verify_read_status(plans[0], ws) == 0


def test_two_calls_at_once_on_two_streams():
    cases = [Case([(2000 + 500 * k, [(30, 2)] * 8)], 16, seed=20 + k).device() for k in range(2)]
    plan = cases[0].plan()
    streams = [torch.cuda.Stream() for _ in cases]
    plans = [c.plan() for c in cases]
    ws = [torch.zeros(p.workspace_bytes, dtype=torch.uint8, device="cuda") for p in plans]
    outs = [c.outputs() for c in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        for c, p, w, out, st in zip(cases, plans, ws, outs, streams):
            c.call(p, w, *out, stream=st)
    torch.cuda.synchronize()
    for c, out in zip(cases, outs):
        n = int(c.qo_indptr[-1])
        c.match(out[0][:n], out[1][:n])
    assert plan.workspace_bytes > 0


def test_a_stalled_gather_times_out_and_the_next_call_is_right():
    c = Case([(300, [(40, 2)] * 3)], 16, seed=30)
    t0 = time.time()
    _, _, status = c.run(B.MLA_VERIFY_TEST_STALL_GATHER)
    assert status & B.MLA_VERIFY_DEV_TIMEOUT
    assert 0.5 < time.time() - t0 < 60  # the waits are bounded at about 2 s
    c.check(0)
