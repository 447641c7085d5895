"""Attention over a 4-bit pool with the work cut into equal pieces (nsplit = 0):
CTAs that end and start in the middle of a request, many short requests per CTA,
requests without tokens or keys, lengths read on the device alone."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import kv4_util as U
from mla_speculative_decode_tree_gb300 import binding as B
from oracle import kv4

pytestmark = pytest.mark.gpu


def lengths(b, t_hi, p_hi, seed, empty=0.0):
    rng = np.random.default_rng(seed)
    t = rng.integers(1, t_hi + 1, b)
    t[rng.random(b) < empty] = 0
    return [int(x) for x in t], [int(x) for x in rng.integers(0, p_hi + 1, b)]


@pytest.mark.parametrize("b,h,t_hi,p_hi,empty", [
    (33, 4, 3, 300, 0.3),    # one request more than a warp scans at once
    (64, 8, 1, 200, 0.0),    # decode, lengths of one and two tiles
    (200, 2, 2, 40, 0.2),    # more requests than SMs, one tile each
    (331, 1, 1, 3, 0.5),     # a few keys each, half of the requests without a token
    (40, 24, 9, 500, 0.1),   # several row groups per request
])
def test_many_requests(b, h, t_hi, p_hi, empty):
    t, p = lengths(b, t_hi, p_hi, b + h, empty)
    U.run_and_check(U.workload(b, h, t, p, sum(p) + sum(t) + 10, seed=b), 0, 0, "%d requests" % b)


@pytest.mark.parametrize("where", ["first", "middle", "last"])
def test_one_long_request_among_empty_ones(where):
    """All the work is one request's: it is cut between the CTAs wherever it stands."""
    b, at = 70, {"first": 0, "middle": 35, "last": 69}[where]
    t, p = [0] * b, [int(x) for x in np.random.default_rng(1).integers(0, 5, b)]
    t[at], p[at] = 5, 9000
    U.run_and_check(U.workload(b, 8, t, p, sum(p) + 50, seed=2), 0, 0, where)


def test_no_request_has_a_token():
    wl = U.workload(5, 8, [1] * 5, [7] * 5, 100, seed=3)
    d, v = U.device(wl), U.verifier(wl)
    d["qo_indptr"] = torch.zeros(6, dtype=torch.int32, device="cuda")
    v.o.fill_(7)
    v.run(d, 5, wl["sm_scale"])
    assert v.status() == 0 and bool((v.o == 7).all())


@pytest.mark.parametrize("rows,keys", [(16, 128 * 152 + 5), (64, 128 * 304), (65, 20001), (9, 20001)])
def test_pieces_of_one_request(rows, keys):
    """One request over about all SMs: pieces of a tile or two, whole and ragged."""
    U.run_and_check(U.workload(1, rows, [1], [keys - 1], keys + 10, seed=rows), 0, 0, "%d keys" % keys)


def test_nsplit_choices_agree():
    """Equal pieces and chunk grids sum in other orders: equal within the bound of one against the 64-bit result."""
    wl = U.workload(3, 16, [4, 1, 9], [700, 3000, 50], 4000, seed=4)
    for ns in (0, 1, 7):
        U.run_and_check(wl, ns, 0, "nsplit %d" % ns)


def test_a_graph_follows_lengths_that_change_on_the_device():
    """The pieces come from the index arrays on the device: a captured call takes new lengths."""
    big = U.workload(4, 8, [3, 3, 3, 3], [900, 20, 500, 300], 3000, seed=5)
    d, v = U.device(big), U.verifier(big)
    d = {k: torch.nn.functional.pad(x.reshape(-1), (0, 64)) if k in ("custom_mask", "kv_indices") else x for k, x in d.items()}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        v.run(d, 4, big["sm_scale"])
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            v.run(d, 4, big["sm_scale"])
    for t, p in (([3, 3, 3, 3], [900, 20, 500, 300]), ([1, 3, 0, 2], [0, 900, 70, 1]), ([0, 0, 0, 3], [3, 0, 1, 600])):
        wl = U.workload(4, 8, t, p, 3000, seed=sum(p) + 6)
        n = wl["n_tokens"]
        for k, x in U.device(wl).items():
            x = x.reshape(-1)[:d[k].numel()]
            d[k].reshape(-1)[:x.numel()].copy_(x)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert v.status() == 0
        o_ref, l_ref = kv4.verify(wl)
        used = np.concatenate([wl["kv_indices"], wl["out_cache_loc"][:n]])
        vmax = np.abs(kv4.decode_rows(wl["pool"][used])[:, :512]).max()
        U.check(v.o[:n], v.lse[:n], o_ref, l_ref, vmax, str((t, p)))


def test_bits_do_not_depend_on_a_neighbours_contents():
    """Sums are taken in a fixed order: another request's keys change nothing but its own rows."""
    wl = U.workload(3, 8, [2, 2, 2], [400, 800, 300], 1600, seed=7)
    d, v = U.device(wl), U.verifier(wl)
    o, lse = (x.clone() for x in v.run(d, 3, wl["sm_scale"]))
    used = torch.from_numpy(wl["kv_indices"][400:1200].astype(np.int64)).cuda()
    d["kv_pool"][used] = d["kv_pool"][used.flip(0)]
    o2, l2 = v.run(d, 3, wl["sm_scale"])
    assert torch.equal(o[:2], o2[:2]) and torch.equal(o[4:6], o2[4:6]) and torch.equal(lse[4:6], l2[4:6])
    assert not torch.equal(o[2:4], o2[2:4])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("heads,keys", [(5, 40), (8, 3000), (64, 20000)])
def test_a_query_that_is_not_finite_makes_its_row_nan(bad, heads, keys):
    """... and no other row of its group."""
    wl = U.workload(2, heads, [2, 1], [keys, 100], keys + 200, seed=heads)
    d, v = U.device(wl), U.verifier(wl)
    o, lse = (x[:3].clone() for x in v.run(d, 2, wl["sm_scale"]))
    d["q_nope"][0, 1, 17] = bad
    d["q_rope"][2, heads - 1, 3] = bad
    o2, l2 = (x[:3] for x in v.run(d, 2, wl["sm_scale"]))
    assert v.status() == 0
    hit = torch.zeros((3, heads), dtype=torch.bool, device="cuda")
    hit[0, 1] = hit[2, heads - 1] = True
    assert bool(o2[hit].isnan().all()) and bool(l2[hit].isnan().all())
    assert torch.equal(o2[~hit], o[~hit]) and torch.equal(l2[~hit], lse[~hit])
