"""Queries that are not finite, over a 4-bit pool: their row is NaN however the keys are cut up, and no other row is."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import numpy as np  # noqa: E402

import kv4_util as U  # noqa: E402
from mla_speculative_decode_tree_gb300 import binding as B  # noqa: E402


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("heads,keys,max_batch", [(8, 3000, 2), (8, 3000, 200), (40, 700, 200), (64, 9000, 200)])
@pytest.mark.parametrize("nsplit", [0, 1, 3, 40])
def test_row_is_nan_and_no_other(bad, heads, keys, max_batch, nsplit):
    """(Plans for 2 and for 200 requests: the merges for few and for many rows.)"""
    wl = U.workload(2, heads, [2, 1], [keys, 100], keys + 200, seed=heads)
    d, v = U.device(wl), U.verifier(wl, nsplit, 0, max_batch)
    o, lse = (x[:3].clone() for x in v.run(d, 2, wl["sm_scale"]))
    d["q_nope"][0, 1, 17] = bad
    d["q_rope"][2, heads - 1, 3] = bad
    o2, l2 = (x[:3] for x in v.run(d, 2, wl["sm_scale"]))
    assert v.status() == 0
    hit = torch.zeros((3, heads), dtype=torch.bool, device="cuda")
    hit[0, 1] = hit[2, heads - 1] = True
    assert bool(o2[hit].isnan().all()) and bool(l2[hit].isnan().all())
    assert torch.equal(o2[~hit], o[~hit]) and torch.equal(l2[~hit], lse[~hit])


@pytest.mark.parametrize("nsplit", [0, 1, 3])
def test_a_row_that_sees_nothing_stays_empty(nsplit):
    """Its query may hold anything."""
    wl = U.workload(1, 8, [2], [500], 600, seed=1)
    bits = np.unpackbits(wl["custom_mask"], bitorder="little")
    bits[:502] = 0
    wl["custom_mask"] = np.packbits(bits, bitorder="little")
    d, v = U.device(wl), U.verifier(wl, nsplit)
    d["q_nope"][0] = float("nan")
    o, lse = v.run(d, 1, wl["sm_scale"])
    assert v.status() == 0
    assert not bool(o[0].any()) and bool((lse[0] == float("-inf")).all())
    assert bool(o[1].isfinite().all()) and bool(lse[1].isfinite().all())


def test_the_two_launches_and_the_call_without_a_workspace():
    wl = U.workload(1, 8, [2], [900], 1000, seed=2)
    d, v = U.device(wl), U.verifier(wl, 4)
    del d["qo_indptr"]
    d["q_nope"][1, 3, 5] = float("nan")
    args = (d["q_nope"], d["q_rope"], d["kv_pool"], d["kv_indptr"], d["kv_indices"], d["out_cache_loc"],
            d["custom_mask"], d["mask_indptr"], 1, wl["sm_scale"], 4)
    hit = torch.zeros((2, 8), dtype=torch.bool, device="cuda")
    hit[1, 3] = True
    B.mla_verify_split(v.plan, *args, v.workspace)
    B.mla_verify_merge(v.plan, 1, 4, v.workspace, v.o, v.lse)
    assert torch.equal(v.o.isnan().all(-1), hit) and torch.equal(v.o.isnan().any(-1), hit) and torch.equal(v.lse.isnan(), hit)
    B.mla_verify_run_noalloc(v.plan, *args, v.o.zero_(), v.lse.zero_())
    assert torch.equal(v.o.isnan().all(-1), hit) and torch.equal(v.o.isnan().any(-1), hit) and torch.equal(v.lse.isnan(), hit)
