"""Queries that are not finite, behind shared prefixes: their row and its LSE are NaN whatever the signs of the keys, also where
every key that they see scores -inf; no other row is touched."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from mla_speculative_decode_tree_gb300 import binding as B  # noqa: E402
from shared_util import Case  # noqa: E402

SHAPES = [
    (4, [(0, [(0, 1)])]),                               # one key
    (8, [(1, [(0, 1), (2, 2)])]),
    (16, [(200, [(70, 2), (5, 1)]), (0, [(30, 3)])]),   # several tiles of each part, no prefix
    (64, [(3000, [(40, 2)] * 4)]),                      # many pairs have a partial
]


@pytest.mark.parametrize("flags", [0, B.MLA_VERIFY_FORCE_SIMT], ids=["tc", "simt"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("keys", ["negative", "positive", "mixed"])
@pytest.mark.parametrize("scale", [0.07, -0.07])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "h%d" % s[0])
def test_row_is_nan_and_no_other(shape, scale, keys, bad, flags):
    c = Case(shape[1], shape[0], seed=shape[0], scale=scale)
    sign = {"negative": -1, "positive": 1, "mixed": None}[keys]
    for col in (17, 512 + 3):  # (a column of the latent and one of RoPE)
        if sign:
            c.pool[:, col] = sign * (c.pool[:, col].abs() + 0.5)
    good, lse, status = c.run(flags)
    n = good.shape[0]
    assert status == 0 and bool(good.isfinite().all()) and bool(lse.isfinite().all())
    hit = torch.zeros((n, c.H), dtype=torch.bool, device="cuda")
    c.q_nope[0, 1, 17] = bad
    hit[0, 1] = True
    c.q_rope[n - 1, c.H - 1, 3] = bad
    hit[n - 1, c.H - 1] = True
    o, lse2, status = c.run(flags)
    assert status == 0
    assert bool(o[hit].isnan().all()) and bool(lse2[hit].isnan().all())
    assert torch.equal(o[~hit], good[~hit]) and torch.equal(lse2[~hit], lse[~hit])


@pytest.mark.parametrize("flags", [0, B.MLA_VERIFY_FORCE_SIMT], ids=["tc", "simt"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_row_that_sees_nothing_stays_empty(bad, flags):
    """Its query may hold anything."""
    c = Case([(0, [(80, 3), (0, 2)])], 8, seed=5)
    c.masks[0][2] = False
    c.masks[1][:] = False
    c.q_nope[2:5, :, 9] = bad
    o, lse, status = c.run(flags)
    assert status == 0 and not bool(o[2:].any()) and bool((lse[2:] == -float("inf")).all())
    assert bool(o[:2].isfinite().all()) and bool(lse[:2].isfinite().all())
