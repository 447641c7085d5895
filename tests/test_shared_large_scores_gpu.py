"""Scores far outside the usual, above and below zero: the key with the largest one takes all, as the definition has it."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from mla_speculative_decode_tree_gb300 import binding as B  # noqa: E402
from shared_util import Case  # noqa: E402


@pytest.mark.parametrize("flags", [0, B.MLA_VERIFY_FORCE_SIMT], ids=["tc", "simt"])
@pytest.mark.parametrize("order", ["up", "down", "shuffled"])
@pytest.mark.parametrize("sign", [1, -1], ids=["above", "below"])
@pytest.mark.parametrize("size", [12, 22, 24, 30, 60])
def test_the_largest_takes_all(size, sign, order, flags):
    """Each key has a value of its own, 2^-8 to 2^8 with neighbours 2^-8 apart or more, against a query's 2^size."""
    c = Case([(300, [(70, 2), (5, 1)]), (0, [(100, 3)]), (1500, [(0, 1)] * 3)], 16, seed=3)
    rows = torch.cat([c.shared_indices, c.kv_indices, c.loc[:int(c.qo_indptr[-1])]]).long()
    rank = torch.arange(rows.numel(), device="cuda")
    if order == "shuffled":
        rank = torch.randperm(rows.numel(), generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    elif order == "down":
        rank = rank.flip(0)
    assert rows.numel() <= 2048
    c.pool[rows, 512] = (torch.exp2((rank // 128 - 8).double()) * (1 + (rank % 128) / 128)).to(torch.bfloat16)
    c.q_rope[..., 0] = sign * 2.0 ** size
    o, lse, status = c.run(flags)
    exact, exact_lse = c.exact()
    assert status == 0
    # Where one key has all the weight in 64 bits, O is its row in every bit: w v / w, and products of bf16 are exact.  Scores
    # are off by 36 cut-off steps of 2^-23 and neighbours 2^-8 of themselves apart, so no other key comes in front.
    alone = (exact == exact.to(torch.bfloat16).double()).all(-1)
    assert bool(alone.all() if size >= 30 else alone.any() or size == 12)
    assert torch.equal(o[alone].double(), exact[alone])
    assert bool(lse.isfinite().all())
    slack = (36 + 4) * 2.0 ** -23  # the same steps; the scale, the base's change and the LSE's own roundings
    assert bool(((lse.double() - exact_lse).abs() <= 1e-3 + slack * exact_lse.abs()).all())
