"""Draft verification by clusters of every size, alone and while other work keeps SMs busy, so that the CTAs of a cluster
begin at different times."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from mla_speculative_decode_tree_gb300 import binding as B  # noqa: E402
from test_step_gpu import Drafts, i32, plan_ws  # noqa: E402


@pytest.mark.parametrize("drawn", [True, False], ids=["drawn", "proposed"])
@pytest.mark.parametrize("vocab,requests", [(6999, 3), (9000, 3), (20001, 2), (30000, 2), (60001, 1), (57000, 38)])
def test_busy_neighbours(drawn, vocab, requests):
    """(Clusters of 1, 2, 4, 8, 16 and, of many requests, 8.)  A request in four has no child: its first pass comes at once."""
    d = Drafts([(1, 5, 3, 6)[b % 4] for b in range(requests)] + [4], vocab, drawn, seed=vocab % 97 + requests)
    n = len(d.counts)
    plan, ws = plan_ws(n, d.q_len)
    fixed = [torch.from_numpy(d.target).cuda(), torch.from_numpy(d.draft).cuda() if drawn else None, i32(d.tokens),
             i32(d.parents), i32(d.qo), torch.from_numpy(d.u).cuda(), torch.from_numpy(d.u_next).cuda()]
    ref, other = d.oracle(), torch.cuda.Stream()
    x = torch.randn((1024, 1024), device="cuda")
    y = torch.randn((3_000_001,), device="cuda")
    outs = []
    torch.cuda.synchronize()
    for k in range(40):
        if k >= 8:
            with torch.cuda.stream(other):
                (x @ x, y.sin())[k % 2]
        out = [torch.full(s, -9, dtype=torch.int32, device="cuda") for s in ((n, d.q_len), (n,), (n,))]
        B.mla_verify_accept_drafts(plan, *fixed, n, *out, ws)
        outs.append(out)
    torch.cuda.synchronize()
    for out in outs:
        for g, r in zip(out, ref):
            assert np.array_equal(g.cpu().numpy(), r)
