"""mla_verify_run_shared and mla_verify_run_varlen on the same keys and visibilities: O and LSE of the one against the other's."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from mla_speculative_decode_tree_gb300 import binding as B  # noqa: E402
from shared_util import Case, i32  # noqa: E402


def unshared(c, nsplit):
    """The case as a call without groups: each request's prefix in front of its own keys."""
    rows, masks, lens = [], [], []
    for g in range(len(c.groups)):
        sh = c.shared_indices[int(c.shared_indptr[g]):int(c.shared_indptr[g + 1])]
        for b in range(int(c.group_indptr[g]), int(c.group_indptr[g + 1])):
            rows += [sh, c.kv_indices[int(c.kv_indptr[b]):int(c.kv_indptr[b + 1])]]
            lens.append(c.S[g] + c.P[b])
            masks.append(np.concatenate([np.ones((c.T[b], c.S[g]), bool), c.masks[b]], 1).reshape(-1))
    plan = B.mla_verify_plan(c.batch, c.H, c.q_len, max(lens) + c.q_len, c.pool.shape[0], nsplit)
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    o, lse = c.outputs()
    start = np.cumsum([0] + [m.size for m in masks])[:-1]
    mask = torch.from_numpy(np.packbits(np.concatenate(masks), bitorder="little")).cuda()
    B.mla_verify_run_varlen(plan, c.q_nope, c.q_rope, c.pool, i32(np.cumsum([0] + lens)), torch.cat(rows), c.d_qo, c.loc, mask,
                            i32(start), c.batch, c.scale, nsplit, ws, o, lse)
    assert B.mla_verify_read_status(plan, ws) == 0
    n = int(c.qo_indptr[-1])
    return o[:n], lse[:n]


@pytest.mark.parametrize("flags", [0, B.MLA_VERIFY_FORCE_SIMT], ids=["tc", "simt"])
@pytest.mark.parametrize("groups,heads", [([(600, [(40, 3), (0, 2)]), (77, [(130, 4)])], 32), ([(2000, [(30, 1)] * 9)], 8),
                                          ([(0, [(100, 5)]), (400, [(3, 2), (0, 0), (70, 7)])], 64)])
def test_the_same_attention(groups, heads, flags):
    c = Case(groups, heads, seed=heads)
    o, lse, status = c.run(flags)
    o2, lse2 = unshared(c, 4)
    exact, _ = c.exact()
    # sum p |v| of each row
    size = torch.zeros_like(exact)
    for g in range(len(c.groups)):
        sh = c.shared_indices[int(c.shared_indptr[g]):int(c.shared_indptr[g + 1])].long()
        for b in range(int(c.group_indptr[g]), int(c.group_indptr[g + 1])):
            t0, t1 = int(c.qo_indptr[b]), int(c.qo_indptr[b + 1])
            rows = torch.cat([sh, c.kv_indices[int(c.kv_indptr[b]):int(c.kv_indptr[b + 1])].long(), c.loc[t0:t1].long()])
            k, q = c.pool[rows].double(), torch.cat([c.q_nope[t0:t1], c.q_rope[t0:t1]], -1).double()
            see = torch.cat([torch.ones((t1 - t0, sh.numel()), dtype=torch.bool, device="cuda"),
                             torch.from_numpy(c.masks[b]).cuda()], 1)
            s = (torch.einsum("thd,kd->thk", q, k) * c.scale).masked_fill(~see[:, None], -float("inf"))
            size[t0:t1] = torch.softmax(s, -1) @ k[:, :512].abs()
    # Each call: weights in bf16, off by at most 2^-8 of themselves, in the sum of p v and, where it is the divisor, in that of
    # p; then O's own rounding, 2^-8 of it: 2^-8 (size + 2 |O|).  1e-4 for what is added up in fp32 (2,000 terms of up to
    # `size`, 2^-24 each) and for products of these errors.
    bound = 2 * 2.0 ** -8 * (size + 2 * exact.abs()) + 1e-4
    assert status == 0
    assert bool(((o.double() - o2.double()).abs() <= bound).all())
    # 2e-3: within the 1e-3 that each call's LSE is held to against the definition
    assert float((lse - lse2).abs().max()) <= 2e-3
