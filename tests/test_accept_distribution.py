"""What verification has to keep: the token behind the root has the target's distribution, whatever was drafted.  The oracle's
walk and the kernel's, drawn and proposed children, and calls that break the rules, which the same count has to see."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from mla_speculative_decode_tree_gb300 import binding as B  # noqa: E402
from oracle import step as S  # noqa: E402

V = 5
PARENTS = {0: [-1], 1: [-1, 0], 2: [-1, 0, 0], 3: [-1, 0, 0, 0]}


def distributions(seed):
    rng = np.random.default_rng(seed)
    x = rng.exponential(size=(2, V)) ** 2
    p, q = (x / x.sum(1, keepdims=True)).astype(np.float32)
    return rng, p, q


def drafts(rng, n, children, q):
    """[n, children] tokens: drawn from q, or (None) the same different ones for all."""
    if q is None:
        return np.tile((np.arange(children) * 2 + 1) % V, (n, 1))
    return rng.choice(V, (n, children), p=q.astype(np.float64) / q.astype(np.float64).sum())


def far(counts, p):
    """The largest deviation from n * p, in standard deviations (one count more for the roundings of p and the numbers)."""
    n, p = counts.sum(), p.astype(np.float64) / p.astype(np.float64).sum()
    return ((np.abs(counts - n * p) - 1) / np.sqrt(n * p * (1 - p))).max()


def walk_oracle(p, q, tokens, u, u_next):
    n, children = tokens.shape
    target, draft = np.tile(p, (children + 1, 1)), None if q is None else np.tile(q, (children + 1, 1))
    first = []
    for i in range(n):
        path, nxt = S.accept_one(target, draft, np.concatenate([[0], tokens[i]]), PARENTS[children], u[i], u_next[i])
        first.append(tokens[i, path[1] - 1] if len(path) > 1 else nxt)
    return np.bincount(first, minlength=V)


def walk_kernel(p, q, tokens, u, u_next):
    n, children = tokens.shape
    plan = B.mla_verify_plan(n, 1, children + 1, children + 1, 1, 1)
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    rows = n * (children + 1)

    def i32(a):
        return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()

    def tiled(x):
        return torch.from_numpy(np.tile(x, (rows, 1))).cuda()

    out = [torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((n, children + 1), (n,), (n,))]
    B.mla_verify_accept_drafts(plan, tiled(p), None if q is None else tiled(q), i32(np.hstack([np.zeros((n, 1)), tokens])),
                               i32(np.tile(PARENTS[children], n)), None, torch.from_numpy(u.reshape(-1)).cuda(),
                               torch.from_numpy(u_next).cuda(), n, *out, ws)
    acc, num, nxt = (x.cpu().numpy() for x in out)
    first = np.where(num > 1, tokens[np.arange(n), np.maximum(acc[:, 1] - 1, 0)], nxt)
    return np.bincount(first, minlength=V)


def numbers(rng, n, children):
    k = rng.integers(0, 1 << 24, (n, children + 2)).astype(np.float32) / np.float32(1 << 24)
    return k[:, :-1].copy(), k[:, -1].copy()


@pytest.mark.parametrize("walk,n", [pytest.param(walk_oracle, 20_000, id="oracle"),
                                    pytest.param(walk_kernel, 200_000, id="kernel", marks=pytest.mark.gpu)])
@pytest.mark.parametrize("drawn", [True, False], ids=["drawn", "proposed"])
@pytest.mark.parametrize("children", [1, 2, 3])
def test_the_first_new_token(walk, n, drawn, children):
    rng, p, q = distributions(10 * children + drawn)
    q = q if drawn else None
    assert far(walk(p, q, drafts(rng, n, children, q), *numbers(rng, n, children)), p) <= 5


@pytest.mark.parametrize("mistake", ["another draft", "no remainder", "proposed as if drawn"])
def test_calls_that_break_the_rules_are_seen(mistake):
    rng, n = np.random.default_rng(3), 20_000
    p, q = np.array([0.5, 0.2, 0.1, 0.1, 0.1], np.float32), np.array([0.1, 0.4, 0.3, 0.1, 0.1], np.float32)
    tokens = drafts(rng, n, 1, {"another draft": p, "proposed as if drawn": None}.get(mistake, q))
    u, u_next = numbers(rng, n, 1)
    if mistake == "no remainder":  # what is rejected is followed by a draw from the target itself
        kept = np.array([S.accept_one(np.tile(p, (2, 1)), np.tile(q, (2, 1)), [0, t[0]], [-1, 0], x, 0.0)[0] == [0, 1]
                         for t, x in zip(tokens, u)])
        counts = np.bincount(tokens[kept, 0], minlength=V) + walk_oracle(p, None, tokens[~kept][:, :0], u[~kept], u_next[~kept])
    else:
        counts = walk_oracle(p, q, tokens, u, u_next)
    assert counts.sum() == n and far(counts, p) > 10
