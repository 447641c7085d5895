"""Pins of the step oracles: what verification has to keep (the target's distribution), worked examples."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import step as S


def dist(rng, n):
    x = rng.exponential(size=n) ** 2
    return (x / x.sum()).astype(np.float32)


def test_weights_round_to_even():
    assert S.weight(1.0) == 1 << 38 and S.weight(2.0) == 1 << 38 and S.weight(-1.0) == 0 and S.weight(float("nan")) == 0
    assert [S.weight(np.float32(k * 2.0 ** -39)) for k in (1, 2, 3, 4, 5)] == [0, 1, 2, 2, 2]
    assert S.random24(0.0) == 0 and S.random24(1.0) == (1 << 24) - 1 and S.random24(0.5) == 1 << 23


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("children", [1, 2, 3])
def test_the_first_new_token_has_the_targets_distribution(drawn, children):
    """Sum over what was drafted, of the chance of each outcome at the root: the target's probabilities, up to the
    roundings to 2^-38 and 2^-24 (the oracle's own steps, with chances in place of random numbers)."""
    rng = np.random.default_rng(children)
    V = 5
    p, q = dist(rng, V), dist(rng, V)
    w, wq = [S.weight(x) for x in p], [S.weight(x) for x in q]
    out = [Fraction(0)] * V

    def go(k, r, z, chance):
        if k == children:
            for t in range(V):
                out[t] += chance * Fraction(r[t], max(sum(r), 1))
            return
        for x in range(V) if drawn else [(2 * k + 1) % V]:
            s = [y * z >> 38 for y in wq] if drawn else [z if t == x else 0 for t in range(V)]
            drawn_chance = Fraction(wq[x], sum(wq)) if drawn else 1
            ok = min(Fraction(1), Fraction(r[x], s[x])) if s[x] else Fraction(int(r[x] > 0))
            out[x] += chance * drawn_chance * ok
            left = [max(a - b, 0) for a, b in zip(r, s)]
            go(k + 1, left, max(z - sum(min(a, b) for a, b in zip(r, s)), 0), chance * drawn_chance * (1 - ok))

    go(0, w, S.ONE, Fraction(1))
    # V * (children + 1) roundings of 2^-38 each, and float32 rows whose sums are 1 up to V * 2^-25
    assert max(abs(float(a) - float(b)) for a, b in zip(out, p)) < V * (children + 1) * 2.0 ** -24


def test_a_chain_with_the_targets_own_drafts_is_accepted_whole():
    rng = np.random.default_rng(0)
    t = np.stack([dist(rng, 7) for _ in range(4)])
    path, nxt = S.accept_one(t, t, np.array([0, 3, 1, 6]), np.array([-1, 0, 1, 2]), np.full(4, 0.999999), 0.0)
    assert path == [0, 1, 2, 3] and nxt == 0


def test_worked_tree():
    """Two children proposed at the root: 0.5 fails against 1/4, then 1/2 of what is left (3/4) passes 0.6."""
    t = np.zeros((4, 4), np.float32)
    t[0] = [0.25, 0.5, 0.25, 0]
    t[2] = [0, 0, 0, 1]
    tokens, parents = np.array([9, 0, 1, 2]), np.array([-1, 0, 0, 1])
    path, nxt = S.accept_one(t, None, tokens, parents, np.array([0, 0.5, 0.6, 0], np.float32), 0.3)
    assert path == [0, 2] and nxt == 3
    path, nxt = S.accept_one(t, None, tokens, parents, np.array([0, 0.5, 0.7, 0], np.float32), 0.3)
    assert path == [0] and nxt == 2  # tokens 0 and 1 are gone


def test_commit_moves_the_path_to_the_front():
    pool = np.arange(8)[None, :, None] * np.ones((2, 8, 1), int)
    table, refs = np.array([[0, 1, 2, 3]]), np.array([1, 0, 0, 0])
    got, lens, refs, bad = S.commit(pool, [0, 5], np.array([1, 2, 3, 4, 5]), np.array([[0, 2, 4, -1, -1]]), [3], 1, [1], 2,
                                    table, refs)
    assert got[0, :, 0].tolist() == [0, 1, 3, 5, 4, 5, 6, 7] and lens.tolist() == [4] and not bad
    assert refs.tolist() == [1, 1, 0, 0]  # four tokens: two pages


def test_fork_then_release_leaves_the_counts():
    rng = np.random.default_rng(1)
    pool = rng.integers(0, 99, (2, 24, 3))
    table, lens, refs = np.full((3, 4), -1), np.array([7, 0, 0]), np.zeros(8, int)
    table[0, :3] = [5, 1, 3]
    refs[[5, 1, 3]] = 1
    free, n = S.free_list(refs)
    assert free.tolist() == [0, 2, 4, 6, 7, -1, -1, -1] and n == 5
    p2, t2, l2, r2, used, st = S.fork(pool, np.array([0, 0]), np.array([1, 2]), 3, table, lens, refs, free[:n])
    assert used == 2 and st == 0 and t2[1].tolist() == [5, 1, 0, -1] and t2[2].tolist() == [5, 1, 2, -1]
    assert r2.tolist() == [1, 3, 1, 1, 0, 3, 0, 0] and (p2[:, 6] == pool[:, 9]).all() and (p2[:, 0] == pool[:, 9]).all()
    l3, r3, st = S.release(np.array([2, 1, 2]), 3, t2, l2, r2)
    assert l3.tolist() == [7, 0, 0] and r3.tolist() == refs.tolist() and st == 0


@pytest.mark.parametrize("mistake", ["no residual", "strict order", "next from draft"])
def test_planted_mistakes_move_the_distribution(mistake):
    """What the distribution pin would see: one child, a residual that is not taken, a wrong row."""
    p, q = np.array([0.7, 0.2, 0.1], np.float32), np.array([0.1, 0.2, 0.7], np.float32)
    out = np.zeros(3)
    for x in range(3):
        ok = min(1.0, p[x] / q[x])
        r = np.maximum(p - q, 0)
        if mistake == "no residual":
            r = p
        elif mistake == "strict order":
            ok = 1.0 if p[x] > q[x] else 0.0
        else:
            r = q
        out[x] += q[x] * ok
        out += q[x] * (1 - ok) * r / r.sum()
    assert np.abs(out - p).max() > 0.02
