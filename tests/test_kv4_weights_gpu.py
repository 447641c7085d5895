"""Attention over a 4-bit pool where the weights of a row lie far apart: attention sinks above long flat tails.

What the kernel may lose, for any row and any number of keys.  With V = max |v|:
  - a weight p of 2^-6 or more, in its column's scale, carries its e4m3 part and the rest of it to 2 or 3 more bits, after
    a rounding to 11 bits: it is off by at most (2^-8 + 2^-11) p;
  - a smaller one by at most 2^-14.  After 1, 3, 5, 9, 13, ... tiles a column's mean is at least 2^-5, or the scale is
    raised within a tile: after k tiles of which that was so, at most 4, 6, 10, 14, ... tiles have lost 2^-14 a key
    against a sum of 128 k * 2^-5, and of 8 (the first maximum): 2^-8 at most.  A maximum of 2^6 that lowers the
    scale faces six tiles: 2^-10.4;
  - O is rounded to bf16 once: 2^-9.
All of them: (2^-8 + 2^-11 + 2^-8 + 2^-9) V for an element.  The values here have a mean, so that nothing of it averages
out over the keys."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from mla_speculative_decode_tree_gb300 import binding as B  # noqa: E402
from mla_speculative_decode_tree_gb300 import workloads as W  # noqa: E402
from oracle import kv4  # noqa: E402
import kv4_util as U  # noqa: E402

LOSS = 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -8 + 2.0 ** -9
ROWS = 2000  # distinct pool rows of the tail; keys name them over and over
SCALE = 192.0 ** -0.5


def make_pool(sink_value, seed):
    """Rows 0 .. ROWS-1: values 1 +- 0.3; row ROWS: the sink, 6 in RoPE channel 0; row ROWS + 1: another one."""
    x = np.zeros((ROWS + 2, 576))
    x[:, :512] = 1 + 0.3 * np.random.default_rng(seed).standard_normal((ROWS + 2, 512))
    x[ROWS:, :512] = sink_value
    x[ROWS, 512] = 6.0
    x[ROWS + 1, 513] = 6.0
    return kv4.encode_rows(x[:, :512], x[:, 512:])


def bf16(x):
    return W.f32_to_bf16_bits(np.asarray(x, np.float32))


def reference(pool, ids, qn, qr):
    """O and LSE in fp64, [n, 512] and [n]: a row that is named k times counts k times."""
    v = kv4.decode_rows(pool)
    n = np.bincount(ids, minlength=pool.shape[0]).astype(np.float64)
    f = lambda b: W.bf16_bits_to_f32(b).astype(np.float64)  # noqa: E731
    s = np.concatenate([f(qn), f(qr)], -1) @ v.T * SCALE
    s = np.where(n > 0, s, -np.inf)
    m = s.max(-1, keepdims=True)
    p = np.exp(s - m) * n
    l = p.sum(-1)
    return p @ v[:, :512] / l[:, None], m[:, 0] + np.log(l)


def run(pool, ids, qn, qr, requests, nsplit, max_batch, flags=0):
    """`requests` requests of the same keys (the last one the draft's) and one token; qn [H, 512], qr [H, 64]."""
    H, P = qn.shape[0], ids.size - 1
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    tok = lambda b: t(np.tile(b.view(np.int16), (requests, 1, 1))).view(torch.bfloat16)  # noqa: E731
    idx = lambda a: t(np.asarray(a, np.int32))  # noqa: E731
    L = P + 1
    v = B.Verifier(max_batch, H, 1, L, pool.shape[0], nsplit, B.MLA_VERIFY_KV4 | flags)
    d = dict(q_nope=tok(qn[None]), q_rope=tok(qr[None]), kv_pool=t(pool), kv_indptr=idx(np.arange(requests + 1) * P),
             kv_indices=idx(np.tile(ids[:P], requests)), out_cache_loc=idx([ids[P]] * requests),
             custom_mask=torch.full(((requests * L + 7) // 8,), 255, dtype=torch.uint8, device="cuda"),
             mask_indptr=idx(np.arange(requests) * L))
    o, lse = (x.clone() for x in v.run(d, requests, SCALE))
    for _ in range(2):  # the same bits again
        o2, lse2 = v.run(d, requests, SCALE)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert v.status() == 0
    return o.double().cpu().numpy(), lse.double().cpu().numpy(), v.plan.describe()


def check(o, lse, pool, ids, qn, qr):
    o_ref, l_ref = reference(pool, ids, qn, qr)
    vmax = np.abs(kv4.decode_rows(pool)[:, :512]).max()
    err = np.abs(o - o_ref[None]).max(-1)
    assert err.max() <= LOSS * vmax, err.max() / vmax
    assert np.linalg.norm(o - o_ref[None]) <= LOSS * np.linalg.norm(np.ones_like(o) * np.abs(o_ref[None]).max(-1, keepdims=True))
    assert np.abs(lse - l_ref[None]).max() <= U.LSE_ABS


def queries(gaps, spread, seed):
    """Row i scores key ROWS gaps[i] above the tail, whose scores have the given deviation."""
    n = len(gaps)
    qn = spread / (0.3 * np.sqrt(512) * SCALE) * np.random.default_rng(seed).standard_normal((n, 512))
    qn -= qn.mean(-1, keepdims=True)  # (the values' mean is no part of the tail's scores)
    qr = np.zeros((n, 64))
    qr[:, 0] = (np.asarray(gaps) + 0.5 * spread ** 2) / (6 * SCALE)
    return bf16(qn), bf16(qr)


def tail(keys, seed):
    return np.random.default_rng(seed).integers(0, ROWS, keys).astype(np.int32)


@pytest.mark.parametrize("rows,nq", [(16, 16), (31, 32), (47, 48), (64, 64)])
@pytest.mark.parametrize("keys,spread", [(1000, 0.0), (7500, 0.0), (32767, 0.0), (32767, 1.0), (65535, 1.0), (185000, 0.0),
                                         (185000, 1.0), (185000, 2.0)])
def test_sink_in_the_first_tile(rows, nq, keys, spread):
    """One CTA holds all keys; the rows' sinks stand 7 to 16 above the tail."""
    pool, ids = make_pool(-1.0, 1), tail(keys, keys)
    ids[17] = ROWS
    qn, qr = queries(np.linspace(7, 16, rows), spread, rows)
    o, lse, info = run(pool, ids, qn, qr, 1, 1, 200)
    assert info.rows_per_cta == nq
    check(o, lse, pool, ids, qn, qr)


@pytest.mark.parametrize("where", [[130], [128 * 40 + 5], [32000], list(range(0, 32767, 1000)), [5, 6, 7, 20000]])
@pytest.mark.parametrize("rows", [16, 64])
def test_sinks_elsewhere(rows, where):
    """... in the second tile, in the middle, at the end, every thousand keys, a few."""
    pool, ids = make_pool(3.0, 2), tail(32767, 3)
    ids[where] = ROWS
    qn, qr = queries(np.linspace(7, 16, rows), 0.0, rows)
    o, lse, _ = run(pool, ids, qn, qr, 1, 1, 200)
    check(o, lse, pool, ids, qn, qr)


@pytest.mark.parametrize("rows,requests", [(16, 160), (64, 152), (5, 320)])
def test_a_large_batch_in_equal_pieces(rows, requests):
    """A request or two to a CTA."""
    pool, ids = make_pool(-1.0, 4), tail(7500, 5)
    ids[17] = ROWS
    qn, qr = queries(np.linspace(8, 14, rows), 0.3, rows)
    o, lse, _ = run(pool, ids, qn, qr, requests, 0, requests)
    check(o, lse, pool, ids, qn, qr)


@pytest.mark.parametrize("rows", [16, 31, 47, 64])
def test_second_sink_above_the_first(rows):
    """The scale follows the tail after the first sink, then a key far above both comes, then the tail again."""
    pool, ids = make_pool(-2.0, 6), tail(20000, 7)
    ids[3] = ROWS
    ids[11000] = ROWS + 1
    qn, qr = queries(np.linspace(4, 12, rows), 0.5, rows)
    second = W.bf16_bits_to_f32(qr).copy()
    second[:, 1] = second[:, 0] * np.linspace(0.8, 1.5, rows)
    qr = bf16(second)
    o, lse, _ = run(pool, ids, qn, qr, 1, 1, 200)
    check(o, lse, pool, ids, qn, qr)


@pytest.mark.parametrize("rows", [16, 64])
@pytest.mark.parametrize("gap", [25.0, 45.0, 61.0, 120.0])
def test_a_tail_that_counts_for_nothing(rows, gap):
    """The scale is raised as far as the sums in 32 bits allow, and not further."""
    pool, ids = make_pool(-1.0, 8), tail(30000, 9)
    ids[0] = ROWS
    qn, qr = queries(np.full(rows, gap), 1.0, rows)
    o, lse, _ = run(pool, ids, qn, qr, 1, 1, 200)
    check(o, lse, pool, ids, qn, qr)


def test_both_kernels_agree():
    pool, ids = make_pool(-1.0, 10), tail(15000, 11)
    ids[17] = ROWS
    qn, qr = queries(np.linspace(8, 14, 16), 0.5, 12)
    for flags in (0, B.MLA_VERIFY_FORCE_SIMT):
        o, lse, _ = run(pool, ids, qn, qr, 1, 1, 1, flags)
        check(o, lse, pool, ids, qn, qr)
