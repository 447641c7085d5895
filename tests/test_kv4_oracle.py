"""Pins of the 4-bit oracle: the row format by hand, the rounding rule, decode of what was encoded, attention
against a two-key closed form, slot maps of a worked example."""

import numpy as np
import pytest

from oracle import kv4


def test_row_layout_by_hand():
    """One value per block, at a code index whose byte and bits are worked out from the header's text."""
    x, r = np.zeros((1, 512)), np.zeros((1, 64))
    x[0, 0] = 6.0      # block 0, code 0: magnitude index 7 in bits 0..2 of byte 0
    x[0, 133] = -3.0   # block 1, code 5: word at byte 64, bits 20..22, sign bit 11 (code 5 = 4 + 1)
    x[0, 495] = 1.5    # block 3, q = 3, h = 0: alone in its group, so e = -2 (1.5 = 6 * 2^-2)
    r[0, 17] = -0.75   # code 529: block 4, code 17: word at byte 264, code 1: bits 4..6, sign bit 15
    row = kv4.encode_rows(x, r)[0]
    assert row[0] == 7
    word = int.from_bytes(row[64:68].tobytes(), "little")
    assert word == (7 << 20) | (1 << 11)          # -3 = -6 * 2^-1
    assert row[320 + 2 * 0 + 0] == 127            # codes 0..15: e = 0
    assert row[320 + 2 * 1 + 0] == 126            # codes 128..143
    assert row[320 + 16 * 3 + 2 * 3 + 0] == 125   # codes 480..495
    word = int.from_bytes(row[264:268].tobytes(), "little")
    assert word == (7 << 4) | (1 << 15)           # -0.75 = -6 * 2^-3
    assert row[320 + 16 * 0 + 2 * 4 + 1] == 124   # codes 528..543
    unused = [320 + 16 * q + k for q in range(4) for k in range(10, 16)]
    assert not row[unused].any()


@pytest.mark.parametrize("x,expected", [
    (0.25, 0.0), (0.26, 0.5), (0.74, 0.5), (0.75, 1.0), (1.25, 1.0), (1.26, 1.5), (1.75, 2.0), (1.74, 1.5),
    (2.5, 2.0), (2.51, 3.0), (3.5, 4.0), (3.49, 3.0), (5.0, 4.0), (5.01, 6.0), (-2.5, -2.0), (-3.5, -4.0)])
def test_nearest_code_ties_to_even(x, expected):
    g = np.zeros((1, 16))
    g[0, 0], g[0, 1] = 6.0, x  # the 6 holds the group's exponent at 0
    assert kv4.value(*kv4.quantise(g))[0, 1] == expected


@pytest.mark.parametrize("top,e", [(6.0, 0), (6.01, 1), (3.0, -1), (3.01, 0), (0.0, -13), (2.0 ** -14, -13),
                                   (6.0 * 2 ** 13, 13), (1e9, 13), (np.inf, 13)])
def test_exponent_rule(top, e):
    g = np.zeros((1, 16))
    g[0, 3] = top
    assert kv4.quantise(g)[2][0, 0] == e


def test_non_finite_values():
    g = np.zeros((1, 16))
    g[0, :3] = [np.nan, 1.0, -np.inf]
    v = kv4.value(*kv4.quantise(g))[0]
    assert v[0] == 0 and v[2] == -6 * 2.0 ** 13


def test_round_trip_error_and_idempotence():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((40, 576)) * np.exp(rng.standard_normal(576))
    rows = kv4.encode_rows(x[:, :512], x[:, 512:])
    y = kv4.decode_rows(rows)
    top = np.abs(x.reshape(40, -1, 16)).max(-1, keepdims=True)
    err = np.abs((y - x).reshape(40, -1, 16)) / top
    assert err[:, :32].max() <= 1 / 3 + 1e-12  # widest gap 4..6: off by 1 of at least 3
    assert err[:, 32:].max() <= 1 / 9 + 1e-12  # and the residual's by a third of that
    again = kv4.decode_codes(kv4.encode_rows(y[:, :512], np.zeros((40, 64))))[:, :512]
    assert np.array_equal(again, y[:, :512])


def test_garbage_scales_decode_to_finite_values():
    rows = np.random.default_rng(1).integers(0, 256, (8, 384)).astype(np.uint8)
    assert np.isfinite(kv4.decode_rows(rows)).all()
    assert np.abs(kv4.decode_rows(rows)).max() <= 2 * 6 * 2.0 ** 13


def test_attention_two_keys():
    """One query, two keys with scores 0 and ln 3: weights 1/4 and 3/4."""
    lat = np.zeros((2, 512))
    lat[0, 7], lat[1, 9] = 4.0, 4.0
    rope = np.zeros((2, 64))
    rope[1, 0] = 2.0
    bits = lambda x: (np.asarray(x, np.float32).view(np.uint32) >> 16).astype(np.uint16)  # noqa: E731
    qr = np.zeros((1, 1, 64), np.float32)
    qr[0, 0, 0] = 1.0
    wl = dict(B=1, H=1, T=1, pool=kv4.encode_rows(lat, rope), q_nope=bits(np.zeros((1, 1, 512))), q_rope=bits(qr),
              kv_indptr=np.array([0, 1]), kv_indices=np.array([0]), out_cache_loc=np.array([1]),
              custom_mask=np.array([3], np.uint8), mask_indptr=np.array([0]), sm_scale=np.log(3.0) / 2.0)
    o, lse = kv4.verify(wl)
    assert np.isclose(o[0, 7], 1.0) and np.isclose(o[0, 9], 3.0) and np.isclose(lse[0], np.log(4.0))
    wl["custom_mask"] = np.array([0], np.uint8)
    o, lse = kv4.verify(wl)
    assert not o.any() and lse[0] == -np.inf


def test_slots_worked_example():
    """Pages of 4: request 0 has 5 tokens (pages 7, 2) and takes 4 (one fresh page), request 1 is new with 1."""
    r, no_page, bad = kv4.build_slots([5, 0], [4, 1], 4, [[7, 2, -1], [-1, -1, -1]], [9, 1, 3], 64)
    assert r["kv_indptr"] == [0, 5, 5] and r["qo_indptr"] == [0, 4, 5] and r["pages_used"] == 2
    assert r["kv_indices"] == [28, 29, 30, 31, 8]
    assert r["out_cache_loc"] == [9, 10, 11, 36, 4]
    assert r["block_table"].tolist() == [[7, 2, 9], [1, -1, -1]]
    assert not no_page and not bad
