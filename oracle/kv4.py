"""The 4-bit latent cache in plain numpy, fp64 -- test infrastructure.

Written from the row format in ``include/mla_verify.h`` (MLA_VERIFY_KV4): value by value, without the package's
code.  ``encode_rows`` / ``decode_rows`` are the store and the load, ``verify`` is tree-verify attention on decoded
rows, ``build_slots`` the index arrays of a step.
"""

from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E_MIN, E_MAX = -13, 13
ROW_BYTES = 384


def scale_offset(code: int) -> int:
    m, rest = divmod(code, 128)
    q, rest = divmod(rest, 32)
    return 320 + 16 * q + 2 * m + rest // 16


def magnitude_bit(code: int) -> int:
    """First bit (of the row) of a code's 3-bit magnitude."""
    return 32 * (code // 8) + 4 * (code % 8)


def sign_bit(code: int) -> int:
    i = code % 8
    return 32 * (code // 8) + (8 * i + 7 if i < 4 else 8 * (i - 4) + 3)


_SCALE_AT = np.array([scale_offset(c) for c in range(640)])
_MAG_AT = np.array([magnitude_bit(c) for c in range(640)])
_SIGN_AT = np.array([sign_bit(c) for c in range(640)])


def quantise(x: np.ndarray):
    """float64 [n, 16k] -> (magnitude index, negative, exponent per value), by the store's rule."""
    n, w = x.shape
    g = np.where(np.isnan(x), 0.0, x).reshape(n, -1, 16)
    top = np.abs(g).max(-1, keepdims=True)
    e = np.full(top.shape, E_MAX)
    for k in range(E_MAX, E_MIN - 1, -1):  # the least k with top <= 6 * 2^k
        e = np.where(top <= 6.0 * 2.0 ** k, k, e)
    y = np.minimum(np.abs(g) / np.exp2(e.astype(np.float64)), 6.0)
    d = np.abs(y[..., None] - GRID)
    even_first = np.array([0, 2, 4, 6, 1, 3, 5, 7])
    c = even_first[np.argmin(d[..., even_first], axis=-1)]  # argmin keeps the first: the even index
    neg = (g < 0) & (c > 0)
    return c.reshape(n, w), neg.reshape(n, w), np.broadcast_to(e, g.shape).reshape(n, w)


def value(c, neg, e):
    return GRID[c] * np.where(neg, -1.0, 1.0) * np.exp2(e.astype(np.float64))


def encode_rows(latent: np.ndarray, rope: np.ndarray) -> np.ndarray:
    """float64 latents [n, 512], RoPE keys [n, 64] -> uint8 [n, 384]."""
    n = latent.shape[0]
    with np.errstate(invalid="ignore"):
        c0, s0, e0 = quantise(latent)
        c1, s1, e1 = quantise(rope)
        c2, s2, e2 = quantise(rope - value(c1, s1, e1))
    c, s, e = (np.concatenate(t, 1) for t in ((c0, c1, c2), (s0, s1, s2), (e0, e1, e2)))
    bits = np.zeros((n, 2560), np.uint8)
    for k in range(3):
        bits[:, _MAG_AT + k] = (c >> k) & 1
    bits[:, _SIGN_AT] = s
    rows = np.zeros((n, ROW_BYTES), np.uint8)
    rows[:, :320] = np.packbits(bits, axis=1, bitorder="little")
    rows[:, _SCALE_AT] = e + 127
    return rows


def decode_codes(rows: np.ndarray) -> np.ndarray:
    """uint8 [n, 384] -> float64 [n, 640]."""
    bits = np.unpackbits(np.ascontiguousarray(rows[:, :320]), axis=1, bitorder="little").astype(np.int64)
    c = bits[:, _MAG_AT] + 2 * bits[:, _MAG_AT + 1] + 4 * bits[:, _MAG_AT + 2]
    e = np.clip(rows[:, _SCALE_AT].astype(np.int64) - 127, E_MIN, E_MAX)
    return value(c, bits[:, _SIGN_AT] != 0, e)


def decode_rows(rows: np.ndarray) -> np.ndarray:
    """uint8 [n, 384] -> float64 [n, 576]: latents, then RoPE value plus residual."""
    v = decode_codes(rows)
    return np.concatenate([v[:, :512], v[:, 512:576] + v[:, 576:]], 1)


def verify(wl: dict, keys_of=None):
    """Attention of a host workload (its layout: ``workloads``) whose ``pool`` holds 4-bit rows, in fp64.

    Returns (O [n, 512], LSE [n]) for the call's token rows.  ``keys_of(b)`` may name the usable key positions
    (a bool array); by default all are."""
    B, H, T = wl["B"], wl["H"], wl["T"]
    qo = wl.get("qo_indptr")
    qo = np.arange(B + 1) * T if qo is None else np.asarray(qo, np.int64)
    from_bits = lambda a: (a.astype(np.uint32) << 16).view(np.float32).astype(np.float64)  # noqa: E731
    mask_bits = np.unpackbits(np.asarray(wl["custom_mask"], np.uint8), bitorder="little")
    O = np.zeros((int(qo[-1]) * H, 512))
    LSE = np.full(int(qo[-1]) * H, -np.inf)
    for b in range(B):
        t0, t1 = int(qo[b]), int(qo[b + 1])
        if t0 == t1:
            continue
        ids = np.concatenate([wl["kv_indices"][wl["kv_indptr"][b]:wl["kv_indptr"][b + 1]], wl["out_cache_loc"][t0:t1]])
        L = ids.size
        ok = (ids >= 0) & (ids < wl["pool"].shape[0])
        k = np.zeros((L, 576))
        k[ok] = decode_rows(wl["pool"][ids[ok]])
        if keys_of is not None:
            ok &= keys_of(b)
        at = int(wl["mask_indptr"][b])
        vis = mask_bits[at:at + (t1 - t0) * L].reshape(t1 - t0, L).astype(bool) & ok
        q = np.concatenate([from_bits(wl["q_nope"][t0:t1]), from_bits(wl["q_rope"][t0:t1])], -1)
        s = q.reshape(-1, 576) @ k.T * wl["sm_scale"]
        s = np.where(np.repeat(vis, H, axis=0), s, -np.inf)
        m = s.max(-1, keepdims=True)
        some = np.isfinite(m[:, 0])
        p = np.exp(s[some] - m[some])
        l = p.sum(-1)
        rows = slice(t0 * H, t1 * H)
        O[rows][some] = (p @ k[:, :512]) / l[:, None]
        LSE[rows][some] = m[some, 0] + np.log(l)
    return O, LSE


def build_slots(seq_lens, new_lens, page_size, table, free_pages, pool_rows):
    """Index arrays of a step, request by request.  Returns a dict and whether (a page, a row) was missing."""
    table = np.array(table, np.int64)
    kv, qo, kv_idx, loc = [0], [0], [], []
    used = 0
    no_page = bad_row = False
    for b, (P, T) in enumerate(zip(seq_lens, new_lens)):
        P, T = max(0, int(P)), max(0, int(T))
        have = -(-P // page_size)
        for c in range(have, -(-(P + T) // page_size)):
            page = -1
            if used < len(free_pages):
                page = int(free_pages[used])
            else:
                no_page = True
            used += 1
            if c < table.shape[1]:
                table[b, c] = page
        for pos in range(P + T):
            c, r = pos // page_size, -1
            if c >= table.shape[1]:
                no_page = True
            elif table[b, c] >= 0:
                r = int(table[b, c]) * page_size + pos % page_size
                if r >= pool_rows:
                    r, bad_row = -1, True
            elif c < have:
                bad_row = True
            (kv_idx if pos < P else loc).append(r)
        kv.append(kv[-1] + P)
        qo.append(qo[-1] + T)
    return dict(block_table=table, kv_indptr=kv, qo_indptr=qo, kv_indices=kv_idx, out_cache_loc=loc,
                pages_used=min(used, len(free_pages))), no_page, bad_row
