"""The operators of the 4-bit latent cache: cases, inputs, plain forms and 64-bit definitions.

Four operators work on one page_size = 1 pool of 4-bit rows: the slot maps of a step (``slots``), tokens stored
into the pool and read back (``store``), rows read back alone (``load``), and tree-verify attention over the pool
(``verify``).  ``run`` computes them in elementary torch operations in 32 bits, or, where ``own`` is true, through
the package's entry points.

The row (384 bytes): 640 codes of 4 bits in 5 blocks of 128 -- 512 latent channels, 64 RoPE channels, and the
64 RoPE channels' residuals -- then one scale byte (a power of two, exponent + 127) per 16 codes.  A code is a
magnitude of {0, 0.5, 1, 1.5, 2, 3, 4, 6} and a sign.  In each 32-bit word of 8 channels, channel i's magnitude
is bits 4i..4i+2; the signs of channels 0..3 are bits 7, 15, 23, 31 and those of channels 4..7 bits 3, 11, 19, 27.
The scale of codes 128m + 32q + 16h .. + 15 is byte 320 + 16q + 2m + h.
"""

import math

import numpy as np
import torch

own = False

D_LATENT, D_ROPE, ROW = 512, 64, 384
CODES = D_LATENT + 2 * D_ROPE
E_MIN, E_MAX = -13, 13
SM_SCALE = 1.0 / math.sqrt(192.0)


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # the smallest verify call: 16 heads, a chain of 4 drafts behind a short prompt; latency alone
        dict(name="verify_tiny", op="verify", B=1, H=16, T=4, ragged=False, P_lo=256, P_hi=256, pool=4096, holes=False),
        # the headline verify step: a 9-token draft tree, 64 heads, one 4k context
        dict(name="verify_4k", op="verify", B=1, H=64, T=9, ragged=False, P_lo=4096, P_hi=4096, pool=262144, holes=False),
        # the same step deep in a 64k context: bound by the products
        dict(name="verify_64k", op="verify", B=1, H=64, T=9, ragged=False, P_lo=65536, P_hi=65536, pool=1048576, holes=False),
        # one tensor-parallel shard (8 heads) of a very long context: bound by reading the cache
        dict(name="verify_185k_h8", op="verify", B=1, H=8, T=9, ragged=False, P_lo=185000, P_hi=185000, pool=1048576, holes=False),
        # a serving batch whose requests draft 0 to 16 tokens each, some of them padding that sees nothing
        dict(name="verify_varlen_b16", op="verify", B=16, H=64, T=16, ragged=True, P_lo=1024, P_hi=32768, pool=1048576, holes=True),
        # single-token decode of a batch on one tensor-parallel shard
        dict(name="decode_h8_b16", op="verify", B=16, H=8, T=1, ragged=False, P_lo=1024, P_hi=32768, pool=1048576, holes=False),
        # the drafts of one batched verify step written into the cache (and read back)
        dict(name="store_step", op="store", n=144, pool=262144, pad=0),
        # a prompt written into the cache, some of its rows padding without a slot
        dict(name="store_prompt", op="store", n=32768, pool=1048576, pad=37),
        # a short shared prefix read back
        dict(name="load_257", op="load", n=257, pool=65536),
        # a long context read back, e.g. to recompute with it in bf16
        dict(name="load_64k", op="load", n=65545, pool=1048576),
        # the index arrays of one batched verify step, rows allocated one by one
        dict(name="slots_step", op="slots", B=16, T=9, P_lo=1024, P_hi=32768, page=1),
        # the index arrays of a large batch with pages of 64 rows, new requests among it
        dict(name="slots_b512", op="slots", B=512, T=16, P_lo=0, P_hi=8191, page=64),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["verify", "verify", "verify", "store", "load", "slots"])
    if op == "verify":
        while True:
            B, H, T = _log(rng, 1, 32), rng.choice([1, 5, 8, 13, 16, 32, 64, 128]), rng.randint(1, 16)
            hi = _log(rng, 16, 185000)
            lo = rng.choice([hi, rng.randint(0, hi), max(0, hi // 32)])
            # no more products, keys or padded scores than the largest listed case has
            if B * T * H * (hi + T) <= 4.0e8 and B * (hi + T) <= 360000 and T * H <= 1024:
                break
        need = B * (hi + T)
        return dict(op=op, B=B, H=H, T=T, ragged=rng.random() < 0.5, P_lo=lo, P_hi=hi,
                    pool=need + _log(rng, 1, 500000), holes=rng.random() < 0.3)
    if op == "slots":
        B = _log(rng, 1, 1024)
        hi = _log(rng, 1, max(1, 4000000 // B))
        return dict(op=op, B=B, T=rng.randint(1, 64), P_lo=rng.randint(0, hi), P_hi=hi,
                    page=rng.choice([1, 1, 5, 16, 64, 256]))
    n = _log(rng, 1, 65536 if op == "load" else 32768)
    case = dict(op=op, n=n, pool=n + _log(rng, 1, 900000))
    if op == "store":
        case["pad"] = rng.choice([0, rng.randint(0, n - 1)])
    return case


# ---- inputs -------------------------------------------------------------------

def _tokens(n, g):
    """Latents after their norm (channels of unequal spread) and rotated keys, one bf16 [n, 576] projection output."""
    x = torch.randn((n, D_LATENT + D_ROPE), generator=g, device="cuda")
    spread = torch.exp(0.35 * torch.randn((D_LATENT + D_ROPE,), generator=g, device="cuda"))
    return (x * spread).to(torch.bfloat16)


def _noise_pool(rows, g):
    """Rows that nothing refers to hold anything."""
    words = torch.randint(-(2 ** 31), 2 ** 31 - 1, (rows, ROW // 4), generator=g, device="cuda", dtype=torch.int32)
    return words.view(torch.uint8).view(rows, ROW)


def _lengths(case):
    """Cached and new tokens of each request: the same for every seed, as they are the case's sizes."""
    B, T = case["B"], case["T"]
    r = np.random.default_rng([B, T, case["P_lo"], case["P_hi"]])
    P = r.integers(case["P_lo"], case["P_hi"] + 1, B).astype(np.int64)
    if case["op"] == "slots":
        return P, r.integers(1, T + 1, B).astype(np.int64)
    if not case["ragged"]:
        return P, np.full(B, T, np.int64)
    Tn = r.integers(0, T + 1, B).astype(np.int64)
    Tn[0] = max(Tn[0], 1)
    return P, Tn


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _prepare_verify(case, g, r):
    B, H, T = case["B"], case["H"], case["T"]
    P, Tn = _lengths(case)
    L = P + Tn
    n_tok, n_pre = int(Tn.sum()), int(P.sum())
    rows = torch.randperm(case["pool"], generator=g, device="cuda")[:n_pre + n_tok].to(torch.int32)
    pool = _noise_pool(case["pool"], g)
    step = 1 << 17
    for s in range(0, n_pre + n_tok, step):
        at = rows[s:s + step].long()
        tok = _tokens(at.numel(), g)
        pool[at] = _pack(tok[:, :D_LATENT].float(), tok[:, D_LATENT:].float())
    # visibility: the whole prefix and the ancestors in a random draft tree, packed LSB first
    bits, mask_start = [], np.zeros(B, np.int64)
    total = 0
    for b in range(B):
        t = int(Tn[b])
        see = np.zeros((t, t), bool)
        for i in range(t):
            if i:
                see[i] = see[int(r.integers(0, i))]
            see[i, i] = True
        m = np.ones((t, int(L[b])), bool)
        m[:, int(P[b]):] = see
        if case["holes"] and t:
            m[r.random(t) < 0.15] = False
        mask_start[b] = total
        total += m.size
        bits.append(m.reshape(-1))
    mask = np.packbits(np.concatenate(bits), bitorder="little")
    loc = torch.zeros(B * T, dtype=torch.int32, device="cuda")
    loc[:n_tok] = rows[n_pre:]
    s = dict(op="verify", B=B, H=H, T=T, n_tok=n_tok, L_max=int(L.max()), pool_rows=case["pool"], kv_pool=pool,
             q_nope=torch.randn((B * T, H, D_LATENT), generator=g, device="cuda").to(torch.bfloat16),
             q_rope=torch.randn((B * T, H, D_ROPE), generator=g, device="cuda").to(torch.bfloat16),
             kv_indptr=_dev(np.concatenate([[0], np.cumsum(P)])), qo_indptr=_dev(np.concatenate([[0], np.cumsum(Tn)])),
             kv_indices=rows[:max(1, n_pre)].clone(), out_cache_loc=loc, mask_indptr=_dev(mask_start),
             custom_mask=torch.from_numpy(mask).cuda())
    s["o"] = torch.empty((B * T, H, D_LATENT), dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.empty((B * T, H), dtype=torch.float32, device="cuda")
    if own:
        from mla_speculative_decode_tree_gb300 import binding as M
        s["plan"] = M.mla_verify_plan(B, H, T, max(T, s["L_max"]), case["pool"], 0, flags=M.MLA_VERIFY_KV4)
        s["workspace"] = torch.zeros(s["plan"].workspace_bytes, dtype=torch.uint8, device="cuda")
    return s


def _prepare_rows(case, g, r):
    n, pool = case["n"], case["pool"]
    tok = _tokens(n, g)
    rows = torch.randperm(pool, generator=g, device="cuda")[:n].to(torch.int32)
    s = dict(op=case["op"], n=n, pool_rows=pool, kv_pool=_noise_pool(pool + 1, g), slots=rows, read=rows,
             out=torch.zeros((n, D_LATENT + D_ROPE), dtype=torch.bfloat16, device="cuda"))
    if case["op"] == "load":
        s["kv_pool"][rows.long()] = _pack(tok[:, :D_LATENT].float(), tok[:, D_LATENT:].float())
    else:
        s["tokens"] = tok
        if case["pad"]:  # padding tokens have no slot; reading a row of theirs back reads nothing
            s["slots"] = rows.clone()
            s["slots"][torch.from_numpy(r.choice(n, case["pad"], replace=False)).cuda()] = -1
            s["read"] = s["slots"]
    if own:
        from mla_speculative_decode_tree_gb300 import binding as M
        s["plan"] = M.mla_verify_plan(1, 1, 1, 1, pool, 1, flags=M.MLA_VERIFY_KV4)
        s["workspace"] = torch.zeros(s["plan"].workspace_bytes, dtype=torch.uint8, device="cuda")
    return s


def _prepare_slots(case, g, r):
    B, page = case["B"], case["page"]
    P, Tn = _lengths(case)
    have, want = -(-P // page), -(-(P + Tn) // page)
    max_pages = int(want.max()) + 3
    num_pages = int(want.sum()) + 64
    order = r.permutation(num_pages).astype(np.int32)
    table = np.full((B, max_pages), -1, np.int32)
    held = np.arange(max_pages)[None, :] < have[:, None]
    table[held] = order[:int(have.sum())]
    free = order[int(have.sum()):]
    s = dict(op="slots", B=B, page=page, max_pages=max_pages, n_pre=int(P.sum()), n_tok=int(Tn.sum()),
             pool_rows=num_pages * page, seq_lens=_dev(P), new_lens=_dev(Tn), block_table=_dev(table), free_pages=_dev(free))
    for name, size in (("kv_indptr", B + 1), ("qo_indptr", B + 1), ("kv_indices", s["n_pre"] + 1),
                       ("out_cache_loc", s["n_tok"]), ("pages_used", 1)):
        s[name] = torch.zeros(size, dtype=torch.int32, device="cuda")
    if own:
        from mla_speculative_decode_tree_gb300 import binding as M
        s["plan"] = M.mla_verify_plan(B, 1, 1, int((P + Tn).max()), s["pool_rows"], 1, flags=M.MLA_VERIFY_KV4)
        s["workspace"] = torch.zeros(s["plan"].workspace_bytes, dtype=torch.uint8, device="cuda")
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = np.random.default_rng(seed)
    return {"verify": _prepare_verify, "store": _prepare_rows, "load": _prepare_rows,
            "slots": _prepare_slots}[case["op"]](case, g, r)


# ---- the 4-bit row in elementary operations -------------------------------------

def _pow2(e):
    """Exact fp32 powers of two of int32 exponents in [-126, 127]."""
    return ((e + 127) << 23).view(torch.float32)


def _encode(x):
    """fp32 [n, k*16] -> (magnitude codes, signs, exponents, values)."""
    n = x.shape[0]
    v = x.view(n, -1, 16)
    a = v.abs().amax(-1)
    m, e = torch.frexp(a)  # a = m * 2^e, m in [0.5, 1): a <= 6 * 2^k for k = e - 3 + (m > 0.75)
    e = torch.where(a > 0, e - 3 + (m > 0.75).to(e.dtype), torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)
    y = v.abs() * _pow2(-e.unsqueeze(-1))
    # nearest of 0 .5 1 1.5 2 3 4 6; at a midpoint the even code
    c = ((y > 0.25).int() + (y >= 0.75).int() + (y > 1.25).int() + (y >= 1.75).int()
         + (y > 2.5).int() + (y >= 3.5).int() + (y > 5.0).int())
    neg = ((v < 0) & (c > 0)).int()
    return c.view(n, -1), neg.view(n, -1), e, _values(c, neg, e.unsqueeze(-1)).view(n, -1)


def _values(c, neg, e):
    """Magnitude codes, signs and exponents -> fp32 values."""
    half = torch.where(c < 4, c, torch.where(c < 6, 2 * c - 4, 4 * c - 16)).float()  # twice the magnitude
    return half * (1 - 2 * neg).float() * _pow2(e - 1)


def _pack(latent, rope):
    """fp32 latents [n, 512] and RoPE keys [n, 64] -> uint8 rows [n, 384]."""
    n = latent.shape[0]
    cl, nl, el, _ = _encode(latent)
    cr, nr, er, vr = _encode(rope)
    cs, ns, es, _ = _encode(rope - vr)
    c = torch.cat([cl, cr, cs], 1).view(n, CODES // 8, 2, 4)
    neg = torch.cat([nl, nr, ns], 1).view(n, CODES // 8, 2, 4)
    at = torch.arange(4, device=c.device)
    # byte k of a word: magnitudes of channels 2k, 2k+1; signs of channels k (bit 7) and k + 4 (bit 3)
    byte = c.view(n, CODES // 8, 4, 2)[..., 0] | (c.view(n, CODES // 8, 4, 2)[..., 1] << 4)
    byte = byte | (neg[:, :, 0, at] << 7) | (neg[:, :, 1, at] << 3)
    # scales: groups 8m + 2q + h -> byte 16q + 2m + h
    e = torch.cat([el, er, es], 1).view(n, 5, 4, 2).permute(0, 2, 1, 3).reshape(n, 4, 10)
    pad = torch.zeros((n, 4, 6), dtype=torch.uint8, device=c.device)
    scales = torch.cat([(e + 127).to(torch.uint8), pad], 2).view(n, 64)
    return torch.cat([byte.to(torch.uint8).view(n, CODES // 2), scales], 1)


def _unpack(rows):
    """uint8 rows [n, 384] -> fp32 [n, 576]: latents, then RoPE value plus residual."""
    n = rows.shape[0]
    byte = rows[:, :CODES // 2].int().view(n, CODES // 8, 4)
    c = torch.stack([byte & 7, (byte >> 4) & 7], -1).view(n, CODES // 8, 8)
    neg = torch.cat([byte >> 7, (byte >> 3) & 1], -1)
    e = rows[:, CODES // 2:].view(n, 4, 16)[:, :, :10].int().view(n, 4, 5, 2).permute(0, 2, 1, 3).reshape(n, 40, 1)
    v = _values(c.view(n, 40, 16), neg.view(n, 40, 16), (e - 127).clamp(E_MIN, E_MAX)).view(n, CODES)
    return torch.cat([v[:, :D_LATENT], v[:, D_LATENT:D_LATENT + D_ROPE] + v[:, D_LATENT + D_ROPE:]], 1)


# ---- plain forms ------------------------------------------------------------------

def _plain_verify(s):
    B, H, T, L_max, n = s["B"], s["H"], s["T"], s["L_max"], s["n_tok"]
    kv0, qo0 = s["kv_indptr"][:-1].long()[:, None], s["qo_indptr"][:-1].long()[:, None]
    P = s["kv_indptr"][1:].long()[:, None] - kv0
    Tn = s["qo_indptr"][1:].long()[:, None] - qo0
    j = torch.arange(L_max, device="cuda")[None, :]
    pre = s["kv_indices"].long()[(kv0 + j).clamp(0, s["kv_indices"].numel() - 1)]
    new = s["out_cache_loc"].long()[(qo0 + j - P).clamp(0, B * T - 1)]
    rows = torch.where(j < P, pre, new)
    k = _unpack(s["kv_pool"][rows.view(-1)]).view(B, L_max, D_LATENT + D_ROPE)
    i = torch.arange(T, device="cuda")[None, :]
    at = (qo0 + i).clamp(0, B * T - 1).view(-1)
    q = torch.cat([s["q_nope"][at], s["q_rope"][at]], -1).float().view(B, T * H, D_LATENT + D_ROPE)
    bit = s["mask_indptr"].long()[:, None, None] + i[:, :, None] * (P + Tn)[:, :, None] + j[:, None, :]
    inside = (j < P + Tn)[:, None, :] & (i < Tn)[:, :, None]
    bit = torch.where(inside, bit, torch.zeros_like(bit))
    sees = ((s["custom_mask"][bit >> 3].int() >> (bit & 7).int()) & 1).bool() & inside
    sc = (torch.bmm(q, k.transpose(1, 2)) * SM_SCALE).view(B, T, H, L_max)
    sc = sc.masked_fill_(~sees[:, :, None, :], -math.inf)
    top = sc.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = sc.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.bmm(p.view(B, T * H, L_max), k[:, :, :D_LATENT]).view(B, T, H, D_LATENT)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (top + torch.log(total)).squeeze(-1)  # log(0) is -inf: nothing seen
    tok = torch.arange(n, device="cuda")
    b = torch.searchsorted(s["qo_indptr"][1:].long(), tok, right=True)
    i = tok - s["qo_indptr"].long()[b]
    return o[b, i].to(torch.bfloat16), lse[b, i]


def _plain_store(s):
    rows = _pack(s["tokens"][:, :D_LATENT].float(), s["tokens"][:, D_LATENT:].float())
    # a token without a slot is not stored: its place goes to a row past the pool's end
    at = torch.where(s["slots"] >= 0, s["slots"], s["pool_rows"]).long()
    s["kv_pool"][at] = rows
    return _plain_load(s["kv_pool"], s["read"])


def _plain_load(pool, read):
    x = _unpack(pool[read.clamp(min=0).long()])
    return torch.where(read[:, None] >= 0, x, torch.zeros_like(x)).to(torch.bfloat16)


def _plain_slots(s):
    B, page = s["B"], s["page"]
    P, Tn = s["seq_lens"].long(), s["new_lens"].long()
    zero = torch.zeros(1, dtype=torch.long, device="cuda")
    kv, qo = torch.cat([zero, P.cumsum(0)]), torch.cat([zero, Tn.cumsum(0)])
    have, want = (P + page - 1) // page, (P + Tn + page - 1) // page
    first = torch.cat([zero, (want - have).cumsum(0)])
    c = torch.arange(s["max_pages"], device="cuda")[None, :]
    fresh = (c >= have[:, None]) & (c < want[:, None])
    pick = (first[:-1, None] + c - have[:, None]).clamp(0, s["free_pages"].numel() - 1)
    table = torch.where(fresh, s["free_pages"][pick], s["block_table"])

    def rows(start, n, offset):
        x = torch.arange(n, device="cuda")
        b = torch.searchsorted(start[1:], x, right=True)
        pos = x - start[b] + offset[b]
        return (table[b, pos // page] * page + pos % page).to(torch.int32)

    return dict(block_table=table, kv_indptr=kv.to(torch.int32), qo_indptr=qo.to(torch.int32),
                kv_indices=rows(kv, s["n_pre"], torch.zeros_like(P)), out_cache_loc=rows(qo, s["n_tok"], P),
                pages_used=first[-1:].to(torch.int32))


# ---- one pass -----------------------------------------------------------------------

def run(state):
    s, op = state, state["op"]
    if not own:
        if op == "verify":
            return _plain_verify(s)
        if op == "store":
            return _plain_store(s)
        return _plain_load(s["kv_pool"], s["read"]) if op == "load" else _plain_slots(s)
    from mla_speculative_decode_tree_gb300 import binding as M
    if op == "verify":
        M.mla_verify_run_varlen(s["plan"], s["q_nope"], s["q_rope"], s["kv_pool"], s["kv_indptr"], s["kv_indices"],
                                s["qo_indptr"], s["out_cache_loc"], s["custom_mask"], s["mask_indptr"], s["B"],
                                SM_SCALE, 0, s["workspace"], s["o"], s["lse"])
        return s["o"][:s["n_tok"]], s["lse"][:s["n_tok"]]
    if op == "slots":
        M.mla_verify_build_slots(s["plan"], s["seq_lens"], s["new_lens"], s["B"], s["page"], s["block_table"],
                                 s["free_pages"], s["pages_used"], s["kv_indptr"], s["kv_indices"], s["qo_indptr"],
                                 s["out_cache_loc"], s["workspace"])
        return dict(block_table=s["block_table"], kv_indptr=s["kv_indptr"], qo_indptr=s["qo_indptr"],
                    kv_indices=s["kv_indices"][:s["n_pre"]], out_cache_loc=s["out_cache_loc"],
                    pages_used=s["pages_used"])
    if op == "store":
        M.mla_verify_store_kv4(s["plan"], s["tokens"][:, :D_LATENT], s["tokens"][:, D_LATENT:], s["slots"],
                               s["kv_pool"], s["workspace"])
    M.mla_verify_load_kv4(s["plan"], s["kv_pool"], s["read"], s["out"][:, :D_LATENT], s["out"][:, D_LATENT:],
                          s["workspace"])
    return s["out"]


# ---- what a pass cannot do without -----------------------------------------------------

def work(case):
    if case["op"] == "verify":
        (P, Tn), H = _lengths(case), case["H"]
        keys, tokens = int((P + Tn).sum()), int(Tn.sum())
        pairs = int((Tn * (P + Tn)).sum())
        return {"bytes": keys * (360 + 4) + pairs / 8 + tokens * H * (1152 + 1024 + 4), "flops": 2.0 * (576 + 512) * H * pairs}
    if case["op"] == "slots":
        (P, Tn), page = _lengths(case), case["page"]
        pages = int((-(-(P + Tn) // page)).sum())
        return {"bytes": 4.0 * (int(P.sum()) + int(Tn.sum()) + pages + 4 * case["B"]), "flops": 0}
    n = case["n"]
    read_back = 360 + 4 + 1152
    return {"bytes": n * (read_back if case["op"] == "load" else read_back + 1152 + 4 + 360), "flops": 0}


# ---- the definitions in 64 bits -----------------------------------------------------------

_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _exact_rows(rows):
    """uint8 rows -> float64 [n, 576], code by code from the row's definition."""
    n = rows.shape[0]
    word = rows[:, :320].contiguous().view(torch.int32).long().view(n, 80, 1)
    ch = torch.arange(8, device=rows.device)
    sign_at = torch.where(ch < 4, 8 * ch + 7, 8 * (ch - 4) + 3)
    grid = torch.tensor(_GRID, dtype=torch.float64, device=rows.device)
    v = grid[(word >> (4 * ch)) & 7] * (1 - 2 * ((word >> sign_at) & 1)).double()
    code = torch.arange(640, device=rows.device)
    at = 320 + 16 * (code % 128 // 32) + 2 * (code // 128) + code % 32 // 16
    powers = torch.tensor([2.0 ** (k - 127) for k in range(256)], dtype=torch.float64, device=rows.device)
    v = v.view(n, 640) * powers[rows[:, at].long()]
    return torch.cat([v[:, :512], v[:, 512:576] + v[:, 576:]], 1)


def _exact_round(x):
    """float64 [n, 16k] -> the values that the 4-bit code of each group of 16 stands for."""
    v = x.view(x.shape[0], -1, 16)
    powers = torch.tensor([2.0 ** k for k in range(E_MIN, E_MAX + 1)], dtype=torch.float64, device=x.device)
    big = (v.abs().amax(-1, keepdim=True) > 6 * powers).sum(-1, keepdim=True).clamp(max=E_MAX - E_MIN)
    scale = powers[big]
    grid = torch.tensor(_GRID, dtype=torch.float64, device=x.device)
    best, val = torch.full_like(v, math.inf), torch.zeros_like(v)
    for k in (0, 2, 4, 6, 1, 3, 5, 7):  # even codes first: a tie keeps the even one
        d = (v.abs() / scale - grid[k]).abs()
        val = torch.where(d < best, grid[k].expand_as(v), val)
        best = torch.minimum(best, d)
    return (val * scale * torch.sign(v)).view_as(x)


def _exact_verify(s):
    n, H = s["n_tok"], s["H"]
    o = torch.zeros((n, H, D_LATENT), dtype=torch.float64, device="cuda")
    lse = torch.full((n, H), -math.inf, dtype=torch.float64, device="cuda")
    kv, qo, start = s["kv_indptr"].tolist(), s["qo_indptr"].tolist(), s["mask_indptr"].tolist()
    for b in range(s["B"]):
        t0, t1 = qo[b], qo[b + 1]
        if t0 == t1:
            continue
        rows = torch.cat([s["kv_indices"][kv[b]:kv[b + 1]], s["out_cache_loc"][t0:t1]]).long()
        L = rows.numel()
        k = _exact_rows(s["kv_pool"][rows])
        q = torch.cat([s["q_nope"][t0:t1], s["q_rope"][t0:t1]], -1).double()
        sc = (q.view(-1, 576) @ k.T).view(t1 - t0, H, L) * SM_SCALE
        bit = start[b] + torch.arange((t1 - t0) * L, device="cuda")
        sees = ((s["custom_mask"][bit // 8].long() >> (bit % 8)) & 1).bool().view(t1 - t0, 1, L)
        some = sees.any(-1).squeeze(-1)
        if not bool(some.any()):
            continue
        sc = sc.masked_fill(~sees, -math.inf)[some]
        lse[t0:t1][some] = torch.logsumexp(sc, -1)
        o[t0:t1][some] = (torch.softmax(sc, -1).view(-1, L) @ k[:, :512]).view(-1, H, 512)
    return o, lse


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "verify":
        return _exact_verify(s)
    if op == "load":
        return _exact_rows(s["kv_pool"][s["read"].long()])
    if op == "store":
        x = s["tokens"].double()
        rope = _exact_round(x[:, 512:])
        y = torch.cat([_exact_round(x[:, :512]), rope + _exact_round(x[:, 512:] - rope)], 1)
        return torch.where(s["read"][:, None] >= 0, y, torch.zeros_like(y))
    return None  # whole numbers
