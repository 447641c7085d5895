"""Operators of a step over shared prefixes: cases, inputs, plain forms and 64-bit definitions.

Four operators of speculative decoding, from the attention to the pages that are left behind it:

``shared``   tree-verify attention for requests in groups, each group with one prefix that is read once for all of
             its requests, and each request with keys of its own behind it;
``accept``   the draft trees' tokens verified against the target's probabilities, from given random numbers;
``commit``   the accepted path's cache rows moved to the front of the new ones, in every layer, with the lengths and
             the pages' reference counts;
``turnover`` requests forked (pages shared, the last one copied where it is not full), then released, on a free list
             that is made from the reference counts.

``run`` computes them in elementary torch operations, or, where ``own`` is true, through the package's entry points.

Verification is defined in whole numbers, so that no order of summation changes a token.  Probabilities are held as
round(p * 2^38), random numbers as k = floor(u * 2^24).  The walk starts at node 0 of a request's tree with r = p(node)
and Z = 2^38.  The children of the node that the walk is at are tried in ascending order: with s = q(node) * Z >> 38
(without draft probabilities: Z at the child's token, else 0) child c with token x is accepted when k[c] * s(x) <
r(x) * 2^24.  Then the walk goes on from c, else Z = max(Z - sum(min(r, s)), 0) and r = max(r - s, 0).  The next token is the first
one at which the running sum of r exceeds floor(k * sum(r) / 2^24).
"""

import math

import numpy as np
import torch

own = False

D_LATENT, D_ROPE = 512, 64
D_ROW = D_LATENT + D_ROPE
SM_SCALE = 1.0 / math.sqrt(192.0)
ONE = 38  # bits of a probability
KV4_ROW = 384


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # the smallest call: four requests behind a short system prompt, two drafts each; latency alone
        dict(name="shared_tiny", op="shared", groups=1, per=4, H=16, T=2, ragged=False, S_lo=256, S_hi=256, P_lo=8, P_hi=40),
        # single-token decode of 64 requests on one tensor-parallel shard (8 heads) behind a 32k document
        dict(name="shared_decode_h8", op="shared", groups=1, per=64, H=8, T=1, ragged=False, S_lo=32768, S_hi=32768, P_lo=64, P_hi=2048),
        # a verify step of a batch behind a prompt with many examples
        dict(name="shared_verify_8k", op="shared", groups=1, per=16, H=64, T=9, ragged=False, S_lo=8192, S_hi=8192, P_lo=128, P_hi=1024),
        # decode behind a very long common context: bound by the products
        dict(name="shared_decode_128k", op="shared", groups=1, per=32, H=64, T=1, ragged=False, S_lo=131072, S_hi=131072, P_lo=512, P_hi=4096),
        # several prompts at once, each with its samples; requests draft 0 to 8 tokens
        dict(name="shared_groups", op="shared", groups=8, per=4, H=32, T=8, ragged=True, S_lo=1000, S_hi=30000, P_lo=0, P_hi=700),
        # one request's chain of 5 drafts, fixed (not drawn): only the target's probabilities count
        dict(name="accept_one", op="accept", B=1, T=6, ragged=False, V=32000, drawn=False),
        # the headline draft tree (9 nodes) for a batch, drafts drawn from the draft model
        dict(name="accept_b16", op="accept", B=16, T=9, ragged=False, V=131072, drawn=True),
        # a large batch with trees of up to 16 nodes and an odd vocabulary
        dict(name="accept_b64", op="accept", B=64, T=16, ragged=True, V=150001, drawn=True),
        # a batched step's accepted rows in one pool
        dict(name="commit_step", op="commit", B=16, T=9, layers=1, page=1, kv4=False, P_lo=1024, P_hi=32768),
        # a large batch, all layers of a model, 4-bit rows in pages of 64
        dict(name="commit_layers", op="commit", B=256, T=16, layers=32, page=64, kv4=True, P_lo=0, P_hi=8191),
        # four samples forked from one prompt: a small pool
        dict(name="turnover_4", op="turnover", n=4, sources=1, page=16, layers=1, kv4=False, P_lo=700, P_hi=700, pages=2048),
        # many forks of long requests in a larger pool, several layers at once
        dict(name="turnover_64", op="turnover", n=64, sources=8, page=64, layers=8, kv4=False, P_lo=2000, P_hi=20000, pages=2600),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["shared", "shared", "shared", "accept", "accept", "commit", "turnover"])
    if op == "shared":
        while True:
            case = dict(op=op, groups=_log(rng, 1, 24), per=_log(rng, 1, 64), H=rng.choice([1, 5, 8, 16, 32, 64, 128]),
                        T=rng.choice([1, 1, rng.randint(1, 16)]), ragged=rng.random() < 0.4)
            hi = _log(rng, 1, 131072)
            case.update(S_lo=rng.choice([hi, rng.randint(0, hi)]), S_hi=hi)
            hi = _log(rng, 1, 4096)
            case.update(P_lo=rng.choice([hi, rng.randint(0, hi)]), P_hi=hi)
            B, rows = case["groups"] * case["per"], case["per"] * case["T"] * case["H"]
            if (work(case)["flops"] <= 5.8e11 and B <= 256 and rows * case["S_hi"] <= 2.7e8
                    and B * case["T"] * case["H"] * (case["P_hi"] + case["T"]) <= 2.7e8
                    and case["groups"] * case["S_hi"] + B * (case["P_hi"] + case["T"]) <= 400000):
                return case
    if op == "accept":
        while True:
            case = dict(op=op, B=_log(rng, 1, 128), T=rng.choice([1, rng.randint(1, 16), rng.randint(1, 32)]),
                        ragged=rng.random() < 0.5, V=_log(rng, 100, 200000), drawn=rng.random() < 0.6)
            if case["B"] * case["T"] * case["V"] <= 1.5e8:
                return case
    page = rng.choice([1, 5, 16, 64, 256])
    kv4 = rng.random() < 0.4
    if op == "commit":
        while True:
            case = dict(op=op, B=_log(rng, 1, 512), T=rng.randint(1, 32), layers=_log(rng, 1, 48), page=page, kv4=kv4)
            if case["B"] * case["T"] * case["layers"] <= 131072:
                hi = _log(rng, 1, 32768)
                return dict(case, P_lo=rng.randint(0, hi), P_hi=hi)
    while True:
        hi = _log(rng, 1, 20000)
        case = dict(op=op, n=_log(rng, 1, 64), sources=_log(rng, 1, 16), page=page, layers=_log(rng, 1, 32), kv4=kv4,
                    P_lo=rng.randint(0, hi), P_hi=hi)
        need = case["sources"] * -(-hi // page) + case["n"]
        case["pages"] = need + _log(rng, 1, max(2, need))
        if case["pages"] * page * case["layers"] <= 1.3e6:
            return case


# ---- inputs -------------------------------------------------------------------

def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _scan(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int64)


def _sizes(case):
    """Shared, own and new tokens: the same for every seed, as they are the case's sizes."""
    G, B = case["groups"], case["groups"] * case["per"]
    r = np.random.default_rng([G, B, case["T"], case["S_lo"], case["S_hi"], case["P_lo"], case["P_hi"]])
    S = r.integers(case["S_lo"], case["S_hi"] + 1, G).astype(np.int64)
    P = r.integers(case["P_lo"], case["P_hi"] + 1, B).astype(np.int64)
    T = np.full(B, case["T"], np.int64)
    if case["ragged"]:
        T = r.integers(0, case["T"] + 1, B).astype(np.int64)
        T[0] = max(T[0], 1)
    return S, P, T


def _tokens(n, g):
    """Latents after their norm (channels of unequal spread) and rotated keys, as a projection leaves them."""
    x = torch.randn((n, D_ROW), generator=g, device="cuda")
    spread = torch.exp(0.35 * torch.randn((D_ROW,), generator=g, device="cuda"))
    return (x * spread).to(torch.bfloat16)


def _trees(T, r):
    """Parents of random draft trees, node 0 the root, one after the other."""
    return [np.array([-1] + [int(r.integers(0, i)) for i in range(1, t)][:max(0, t - 1)], np.int64)[:t] for t in T.tolist()]


def _prepare_shared(case, g, r):
    G, per, H, T = case["groups"], case["per"], case["H"], case["T"]
    B = G * per
    S, P, Tn = _sizes(case)
    L = P + Tn
    n_sh, n_pre, n_tok = int(S.sum()), int(P.sum()), int(Tn.sum())
    need = n_sh + n_pre + n_tok
    pool_rows = need + need // 4 + 16
    rows = torch.randperm(pool_rows, generator=g, device="cuda")[:need].to(torch.int32)
    pool = _tokens(pool_rows, g)
    bits, start, total = [], np.zeros(B, np.int64), 0
    for b, tree in enumerate(_trees(Tn, r)):  # the own prefix and the ancestors, packed LSB first
        t = int(Tn[b])
        m = np.ones((t, int(L[b])), bool)
        see = np.eye(t, dtype=bool)
        for i in range(1, t):
            see[i] |= see[tree[i]]
        m[:, int(P[b]):] = see
        start[b] = total
        total += m.size
        bits.append(m.reshape(-1))
    mask = np.packbits(np.concatenate(bits + [np.zeros(8, bool)]), bitorder="little")
    loc = torch.zeros(B * T, dtype=torch.int32, device="cuda")
    loc[:n_tok] = rows[n_sh + n_pre:]
    s = dict(op="shared", G=G, B=B, H=H, T=T, n_tok=n_tok, S=S.tolist(), L_max=int(L.max()), qo=_scan(Tn).tolist(), per=per,
             pool_rows=pool_rows, kv_pool=pool, group_indptr=_dev(np.arange(G + 1) * per), shared_indptr=_dev(_scan(S)),
             shared_indices=rows[:max(1, n_sh)].clone(), kv_indptr=_dev(_scan(P)),
             kv_indices=rows[n_sh:n_sh + max(1, n_pre)].clone(), qo_indptr=_dev(_scan(Tn)), out_cache_loc=loc,
             mask_indptr=_dev(start), custom_mask=torch.from_numpy(mask).cuda(),
             q_nope=torch.randn((B * T, H, D_LATENT), generator=g, device="cuda").to(torch.bfloat16),
             q_rope=torch.randn((B * T, H, D_ROPE), generator=g, device="cuda").to(torch.bfloat16),
             o=torch.empty((B * T, H, D_LATENT), dtype=torch.bfloat16, device="cuda"),
             lse=torch.empty((B * T, H), dtype=torch.float32, device="cuda"))
    if own:
        from mla_speculative_decode_tree_gb300 import binding as M
        s["plan"] = M.mla_verify_plan(B, H, T, s["L_max"] if s["L_max"] > T else T, pool_rows, 0, flags=M.MLA_VERIFY_SHARED)
        s["workspace"] = torch.zeros(s["plan"].workspace_bytes, dtype=torch.uint8, device="cuda")
    return s


def _prepare_accept(case, g, r):
    B, T, V = case["B"], case["T"], case["V"]
    size = np.random.default_rng([B, T, V])
    Tn = size.integers(0, T + 1, B).astype(np.int64) if case["ragged"] else np.full(B, T, np.int64)
    Tn[0] = max(Tn[0], 1)
    qo, n = _scan(Tn), int(Tn.sum())
    trees = _trees(Tn, r)
    # a target of a few likely tokens before a long tail, and a draft model near it
    target = torch.empty((B * T, V), dtype=torch.float32, device="cuda")
    draft = torch.empty((B * T, V), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 26) // V)
    for a in range(0, B * T, step):
        z = 2.5 * torch.randn((min(step, B * T - a), V), generator=g, device="cuda")
        target[a:a + step] = torch.softmax(z, -1)
        draft[a:a + step] = torch.softmax(z + 0.7 * torch.randn(z.shape, generator=g, device="cuda"), -1)
    at = np.concatenate([qo[b] + np.maximum(t, 0) for b, t in enumerate(trees)]).astype(np.int64)  # each node's parent's row
    tokens = torch.zeros(B * T, dtype=torch.int32, device="cuda")
    edge = torch.from_numpy(at).cuda()
    for a in range(0, n, step):
        tokens[a:min(n, a + step)] = torch.multinomial(draft[edge[a:a + step]], 1, generator=g).view(-1).to(torch.int32)
    if not case["drawn"]:
        draft = None
    parents = np.full(B * T, -1, np.int64)
    parents[:n] = np.concatenate(trees)
    s = dict(op="accept", B=B, T=T, V=V, target=target, draft=draft, tokens=tokens, parents=_dev(parents), qo_indptr=_dev(qo),
             u=torch.rand(B * T, generator=g, device="cuda"), u_next=torch.rand(B, generator=g, device="cuda"),
             accepted=torch.zeros((B, T), dtype=torch.int32, device="cuda"),
             num_accepted=torch.zeros(B, dtype=torch.int32, device="cuda"),
             next_tokens=torch.zeros(B, dtype=torch.int32, device="cuda"))
    if own:
        from mla_speculative_decode_tree_gb300 import binding as M
        s["plan"] = M.mla_verify_plan(B, 1, T, T, 1, 1)
        s["workspace"] = torch.zeros(s["plan"].workspace_bytes, dtype=torch.uint8, device="cuda")
    return s


def _pool(layers, rows, kv4, g):
    if kv4:
        x = torch.randint(0, 2 ** 31 - 1, (layers, rows, KV4_ROW // 4), generator=g, device="cuda", dtype=torch.int32)
        return x.view(torch.uint8)
    return torch.randn((layers, rows, D_ROW), generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _page_plan(case, s, max_batch, T, pool_rows):
    if own:
        from mla_speculative_decode_tree_gb300 import binding as M
        s["plan"] = M.mla_verify_plan(max_batch, 1, T, T, pool_rows, 1, flags=M.MLA_VERIFY_KV4 if case["kv4"] else 0)
        s["workspace"] = torch.zeros(s["plan"].workspace_bytes, dtype=torch.uint8, device="cuda")
    return s


def _prepare_commit(case, g, r):
    """A step's new rows; of the cached ones only the page numbers matter, so the pool holds pages of new tokens alone."""
    B, T, page, layers = case["B"], case["T"], case["page"], case["layers"]
    size = np.random.default_rng([B, T, page, case["P_lo"], case["P_hi"]])
    P = size.integers(case["P_lo"], case["P_hi"] + 1, B).astype(np.int64)
    Tn = size.integers(1, T + 1, B).astype(np.int64)
    first, last = P // page, (P + Tn - 1) // page  # pages that hold new tokens
    count = last - first + 1
    pages = r.permutation(int(count.sum())).astype(np.int64)
    held = -(-P // page)
    max_pages = int(last.max()) + 2
    table = np.full((B, max_pages), -1, np.int64)
    loc, refs, k = np.zeros(B * T, np.int64), np.zeros(pages.size, np.int64), 0
    qo = _scan(Tn)
    accepted, num = np.full((B, T), -1, np.int64), np.zeros(B, np.int64)
    for b, tree in enumerate(_trees(Tn, r)):
        mine = pages[k:k + int(count[b])]
        k += int(count[b])
        table[b, first[b]:last[b] + 1] = mine
        pos = P[b] + np.arange(Tn[b])
        loc[qo[b]:qo[b + 1]] = mine[pos // page - first[b]] * page + pos % page
        if held[b] > first[b]:
            refs[mine[0]] = 1
        path, i = [], int(r.integers(0, Tn[b]))
        while i >= 0:
            path.append(i)
            i = int(tree[i])
        accepted[b, :len(path)], num[b] = path[::-1], len(path)
    rows = pages.size * page
    s = dict(op="commit", B=B, T=T, page=page, layers=layers, max_pages=max_pages, kv_pool=_pool(layers, rows, case["kv4"], g),
             qo_indptr=_dev(qo), out_cache_loc=_dev(loc), accepted=_dev(accepted), num_accepted=_dev(num), seq_lens=_dev(P),
             new_seq_lens=torch.zeros(B, dtype=torch.int32, device="cuda"), block_table=_dev(table), page_refs=_dev(refs))
    return _page_plan(case, s, B, T, rows)


def _prepare_turnover(case, g, r):
    n, src_n, page, layers, pages = case["n"], case["sources"], case["page"], case["layers"], case["pages"]
    size = np.random.default_rng([n, src_n, page, case["P_lo"], case["P_hi"]])
    P = size.integers(case["P_lo"], case["P_hi"] + 1, src_n).astype(np.int64)
    src = size.integers(0, src_n, n)
    held = -(-P // page)
    B, max_pages = src_n + n, int(held.max()) + 2
    order = r.permutation(pages).astype(np.int64)
    table, refs, k = np.full((B, max_pages), -1, np.int64), np.zeros(pages, np.int64), 0
    slots = r.permutation(B)  # sources and free places, mixed
    lens = np.zeros(B, np.int64)
    for i in range(src_n):
        mine = order[k:k + int(held[i])]
        k += int(held[i])
        table[slots[i], :held[i]], lens[slots[i]] = mine, P[i]
        refs[mine] = 1
    s = dict(op="turnover", n=n, B=B, page=page, layers=layers, pages=pages, max_pages=max_pages,
             kv_pool=_pool(layers, pages * page + 1, case["kv4"], g), src=_dev(slots[src]), dst=_dev(slots[src_n:]),
             seq_lens=_dev(lens), block_table=_dev(table), page_refs=_dev(refs),
             free_pages=torch.zeros(pages, dtype=torch.int32, device="cuda"),
             num_free=torch.zeros(1, dtype=torch.int32, device="cuda"), pages_used=torch.zeros(1, dtype=torch.int32, device="cuda"))
    return _page_plan(case, s, B, 1, pages * page + 1)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = np.random.default_rng(seed)
    return {"shared": _prepare_shared, "accept": _prepare_accept, "commit": _prepare_commit,
            "turnover": _prepare_turnover}[case["op"]](case, g, r)


# ---- plain forms ------------------------------------------------------------------

def _rows_of(s):
    """Rows of the own keys, [B, L_max], and who sees them, [B, T, L_max]."""
    B, T = s["B"], s["T"]
    kv0, qo0 = s["kv_indptr"][:-1].long()[:, None], s["qo_indptr"][:-1].long()[:, None]
    P, Tn = s["kv_indptr"][1:].long()[:, None] - kv0, s["qo_indptr"][1:].long()[:, None] - qo0
    j = torch.arange(s["L_max"], device="cuda")[None, :]
    pre = s["kv_indices"].long()[(kv0 + j).clamp(0, s["kv_indices"].numel() - 1)]
    new = s["out_cache_loc"].long()[(qo0 + j - P).clamp(0, B * T - 1)]
    i = torch.arange(T, device="cuda")[None, :]
    bit = s["mask_indptr"].long()[:, None, None] + i[:, :, None] * (P + Tn)[:, :, None] + j[:, None, :]
    inside = (j < P + Tn)[:, None, :] & (i < Tn)[:, :, None]
    bit = torch.where(inside, bit, torch.zeros_like(bit))
    sees = ((s["custom_mask"][bit >> 3].int() >> (bit & 7).int()) & 1).bool() & inside
    return torch.where(j < P, pre, new), sees, (qo0 + i).clamp(0, B * T - 1)


def _plain_shared(s):
    B, H, T, n = s["B"], s["H"], s["T"], s["n_tok"]
    q_all = torch.cat([s["q_nope"], s["q_rope"]], -1).float()  # [B*T, H, 576]
    # the requests' own keys, padded to the longest
    rows, sees, at = _rows_of(s)
    k = s["kv_pool"][rows.view(-1)].float().view(B, s["L_max"], D_ROW)
    q = q_all[at.view(-1)].view(B, T * H, D_ROW)
    sc = (torch.bmm(q, k.transpose(1, 2)) * SM_SCALE).view(B, T, H, s["L_max"])
    sc = sc.masked_fill_(~sees[:, :, None, :], -math.inf)
    top = sc.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = sc.sub_(top).exp_()
    total = p.sum(-1)
    o = torch.bmm(p.view(B, T * H, s["L_max"]), k[:, :, :D_LATENT]).view(B, T, H, D_LATENT)
    tok = torch.arange(n, device="cuda")
    b = torch.searchsorted(s["qo_indptr"][1:].long(), tok, right=True)
    i = tok - s["qo_indptr"].long()[b]
    o, total, top = o[b, i], total[b, i], top.view(B, T, H)[b, i]  # [n, H, ...]
    out, lse = [], []
    at = 0
    for g in range(s["G"]):  # each group's rows against its prefix, and the two joined
        t0, t1 = s["qo"][g * s["per"]], s["qo"][(g + 1) * s["per"]]
        og, tg, mg = o[t0:t1], total[t0:t1], top[t0:t1]
        if s["S"][g] and t1 > t0:
            k = s["kv_pool"][s["shared_indices"][at:at + s["S"][g]].long()].float()
            sc = (q_all[t0:t1].reshape(-1, D_ROW) @ k.T) * SM_SCALE
            m = sc.amax(-1, keepdim=True)
            p = sc.sub_(m).exp_()
            os = (p @ k[:, :D_LATENT]).view(t1 - t0, H, D_LATENT)
            ts, m = p.sum(-1).view(t1 - t0, H), m.view(t1 - t0, H)
            mx = torch.where(tg > 0, torch.maximum(mg, m), m)
            a, c = torch.where(tg > 0, (mg - mx).exp(), torch.zeros_like(tg)), (m - mx).exp()
            og, tg, mg = og * a[..., None] + os * c[..., None], tg * a + ts * c, mx
        at += s["S"][g]
        out.append(torch.where(tg[..., None] > 0, og / tg[..., None], torch.zeros_like(og)))
        lse.append(mg + torch.log(tg))
    return torch.cat(out).to(torch.bfloat16), torch.cat(lse)


def _weights(p):
    return torch.round(p.double() * 2.0 ** ONE).long()


def _scaled(q, Z):
    """q * Z >> 38 for whole numbers up to 2^38, in 64 bits."""
    half = ONE // 2
    hi, lo = q >> half, q & ((1 << half) - 1)
    return (hi * Z + ((lo * Z) >> half)) >> half


def _plain_accept(s):
    B, T, V = s["B"], s["T"], s["V"]
    dev = "cuda"
    qo = s["qo_indptr"].long()
    first, Tn = qo[:-1], qo[1:] - qo[:-1]
    batch = torch.arange(B, device=dev)
    k, k_next = (s["u"].double() * 2 ** 24).floor().long(), (s["u_next"].double() * 2 ** 24).floor().long()
    cur = torch.zeros(B, dtype=torch.long, device=dev)
    node = first.clamp(max=B * T - 1)
    r = _weights(s["target"][node])
    Z = torch.full((B, 1), 1 << ONE, dtype=torch.long, device=dev)
    accepted = torch.full((B, T), -1, dtype=torch.int32, device=dev)
    num = (Tn > 0).int()
    accepted[:, 0] = num - 1
    for c in range(1, T):
        at = (first + c).clamp(max=B * T - 1)
        tries = (c < Tn) & (s["parents"][at].long() == cur)
        x = s["tokens"][at].long()[:, None]
        if s["draft"] is not None:
            sc = _scaled(_weights(s["draft"][(first + cur).clamp(max=B * T - 1)]), Z)
        else:
            sc = torch.zeros((B, V), dtype=torch.long, device=dev).scatter_(1, x, Z)
        takes = tries & (k[at] * sc.gather(1, x)[:, 0] < r.gather(1, x)[:, 0] << 24)
        fails = (tries & ~takes)[:, None]
        Z = torch.where(fails, (Z - torch.minimum(r, sc).sum(1, keepdim=True)).clamp(min=0), Z)
        r = torch.where(fails, (r - sc).clamp(min=0), r)
        cur = torch.where(takes, torch.full_like(cur, c), cur)
        Z = torch.where(takes[:, None], torch.full_like(Z, 1 << ONE), Z)
        r = torch.where(takes[:, None], _weights(s["target"][(first + cur).clamp(max=B * T - 1)]), r)
        accepted[batch, num.long().clamp(max=T - 1)] = torch.where(
            takes, torch.full_like(num, c), accepted[batch, num.long().clamp(max=T - 1)])
        num = num + takes.int()
    t = (k_next[:, None] * r.sum(1, keepdim=True)) >> 24
    nxt = (r.cumsum(1) <= t).sum(1)
    nxt = torch.where(Tn > 0, nxt, torch.full_like(nxt, -1))
    return dict(accepted=accepted, num_accepted=num, next_tokens=nxt.to(torch.int32))


def _plain_commit(s):
    B, T, page = s["B"], s["T"], s["page"]
    first, n = s["qo_indptr"][:-1].long()[:, None], s["num_accepted"].long()[:, None]
    j = torch.arange(T, device="cuda")[None, :]
    keep = j < n
    loc = s["out_cache_loc"].long()
    src = loc[(first + torch.where(keep, s["accepted"].long(), torch.zeros_like(j))).clamp(max=B * T - 1)]
    dst = loc[(first + torch.where(keep, j, torch.zeros_like(j))).clamp(max=B * T - 1)]
    src = torch.where(keep, src, dst)  # (a row that is not kept is node 0's, which stays where it is)
    s["kv_pool"][:, dst.view(-1)] = s["kv_pool"][:, src.view(-1)]
    P = s["seq_lens"].long()[:, None]
    c = torch.arange(s["max_pages"], device="cuda")[None, :]
    fresh = (c >= (P + page - 1) // page) & (c < (P + n + page - 1) // page)
    at = torch.where(fresh, s["block_table"].long(), torch.full_like(c, s["page_refs"].numel()))
    refs = torch.cat([s["page_refs"], s["page_refs"].new_zeros(1)])
    refs[at.view(-1)] = 1
    s["page_refs"].copy_(refs[:-1])
    return dict(kv_pool=s["kv_pool"].view(torch.int16), new_seq_lens=(P + n).view(-1).to(torch.int32), page_refs=s["page_refs"])


def _plain_turnover(s):
    n, page, pages, mp = s["n"], s["page"], s["pages"], s["max_pages"]
    refs, table, lens = s["page_refs"], s["block_table"], s["seq_lens"]
    ids = torch.arange(pages, device="cuda", dtype=torch.int32)
    free = refs == 0
    num_free = free.sum().to(torch.int32).view(1)
    place = torch.where(free, torch.cumsum(free, 0) - 1, torch.full_like(ids, pages).long())
    free_pages = torch.full((pages + 1,), -1, dtype=torch.int32, device="cuda")
    free_pages[place] = ids
    free_pages[pages:] = -1
    free_pages = free_pages[:pages]
    # fork: full pages are shared, the rows of one that is not full go to a fresh page
    src, dst = s["src"].long(), s["dst"].long()
    P = lens[src].long()
    full, part = P // page, (P % page > 0).long()
    fresh = free_pages[(torch.cumsum(part, 0) - part).clamp(max=pages - 1)].long()
    c = torch.arange(mp, device="cuda")[None, :]
    shared = c < full[:, None]
    new = torch.where(shared, table[src], table[dst])
    last = (c == full[:, None]) & (part > 0)[:, None]
    new = torch.where(last, fresh[:, None].to(torch.int32), new)
    counted = torch.where(shared | last, new.long(), torch.full_like(new, pages).long()).view(-1)
    old = table[src, full.clamp(max=mp - 1)].long()
    x = torch.arange(page, device="cuda")[None, :]
    within = x < (P % page)[:, None]
    # (past the last row, the page's first row once more)
    to, frm = fresh[:, None] * page + torch.where(within, x, 0 * x), old[:, None] * page + torch.where(within, x, 0 * x)
    # (a fork whose pages are all full copies the row behind the last page onto itself)
    spare = torch.full_like(to, pages * page)
    to, frm = torch.where((part > 0)[:, None], to, spare), torch.where((part > 0)[:, None], frm, spare)
    s["kv_pool"][:, to.view(-1)] = s["kv_pool"][:, frm.view(-1)]
    table[dst] = new
    refs1 = torch.cat([refs, refs.new_zeros(1)])
    refs1.index_add_(0, counted, torch.ones_like(counted, dtype=torch.int32))
    lens[dst] = lens[src]
    pages_used = part.sum().to(torch.int32).view(1)
    # release the copies again
    refs1.index_add_(0, counted, torch.full_like(counted, -1, dtype=torch.int32))
    refs.copy_(refs1[:pages])
    lens[dst] = 0
    return dict(free_pages=free_pages, num_free=num_free, block_table=table, seq_lens=lens, pages_used=pages_used,
                page_refs=refs, kv_pool=s["kv_pool"].view(torch.int16))


# ---- one pass -----------------------------------------------------------------------

def run(state):
    # (pool rows are moved as they are: they come back as the bits that they are)
    s, op = state, state["op"]
    if not own:
        return {"shared": _plain_shared, "accept": _plain_accept, "commit": _plain_commit,
                "turnover": _plain_turnover}[op](s)
    from mla_speculative_decode_tree_gb300 import binding as M
    if op == "shared":
        M.mla_verify_run_shared(s["plan"], s["q_nope"], s["q_rope"], s["kv_pool"], s["group_indptr"], s["shared_indptr"],
                                s["shared_indices"], s["kv_indptr"], s["kv_indices"], s["qo_indptr"], s["out_cache_loc"],
                                s["custom_mask"], s["mask_indptr"], s["B"], s["G"], SM_SCALE, s["workspace"], s["o"], s["lse"])
        return s["o"][:s["n_tok"]], s["lse"][:s["n_tok"]]
    if op == "accept":
        M.mla_verify_accept_drafts(s["plan"], s["target"], s["draft"], s["tokens"], s["parents"], s["qo_indptr"], s["u"],
                                   s["u_next"], s["B"], s["accepted"], s["num_accepted"], s["next_tokens"], s["workspace"])
        return dict(accepted=s["accepted"], num_accepted=s["num_accepted"], next_tokens=s["next_tokens"])
    if op == "commit":
        M.mla_verify_commit_drafts(s["plan"], s["kv_pool"], s["qo_indptr"], s["out_cache_loc"], s["accepted"],
                                   s["num_accepted"], s["B"], s["seq_lens"], s["new_seq_lens"], s["page"], s["block_table"],
                                   s["page_refs"], s["workspace"])
        return dict(kv_pool=s["kv_pool"].view(torch.int16), new_seq_lens=s["new_seq_lens"], page_refs=s["page_refs"])
    M.mla_verify_list_free_pages(s["plan"], s["page_refs"], s["free_pages"], s["num_free"])
    M.mla_verify_fork(s["plan"], s["kv_pool"], s["src"], s["dst"], s["page"], s["block_table"], s["seq_lens"],
                      s["page_refs"], s["free_pages"], s["pages_used"], s["workspace"])
    M.mla_verify_release(s["plan"], s["dst"], s["page"], s["block_table"], s["seq_lens"], s["page_refs"], s["workspace"])
    return dict(free_pages=s["free_pages"], num_free=s["num_free"], block_table=s["block_table"], seq_lens=s["seq_lens"],
                pages_used=s["pages_used"], page_refs=s["page_refs"], kv_pool=s["kv_pool"].view(torch.int16))


# ---- what a pass cannot do without -----------------------------------------------------

def work(case):
    if case["op"] == "shared":
        S, P, Tn = _sizes(case)
        H, per = case["H"], case["per"]
        pairs = int((Tn * (P + Tn)).sum()) + int((S * Tn.reshape(-1, per).sum(1)).sum())
        keys = int(S.sum()) + int((P + Tn).sum())
        return {"bytes": keys * (1152 + 4) + int((Tn * (P + Tn)).sum()) / 8 + int(Tn.sum()) * H * (1152 + 1024 + 4),
                "flops": 2.0 * (576 + 512) * H * pairs}
    if case["op"] == "accept":  # the row that the next token is drawn from, with drawn drafts its draft row as well
        return {"bytes": case["B"] * case["V"] * 4.0 * (2 if case["drawn"] else 1), "flops": 0}
    row = KV4_ROW if case["kv4"] else 2 * D_ROW
    if case["op"] == "commit":  # a path of a random tree of T nodes has about ln T nodes behind the root
        return {"bytes": case["B"] * (2.0 * row * case["layers"] * math.log(case["T"] + 1) + 40), "flops": 0}
    size = np.random.default_rng([case["n"], case["sources"], case["page"], case["P_lo"], case["P_hi"]])
    P = size.integers(case["P_lo"], case["P_hi"] + 1, case["sources"]).astype(np.int64)[
        size.integers(0, case["sources"], case["n"])]
    page = case["page"]
    return {"bytes": 8.0 * case["pages"] + float((P % page).sum()) * 2 * row * case["layers"] + 24.0 * float((-(-P // page)).sum()),
            "flops": 0}


# ---- the definition in 64 bits -----------------------------------------------------------

def exact(case, seed):
    if case["op"] != "shared":
        return None  # whole numbers, and rows that are moved as they are
    s = prepare(case, seed)
    n, H = s["n_tok"], s["H"]
    o = torch.zeros((n, H, D_LATENT), dtype=torch.float64, device="cuda")
    lse = torch.full((n, H), -math.inf, dtype=torch.float64, device="cuda")
    sh, kv, start = s["shared_indptr"].tolist(), s["kv_indptr"].tolist(), s["mask_indptr"].tolist()
    for g in range(s["G"]):
        common = s["kv_pool"][s["shared_indices"][sh[g]:sh[g + 1]].long()].double()
        for b in range(g * s["per"], (g + 1) * s["per"]):
            t0, t1 = s["qo"][b], s["qo"][b + 1]
            if t0 == t1:
                continue
            own_rows = torch.cat([s["kv_indices"][kv[b]:kv[b + 1]], s["out_cache_loc"][t0:t1]]).long()
            k = torch.cat([common, s["kv_pool"][own_rows].double()])
            L, S = own_rows.numel(), common.shape[0]
            q = torch.cat([s["q_nope"][t0:t1], s["q_rope"][t0:t1]], -1).double()
            sc = (q.view(-1, D_ROW) @ k.T).view(t1 - t0, H, S + L) * SM_SCALE
            bit = start[b] + torch.arange((t1 - t0) * L, device="cuda")
            sees = ((s["custom_mask"][bit // 8].long() >> (bit % 8)) & 1).bool().view(t1 - t0, 1, L)
            sc[:, :, S:] = sc[:, :, S:].masked_fill(~sees, -math.inf)
            lse[t0:t1] = torch.logsumexp(sc, -1)
            o[t0:t1] = (torch.softmax(sc, -1).view(-1, S + L) @ k[:, :D_LATENT]).view(-1, H, D_LATENT)
    return o, lse
