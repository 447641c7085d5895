"""Oracles of the operators around a verify step (test infrastructure only).

Draft trees verified against the target's probabilities, accepted rows
committed, the free list, requests forked and released: each written out
request by request in Python's whole numbers.
"""

from __future__ import annotations

import numpy as np

ONE = 1 << 38


def weight(p) -> int:
    """round(p * 2^38), ties to even, of a float32 probability; NaN and negative ones 0, above 1: 1."""
    p = float(np.float32(p))
    if not p > 0:
        return 0
    p = min(p, 1.0)
    return round(p * ONE)  # exact in float64: 24 bits; Python rounds ties to even


def random24(u) -> int:
    u = float(np.float32(u))
    if not u > 0:
        return 0
    return min(int(u * (1 << 24)), (1 << 24) - 1)


def accept_one(target, draft, tokens, parents, u, u_next):
    """One request: target [n, V] (and draft [n, V] or None), tokens, parents, u [n] -> (path, next token)."""
    n, vocab = target.shape
    if n == 0:
        return [], -1
    path, cur = [0], 0
    w = [weight(x) for x in target[0]]
    r, z = list(w), ONE
    for c in range(1, n):
        if int(parents[c]) != cur:
            continue
        x = int(tokens[c])
        if not 0 <= x < vocab:
            continue
        if draft is not None:
            s = [weight(q) * z >> 38 for q in draft[cur]]
        else:
            s = [0] * vocab
            s[x] = z
        if random24(u[c]) * s[x] < r[x] << 24:
            path.append(c)
            cur = c
            w = [weight(y) for y in target[c]]
            r, z = list(w), ONE
        else:
            z = max(z - sum(min(a, b) for a, b in zip(r, s)), 0)
            r = [max(a - b, 0) for a, b in zip(r, s)]
    if sum(r) == 0:
        r = w
    total = sum(r)
    if total == 0:
        return path, -1
    aim = random24(u_next) * total >> 24
    at = 0
    for t, a in enumerate(r):
        at += a
        if at > aim:
            return path, t
    raise AssertionError("unreachable")


def accept(target, draft, tokens, parents, qo_indptr, u, u_next, batch, q_len):
    """All requests -> accepted int32 [batch, q_len], num_accepted, next_tokens."""
    accepted = np.full((batch, q_len), -1, np.int32)
    num, nxt = np.zeros(batch, np.int32), np.zeros(batch, np.int32)
    for b in range(batch):
        s = slice(int(qo_indptr[b]), int(qo_indptr[b + 1]))
        path, nxt[b] = accept_one(target[s], None if draft is None else draft[s], tokens[s], parents[s], u[s], u_next[b])
        accepted[b, :len(path)] = path
        num[b] = len(path)
    return accepted, num, nxt


def commit(pool, qo_indptr, loc, accepted, num, batch, seq_lens, page=None, table=None, refs=None):
    """pool [layers, rows, ...] -> (pool, new_seq_lens, refs, bad)."""
    pool, bad = pool.copy(), False
    refs = None if refs is None else refs.copy()
    new = np.zeros(batch, np.int64)
    for b in range(batch):
        q0, t = int(qo_indptr[b]), int(qo_indptr[b + 1]) - int(qo_indptr[b])
        path, last = [], -1
        bad |= not 0 <= num[b] <= t
        for j in range(min(max(int(num[b]), 0), t)):
            i = int(accepted[b][j])
            if not last < i < t:
                bad = True
                break
            path.append(i)
            last = i
        rows = [pool[:, loc[q0 + i]].copy() if 0 <= loc[q0 + i] < pool.shape[1] else None for i in path]
        for j, row in enumerate(rows):
            if path[j] == j:
                continue
            to = int(loc[q0 + j])
            if row is None or not 0 <= to < pool.shape[1]:
                bad = True
            else:
                pool[:, to] = row
        P = max(int(seq_lens[b]), 0)
        new[b] = P + len(path)
        if refs is not None:
            for c in range(-(-P // page), min(-(-int(new[b]) // page), table.shape[1])):
                if 0 <= table[b, c] < refs.size:
                    refs[table[b, c]] = 1
                else:
                    bad = True
    return pool, new.astype(np.int32), refs, bad


def free_list(refs):
    free = [p for p in range(refs.size) if refs[p] == 0]
    return np.array(free + [-1] * (refs.size - len(free)), np.int32), len(free)


def fork(pool, src, dst, page, table, lens, refs, free):
    """-> (pool, table, lens, refs, entries of the list gone through, status bits: 1 bad row, 4 no page).  A fork whose source
    has a last page in part has an entry of the list, whether it is left out for a clash or not."""
    pool, table, lens, refs = pool.copy(), table.copy(), lens.copy(), refs.copy()
    requests, status, taken = table.shape[0], 0, 0
    free = [int(p) for p in free]
    free = free[:next((k for k, p in enumerate(free) if p < 0), len(free))]  # -1 ends the list
    for i, (s, d) in enumerate(zip(src.tolist(), dst.tolist())):
        if not 0 <= s < requests or not 0 <= d < requests or s == d:
            status |= 1
            continue
        P = max(int(lens[s]), 0)
        full, tail = P // page, P % page
        mine = taken
        taken += tail > 0
        if d in dst[:i].tolist() or d in src.tolist():
            status |= 1
            continue
        for c in range(full):
            table[d, c] = table[s, c]
            refs[table[s, c]] += 1
        lens[d] = P
        if tail:
            fresh = free[mine] if mine < len(free) else -1
            if not 0 <= fresh < refs.size or fresh * page + tail > pool.shape[1]:
                status |= 4
                table[d, full] = -1
                lens[d] = full * page
            else:
                table[d, full] = fresh
                refs[fresh] = 1
                old = int(table[s, full])
                pool[:, fresh * page:fresh * page + tail] = pool[:, old * page:old * page + tail]
    return pool, table, lens, refs, min(taken, len(free)), status


def release(which, page, table, lens, refs):
    lens, refs, status, seen = lens.copy(), refs.copy(), 0, set()
    for b in which.tolist():
        if not 0 <= b < table.shape[0]:
            status |= 1
        elif b not in seen:
            seen.add(b)
            for c in range(-(-max(int(lens[b]), 0) // page)):
                if 0 <= table[b, c] < refs.size and refs[table[b, c]] > 0:
                    refs[table[b, c]] -= 1
                else:
                    status |= 1
            lens[b] = 0
    return lens, refs, status
