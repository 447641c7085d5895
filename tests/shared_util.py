"""Workloads and references for attention over shared prefixes."""

import numpy as np
import torch

from mla_speculative_decode_tree_gb300 import binding as B
from parity_util import LSE_MAX_ABS, bf16_to_f64, compare

SCALE = 192 ** -0.5


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def scan(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int64)


class Case:
    """Groups of requests: groups[g] = (S_g, [(P_b, T_b), ...]).  Rows are drawn without replacement from the pool."""

    def __init__(self, groups, heads, pool_rows=None, seed=0, q_scale=1.0, scale=SCALE, uniform=None):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.groups, self.H, self.scale = groups, heads, scale
        self.S = [s for s, _ in groups]
        self.P = [p for _, r in groups for p, _ in r]
        self.T = [t for _, r in groups for _, t in r]
        self.batch, self.uniform = len(self.P), uniform
        n_sh, n_pre, n = sum(self.S), sum(self.P), sum(self.T)
        pool_rows = pool_rows or n_sh + n_pre + n + 40
        self.pool = torch.randn((pool_rows, 576), generator=g, device="cuda").to(torch.bfloat16)
        rows = torch.randperm(pool_rows, generator=g, device="cuda")[:n_sh + n_pre + n].to(torch.int32)
        self.q_len = uniform or max(max(self.T), 1)
        cap = self.batch * self.q_len
        self.q_nope = (q_scale * torch.randn((cap, heads, 512), generator=g, device="cuda")).to(torch.bfloat16)
        self.q_rope = (q_scale * torch.randn((cap, heads, 64), generator=g, device="cuda")).to(torch.bfloat16)
        self.group_indptr = scan([len(r) for _, r in groups])
        self.shared_indptr, self.kv_indptr, self.qo_indptr = scan(self.S), scan(self.P), scan(self.T)
        self.shared_indices = rows[:n_sh].clone()
        self.kv_indices = rows[n_sh:n_sh + n_pre].clone()
        self.loc = torch.zeros(cap, dtype=torch.int32, device="cuda")
        self.loc[:n] = rows[n_sh + n_pre:]
        self.masks = []
        for p, t in zip(self.P, self.T):
            m = np.ones((t, p + t), bool)
            see = np.eye(t, dtype=bool)
            for i in range(1, t):
                see[i] |= see[int(rng.integers(0, i))]
            m[:, p:] = see
            self.masks.append(m)

    def device(self):
        bits, start, total = [], [], 0
        for m in self.masks:
            start.append(total)
            total += m.size
            bits.append(m.reshape(-1))
        packed = np.packbits(np.concatenate(bits + [np.zeros(1, bool)]), bitorder="little")
        self.mask, self.mask_indptr = torch.from_numpy(packed).cuda(), i32(start)
        self.d_group, self.d_shared = i32(self.group_indptr), i32(self.shared_indptr)
        self.d_kv, self.d_qo = i32(self.kv_indptr), i32(self.qo_indptr)
        return self

    def plan(self, flags=0, max_batch=None, q_len=None):
        longest = max(p + t for p, t in zip(self.P, self.T))
        q_len = q_len or self.q_len
        return B.mla_verify_plan(max_batch or self.batch, self.H, q_len, max(longest, q_len), self.pool.shape[0], 0,
                                 flags=B.MLA_VERIFY_SHARED | flags)

    def call(self, plan, ws, o, lse, stream=None):
        B.mla_verify_run_shared(plan, self.q_nope, self.q_rope, self.pool, self.d_group, self.d_shared,
                                self.shared_indices if len(self.shared_indices) else None, self.d_kv,
                                self.kv_indices if len(self.kv_indices) else None, None if self.uniform else self.d_qo,
                                self.loc, self.mask, self.mask_indptr, self.batch, len(self.groups), self.scale, ws, o, lse,
                                stream=stream)

    def outputs(self, fill=7.0):
        cap = self.q_nope.shape[0]
        o = torch.full((cap, self.H, 512), fill, dtype=torch.bfloat16, device="cuda")
        return o, torch.full((cap, self.H), fill, dtype=torch.float32, device="cuda")

    def run(self, flags=0, **kw):
        self.device()
        plan = self.plan(flags, **kw)
        ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
        ws[256:].random_(0, 256)  # nothing but the header has to be zero
        o, lse = self.outputs()
        self.call(plan, ws, o, lse)
        status = B.mla_verify_read_status(plan, ws)
        n = int(self.qo_indptr[-1])
        assert bool((o[n:] == 7).all()) and bool((lse[n:] == 7).all())  # rows behind the last token stay
        return o[:n], lse[:n], status

    def exact(self):
        """(O, LSE) in float64, from the definition; rows outside the pool are left out."""
        n, rows_all = int(self.qo_indptr[-1]), self.pool.shape[0]
        o = torch.zeros((n, self.H, 512), dtype=torch.float64, device="cuda")
        lse = torch.full((n, self.H), -float("inf"), dtype=torch.float64, device="cuda")
        for g in range(len(self.groups)):
            sh = self.shared_indices[int(self.shared_indptr[g]):int(self.shared_indptr[g + 1])].long()
            for b in range(int(self.group_indptr[g]), int(self.group_indptr[g + 1])):
                t0, t1 = int(self.qo_indptr[b]), int(self.qo_indptr[b + 1])
                if t0 == t1:
                    continue
                own = torch.cat([self.kv_indices[int(self.kv_indptr[b]):int(self.kv_indptr[b + 1])], self.loc[t0:t1]]).long()
                rows = torch.cat([sh, own])
                inside = (rows >= 0) & (rows < rows_all)
                k = self.pool[rows.clamp(0, rows_all - 1)].double()
                q = torch.cat([self.q_nope[t0:t1], self.q_rope[t0:t1]], -1).double()
                s = torch.einsum("thd,kd->thk", q, k) * self.scale
                see = torch.cat([torch.ones((t1 - t0, sh.numel()), dtype=torch.bool, device="cuda"),
                                 torch.from_numpy(self.masks[b]).cuda()], 1) & inside
                s = s.masked_fill(~see[:, None, :], -float("inf"))
                some = see.any(1)
                if bool(some.any()):
                    lse[t0:t1][some] = torch.logsumexp(s[some], -1)
                    o[t0:t1][some] = torch.softmax(s[some], -1) @ k[:, :512]
        return o, lse

    def check(self, flags=0, what="", lse_slack=0.0, **kw):
        o, lse, status = self.run(flags, **kw)
        assert status == 0, (what, status)
        self.match(o, lse, what, lse_slack)

    def match(self, o, lse, what="", lse_slack=0.0):
        ro, rl = (x.cpu().numpy() for x in self.exact())
        got = lse.cpu().numpy().astype(np.float64)
        if lse_slack:
            fin = np.isfinite(rl)
            assert np.abs(got[fin] - rl[fin]).max() <= LSE_MAX_ABS + lse_slack, what
            got = np.where(fin, rl, got)
        if ro.size:
            compare(bf16_to_f64(o).reshape(-1, 512), got.reshape(-1), ro.reshape(-1, 512), rl.reshape(-1), what)
