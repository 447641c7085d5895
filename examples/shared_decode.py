"""Speculative decoding of several samples per prompt, every array on the GPU.

The samples of a prompt read its keys once together.  One step is one CUDA graph: the free pages, slot maps, the drafts'
keys, tree masks, attention in every layer, the verification of the drafts against the target's probabilities, and the
commit of what was accepted.  Between steps samples are released and others forked into their places: a fork shares
the pages that it has in common with its source.

    python examples/shared_decode.py         # random weights; prints the step time and an error

Synthetic: keys, queries and both models' probabilities are random.
"""

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from mla_speculative_decode_tree_gb300 import binding as B  # noqa: E402


class SharedDecoder:
    """`samples` requests for each of the prompts (lengths `prompts`), at most `drafts` new tokens per request and step.
    Every layer has a pool of the prompts' rows, `pages` pages of `page` rows and one row more that nothing reads."""

    def __init__(self, prompts, samples, heads, drafts, vocab, max_len, pages, page=16, layers=2, device="cuda"):
        self.batch, self.drafts, self.page, self.pages = len(prompts) * samples, drafts, page, pages
        self.groups, self.scale = len(prompts), 192 ** -0.5
        total = sum(prompts)
        rows = pages * page + total + 1
        self.v = [B.Verifier(self.batch, heads, drafts, max_len, rows, 0, B.MLA_VERIFY_SHARED, device) for _ in range(layers)]
        n, columns = self.batch * drafts, -(-max_len // page)

        def i32(*shape):
            return torch.zeros(shape, dtype=torch.int32, device=device)

        def f(dtype, *shape):
            return torch.zeros(shape, dtype=dtype, device=device)

        self.pool = f(torch.bfloat16, layers, rows, 576)
        self.group_indptr = torch.arange(0, self.batch + 1, samples, dtype=torch.int32, device=device)
        self.shared_indptr = torch.tensor([0] + np.cumsum(prompts).tolist(), dtype=torch.int32, device=device)
        self.shared_indices = torch.arange(pages * page, rows - 1, dtype=torch.int32, device=device)
        # lengths, tables and rows are those behind the prompts
        self.seq_lens, self.new_lens, self.table, self.refs = i32(self.batch), i32(self.batch), i32(self.batch, columns), i32(pages)
        self.free, self.num_free, self.used = i32(pages), i32(1), i32(1)
        self.kv_indptr, self.qo_indptr, self.mask_indptr = i32(self.batch + 1), i32(self.batch + 1), i32(self.batch)
        self.kv_indices, self.slots = i32(self.batch * max_len), i32(n)
        self.mask = f(torch.uint8, self.batch * (drafts * max_len + 7) // 8 + 8)
        self.parents, self.draft_tokens = i32(n), i32(n)
        self.tokens = f(torch.bfloat16, layers, n, 576)
        self.q_nope, self.q_rope = f(torch.bfloat16, layers, n, heads, 512), f(torch.bfloat16, layers, n, heads, 64)
        self.target, self.draft = f(torch.float32, n, vocab), f(torch.float32, n, vocab)
        self.uniform, self.uniform_next = f(torch.float32, n), f(torch.float32, self.batch)
        self.accepted, self.num_accepted, self.next_tokens = i32(self.batch, drafts), i32(self.batch), i32(self.batch)
        self._calls()  # warm up; without tokens nothing changes
        torch.cuda.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.out = self._calls()

    def _calls(self):
        v, ws = self.v[0], self.v[0].workspace
        B.mla_verify_list_free_pages(v.plan, self.refs, self.free, self.num_free)
        self.slots.fill_(-1)
        B.mla_verify_build_slots(v.plan, self.seq_lens, self.new_lens, self.batch, self.page, self.table, self.free, self.used,
                                 self.kv_indptr, self.kv_indices, self.qo_indptr, self.slots, ws)
        B.mla_verify_build_tree_mask_varlen(v.plan, self.parents, self.kv_indptr, self.qo_indptr, self.batch, self.mask,
                                            self.mask_indptr)
        rows = torch.where(self.slots < 0, self.pool.shape[1] - 1, self.slots).long()  # (past the step's tokens: the spare row)
        out = []
        for k, verifier in enumerate(self.v):
            self.pool[k].index_copy_(0, rows, self.tokens[k])
            out.append(verifier.run(dict(
                q_nope=self.q_nope[k], q_rope=self.q_rope[k], kv_pool=self.pool[k], group_indptr=self.group_indptr,
                shared_indptr=self.shared_indptr, shared_indices=self.shared_indices, kv_indptr=self.kv_indptr,
                kv_indices=self.kv_indices, qo_indptr=self.qo_indptr, out_cache_loc=self.slots, custom_mask=self.mask,
                mask_indptr=self.mask_indptr), self.batch, self.scale))
        # (a model's last layer would leave self.target here)
        B.mla_verify_accept_drafts(v.plan, self.target, self.draft, self.draft_tokens, self.parents, self.qo_indptr,
                                   self.uniform, self.uniform_next, self.batch, self.accepted, self.num_accepted,
                                   self.next_tokens, ws)
        B.mla_verify_commit_drafts(v.plan, self.pool, self.qo_indptr, self.slots, self.accepted, self.num_accepted, self.batch,
                                   self.seq_lens, self.seq_lens, self.page, self.table, self.refs, ws)
        return out

    def _check(self):
        for v in self.v:
            status = v.status()  # (waits for the calls)
            if status:
                raise RuntimeError("status 0x%x" % status)

    def prefill(self, g, keys):
        """The keys of prompt g: bf16 [layers, n, 576]."""
        a, b = self.shared_indptr[g:g + 2].tolist()
        self.pool[:, self.pages * self.page + a:self.pages * self.page + b] = keys

    def step(self):
        """One step of what is in the buffers -> [(O, LSE)] per layer; the paths and next tokens stand in `accepted`,
        `num_accepted` and `next_tokens`."""
        self.graph.replay()
        self._check()
        return self.out

    def replace(self, drop, src, dst):
        """Release the requests `drop`, then fork src[i] into dst[i]."""
        v, ws = self.v[0], self.v[0].workspace
        drop, src, dst = (torch.tensor(x, dtype=torch.int32, device=self.refs.device) for x in (drop, src, dst))
        B.mla_verify_release(v.plan, drop, self.page, self.table, self.seq_lens, self.refs, ws)
        B.mla_verify_list_free_pages(v.plan, self.refs, self.free, self.num_free)
        B.mla_verify_fork(v.plan, self.pool, src, dst, self.page, self.table, self.seq_lens, self.refs, self.free, self.used, ws)
        self._check()


def exact(dec, layer, g, own, t0, t1):
    """O of a request's new tokens in float64: prompt g's keys, the request's own ones, its drafts."""
    a, b = dec.shared_indptr[g:g + 2].tolist()
    base = dec.pages * dec.page
    kv = torch.cat([dec.pool[layer, base + a:base + b], own, dec.tokens[layer, t0:t1]]).double()
    n, prefix = t1 - t0, kv.shape[0] - (t1 - t0)
    see = torch.zeros((n, kv.shape[0]), dtype=torch.bool, device=kv.device)
    see[:, :prefix] = True
    for i, p in enumerate(dec.parents[t0:t1].tolist()):
        if p >= 0:
            see[i] = see[p]
        see[i, prefix + i] = True
    q = torch.cat([dec.q_nope[layer, t0:t1], dec.q_rope[layer, t0:t1]], 2).double()
    s = torch.einsum("nhd,kd->nhk", q, kv) * dec.scale
    return torch.einsum("nhk,kd->nhd", torch.softmax(s.masked_fill(~see[:, None, :], float("-inf")), -1), kv[:, :512])


def main(prompts=(4000, 1500), samples=8, heads=16, drafts=5, vocab=2000, steps=8, page=16, layers=2, seed=0):
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    max_len = (steps + 1) * drafts
    batch = len(prompts) * samples
    dec = SharedDecoder(prompts, samples, heads, drafts, vocab, max_len, batch * (max_len // page + 2), page, layers)
    for k, n in enumerate(prompts):
        dec.prefill(k, torch.randn((layers, n, 576), generator=g, device="cuda").to(torch.bfloat16))
    own = [torch.zeros((layers, 0, 576), dtype=torch.bfloat16, device="cuda") for _ in range(batch)]  # what each should hold
    live = [b % samples == 0 for b in range(batch)]  # one sample of each prompt to begin with
    worst, times, grown = 0.0, [], 0
    for _ in range(steps):
        new = np.where(live, rng.integers(1, drafts + 1, batch), 0)
        parents = [int(rng.integers(0, i)) if i else -1 for t in new for i in range(t)]
        n = len(parents)
        dec.new_lens.copy_(torch.from_numpy(new.astype(np.int32)))
        dec.parents[:n] = torch.tensor(parents, dtype=torch.int32, device="cuda")
        for x in (dec.tokens, dec.q_nope, dec.q_rope):
            x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        logits = 2 * torch.randn(dec.target.shape, generator=g, device="cuda")
        dec.target.copy_(torch.softmax(logits, -1))
        dec.draft.copy_(torch.softmax(logits + 0.5 * torch.randn(logits.shape, generator=g, device="cuda"), -1))
        at = np.concatenate([[0], np.cumsum(new)])
        parent_rows = torch.tensor([int(at[b]) + max(parents[at[b] + i], 0) for b in range(batch) for i in range(new[b])],
                                   device="cuda")
        dec.draft_tokens[:n] = torch.multinomial(dec.draft[parent_rows], 1, generator=g).view(-1).to(torch.int32)
        dec.uniform.copy_(torch.rand(dec.uniform.shape, generator=g, device="cuda"))
        dec.uniform_next.copy_(torch.rand(dec.uniform_next.shape, generator=g, device="cuda"))
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        out = dec.step()
        end.record()
        torch.cuda.synchronize()
        times.append(start.elapsed_time(end) * 1e3)
        accepted, num = dec.accepted.tolist(), dec.num_accepted.tolist()
        for b in range(batch):
            for k in range(layers if new[b] else 0):
                ref = exact(dec, k, b // samples, own[b][k], int(at[b]), int(at[b + 1]))
                worst = max(worst, float((out[k][0][at[b]:at[b + 1]].double() - ref).norm() / ref.norm()))
            path = [int(at[b]) + i for i in accepted[b][:num[b]]]
            own[b] = torch.cat([own[b], dec.tokens[:, path]], 1)
            grown += num[b]
        # end a few samples, and continue others in every place that is free
        drop = [b for b in range(batch) if live[b] and b % samples and rng.random() < 0.3]
        for b in drop:
            live[b], own[b] = False, own[b][:, :0]
        src, dst = [], []
        for b in range(batch):
            if not live[b] and rng.random() < 0.7:
                src.append(int(rng.choice([x for x in range(b - b % samples, b - b % samples + samples)
                                           if live[x] and x not in dst])))
                dst.append(b)
        dec.replace(drop, src, dst)
        for s, d in zip(src, dst):
            live[d], own[d] = True, own[s]
        for b in range(batch):
            if live[b] and own[b].shape[1] + drafts > max_len:
                raise AssertionError("longer than planned")
    return worst, float(np.median(times)), dec, own, grown


def held_rows(dec, b):
    """What request b holds in the pool: bf16 [layers, seq_lens[b], 576]."""
    n = int(dec.seq_lens[b])
    pages = dec.table[b, :-(-n // dec.page)].long()
    rows = (pages[:, None] * dec.page + torch.arange(dec.page, device=pages.device)).reshape(-1)[:n]
    return dec.pool[:, rows]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("samples", 8), ("heads", 16), ("drafts", 5), ("vocab", 2000), ("steps", 8), ("page", 16)):
        ap.add_argument("--" + name, type=int, default=value)
    error, us, dec, own, grown = main(**vars(ap.parse_args()))
    print("step %.1f us (slot maps, masks, attention in %d layers, verification, commit in one graph), relative error of O "
          "%.1e, %d tokens kept, pages in use %d of %d" % (us, len(dec.v), error, grown, int((dec.refs > 0).sum()), dec.pages))
