"""Speculative decoding over a 4-bit paged latent cache, every array on the GPU.

One step is four calls in one CUDA graph: block tables and slot maps from the
requests' lengths, the drafts' keys stored into the 4-bit pool, the drafts' tree
masks, the verify attention.  Lengths change from step to step; the captured
graph reads them on the device.  Between steps the rows of the accepted path
move to the front of the new ones, and the host hands back the pages that only
rejected drafts used.

    python examples/kv4_decode.py            # random weights; prints the step time and an error

Synthetic: tokens and queries are random, and so are the draft trees and the path through each that is accepted.
"""

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from mla_speculative_decode_tree_gb300 import binding as B  # noqa: E402


class Kv4Decoder:
    """Requests over one 4-bit pool of `pages` pages of `page` rows; at most `drafts` new tokens per request and step."""

    def __init__(self, batch, heads, drafts, max_len, pages, page=64, device="cuda"):
        self.batch, self.drafts, self.page = batch, drafts, page
        self.scale = 192 ** -0.5
        self.v = B.Verifier(batch, heads, drafts, max_len, pages * page, 0, B.MLA_VERIFY_KV4, device)

        def i32(*shape):
            return torch.zeros(shape, dtype=torch.int32, device=device)

        n = batch * drafts
        columns = -(-max_len // page)
        self.pool = torch.zeros((pages * page, B.MLA_VERIFY_KV4_ROW_BYTES), dtype=torch.uint8, device=device)
        self.seq_lens, self.new_lens, self.parents = i32(batch), i32(batch), i32(n)
        self.table, self.free, self.used = i32(batch, columns), i32(pages), i32(1)
        self.kv_indptr, self.qo_indptr, self.mask_indptr = i32(batch + 1), i32(batch + 1), i32(batch)
        self.kv_indices, self.slots = i32(pages * page), i32(n)
        self.mask = torch.zeros(batch * (drafts * max_len + 7) // 8 + 8, dtype=torch.uint8, device=device)
        bf16 = dict(dtype=torch.bfloat16, device=device)
        self.tokens = torch.zeros((n, 576), **bf16)  # latent and RoPE key of each draft, as a projection leaves them
        self.q_nope, self.q_rope = torch.zeros((n, heads, 512), **bf16), torch.zeros((n, heads, 64), **bf16)
        self.table_host = [[] for _ in range(batch)]
        self.free_host = list(range(pages))
        self.graph = None

    def _calls(self):
        v, ws = self.v, self.v.workspace
        self.slots.fill_(-1)  # a slot past the step's tokens stores nothing
        B.mla_verify_build_slots(v.plan, self.seq_lens, self.new_lens, self.batch, self.page, self.table, self.free,
                                 self.used, self.kv_indptr, self.kv_indices, self.qo_indptr, self.slots, ws)
        B.mla_verify_store_kv4(v.plan, self.tokens[:, :512], self.tokens[:, 512:], self.slots, self.pool, ws)
        B.mla_verify_build_tree_mask_varlen(v.plan, self.parents, self.kv_indptr, self.qo_indptr, self.batch,
                                            self.mask, self.mask_indptr)
        return v.run(dict(q_nope=self.q_nope, q_rope=self.q_rope, kv_pool=self.pool, kv_indptr=self.kv_indptr,
                          kv_indices=self.kv_indices, qo_indptr=self.qo_indptr, out_cache_loc=self.slots,
                          custom_mask=self.mask, mask_indptr=self.mask_indptr), self.batch, self.scale)

    def prefill(self, b, latent, rope):
        """Store a prompt as request b's, in place of what it held: latent bf16 [n, 512], rope bf16 [n, 64]."""
        n = latent.shape[0]
        need = -(-n // self.page)
        if need > len(self.free_host) + len(self.table_host[b]) or need > self.table.shape[1]:
            raise ValueError("no room for a prompt of %d tokens" % n)
        self.free_host.extend(self.table_host[b])
        pages = [self.free_host.pop() for _ in range(need)]
        self.table_host[b] = pages
        row = (np.array(pages, np.int32)[:, None] * self.page + np.arange(self.page, dtype=np.int32)).reshape(-1)[:n]
        B.mla_verify_store_kv4(self.v.plan, latent, rope, torch.from_numpy(row).to(latent.device), self.pool,
                               self.v.workspace)
        self.seq_lens[b] = n
        self.table[b, :len(pages)] = torch.tensor(pages, dtype=torch.int32, device=latent.device)

    def step(self):
        """One verify step of the lengths, parents, tokens and queries now in the buffers -> (O, LSE)."""
        self.free.fill_(-1)  # (a step that needs more pages than there are reports it)
        self.free[:len(self.free_host)] = torch.tensor(self.free_host[::-1], dtype=torch.int32, device=self.free.device)
        if self.graph is None:
            self._calls()  # warm up; a repeated build and store change nothing
            torch.cuda.synchronize()
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self.out = self._calls()
        self.graph.replay()
        return self.out

    def accept(self, paths):
        """Of request b's new tokens those on paths[b] stay: a path of its draft tree, node numbers from a root on (empty:
        none).  Their rows move to the first of the new rows; pages past them are free again."""
        status = self.v.status()  # (waits for the step)
        if status:
            raise RuntimeError("verify step reported status 0x%x" % status)
        old, new, at, k = self.seq_lens.tolist(), self.new_lens.tolist(), self.qo_indptr.tolist(), 0
        src = [at[b] + i for b, path in enumerate(paths) for i in path]
        dst = [at[b] + i for b, path in enumerate(paths) for i in range(len(path))]
        if src != dst:
            src, dst = (self.slots[torch.tensor(x, device=self.slots.device)].long() for x in (src, dst))
            self.pool[dst] = self.pool[src]  # (all read before any is written: a row may be both)
        taken = self.free_host[::-1][:int(self.used)]
        del self.free_host[len(self.free_host) - len(taken):]
        for b in range(self.batch):
            have = len(self.table_host[b])
            fresh = -(-(old[b] + new[b]) // self.page) - have
            pages = self.table_host[b] + taken[k:k + fresh]
            k += fresh
            keep = -(-(old[b] + len(paths[b])) // self.page)
            self.table_host[b], back = pages[:keep], pages[keep:]
            self.free_host.extend(back)
        self.seq_lens += torch.tensor([len(path) for path in paths], dtype=torch.int32, device=self.seq_lens.device)


def exact(dec, b, t0, t1):
    """O of request b's new tokens in float64, from the pool's rows read back."""
    rows = torch.cat([dec.kv_indices[dec.kv_indptr[b]:dec.kv_indptr[b + 1]], dec.slots[t0:t1]])
    kv = torch.empty((rows.numel(), 576), dtype=torch.bfloat16, device=rows.device)
    B.mla_verify_load_kv4(dec.v.plan, dec.pool, rows, kv[:, :512], kv[:, 512:], dec.v.workspace)
    n, prefix = t1 - t0, rows.numel() - (t1 - t0)
    see = torch.zeros((n, rows.numel()), dtype=torch.bool, device=rows.device)
    see[:, :prefix] = True
    for i, p in enumerate(dec.parents[t0:t1].tolist()):
        if p >= 0:
            see[i] = see[p]
        see[i, prefix + i] = True
    q = torch.cat([dec.q_nope[t0:t1], dec.q_rope[t0:t1]], 2).double()
    s = torch.einsum("nhd,kd->nhk", q, kv.double()) * dec.scale
    p = torch.softmax(s.masked_fill(~see[:, None, :], float("-inf")), -1)
    return torch.einsum("nhk,kd->nhd", p, kv[:, :512].double())


def random_path(parents, rng):
    """Node numbers from a root to a random node of a draft tree, or none."""
    path, i = [], int(rng.integers(-1, len(parents)))
    while i >= 0:
        path.append(i)
        i = int(parents[i])
    return path[::-1]


def main(batch=8, heads=16, drafts=6, prompt=2000, steps=6, page=64, seed=0):
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

    max_len = 2 * prompt + steps * drafts
    dec = Kv4Decoder(batch, heads, drafts, max_len, batch * (max_len // page + 2), page)
    for b in range(batch):
        x = normal(int(rng.integers(1, 2 * prompt)), 576)
        dec.prefill(b, x[:, :512], x[:, 512:])
    worst, times = 0.0, []
    for _ in range(steps):
        new = rng.integers(0, drafts + 1, batch)
        n = int(new.sum())
        parents = np.concatenate([[int(rng.integers(-1, i)) if i else -1 for i in range(t)] for t in new] + [[]])
        dec.new_lens.copy_(torch.from_numpy(new.astype(np.int32)))
        dec.parents[:n] = torch.from_numpy(parents.astype(np.int32)).cuda()
        dec.tokens.copy_(normal(*dec.tokens.shape))
        dec.q_nope.copy_(normal(*dec.q_nope.shape))
        dec.q_rope.copy_(normal(*dec.q_rope.shape))
        o, _ = dec.step()
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        dec.graph.replay()  # the same step once more, for its time
        end.record()
        torch.cuda.synchronize()
        times.append(start.elapsed_time(end) * 1e3)
        at = dec.qo_indptr.tolist()
        for b in range(batch):
            if at[b + 1] > at[b]:
                ref = exact(dec, b, at[b], at[b + 1])
                worst = max(worst, float((o[at[b]:at[b + 1]].double() - ref).norm() / ref.norm()))
        dec.accept([random_path(parents[at[b]:at[b + 1]], rng) for b in range(batch)])
    return worst, float(np.median(times)), dec


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("batch", 8), ("heads", 16), ("drafts", 6), ("prompt", 2000), ("steps", 6), ("page", 64)):
        ap.add_argument("--" + name, type=int, default=value)
    error, us, dec = main(**vars(ap.parse_args()))
    print("step %.1f us (slot maps, store, masks, attention in one graph), relative error of O %.1e, cache %.1f MB in 4 bits "
          "(%.1f in bf16)" % (us, error, dec.pool.numel() / 1e6, dec.pool.shape[0] * 1152 / 1e6))
