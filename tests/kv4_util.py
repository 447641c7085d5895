"""Helpers of the 4-bit cache tests: host workloads over a 4-bit pool and their device buffers."""

import numpy as np

from mla_speculative_decode_tree_gb300 import binding as B
from mla_speculative_decode_tree_gb300 import workloads as W
from oracle import kv4

# O is bf16: each value may be off by half its last place (2^-9 of it) from rounding once; the weights p carry at
# least 8 significant bits, so a convex sum of values v is off by at most 2^-8 * sum w |v| <= 2^-8 * max |v| more,
# plus fp32 sums.  LSE: the scores are fp32 sums of exact products and p is not rounded before its sum: an absolute
# error of about 2^-20 times the largest |score| (576 products), plus exp2 and log2 of 2^-21; 2e-4 covers |score| < 100.
LSE_ABS = 2e-4


def check(o, lse, o_ref, lse_ref, vmax, what=""):
    o = o.detach().float().cpu().numpy().astype(np.float64).reshape(o_ref.shape)
    lse = lse.detach().cpu().numpy().astype(np.float64).reshape(lse_ref.shape)
    fin = np.isfinite(lse_ref)
    assert np.array_equal(np.isfinite(lse), fin), what + ": -inf pattern of LSE differs"
    assert np.all(lse[~fin] == -np.inf) and np.all(o[~fin] == 0), what + ": rows with nothing visible"
    if fin.any():
        assert np.abs(lse - lse_ref)[fin].max() <= LSE_ABS, (what, np.abs(lse - lse_ref)[fin].max())
        bound = 2.0 ** -8 * np.abs(o_ref[fin]) + 2.0 ** -8 * vmax
        excess = np.abs(o - o_ref)[fin] - bound
        assert excess.max() <= 0, (what, excess.max(), vmax)
        norm = np.linalg.norm(o_ref[fin])
        assert np.linalg.norm((o - o_ref)[fin]) <= 2.0 ** -8 * norm + 1e-12, (what, norm)


def workload(B_, H, T_list, P_list, pool_rows, seed, spread=True, q_scale=1.0):
    """A varlen workload whose pool holds 4-bit rows (and garbage where nothing refers to)."""
    wl = W.varlen_workload(B_, H, T_list, P_list, pool_rows, seed)
    rng = np.random.default_rng(seed + 100)
    x = W.bf16_bits_to_f32(wl["pool"]).astype(np.float64)
    if spread:
        x = x * np.exp(0.4 * rng.standard_normal(576))
        x = W.bf16_bits_to_f32(W.f32_to_bf16_bits(x.astype(np.float32))).astype(np.float64)
    rows = rng.integers(0, 256, (pool_rows, kv4.ROW_BYTES)).astype(np.uint8)
    used = np.unique(np.concatenate([wl["kv_indices"], wl["out_cache_loc"][:wl["n_tokens"]]]))
    rows[used] = kv4.encode_rows(x[used, :512], x[used, 512:])
    wl["pool"] = rows
    if q_scale != 1.0:
        for k in ("q_nope", "q_rope"):
            wl[k] = W.f32_to_bf16_bits(W.bf16_bits_to_f32(wl[k]) * np.float32(q_scale))
    return wl


def device(wl):
    import torch
    t = lambda a, d: torch.from_numpy(np.ascontiguousarray(a)).cuda().view(d)  # noqa: E731
    idx = wl["kv_indices"] if wl["kv_indices"].size else np.zeros(1, np.int32)
    d = dict(q_nope=t(wl["q_nope"].view(np.int16), torch.bfloat16), q_rope=t(wl["q_rope"].view(np.int16), torch.bfloat16),
             kv_pool=t(wl["pool"], torch.uint8), kv_indptr=t(wl["kv_indptr"], torch.int32),
             kv_indices=t(idx.astype(np.int32), torch.int32),
             out_cache_loc=t(wl["out_cache_loc"], torch.int32), custom_mask=t(wl["custom_mask"], torch.uint8),
             mask_indptr=t(wl["mask_indptr"], torch.int32))
    if wl.get("qo_indptr") is not None:
        d["qo_indptr"] = t(wl["qo_indptr"].astype(np.int32), torch.int32)
    return d


def verifier(wl, nsplit=0, flags=0, max_batch=None):
    L = int(max([p + t for p, t in zip(wl["prefix_lens"], wl["T_list"])] + [wl["T"]]))
    return B.Verifier(max_batch or wl["B"], wl["H"], wl["T"], L, wl["pool"].shape[0], nsplit, flags | B.MLA_VERIFY_KV4)


def run_and_check(wl, nsplit=0, flags=0, what="", status=0, max_batch=None):
    import torch
    d, v = device(wl), verifier(wl, nsplit, flags, max_batch)
    v.o.fill_(float("nan"))
    v.lse.fill_(float("nan"))
    o, lse = v.run(d, wl["B"], wl["sm_scale"])
    torch.cuda.synchronize()
    assert v.status() == status, what
    n = wl["n_tokens"]
    o_ref, lse_ref = kv4.verify(wl)
    used = np.concatenate([wl["kv_indices"], wl["out_cache_loc"][:n]])
    used = used[(used >= 0) & (used < wl["pool"].shape[0])]
    vmax = np.abs(kv4.decode_rows(wl["pool"][used])[:, :512]).max() if used.size else 0.0
    check(o[:n], lse[:n], o_ref, lse_ref, vmax, what)
    if n < v.o.shape[0]:
        assert torch.isnan(v.o[n:]).all(), what + ": rows past the call's tokens were written"
    return v, o[:n], lse[:n]
