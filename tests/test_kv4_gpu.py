"""The 4-bit latent cache on the GPU against the fp64 oracle: store, load, tree-verify attention (both kernels,
every row-group size), KV relocation, streams, graphs, refused arguments, bounded waits."""

import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from mla_speculative_decode_tree_gb300 import binding as B  # noqa: E402
from mla_speculative_decode_tree_gb300 import workloads as W  # noqa: E402
from oracle import kv4  # noqa: E402
import kv4_util as U  # noqa: E402


# ---- attention --------------------------------------------------------------

SHAPES = [
    # B, H, T_list, P_list, nsplit
    (1, 16, [4], [256], 0),             # one row group, two tiles
    (1, 64, [9], [21], 0),              # prefix shorter than a tile
    (1, 8, [1], [0], 1),                # a single key: the draft itself
    (1, 1, [1], [1], 1),                # one row
    (1, 64, [9], [119], 3),             # 128 keys: one whole tile; empty splits
    (1, 64, [9], [120], 2),             # 129 keys: one key into the second tile
    (1, 5, [7], [1000], 4),             # odd heads
    (2, 13, [3, 7], [100, 700], 5),     # ragged
    (3, 8, [0, 2, 5], [40, 0, 333], 0),  # no drafts; no prefix
    (1, 128, [8], [515], 0),            # 1024 rows
    (4, 8, [1, 1, 1, 1], [1, 127, 128, 1025], 4),  # decode
    (1, 3, [64], [300], 2),             # the longest draft tree
    (1, 64, [9], [4096], 0),            # several tiles per split
    (1, 8, [9], [9000], 3),             # many tiles per split: the ring wraps
    (1, 16, [1], [9000], 2),
    (1, 24, [2], [9000], 2),
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("flags", [0, B.MLA_VERIFY_FORCE_SIMT], ids=["tc", "simt"])
def test_verify(shape, flags):
    b, h, t, p, ns = shape
    wl = U.workload(b, h, t, p, sum(p) + sum(t) + 50, seed=sum(p) + h)
    U.run_and_check(wl, ns, flags, str(shape))


@pytest.mark.parametrize("rows,nq", [(1, 16), (16, 16), (31, 32), (47, 48), (64, 64), (96, 48), (125, 64)])
@pytest.mark.parametrize("keys", [1, 130, 1500])
def test_every_row_group_size(rows, nq, keys):
    """A plan for many requests picks the row-group size of least work: each kernel built, the last group partial."""
    wl = U.workload(1, rows, [1], [keys - 1], 3000, seed=rows)
    v, _, _ = U.run_and_check(wl, 1, 0, "rows %d" % rows, max_batch=200)
    assert v.plan.describe().rows_per_cta == nq


@pytest.mark.parametrize("q_scale", [0.0, 1e-30, 0.1, 6.0, 40.0])
def test_score_ranges(q_scale):
    """From a flat softmax to one key that takes all the weight; queries far below and above one.

    (LSE tolerance: scores up to ~40 * 24 * 3 / 14; the relative part is 2^-20 of that.)"""
    wl = U.workload(1, 16, [3], [700], 900, seed=3, q_scale=q_scale)
    d, v = U.device(wl), U.verifier(wl, 3)
    o, lse = v.run(d, 1, wl["sm_scale"])
    o_ref, lse_ref = kv4.verify(wl)
    vmax = np.abs(kv4.decode_rows(wl["pool"][wl["kv_indices"]])[:, :512]).max()
    U.check(o, lse, o_ref, lse_ref, vmax, "q_scale %g" % q_scale)


def test_growing_scores_raise_the_running_max():
    """Scores that climb along the keys: every tile raises the maximum, so O is rescaled in every tile."""
    wl = U.workload(1, 16, [4], [1700], 2000, seed=9)
    x = np.zeros((2000, 576))
    rng = np.random.default_rng(5)
    x[:, :512] = rng.standard_normal((2000, 512))
    for j, r in enumerate(wl["kv_indices"]):
        x[r, 512] = 0.05 * j
    wl["pool"] = kv4.encode_rows(x[:, :512], x[:, 512:])
    qr = W.bf16_bits_to_f32(wl["q_rope"])
    qr[..., 0] = 14.0
    wl["q_rope"] = W.f32_to_bf16_bits(qr)
    U.run_and_check(wl, 2, 0, "climbing")


def test_one_key_above_many_small_ones():
    """One key ten above the rest, whose many small weights together still count."""
    wl = U.workload(1, 16, [1], [30000], 31000, seed=11, q_scale=0.02)
    x = np.random.default_rng(2).standard_normal((31000, 576))
    x[:, 512:] = 0
    x[wl["kv_indices"][17], 512] = 6.0
    wl["pool"] = kv4.encode_rows(x[:, :512], x[:, 512:])
    qr = np.zeros((1, 16, 64), np.float32)
    qr[..., 0] = 10 * np.sqrt(192.0) / 6
    wl["q_rope"] = W.f32_to_bf16_bits(qr)
    U.run_and_check(wl, 4, 0, "sink")


def test_rows_whose_mask_leaves_nothing():
    wl = U.workload(2, 8, [4, 3], [300, 17], 400, seed=2)
    bits = np.unpackbits(wl["custom_mask"], bitorder="little")
    L = [304, 20]
    bits[1 * L[0]:2 * L[0]] = 0                      # request 0, token 1 sees nothing
    at = int(wl["mask_indptr"][1])
    bits[at:at + 3 * L[1]] = 0                       # request 1 sees nothing at all
    bits[0:128] = 0                                  # request 0, token 0: nothing in the first tile
    wl["custom_mask"] = np.packbits(bits, bitorder="little")
    for flags in (0, B.MLA_VERIFY_FORCE_SIMT):
        for ns in (1, 2, 0):
            U.run_and_check(wl, ns, flags, "empty rows")


def test_masked_rows_may_hold_anything():
    """Rows that are masked for every token hold bytes that no store wrote (scales far outside the format)."""
    wl = U.workload(1, 16, [2], [400], 500, seed=4)
    bits = np.unpackbits(wl["custom_mask"], bitorder="little")
    m = bits[:2 * 402].reshape(2, 402)
    m[:, 100:260] = 0
    bits[:2 * 402] = m.reshape(-1)
    wl["custom_mask"] = np.packbits(bits, bitorder="little")
    wl["pool"][wl["kv_indices"][100:260]] = 0xFF
    U.run_and_check(wl, 2, 0, "masked garbage")


def test_rows_outside_the_pool_are_left_out_and_reported():
    wl = U.workload(1, 16, [3], [500], 600, seed=6)
    wl["kv_indices"] = wl["kv_indices"].copy()
    wl["kv_indices"][[3, 130, 499]] = [-1, 600, 2 ** 31 - 1]
    for flags in (0, B.MLA_VERIFY_FORCE_SIMT):
        U.run_and_check(wl, 2, flags, "bad rows", status=B.MLA_VERIFY_DEV_BAD_ROW)


def test_uniform_and_varlen_entries_agree():
    wl = U.workload(2, 8, [5, 5], [200, 77], 400, seed=8)
    d, v = U.device(wl), U.verifier(wl, 2)
    o1, l1 = (x.clone() for x in v.run(d, 2, wl["sm_scale"]))
    del d["qo_indptr"]
    o2, l2 = v.run(d, 2, wl["sm_scale"])
    assert torch.equal(o1, o2) and torch.equal(l1, l2)


def test_split_and_merge_entries_and_no_alloc_entry():
    wl = U.workload(1, 16, [4], [900], 1000, seed=12)
    d, v = U.device(wl), U.verifier(wl, 4)
    del d["qo_indptr"]
    o, lse = (x.clone() for x in v.run(d, 1, wl["sm_scale"]))
    args = (d["q_nope"], d["q_rope"], d["kv_pool"], d["kv_indptr"], d["kv_indices"], d["out_cache_loc"],
            d["custom_mask"], d["mask_indptr"], 1, wl["sm_scale"], 4)
    o2, l2 = torch.zeros_like(o), torch.zeros_like(lse)
    B.mla_verify_split(v.plan, *args, v.workspace)
    B.mla_verify_merge(v.plan, 1, 4, v.workspace, o2, l2)
    assert torch.equal(o, o2) and torch.equal(lse, l2)
    B.mla_verify_run_noalloc(v.plan, *args, o2.zero_(), l2.zero_())
    assert torch.equal(o, o2) and torch.equal(lse, l2)


def test_repeated_calls_give_the_same_bits():
    wl = U.workload(2, 64, [9, 4], [3000, 1234], 5000, seed=13)
    d, v = U.device(wl), U.verifier(wl)
    n = wl["n_tokens"]
    o, lse = (x[:n].clone() for x in v.run(d, 2, wl["sm_scale"]))
    for _ in range(3):
        o2, l2 = v.run(d, 2, wl["sm_scale"])
        assert torch.equal(o, o2[:n]) and torch.equal(lse, l2[:n])


def test_captured_graph_replays_with_new_contents_on_another_stream():
    wl = U.workload(1, 16, [4], [600], 700, seed=14)
    d, v = U.device(wl), U.verifier(wl)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        v.run(d, 1, wl["sm_scale"])
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        o, lse = v.run(d, 1, wl["sm_scale"])
    other = U.workload(1, 16, [4], [600], 700, seed=15)
    for k, x in U.device(other).items():
        d[k].copy_(x)
    g.replay()
    torch.cuda.synchronize()
    o_ref, lse_ref = kv4.verify(other)
    U.check(o, lse, o_ref, lse_ref, np.abs(kv4.decode_rows(other["pool"][other["kv_indices"]])[:, :512]).max())


def test_pool_offsets_past_32_bits():
    """Rows whose byte offset passes 2^32 (12 million rows of 384 bytes)."""
    rows = 12_000_000
    wl = U.workload(1, 8, [2], [300], 400, seed=16)
    far = wl["kv_indices"].astype(np.int64) + (rows - 400)
    loc = wl["out_cache_loc"].astype(np.int64) + (rows - 400)
    assert far.min() * 384 > 2 ** 32
    d = U.device(wl)
    pool = torch.zeros((rows, 384), dtype=torch.uint8, device="cuda")
    pool[rows - 400:] = d["kv_pool"]
    d["kv_pool"] = pool
    d["kv_indices"] = torch.from_numpy(far.astype(np.int32)).cuda()
    d["out_cache_loc"] = torch.from_numpy(loc.astype(np.int32)).cuda()
    v = B.Verifier(1, 8, 2, 302, rows, 0, B.MLA_VERIFY_KV4)
    o, lse = v.run(d, 1, wl["sm_scale"])
    o_ref, lse_ref = kv4.verify(wl)
    U.check(o, lse, o_ref, lse_ref, np.abs(kv4.decode_rows(wl["pool"][wl["kv_indices"]])[:, :512]).max())
    out = torch.empty((300, 576), dtype=torch.bfloat16, device="cuda")
    B.mla_verify_load_kv4(v.plan, pool, d["kv_indices"], out[:, :512], out[:, 512:], v.workspace)
    assert np.array_equal(out[:, :512].double().cpu().numpy(), kv4.decode_rows(wl["pool"][wl["kv_indices"]])[:, :512])
    again = torch.zeros_like(pool)
    B.mla_verify_store_kv4(v.plan, out[:, :512], out[:, 512:], d["kv_indices"], again, v.workspace)
    h = host(out)
    assert np.array_equal(again[rows - 400:].cpu().numpy()[far - (rows - 400)], kv4.encode_rows(h[:, :512], h[:, 512:]))
    assert int(again.any(dim=1).sum()) == 300  # and no other row


def test_batch_beyond_and_below_the_plan():
    """A plan for 3 requests runs 0, 1 and 3 of them; the rest is not written."""
    wl = U.workload(3, 8, [2, 3, 1], [50, 60, 70], 300, seed=17)
    d, v = U.device(wl), U.verifier(wl, 2)
    ref_o, ref_l = kv4.verify(wl)
    v.o.fill_(7)
    v.run(d, 0, wl["sm_scale"])
    torch.cuda.synchronize()
    assert bool((v.o == 7).all())
    v.run(d, 1, wl["sm_scale"])
    torch.cuda.synchronize()
    assert bool((v.o[2:] == 7).all())
    vmax = np.abs(kv4.decode_rows(wl["pool"][wl["kv_indices"]])[:, :512]).max()
    U.check(v.o[:2], v.lse[:2], ref_o[:16], ref_l[:16], vmax)
    with pytest.raises(B.MlaVerifyError):
        v.run(d, 4, wl["sm_scale"])


def test_stalled_expansion_times_out_and_reports():
    """A block that is never signalled: every wait gives up after its limit, the call reports it, the next is right."""
    wl = U.workload(1, 16, [4], [300], 400, seed=18)
    d = U.device(wl)
    v = U.verifier(wl, 1, B.MLA_VERIFY_TEST_STALL_GATHER)
    v.run(d, 1, wl["sm_scale"])
    assert v.status() & B.MLA_VERIFY_DEV_TIMEOUT
    U.run_and_check(wl, 1, 0, "after the stall")


def test_relocated_rows_give_the_same_bits():
    wl = U.workload(2, 8, [3, 2], [400, 150], 2000, seed=19)
    # rows below 550 free: move the used ones up
    used = np.concatenate([wl["kv_indices"], wl["out_cache_loc"][:5]])
    new = 600 + np.random.default_rng(0).permutation(1300)[:used.size]
    pool = np.zeros_like(wl["pool"])
    pool[new] = wl["pool"][used]
    wl["pool"] = pool
    wl["kv_indices"], wl["out_cache_loc"][:5] = new[:550].astype(np.int32), new[550:]
    d, v = U.device(wl), U.verifier(wl, 3)
    o, lse = (x[:5].clone() for x in v.run(d, 2, wl["sm_scale"]))
    B.mla_verify_relocate_kv(v.plan, d["kv_pool"], d["kv_indptr"], d["kv_indices"],
                             torch.tensor([0, 400], dtype=torch.int32, device="cuda"), 2, v.workspace)
    assert torch.equal(d["kv_indices"].cpu(), torch.arange(550, dtype=torch.int32))
    assert torch.equal(d["kv_pool"][:550].cpu(), torch.from_numpy(pool[new[:550]]))
    o2, l2 = v.run(d, 2, wl["sm_scale"])
    assert torch.equal(o, o2[:5]) and torch.equal(lse, l2[:5]) and v.status() == 0


# ---- store and load -----------------------------------------------------------

def plan(pool_rows, max_batch=1, max_kv=1, q_len=1):
    p = B.mla_verify_plan(max_batch, 1, q_len, max_kv, pool_rows, 1, flags=B.MLA_VERIFY_KV4)
    return p, torch.zeros(p.workspace_bytes, dtype=torch.uint8, device="cuda")


def host(x):
    return x.float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 63, 1000, 4099])
@pytest.mark.parametrize("layout", ["one", "split", "strided"])
def test_store_then_load(n, layout):
    g = torch.Generator(device="cuda").manual_seed(n)
    x = torch.randn((n, 576), generator=g, device="cuda") * torch.exp(torch.randn(576, generator=g, device="cuda"))
    x = x.to(torch.bfloat16)
    if layout == "one":
        lat, rope = x[:, :512], x[:, 512:]
    elif layout == "split":
        lat, rope = x[:, :512].contiguous(), x[:, 512:].contiguous()
    else:
        big = torch.zeros((n, 4, 640), dtype=torch.bfloat16, device="cuda")
        big[:, 1, 64:] = x
        lat, rope = big[:, 1, 64:576], big[:, 1, 576:]
    p, ws = plan(n + 100)
    slots = torch.randperm(n + 100, generator=g, device="cuda")[:n].to(torch.int32)
    pool = torch.full((n + 100, 384), 0xAB, dtype=torch.uint8, device="cuda")
    B.mla_verify_store_kv4(p, lat, rope, slots, pool, ws)
    expected = np.full((n + 100, 384), 0xAB, np.uint8)
    expected[slots.cpu().numpy()] = kv4.encode_rows(host(lat), host(rope))
    assert np.array_equal(pool.cpu().numpy(), expected)  # bit for bit, and nothing else written
    out = torch.full((n, 3, 704), 7.0, dtype=torch.bfloat16, device="cuda")
    B.mla_verify_load_kv4(p, pool, slots, out[:, 1, 8:520], out[:, 1, 600:664], ws)
    v = kv4.decode_rows(expected[slots.cpu().numpy()])
    as_bf16 = torch.from_numpy(v).float().to(torch.bfloat16)
    assert torch.equal(out[:, 1, 8:520].cpu(), as_bf16[:, :512])
    assert torch.equal(out[:, 1, 600:664].cpu(), as_bf16[:, 512:])
    out[:, 1, 8:520], out[:, 1, 600:664] = 7.0, 7.0
    assert bool((out == 7.0).all())
    assert B.mla_verify_read_status(p, ws) == 0


def test_store_every_bf16_value():
    """All 65536 bit patterns (as latents and as RoPE), infinities, NaN and denormals among them."""
    bits = np.random.default_rng(0).permutation(65536).astype(np.uint16)
    bits = np.concatenate([bits, np.zeros(-65536 % 576, np.uint16)]).reshape(-1, 576)
    sorted_bits = np.sort(bits.reshape(-1)).reshape(-1, 576)  # groups of like magnitude
    for b in (bits, sorted_bits):
        x = torch.from_numpy(b.view(np.int16)).cuda().view(torch.bfloat16)
        n = x.shape[0]
        p, ws = plan(n)
        pool = torch.zeros((n, 384), dtype=torch.uint8, device="cuda")
        B.mla_verify_store_kv4(p, x[:, :512], x[:, 512:], torch.arange(n, dtype=torch.int32, device="cuda"), pool, ws)
        h = W.bf16_bits_to_f32(b).astype(np.float64)
        assert np.array_equal(pool.cpu().numpy(), kv4.encode_rows(h[:, :512], h[:, 512:]))


def test_slots_without_a_row():
    n = 70
    x = torch.randn((n, 576), device="cuda").to(torch.bfloat16)
    p, ws = plan(50)
    slots = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    slots[5], slots[66] = 3, 49
    pool = torch.zeros((51, 384), dtype=torch.uint8, device="cuda")
    B.mla_verify_store_kv4(p, x[:, :512], x[:, 512:], slots, pool, ws)
    assert B.mla_verify_read_status(p, ws) == 0  # -1 is a token without a slot
    assert pool.any(dim=1).nonzero().flatten().tolist() == [3, 49]
    out = torch.full((n, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    B.mla_verify_load_kv4(p, pool, slots, out[:, :512], out[:, 512:], ws)
    assert out.any(dim=1).nonzero().flatten().tolist() == [5, 66]
    for bad in (50, -2, 2 ** 31 - 1):
        slots[0] = bad
        before = pool.clone()
        B.mla_verify_store_kv4(p, x[:, :512], x[:, 512:], slots, pool, ws)
        assert B.mla_verify_read_status(p, ws) == B.MLA_VERIFY_DEV_BAD_ROW
        assert torch.equal(pool, before)
        B.mla_verify_load_kv4(p, pool, slots, out[:, :512], out[:, 512:], ws)
        assert B.mla_verify_read_status(p, ws) == B.MLA_VERIFY_DEV_BAD_ROW and not bool(out[0].any())


def test_no_tokens():
    p, ws = plan(4)
    e = torch.empty((0, 576), dtype=torch.bfloat16, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    pool = torch.zeros((4, 384), dtype=torch.uint8, device="cuda")
    B.mla_verify_store_kv4(p, e[:, :512], e[:, 512:], none, pool, ws)
    B.mla_verify_load_kv4(p, pool, none, e[:, :512], e[:, 512:], ws)


# ---- a whole step -----------------------------------------------------------------

def test_slots_store_mask_verify_in_one_graph():
    """The step as a server runs it: slot maps, store, tree mask, attention, one captured graph."""
    H, T, page = 8, 4, 16
    P, Tn = [33, 0, 200], [4, 2, 3]
    rng = np.random.default_rng(1)
    pages = rng.permutation(40)
    table = np.full((3, 16), -1, np.int32)
    k = 0
    for b, x in enumerate(P):
        n = -(-x // page)
        table[b, :n] = pages[k:k + n]
        k += n
    i32 = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()  # noqa: E731
    v = B.Verifier(3, H, T, 210, 640, 0, B.MLA_VERIFY_KV4)
    z = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    bt, free, used = i32(table), i32(pages[k:]), z(1)
    seq, new, kvp, kvi, qop, loc, mp = i32(P), i32(Tn), z(4), z(300), z(4), z(3 * T), z(3)
    mask = torch.zeros(3 * T * 220 // 8 + 8, dtype=torch.uint8, device="cuda")
    parents = i32([-1, 0, 0, 2, -1, 0, -1, 0, 1] + [0] * 3)
    tokens = torch.from_numpy(rng.standard_normal((3 * T, 576)).astype(np.float32)).cuda().to(torch.bfloat16)
    qn = torch.from_numpy(rng.standard_normal((3 * T, H, 512)).astype(np.float32)).cuda().to(torch.bfloat16)
    qr = torch.from_numpy(rng.standard_normal((3 * T, H, 64)).astype(np.float32)).cuda().to(torch.bfloat16)
    old = rng.standard_normal((640, 576))
    pool = torch.from_numpy(kv4.encode_rows(old[:, :512], old[:, 512:])).cuda()

    def step():
        loc.fill_(-1)
        B.mla_verify_build_slots(v.plan, seq, new, 3, page, bt, free, used, kvp, kvi, qop, loc, v.workspace)
        B.mla_verify_store_kv4(v.plan, tokens[:, :512], tokens[:, 512:], loc, pool, v.workspace)
        B.mla_verify_build_tree_mask_varlen(v.plan, parents, kvp, qop, 3, mask, mp)
        return v.run(dict(q_nope=qn, q_rope=qr, kv_pool=pool, kv_indptr=kvp, kv_indices=kvi, qo_indptr=qop,
                          out_cache_loc=loc, custom_mask=mask, mask_indptr=mp), 3, 192 ** -0.5)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        o, lse = step()
    g.replay()
    torch.cuda.synchronize()
    assert v.status() == 0
    ref, _, _ = kv4.build_slots(P, Tn, page, table, pages[k:], 640)
    assert kvi[:233].tolist() == ref["kv_indices"] and loc[:9].tolist() == ref["out_cache_loc"]
    assert bt.tolist() == ref["block_table"].tolist() and used.item() == ref["pages_used"]
    h_pool = kv4.encode_rows(old[:, :512], old[:, 512:])
    h_tok = host(tokens)[:9]
    h_pool[ref["out_cache_loc"]] = kv4.encode_rows(h_tok[:, :512], h_tok[:, 512:])
    assert np.array_equal(h_pool, pool.cpu().numpy())
    to_bits = lambda x: x.cpu().view(torch.int16).numpy().view(np.uint16)  # noqa: E731
    wl = dict(B=3, H=H, T=T, pool=h_pool, q_nope=to_bits(qn), q_rope=to_bits(qr), kv_indptr=np.array(ref["kv_indptr"]),
              kv_indices=np.array(ref["kv_indices"]), qo_indptr=np.array(ref["qo_indptr"]),
              out_cache_loc=np.array(ref["out_cache_loc"]), custom_mask=mask.cpu().numpy(),
              mask_indptr=mp.cpu().numpy(), sm_scale=192 ** -0.5)
    o_ref, lse_ref = kv4.verify(wl)
    U.check(o[:9], lse[:9], o_ref, lse_ref, np.abs(kv4.decode_rows(h_pool)[:, :512]).max())
