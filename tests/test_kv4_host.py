"""The 4-bit operators' argument checks and plan choices, which need no GPU:
every refused call fails before any device work."""

import ctypes

import pytest
import torch

from mla_speculative_decode_tree_gb300 import binding as B

FAKE = 0x10000  # never dereferenced
EINVAL, EWS, OK = B.MLA_VERIFY_EINVAL, B.MLA_VERIFY_EWORKSPACE, B.MLA_VERIFY_OK


@pytest.fixture(scope="module")
def lib():
    from mla_speculative_decode_tree_gb300 import build
    build.build()
    return B.load()


def plan(**kw):
    args = dict(max_batch=2, num_heads=64, q_len=9, max_kv_len=4105, pool_rows=262144, nsplit=0,
                flags=B.MLA_VERIFY_KV4)
    args.update(kw)
    return B.mla_verify_plan(**args)


def up(x, a):
    return -(-x // a) * a


@pytest.mark.parametrize("flags", [B.MLA_VERIFY_FUSED_MERGE, B.MLA_VERIFY_REFETCH_VALUES,
                                   B.MLA_VERIFY_FUSED_MERGE | B.MLA_VERIFY_REFETCH_VALUES])
def test_flags_of_the_bf16_kernel_are_refused(lib, flags):
    with pytest.raises(B.MlaVerifyError) as e:
        plan(flags=B.MLA_VERIFY_KV4 | flags)
    assert e.value.code == EINVAL


@pytest.mark.parametrize("change", [dict(q_len=0), dict(q_len=65), dict(num_heads=0), dict(max_batch=0),
                                    dict(nsplit=-1), dict(pool_rows=0), dict(max_kv_len=8)])
def test_sizes_that_no_plan_takes(lib, change):
    with pytest.raises(B.MlaVerifyError) as e:
        plan(**change)
    assert e.value.code == EINVAL


@pytest.mark.parametrize("batch,heads,q_len,kv", [(1, 64, 9, 4105), (1, 8, 9, 185009), (16, 8, 1, 33000),
                                                   (3, 128, 64, 5000), (200, 1, 1, 1), (1, 7, 3, 130)])
def test_equal_pieces_workspace(lib, batch, heads, q_len, kv):
    """nsplit = 0: one CTA per SM takes a piece of the work; a partial of
    rows_per_cta rows per piece and per row group, behind a table of 8 bytes per
    row group."""
    p = plan(max_batch=batch, num_heads=heads, q_len=q_len, max_kv_len=kv)
    i = p.describe()
    assert i.kernel == 1 and i.rows_per_cta in (16, 32, 48, 64) and i.keys_per_tile == 128
    assert i.grid_x >= 1 and i.grid_y == 1 and i.grid_z == 1
    spans = batch * -(-heads * q_len // i.rows_per_cta)
    rows = (spans + i.grid_x) * i.rows_per_cta
    off_lse = up(256 + 8 * spans, 256)
    off_o = up(off_lse + 4 * rows, 256)
    assert p.workspace_bytes == i.workspace_bytes == off_o + 4 * rows * 512
    assert i.merge_blocks > 0 and 0 < i.smem_bytes <= 227 * 1024


@pytest.mark.parametrize("flags", [0, B.MLA_VERIFY_FORCE_SIMT])
def test_chunk_grid_workspace(lib, flags):
    """nsplit >= 1: the grid and workspace of a bf16 pool's plan."""
    p = plan(nsplit=16, flags=B.MLA_VERIFY_KV4 | flags)
    i = p.describe()
    rows = 2 * 9 * 64
    assert i.kernel == (0 if flags else 1)
    assert (i.grid_x, i.grid_y, i.grid_z) == (-(-576 // i.rows_per_cta), 16, 2)
    assert p.workspace_bytes == up(256 + 4 * 16 * rows, 256) + 4 * 16 * rows * 512


def test_run_is_checked_as_with_a_bf16_pool(lib):
    p = plan()

    def run(batch=1, nsplit=0, ws=FAKE, short=0, q=FAKE, pool=FAKE, idx=FAKE, o=FAKE, lse=FAKE):
        return lib.mla_verify_run_varlen(ctypes.c_void_p(p.handle), q, q, pool, idx, idx, idx, idx, FAKE, idx, batch,
                                         0.07, nsplit, ws, p.workspace_bytes - short, o, lse, None)

    assert run(batch=0) == OK
    for bad in (dict(batch=3), dict(batch=-1), dict(nsplit=4), dict(q=FAKE + 2), dict(pool=FAKE + 8), dict(pool=None),
                dict(idx=FAKE + 2), dict(o=FAKE + 8), dict(o=None), dict(lse=FAKE + 1), dict(ws=FAKE + 16)):
        assert run(**bad) == EINVAL, bad
    assert run(short=1) == EWS and run(ws=None) == EWS


@pytest.mark.parametrize("name", ["mla_verify_store_kv4", "mla_verify_load_kv4"])
def test_store_and_load_refusals(lib, name):
    p, bf16 = plan(), plan(flags=0, nsplit=4)
    fn = getattr(lib, name)

    def call(pl=p, latent=FAKE, ls=512, rope=FAKE, rs=64, slots=FAKE, n=1, pool=FAKE, ws=FAKE, short=0):
        h = ctypes.c_void_p(pl.handle) if pl else None
        size = (pl or p).workspace_bytes - short
        if name.endswith("store_kv4"):
            return fn(h, latent, ls, rope, rs, slots, n, pool, ws, size, None)
        return fn(h, pool, slots, n, latent, ls, rope, rs, ws, size, None)

    assert call(n=0) == OK
    assert call(n=0, latent=None, rope=None, slots=None, pool=None, ws=None) == OK
    for bad in (dict(pl=None), dict(pl=bf16), dict(n=-1), dict(n=1 << 31), dict(latent=None), dict(rope=None),
                dict(slots=None), dict(pool=None), dict(latent=FAKE + 2), dict(rope=FAKE + 8), dict(slots=FAKE + 2),
                dict(pool=FAKE + 8), dict(ls=511), dict(ls=0), dict(ls=-512), dict(ls=516), dict(rs=63), dict(rs=66),
                dict(ls=(1 << 31) + 8), dict(rs=1 << 40), dict(ws=FAKE + 16)):
        assert call(**bad) == EINVAL, bad
    assert call(ws=None) == EWS and call(short=1) == EWS


@pytest.mark.parametrize("kv4", [True, False])
def test_build_slots_refusals(lib, kv4):
    p = plan(max_batch=8) if kv4 else plan(max_batch=8, flags=0, nsplit=4)

    def call(handle=p.handle, seq=FAKE, new=FAKE, batch=2, page=64, table=FAKE, cols=4, free=FAKE, nfree=3, used=FAKE,
             indptr=FAKE, idx=FAKE, cap=100, qo=FAKE, loc=FAKE, loc_cap=18, ws=FAKE, short=0):
        return lib.mla_verify_build_slots(ctypes.c_void_p(handle), seq, new, batch, page, table, cols, free, nfree,
                                          used, indptr, idx, cap, qo, loc, loc_cap, ws, p.workspace_bytes - short,
                                          None)

    assert call(batch=0) == OK
    for bad in (dict(handle=None), dict(batch=-1), dict(batch=9), dict(page=0), dict(page=-64), dict(cols=0),
                dict(nfree=-1), dict(cap=-1), dict(loc_cap=-1), dict(seq=None), dict(table=None), dict(used=None),
                dict(indptr=None), dict(qo=None), dict(free=None), dict(idx=None), dict(loc=None), dict(ws=FAKE + 16),
                *({k: FAKE + 2} for k in ("seq", "new", "table", "free", "used", "indptr", "idx", "qo", "loc"))):
        assert call(**bad) == EINVAL, bad
    assert call(ws=None) == EWS and call(short=1) == EWS


def test_build_slots_batch_limit(lib):
    p = plan(max_batch=4097, num_heads=1, q_len=1, max_kv_len=64)
    rc = lib.mla_verify_build_slots(ctypes.c_void_p(p.handle), FAKE, FAKE, 4097, 64, FAKE, 1, FAKE, 1, FAKE, FAKE,
                                    FAKE, 1, FAKE, FAKE, 1, FAKE, p.workspace_bytes, None)
    assert rc == EINVAL


def test_python_calls_check_types_shapes_and_strides(lib):
    p = plan()
    ws = torch.zeros(256, dtype=torch.uint8)
    pool = torch.zeros(8, 384, dtype=torch.uint8)
    latent, rope = torch.zeros(4, 512, dtype=torch.bfloat16), torch.zeros(4, 64, dtype=torch.bfloat16)
    slots = torch.zeros(4, dtype=torch.int32)
    for lat, rop, slo in ((latent.float(), rope, slots), (latent[:, :256], rope, slots), (latent[:3], rope, slots),
                          (latent, rope.half(), slots), (latent, rope[:, ::2], slots),
                          (latent.t().contiguous().t(), rope, slots), (latent, rope, slots.long()),
                          (latent, rope, torch.zeros(8, dtype=torch.int32)[::2])):
        with pytest.raises(ValueError):
            B.mla_verify_store_kv4(p, lat, rop, slo, pool, ws)
        with pytest.raises(ValueError):
            B.mla_verify_load_kv4(p, pool, slo, lat, rop, ws)

    def i32(n):
        return torch.zeros(n, dtype=torch.int32)

    good = dict(seq_lens=i32(2), new_lens=i32(2), batch=2, page_size=4, block_table=i32((2, 3)), free_pages=i32(2),
                pages_used=i32(1), kv_indptr=i32(3), kv_indices=i32(9), qo_indptr=i32(3), out_cache_loc=i32(4),
                workspace=ws)
    for bad in (dict(seq_lens=i32(1)), dict(new_lens=i32(1)), dict(kv_indptr=i32(2)), dict(qo_indptr=i32(2)),
                dict(block_table=i32((1, 3))), dict(seq_lens=i32(2).long()), dict(kv_indices=i32(18)[::2]),
                dict(block_table=i32((3, 2)).t())):
        with pytest.raises(ValueError):
            B.mla_verify_build_slots(p, **{**good, **bad})
