"""Argument checks of the operators around a verify step, which need no GPU: every refused call fails before any
device work."""

import ctypes

import pytest
import torch

from mla_speculative_decode_tree_gb300 import binding as B

F = 0x10000  # never dereferenced
EINVAL, EWS, OK = B.MLA_VERIFY_EINVAL, B.MLA_VERIFY_EWORKSPACE, B.MLA_VERIFY_OK


@pytest.fixture(scope="module")
def lib():
    from mla_speculative_decode_tree_gb300 import build
    build.build()
    return B.load()


def plan(**kw):
    args = dict(max_batch=4, num_heads=16, q_len=5, max_kv_len=500, pool_rows=1000, nsplit=0)
    args.update(kw)
    return B.mla_verify_plan(**args)


def shared_plan(**kw):
    return plan(flags=B.MLA_VERIFY_SHARED | kw.pop("flags", 0), **kw)


@pytest.mark.parametrize("change", [dict(nsplit=1), dict(max_batch=1025), dict(flags=B.MLA_VERIFY_KV4),
                                    dict(flags=B.MLA_VERIFY_FUSED_MERGE), dict(flags=B.MLA_VERIFY_REFETCH_VALUES)])
def test_shared_plans_that_are_refused(lib, change):
    with pytest.raises(B.MlaVerifyError) as e:
        shared_plan(**change)
    assert e.value.code == EINVAL


@pytest.mark.parametrize("batch,heads,q_len", [(1, 1, 1), (64, 8, 1), (16, 64, 9), (1024, 1, 64), (3, 128, 7)])
def test_shared_workspace(lib, batch, heads, q_len):
    """A table entry per row and part, then partials: a place per row and part and 128 rows for each CTA pair."""
    p = shared_plan(max_batch=batch, num_heads=heads, q_len=q_len)
    i = p.describe()
    rows = batch * heads * q_len
    assert i.kernel == 1 and i.rows_per_cta == 128 and i.keys_per_tile == 64
    parts = 2 * rows + 128 * i.grid_x
    lse = -(-(256 + 16 * rows) // 256) * 256
    o = -(-(lse + 4 * parts) // 256) * 256
    assert p.workspace_bytes == i.workspace_bytes == o + 2048 * parts
    assert shared_plan(flags=B.MLA_VERIFY_FORCE_SIMT).describe().kernel == 0


def call_shared(lib, p, **change):
    a = dict(q=F, qr=F, kv=F, gp=F, sp=F, si=F, kp=F, ki=F, qo=F, loc=F, cm=F, mp=F, batch=4, groups=2, scale=0.1, ws=F,
             n=p.workspace_bytes, o=F, lse=F)
    a.update(change)
    P = ctypes.c_void_p
    return lib.mla_verify_run_shared(P(p.handle), a["q"], a["qr"], a["kv"], a["gp"], a["sp"], a["si"], a["kp"], a["ki"],
                                     a["qo"], a["loc"], a["cm"], a["mp"], a["batch"], a["groups"], a["scale"], a["ws"],
                                     a["n"], a["o"], a["lse"], None)


@pytest.mark.parametrize("change", [dict(q=None), dict(qr=None), dict(kv=None), dict(gp=None), dict(sp=None), dict(kp=None),
                                    dict(loc=None), dict(cm=None), dict(mp=None), dict(o=None), dict(lse=None),
                                    dict(q=F + 8), dict(kv=F + 8), dict(o=F + 8), dict(gp=F + 2), dict(sp=F + 1),
                                    dict(si=F + 2), dict(qo=F + 2), dict(lse=F + 2), dict(batch=-1), dict(batch=5),
                                    dict(groups=0), dict(groups=5), dict(scale=float("nan")), dict(scale=float("inf")),
                                    dict(ws=F + 128)])
def test_shared_arguments(lib, change):
    assert call_shared(lib, shared_plan(), **change) == EINVAL


def test_shared_workspace_and_plans_of_other_calls(lib):
    p = shared_plan()
    assert call_shared(lib, p, ws=None) == EWS
    assert call_shared(lib, p, n=p.workspace_bytes - 1) == EWS
    assert call_shared(lib, p, batch=0, q=None) == OK
    assert call_shared(lib, plan(nsplit=1)) == EINVAL  # a plan without the flag
    P = ctypes.c_void_p
    args = [P(p.handle)] + [F] * 8 + [1, 0.1, 0, F, p.workspace_bytes]
    assert lib.mla_verify_run(*args, F, F, None) == EINVAL  # and no other run takes a plan with it
    assert lib.mla_verify_split(*args, None) == EINVAL
    assert lib.mla_verify_merge(P(p.handle), 1, 0, F, p.workspace_bytes, F, F, None) == EINVAL
    assert lib.mla_verify_run_noalloc(P(p.handle), *[F] * 8, 1, 0.1, 0, F, F, None) == EINVAL


def call_accept(lib, p, **change):
    a = dict(t=F, ts=100, d=F, ds=100, v=100, tok=F, par=F, qo=F, u=F, un=F, batch=4, acc=F, num=F, nxt=F, ws=F,
             n=p.workspace_bytes)
    a.update(change)
    return lib.mla_verify_accept_drafts(ctypes.c_void_p(p.handle), a["t"], a["ts"], a["d"], a["ds"], a["v"], a["tok"],
                                        a["par"], a["qo"], a["u"], a["un"], a["batch"], a["acc"], a["num"], a["nxt"],
                                        a["ws"], a["n"], None)


@pytest.mark.parametrize("change", [dict(t=None), dict(tok=None), dict(par=None), dict(u=None), dict(un=None), dict(acc=None),
                                    dict(num=None), dict(nxt=None), dict(t=F + 2), dict(d=F + 1), dict(qo=F + 2),
                                    dict(ts=99), dict(ds=99), dict(v=0), dict(v=(1 << 30) + 1), dict(batch=-1),
                                    dict(batch=5), dict(ws=F + 16)])
def test_accept_arguments(lib, change):
    assert call_accept(lib, plan(nsplit=1), **change) == EINVAL


def test_accept_workspace_and_nothing_to_do(lib):
    p = plan(nsplit=1)
    assert call_accept(lib, p, ws=None) == EWS and call_accept(lib, p, n=10) == EWS
    assert call_accept(lib, p, batch=0, t=None) == OK


def call_commit(lib, p, **change):
    a = dict(kv=F, layers=2, stride=1000 * 1152, qo=F, loc=F, acc=F, num=F, batch=4, lens=F, new=F, page=16, tab=F, mp=9,
             refs=F, pages=50, ws=F, n=p.workspace_bytes)
    a.update(change)
    return lib.mla_verify_commit_drafts(ctypes.c_void_p(p.handle), a["kv"], a["layers"], a["stride"], a["qo"], a["loc"],
                                        a["acc"], a["num"], a["batch"], a["lens"], a["new"], a["page"], a["tab"], a["mp"],
                                        a["refs"], a["pages"], a["ws"], a["n"], None)


POOL = [dict(kv=None), dict(kv=F + 8), dict(layers=0), dict(stride=-16), dict(stride=1000 * 1152 + 8),
        dict(stride=1000 * 1152 - 16)]


@pytest.mark.parametrize("change", POOL + [dict(loc=None), dict(acc=None), dict(num=None), dict(lens=None), dict(new=None),
                                           dict(loc=F + 2), dict(qo=F + 2), dict(tab=None), dict(refs=None), dict(page=0),
                                           dict(mp=0), dict(pages=-1), dict(batch=5), dict(batch=-1), dict(ws=F + 64)])
def test_commit_arguments(lib, change):
    assert call_commit(lib, plan(nsplit=1), **change) == EINVAL


def call_fork(lib, p, **change):
    a = dict(kv=F, layers=2, stride=1000 * 1152, src=F, dst=F, m=3, page=16, tab=F, reqs=8, mp=9, lens=F, refs=F, pages=50,
             free=F, nf=20, used=F, ws=F, n=p.workspace_bytes)
    a.update(change)
    return lib.mla_verify_fork(ctypes.c_void_p(p.handle), a["kv"], a["layers"], a["stride"], a["src"], a["dst"], a["m"],
                               a["page"], a["tab"], a["reqs"], a["mp"], a["lens"], a["refs"], a["pages"], a["free"], a["nf"],
                               a["used"], a["ws"], a["n"], None)


@pytest.mark.parametrize("change", POOL + [dict(src=None), dict(dst=None), dict(tab=None), dict(lens=None), dict(refs=None),
                                           dict(used=None), dict(free=None), dict(m=-1), dict(m=4097), dict(page=0),
                                           dict(reqs=0), dict(mp=0), dict(pages=0), dict(nf=-1), dict(src=F + 2),
                                           dict(ws=F + 64)])
def test_fork_arguments(lib, change):
    assert call_fork(lib, plan(nsplit=1), **change) == EINVAL


def test_release_and_free_list_arguments(lib):
    p = plan(nsplit=1)
    P = ctypes.c_void_p(p.handle)
    good = [P, F, 3, 16, F, 8, 9, F, F, 50, F, p.workspace_bytes, None]
    for at, bad in [(1, None), (1, F + 2), (2, -1), (2, 4097), (3, 0), (4, None), (5, 0), (6, 0), (7, None), (8, None),
                    (9, 0), (10, F + 64)]:
        a = list(good)
        a[at] = bad
        assert lib.mla_verify_release(*a) == EINVAL, at
    a = list(good)
    a[10] = None
    assert lib.mla_verify_release(*a) == EWS
    a[2] = 0
    assert lib.mla_verify_release(*a) == OK
    for a in ([None, F, 5, F, F, None], [P, None, 5, F, F, None], [P, F, 5, None, F, None], [P, F, 5, F, None, None],
              [P, F, -1, F, F, None], [P, F + 2, 5, F, F, None]):
        assert lib.mla_verify_list_free_pages(*a) == EINVAL
    p2 = plan(nsplit=1)
    assert call_commit(lib, p2, batch=0, kv=None) == OK and call_fork(lib, p2, m=0, kv=None) == OK
    assert call_commit(lib, p2, ws=None) == EWS and call_fork(lib, p2, n=1) == EWS


def test_the_binding_refuses_other_types_and_shapes():
    p = plan(nsplit=1)
    i32 = dict(dtype=torch.int32)
    n = 4 * 5
    ok = dict(target_probs=torch.zeros(n, 7), draft_probs=None, draft_tokens=torch.zeros(n, **i32),
              parents=torch.zeros(n, **i32), qo_indptr=None, uniform=torch.zeros(n), uniform_next=torch.zeros(4), batch=4,
              accepted=torch.zeros(4, 5, **i32), num_accepted=torch.zeros(4, **i32), next_tokens=torch.zeros(4, **i32),
              workspace=torch.zeros(1))
    for name, bad in (("target_probs", torch.zeros(n, 7).half()), ("target_probs", torch.zeros(7, n).t()),
                      ("target_probs", torch.zeros(n - 1, 7)), ("draft_probs", torch.zeros(n, 6)),
                      ("draft_probs", torch.zeros(n - 1, 7)), ("draft_tokens", torch.zeros(n).long()),
                      ("uniform", torch.zeros(n).double()), ("uniform_next", torch.zeros(3)),
                      ("accepted", torch.zeros(3, 5, **i32)), ("num_accepted", torch.zeros(8, **i32)[::2])):
        with pytest.raises(ValueError):
            B.mla_verify_accept_drafts(p, **{**ok, name: bad}, stream=0)
    pool = torch.zeros(2, 1000, 576, dtype=torch.bfloat16)
    for bad in (pool.float(), pool[:, :999], pool[:, :, :575], torch.zeros(1000, 1152, dtype=torch.bfloat16)[:, :576]):
        with pytest.raises(ValueError):
            B._layers_of(p, bad)
    assert B._layers_of(p, pool) == (2, 1000 * 1152) and B._layers_of(p, pool[0]) == (1, 0)
    with pytest.raises(ValueError):
        B.mla_verify_list_free_pages(p, torch.zeros(5, **i32), torch.zeros(4, **i32), torch.zeros(1, **i32), stream=0)
