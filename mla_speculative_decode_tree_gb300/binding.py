"""Python binding of libmlaverify.so (argument marshalling only).

The functions carry the names of the C ABI in ``include/mla_verify.h`` and
take torch tensors (device memory) or raw integers.  Every step of the verify
path runs in the library's CUDA kernels; there is no Python or CPU fallback:
if the library is missing or the device is unsupported, the call raises.
"""

from __future__ import annotations

import ctypes
import os
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmlaverify.so")

MLA_VERIFY_OK = 0
MLA_VERIFY_EINVAL = 1
MLA_VERIFY_EUNSUPPORTED = 2
MLA_VERIFY_EWORKSPACE = 3
MLA_VERIFY_ECUDA = 4
MLA_VERIFY_DEV_BAD_ROW = 0x1
MLA_VERIFY_DEV_TIMEOUT = 0x2
MLA_VERIFY_DEV_NO_PAGE = 0x4
MLA_VERIFY_DEV_CAPACITY = 0x8
MLA_VERIFY_FORCE_SIMT = 0x1
MLA_VERIFY_FUSED_MERGE = 0x2
MLA_VERIFY_REFETCH_VALUES = 0x4
MLA_VERIFY_KV4 = 0x10
MLA_VERIFY_KV4_ROW_BYTES = 384
MLA_VERIFY_SHARED = 0x20
MLA_VERIFY_TEST_STALL_GATHER = 0x100

EXPORTED = ("mla_verify_plan", "mla_verify_plan_describe", "mla_verify_run", "mla_verify_split",
            "mla_verify_merge", "mla_verify_workspace_init", "mla_verify_read_status", "mla_verify_destroy",
            "mla_verify_strerror", "mla_verify_run_noalloc", "mla_verify_build_tree_mask",
            "mla_verify_run_varlen", "mla_verify_relocate_kv", "mla_verify_build_tree_mask_varlen",
            "mla_verify_store_kv4", "mla_verify_load_kv4", "mla_verify_build_slots", "mla_verify_run_shared",
            "mla_verify_accept_drafts", "mla_verify_commit_drafts", "mla_verify_list_free_pages", "mla_verify_fork",
            "mla_verify_release")


class MlaVerifyParams(ctypes.Structure):
    _fields_ = [("max_batch", ctypes.c_int32), ("num_heads", ctypes.c_int32), ("q_len", ctypes.c_int32),
                ("max_kv_len", ctypes.c_int32), ("pool_rows", ctypes.c_int64), ("nsplit", ctypes.c_int32),
                ("d_latent", ctypes.c_int32), ("d_rope", ctypes.c_int32), ("flags", ctypes.c_int32)]


class MlaVerifyPlanInfo(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int32), ("rows_per_cta", ctypes.c_int32), ("keys_per_tile", ctypes.c_int32),
                ("grid_x", ctypes.c_int32), ("grid_y", ctypes.c_int32), ("grid_z", ctypes.c_int32),
                ("merge_blocks", ctypes.c_int32), ("smem_bytes", ctypes.c_int32),
                ("workspace_bytes", ctypes.c_size_t), ("resident_tile", ctypes.c_int32),
                ("min_chunk", ctypes.c_int32), ("chunk_granule", ctypes.c_int32)]


class MlaVerifyError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__("%s failed with code %d: %s" % (what, code, strerror(code)))
        self.code = code


_lib = None


def load(path: str = LIB_PATH):
    """Load the shared library; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError("libmlaverify.so not built (run `python -c \"import __graft_entry__ as g; g.build()\"` "
                          "or `python mla_speculative_decode_tree_gb300/build.py`)")
    lib = ctypes.CDLL(path)
    P, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    lib.mla_verify_plan.argtypes = [ctypes.POINTER(MlaVerifyParams), ctypes.POINTER(sz), ctypes.POINTER(P)]
    lib.mla_verify_plan_describe.argtypes = [P, ctypes.POINTER(MlaVerifyPlanInfo)]
    run_args = [P, P, P, P, P, P, P, P, P, i32, f32, i32, P, sz]
    lib.mla_verify_run.argtypes = run_args + [P, P, P]
    lib.mla_verify_split.argtypes = run_args + [P]
    lib.mla_verify_run_varlen.argtypes = run_args[:6] + [P] + run_args[6:] + [P, P, P]
    lib.mla_verify_merge.argtypes = [P, i32, i32, P, sz, P, P, P]
    lib.mla_verify_run_noalloc.argtypes = [P, P, P, P, P, P, P, P, P, i32, f32, i32, P, P, P]
    lib.mla_verify_workspace_init.argtypes = [P, P, sz, P]
    lib.mla_verify_build_tree_mask.argtypes = [P, P, P, i32, P, sz, P, P]
    lib.mla_verify_relocate_kv.argtypes = [P, P, P, P, P, i32, P, sz, P]
    lib.mla_verify_build_tree_mask_varlen.argtypes = [P, P, P, P, i32, P, sz, P, P]
    lib.mla_verify_store_kv4.argtypes = [P, P, i64, P, i64, P, i64, P, P, sz, P]
    lib.mla_verify_load_kv4.argtypes = [P, P, P, i64, P, i64, P, i64, P, sz, P]
    lib.mla_verify_build_slots.argtypes = [P, P, P, i32, i32, P, i32, P, i32, P, P, P, i64, P, P, i64, P, sz, P]
    lib.mla_verify_run_shared.argtypes = [P] * 13 + [i32, i32, f32, P, sz, P, P, P]
    lib.mla_verify_accept_drafts.argtypes = [P, P, i64, P, i64, i32, P, P, P, P, P, i32, P, P, P, P, sz, P]
    lib.mla_verify_commit_drafts.argtypes = [P, P, i32, i64, P, P, P, P, i32, P, P, i32, P, i32, P, i32, P, sz, P]
    lib.mla_verify_list_free_pages.argtypes = [P, P, i32, P, P, P]
    lib.mla_verify_fork.argtypes = [P, P, i32, i64, P, P, i32, i32, P, i32, i32, P, P, i32, P, i32, P, P, sz, P]
    lib.mla_verify_release.argtypes = [P, P, i32, i32, P, i32, i32, P, P, i32, P, sz, P]
    lib.mla_verify_read_status.argtypes = [P, P, P, ctypes.POINTER(ctypes.c_uint32)]
    lib.mla_verify_destroy.argtypes = [P]
    lib.mla_verify_strerror.argtypes = [ctypes.c_int]
    lib.mla_verify_strerror.restype = ctypes.c_char_p
    for name in EXPORTED:
        if name != "mla_verify_strerror":
            getattr(lib, name).restype = ctypes.c_int
    _lib = lib
    return lib


def strerror(code: int) -> str:
    return load().mla_verify_strerror(int(code)).decode()


def _check(rc: int, what: str):
    if rc != MLA_VERIFY_OK:
        raise MlaVerifyError(rc, what)


def _ptr(t) -> Optional[int]:
    try:
        return t.data_ptr()
    except AttributeError:  # None, or an address
        return t


_torch = None
_raw_stream = None


def _load_torch():
    global _torch, _raw_stream
    import torch
    # The current stream's handle without a Stream object around it (0.1 against 3 us per call on Grace).
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if _raw_stream is None:
        def _raw_stream(device):
            return torch.cuda.current_stream(device).cuda_stream
    _torch = torch
    return torch


def _stream(stream) -> Optional[int]:
    if stream is None:
        torch = _torch or _load_torch()
        return _raw_stream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


class Plan:
    """Owns a host-side plan handle (mla_verify_destroy on close / GC)."""

    def __init__(self, handle: int, params: MlaVerifyParams, workspace_bytes: int):
        self.handle = handle
        self.params = params
        self.q_len, self.pool_rows = params.q_len, params.pool_rows  # (read at every call)
        self.kv4 = bool(params.flags & MLA_VERIFY_KV4)
        self.workspace_bytes = workspace_bytes

    @property
    def nsplit(self) -> int:
        return self.params.nsplit

    def describe(self) -> MlaVerifyPlanInfo:
        return mla_verify_plan_describe(self)

    def close(self):
        if self.handle:
            load().mla_verify_destroy(ctypes.c_void_p(self.handle))
            self.handle = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def mla_verify_plan(max_batch: int, num_heads: int, q_len: int, max_kv_len: int, pool_rows: int, nsplit: int,
                    flags: int = 0, d_latent: int = 512, d_rope: int = 64) -> Plan:
    p = MlaVerifyParams(max_batch, num_heads, q_len, max_kv_len, pool_rows, nsplit, d_latent, d_rope, flags)
    ws = ctypes.c_size_t(0)
    h = ctypes.c_void_p(0)
    _check(load().mla_verify_plan(ctypes.byref(p), ctypes.byref(ws), ctypes.byref(h)), "mla_verify_plan")
    return Plan(h.value, p, ws.value)


def mla_verify_plan_describe(plan: Plan) -> MlaVerifyPlanInfo:
    info = MlaVerifyPlanInfo()
    _check(load().mla_verify_plan_describe(ctypes.c_void_p(plan.handle), ctypes.byref(info)),
           "mla_verify_plan_describe")
    return info


def mla_verify_run_varlen(plan: Plan, q_nope_absorbed, q_rope, kv_pool, kv_indptr, kv_indices, qo_indptr,
                          out_cache_loc, custom_mask, mask_indptr, batch: int, sm_scale: float, nsplit: int,
                          workspace, o, lse, stream=None, workspace_bytes: Optional[int] = None):
    args = (q_nope_absorbed, q_rope, kv_pool, kv_indptr, kv_indices, qo_indptr, out_cache_loc, custom_mask, mask_indptr,
            workspace, o, lse)
    try:  # all tensors, as a rule
        qn, qr, kv, kp, ki, qo, loc, cm, mp, ws, po, pl = [t.data_ptr() for t in args]
    except AttributeError:
        qn, qr, kv, kp, ki, qo, loc, cm, mp, ws, po, pl = map(_ptr, args)
    rc = (_lib or load()).mla_verify_run_varlen(
        plan.handle, qn, qr, kv, kp, ki, qo, loc, cm, mp, int(batch), float(sm_scale), int(nsplit), ws,
        plan.workspace_bytes if workspace_bytes is None else int(workspace_bytes), po, pl, _stream(stream))
    if rc:
        _check(rc, "mla_verify_run_varlen")


def mla_verify_run(plan: Plan, q_nope_absorbed, q_rope, kv_pool, kv_indptr, kv_indices, out_cache_loc,
                   custom_mask, mask_indptr, batch: int, sm_scale: float, nsplit: int, workspace, o, lse,
                   stream=None, workspace_bytes: Optional[int] = None):
    rc = (_lib or load()).mla_verify_run(
        plan.handle, _ptr(q_nope_absorbed), _ptr(q_rope), _ptr(kv_pool), _ptr(kv_indptr), _ptr(kv_indices),
        _ptr(out_cache_loc), _ptr(custom_mask), _ptr(mask_indptr), int(batch), float(sm_scale), int(nsplit),
        _ptr(workspace), plan.workspace_bytes if workspace_bytes is None else int(workspace_bytes), _ptr(o),
        _ptr(lse), _stream(stream))
    if rc:
        _check(rc, "mla_verify_run")


def mla_verify_split(plan: Plan, q_nope_absorbed, q_rope, kv_pool, kv_indptr, kv_indices, out_cache_loc,
                     custom_mask, mask_indptr, batch: int, sm_scale: float, nsplit: int, workspace, stream=None,
                     workspace_bytes: Optional[int] = None):
    ws_bytes = plan.workspace_bytes if workspace_bytes is None else workspace_bytes
    rc = load().mla_verify_split(ctypes.c_void_p(plan.handle), _ptr(q_nope_absorbed), _ptr(q_rope), _ptr(kv_pool),
                                 _ptr(kv_indptr), _ptr(kv_indices), _ptr(out_cache_loc), _ptr(custom_mask),
                                 _ptr(mask_indptr), int(batch), float(sm_scale), int(nsplit), _ptr(workspace),
                                 int(ws_bytes), _stream(stream))
    _check(rc, "mla_verify_split")


def mla_verify_run_noalloc(plan: Plan, q_nope_absorbed, q_rope, kv_pool, kv_indptr, kv_indices, out_cache_loc,
                           custom_mask, mask_indptr, batch: int, sm_scale: float, nsplit: int, o, lse, stream=None):
    """mla_verify_run on the library's built-in scratch array (no workspace, no allocation)."""
    rc = load().mla_verify_run_noalloc(ctypes.c_void_p(plan.handle), _ptr(q_nope_absorbed), _ptr(q_rope),
                                       _ptr(kv_pool), _ptr(kv_indptr), _ptr(kv_indices), _ptr(out_cache_loc),
                                       _ptr(custom_mask), _ptr(mask_indptr), int(batch), float(sm_scale), int(nsplit),
                                       _ptr(o), _ptr(lse), _stream(stream))
    _check(rc, "mla_verify_run_noalloc")


def mla_verify_merge(plan: Plan, batch: int, nsplit: int, workspace, o, lse, stream=None,
                     workspace_bytes: Optional[int] = None):
    ws_bytes = plan.workspace_bytes if workspace_bytes is None else workspace_bytes
    rc = load().mla_verify_merge(ctypes.c_void_p(plan.handle), int(batch), int(nsplit), _ptr(workspace),
                                 int(ws_bytes), _ptr(o), _ptr(lse), _stream(stream))
    _check(rc, "mla_verify_merge")


def mla_verify_build_tree_mask(plan: Plan, parents, kv_indptr, batch: int, custom_mask, mask_indptr, stream=None,
                               mask_bytes: Optional[int] = None):
    """Device tree-mask build: parents int32 [batch*q_len] -> packed custom_mask, mask_indptr int32 [batch]."""
    nbytes = custom_mask.numel() * custom_mask.element_size() if mask_bytes is None else mask_bytes
    rc = load().mla_verify_build_tree_mask(ctypes.c_void_p(plan.handle), _ptr(parents), _ptr(kv_indptr), int(batch),
                                           _ptr(custom_mask), int(nbytes), _ptr(mask_indptr), _stream(stream))
    _check(rc, "mla_verify_build_tree_mask")


def mla_verify_relocate_kv(plan: Plan, kv_pool, kv_indptr, kv_indices, dst_start, batch: int, workspace,
                           stream=None):
    """KV relocation: request b's prefix rows move to rows dst_start[b].. and kv_indices is rewritten in place."""
    rc = load().mla_verify_relocate_kv(ctypes.c_void_p(plan.handle), _ptr(kv_pool), _ptr(kv_indptr), _ptr(kv_indices),
                                       _ptr(dst_start), int(batch), _ptr(workspace),
                                       workspace.numel() * workspace.element_size(), _stream(stream))
    _check(rc, "mla_verify_relocate_kv")


def mla_verify_build_tree_mask_varlen(plan: Plan, parents, kv_indptr, qo_indptr, batch: int, custom_mask,
                                      mask_indptr, stream=None, mask_bytes: Optional[int] = None):
    """Device tree-mask build for a varlen call: parents int32 [qo_indptr[batch]] (request b's at
    qo_indptr[b]..), blocks [T_b, P_b + T_b]."""
    nbytes = custom_mask.numel() * custom_mask.element_size() if mask_bytes is None else mask_bytes
    rc = load().mla_verify_build_tree_mask_varlen(ctypes.c_void_p(plan.handle), _ptr(parents), _ptr(kv_indptr),
                                                  _ptr(qo_indptr), int(batch), _ptr(custom_mask), int(nbytes),
                                                  _ptr(mask_indptr), _stream(stream))
    _check(rc, "mla_verify_build_tree_mask_varlen")


def _rows_of(x, width: int, n: int, what: str) -> int:
    """Row stride in elements of a bf16 [n, width] tensor (any row stride, contiguous rows)."""
    if x.dtype is (_torch or _load_torch()).bfloat16 and x.shape == (n, width):
        row, col = x.stride()
        if col == 1 or n == 0:
            return row if n > 1 else max(width, row // 8 * 8)
    raise ValueError("%s: bf16 [%d, %d] with contiguous rows expected, got %s %s strides %s"
                     % (what, n, width, x.dtype, tuple(x.shape), x.stride()))


def _int32(x, what: str):
    if x.dtype is not (_torch or _load_torch()).int32 or not x.is_contiguous():
        raise ValueError("%s: a contiguous int32 tensor expected, got %s strides %s" % (what, x.dtype, x.stride()))


def mla_verify_store_kv4(plan: Plan, latent, rope, slots, kv_pool, workspace, stream=None):
    """Code tokens (latent bf16 [n, 512], rope bf16 [n, 64], any row strides) into rows ``slots`` of a 4-bit pool."""
    n = slots.numel()
    _int32(slots, "slots")
    rc = (_lib or load()).mla_verify_store_kv4(
        plan.handle, latent.data_ptr(), _rows_of(latent, 512, n, "latent"), rope.data_ptr(),
        _rows_of(rope, 64, n, "rope"), slots.data_ptr(), n, _ptr(kv_pool), workspace.data_ptr(), workspace.nbytes,
        _stream(stream))
    if rc:
        _check(rc, "mla_verify_store_kv4")


def mla_verify_load_kv4(plan: Plan, kv_pool, slots, latent, rope, workspace, stream=None):
    """Rows ``slots`` of a 4-bit pool as bf16, into latent [n, 512] and rope [n, 64] (any row strides)."""
    n = slots.numel()
    _int32(slots, "slots")
    rc = (_lib or load()).mla_verify_load_kv4(
        plan.handle, _ptr(kv_pool), slots.data_ptr(), n, latent.data_ptr(), _rows_of(latent, 512, n, "latent"),
        rope.data_ptr(), _rows_of(rope, 64, n, "rope"), workspace.data_ptr(), workspace.nbytes, _stream(stream))
    if rc:
        _check(rc, "mla_verify_load_kv4")


def mla_verify_build_slots(plan: Plan, seq_lens, new_lens, batch: int, page_size: int, block_table, free_pages,
                           pages_used, kv_indptr, kv_indices, qo_indptr, out_cache_loc, workspace, stream=None):
    """Block tables and slot maps of a step from the requests' lengths (new_lens None: the plan's q_len each).

    block_table is int32 [>= batch, max_pages]; the capacities are the index tensors' lengths."""
    i32 = (_torch or _load_torch()).int32
    for x in (seq_lens, block_table, free_pages, pages_used, kv_indptr, kv_indices, qo_indptr, out_cache_loc):
        if x.dtype is not i32 or not x.is_contiguous():
            raise ValueError("contiguous int32 tensors expected, got %s strides %s" % (x.dtype, x.stride()))
    if new_lens is not None:
        _int32(new_lens, "new_lens")
        if new_lens.numel() < batch:
            raise ValueError("new_lens is too short for %d requests" % batch)
    rows, max_pages = block_table.shape
    if rows < batch or seq_lens.numel() < batch or kv_indptr.numel() <= batch or qo_indptr.numel() <= batch:
        raise ValueError("an array is too short for %d requests" % batch)
    rc = (_lib or load()).mla_verify_build_slots(
        plan.handle, seq_lens.data_ptr(), _ptr(new_lens), int(batch), int(page_size), block_table.data_ptr(),
        max_pages, free_pages.data_ptr(), free_pages.numel(), pages_used.data_ptr(), kv_indptr.data_ptr(),
        kv_indices.data_ptr(), kv_indices.numel(), qo_indptr.data_ptr(), out_cache_loc.data_ptr(),
        out_cache_loc.numel(), workspace.data_ptr(), workspace.nbytes, _stream(stream))
    if rc:
        _check(rc, "mla_verify_build_slots")


def mla_verify_run_shared(plan: Plan, q_nope_absorbed, q_rope, kv_pool, group_indptr, shared_indptr, shared_indices,
                          kv_indptr, kv_indices, qo_indptr, out_cache_loc, custom_mask, mask_indptr, batch: int,
                          num_groups: int, sm_scale: float, workspace, o, lse, stream=None,
                          workspace_bytes: Optional[int] = None):
    """Verify attention for requests in groups with shared prefixes (qo_indptr None: the plan's q_len tokens each)."""
    args = (q_nope_absorbed, q_rope, kv_pool, group_indptr, shared_indptr, shared_indices, kv_indptr, kv_indices,
            qo_indptr, out_cache_loc, custom_mask, mask_indptr, workspace, o, lse)
    qn, qr, kv, gp, sp, si, kp, ki, qo, loc, cm, mp, ws, po, pl = map(_ptr, args)
    rc = (_lib or load()).mla_verify_run_shared(
        plan.handle, qn, qr, kv, gp, sp, si, kp, ki, qo, loc, cm, mp, int(batch), int(num_groups), float(sm_scale), ws,
        plan.workspace_bytes if workspace_bytes is None else int(workspace_bytes), po, pl, _stream(stream))
    if rc:
        _check(rc, "mla_verify_run_shared")


def _arrays(dtype, *arrays):
    """(tensor, least entries, name) each: contiguous and of this type."""
    for x, n, what in arrays:
        if x.dtype is not dtype or not x.is_contiguous():
            raise ValueError("%s: a contiguous %s tensor expected, got %s strides %s" % (what, dtype, x.dtype, x.stride()))
        if x.numel() < n:
            raise ValueError("%s is too short: %d entries, %d needed" % (what, x.numel(), n))


def _prob_rows(x, vocab: int, what: str) -> int:
    """Row stride of fp32 [rows, vocab] probabilities with contiguous rows."""
    if x.dtype is not (_torch or _load_torch()).float32 or x.dim() != 2 or x.shape[1] != vocab or (
            vocab > 1 and x.stride(1) != 1):
        raise ValueError("%s: fp32 [rows, %d] with contiguous rows expected, got %s %s strides %s"
                         % (what, vocab, x.dtype, tuple(x.shape), x.stride()))
    return x.stride(0) if x.shape[0] > 1 else max(vocab, x.stride(0))


def mla_verify_accept_drafts(plan: Plan, target_probs, draft_probs, draft_tokens, parents, qo_indptr, uniform,
                             uniform_next, batch: int, accepted, num_accepted, next_tokens, workspace, stream=None):
    """Draft trees against the target's probabilities (draft_probs None: proposed, not drawn; qo_indptr None: q_len nodes
    each): accepted int32 [batch, q_len], num_accepted and next_tokens int32 [batch] are written."""
    torch = _torch or _load_torch()
    i32 = torch.int32
    rows, vocab = target_probs.shape[0], target_probs.shape[-1]
    nodes = 0 if qo_indptr is not None else batch * plan.q_len
    _arrays(i32, (draft_tokens, nodes, "draft_tokens"), (parents, nodes, "parents"),
            (accepted, batch * plan.q_len, "accepted"), (num_accepted, batch, "num_accepted"),
            (next_tokens, batch, "next_tokens"))
    _arrays(torch.float32, (uniform, nodes, "uniform"), (uniform_next, batch, "uniform_next"))
    if qo_indptr is not None:
        _arrays(i32, (qo_indptr, batch + 1, "qo_indptr"))
    elif rows < nodes:
        raise ValueError("target_probs has too few rows")
    if draft_probs is not None and draft_probs.shape[0] < rows:
        raise ValueError("draft_probs has fewer rows than target_probs")
    rc = (_lib or load()).mla_verify_accept_drafts(
        plan.handle, target_probs.data_ptr(), _prob_rows(target_probs, vocab, "target_probs"), _ptr(draft_probs),
        0 if draft_probs is None else _prob_rows(draft_probs, vocab, "draft_probs"), vocab, draft_tokens.data_ptr(),
        parents.data_ptr(), _ptr(qo_indptr), uniform.data_ptr(), uniform_next.data_ptr(), int(batch),
        accepted.data_ptr(), num_accepted.data_ptr(), next_tokens.data_ptr(), workspace.data_ptr(), workspace.nbytes,
        _stream(stream))
    if rc:
        _check(rc, "mla_verify_accept_drafts")


def _layers_of(plan: Plan, kv_pool):
    """(layers, bytes from one to the next) of a pool [rows, row] or [layers, rows, row] of whole rows."""
    torch = _torch or _load_torch()
    row, dtype = (MLA_VERIFY_KV4_ROW_BYTES, torch.uint8) if plan.kv4 else (576, torch.bfloat16)
    shape, stride = kv_pool.shape, kv_pool.stride()
    if kv_pool.dtype is not dtype or len(shape) not in (2, 3) or shape[-1] != row or shape[-2] != plan.pool_rows or (
            stride[-1] != 1 or (stride[-2] != row and shape[-2] > 1)):
        raise ValueError("kv_pool: %s [layers, %d, %d] expected, got %s %s strides %s"
                         % (dtype, plan.pool_rows, row, kv_pool.dtype, tuple(shape), stride))
    if len(shape) == 2 or shape[0] == 1:
        return 1, 0
    return shape[0], stride[0] * (1 if plan.kv4 else 2)


def mla_verify_commit_drafts(plan: Plan, kv_pool, qo_indptr, out_cache_loc, accepted, num_accepted, batch: int, seq_lens,
                             new_seq_lens, page_size: int, block_table, page_refs, workspace, stream=None):
    """The accepted paths' rows to the front of the new rows of kv_pool ([rows, row] or [layers, rows, row]), lengths and
    page counts (block_table int32 [>= batch, max_pages] and page_refs None: no pages)."""
    i32 = (_torch or _load_torch()).int32
    tokens = batch * plan.q_len
    _arrays(i32, (out_cache_loc, 0 if qo_indptr is not None else tokens, "out_cache_loc"), (accepted, tokens, "accepted"),
            (num_accepted, batch, "num_accepted"), (seq_lens, batch, "seq_lens"), (new_seq_lens, batch, "new_seq_lens"))
    if qo_indptr is not None:
        _arrays(i32, (qo_indptr, batch + 1, "qo_indptr"))
    max_pages = num_pages = 0
    if (block_table is None) != (page_refs is None):
        raise ValueError("block_table and page_refs go together")
    if block_table is not None:
        _arrays(i32, (block_table, 0, "block_table"), (page_refs, 0, "page_refs"))
        held, max_pages = block_table.shape
        if held < batch:
            raise ValueError("block_table has too few rows")
        num_pages = page_refs.numel()
    layers, stride = _layers_of(plan, kv_pool)
    rc = (_lib or load()).mla_verify_commit_drafts(
        plan.handle, kv_pool.data_ptr(), layers, stride, _ptr(qo_indptr), out_cache_loc.data_ptr(), accepted.data_ptr(),
        num_accepted.data_ptr(), int(batch), seq_lens.data_ptr(), new_seq_lens.data_ptr(), int(page_size),
        _ptr(block_table), max_pages, _ptr(page_refs), num_pages, workspace.data_ptr(), workspace.nbytes,
        _stream(stream))
    if rc:
        _check(rc, "mla_verify_commit_drafts")


def mla_verify_list_free_pages(plan: Plan, page_refs, free_pages, num_free, stream=None):
    """Pages without a reference, ascending, into free_pages (-1 behind them), and their number."""
    n = page_refs.numel()
    _arrays((_torch or _load_torch()).int32, (page_refs, 0, "page_refs"), (free_pages, n, "free_pages"),
            (num_free, 1, "num_free"))
    rc = (_lib or load()).mla_verify_list_free_pages(plan.handle, page_refs.data_ptr(), n, free_pages.data_ptr(),
                                                     num_free.data_ptr(), _stream(stream))
    if rc:
        _check(rc, "mla_verify_list_free_pages")


def mla_verify_fork(plan: Plan, kv_pool, src, dst, page_size: int, block_table, seq_lens, page_refs, free_pages,
                    pages_used, workspace, stream=None):
    """Requests dst become copies of requests src: full pages shared, the last one copied (all layers of kv_pool)."""
    requests, max_pages = block_table.shape
    n = src.numel()
    _arrays((_torch or _load_torch()).int32, (block_table, 0, "block_table"), (seq_lens, requests, "seq_lens"),
            (page_refs, 0, "page_refs"), (src, 0, "src"), (dst, n, "dst"), (free_pages, 0, "free_pages"),
            (pages_used, 1, "pages_used"))
    layers, stride = _layers_of(plan, kv_pool)
    rc = (_lib or load()).mla_verify_fork(
        plan.handle, kv_pool.data_ptr(), layers, stride, src.data_ptr(), dst.data_ptr(), n, int(page_size),
        block_table.data_ptr(), requests, max_pages, seq_lens.data_ptr(), page_refs.data_ptr(), page_refs.numel(),
        free_pages.data_ptr(), free_pages.numel(), pages_used.data_ptr(), workspace.data_ptr(), workspace.nbytes,
        _stream(stream))
    if rc:
        _check(rc, "mla_verify_fork")


def mla_verify_release(plan: Plan, requests, page_size: int, block_table, seq_lens, page_refs, workspace, stream=None):
    """Requests let go of their pages; their lengths become 0."""
    rows, max_pages = block_table.shape
    _arrays((_torch or _load_torch()).int32, (block_table, 0, "block_table"), (seq_lens, rows, "seq_lens"),
            (page_refs, 0, "page_refs"), (requests, 0, "requests"))
    rc = (_lib or load()).mla_verify_release(
        plan.handle, requests.data_ptr(), requests.numel(), int(page_size), block_table.data_ptr(), rows, max_pages,
        seq_lens.data_ptr(), page_refs.data_ptr(), page_refs.numel(), workspace.data_ptr(), workspace.nbytes,
        _stream(stream))
    if rc:
        _check(rc, "mla_verify_release")


def mla_verify_workspace_init(plan: Plan, workspace, stream=None):
    _check(load().mla_verify_workspace_init(ctypes.c_void_p(plan.handle), _ptr(workspace), plan.workspace_bytes,
                                            _stream(stream)), "mla_verify_workspace_init")


def mla_verify_read_status(plan: Plan, workspace, stream=None) -> int:
    st = ctypes.c_uint32(0)
    _check(load().mla_verify_read_status(ctypes.c_void_p(plan.handle), _ptr(workspace), _stream(stream),
                                         ctypes.byref(st)), "mla_verify_read_status")
    return int(st.value)


def mla_verify_destroy(plan: Plan):
    plan.close()


# ---------------------------------------------------------------------------
# Convenience layer over the C calls: device buffers for a host workload and a
# one-shot call that allocates outputs and workspace with torch.

def device_inputs(wl: dict, device="cuda"):
    """Copy a host workload (numpy arrays from ``workloads.make_workload``) to the device."""
    import numpy as np
    import torch

    def t(a, dtype):
        return torch.from_numpy(np.ascontiguousarray(a)).to(device=device).view(dtype)

    kv_idx = wl["kv_indices"] if wl["kv_indices"].size else np.zeros(1, np.int32)
    return dict(
        q_nope=t(wl["q_nope"].view(np.int16), torch.bfloat16),
        q_rope=t(wl["q_rope"].view(np.int16), torch.bfloat16),
        kv_pool=t(wl["pool"].view(np.int16), torch.bfloat16),
        kv_indptr=t(wl["kv_indptr"].astype(np.int32), torch.int32),
        kv_indices=t(kv_idx.astype(np.int32), torch.int32),
        out_cache_loc=t(wl["out_cache_loc"].astype(np.int32), torch.int32),
        custom_mask=t(wl["custom_mask"].astype(np.uint8), torch.uint8),
        mask_indptr=t(wl["mask_indptr"].astype(np.int32), torch.int32),
        **({"qo_indptr": t(wl["qo_indptr"].astype(np.int32), torch.int32)} if wl.get("qo_indptr") is not None
           else {}),
    )


class Verifier:
    """A plan plus its workspace and output buffers on one device."""

    def __init__(self, max_batch: int, num_heads: int, q_len: int, max_kv_len: int, pool_rows: int, nsplit: int,
                 flags: int = 0, device="cuda"):
        import torch
        self.plan = mla_verify_plan(max_batch, num_heads, q_len, max_kv_len, pool_rows, nsplit, flags)
        self.workspace = torch.zeros(self.plan.workspace_bytes, dtype=torch.uint8, device=device)
        rows = max_batch * q_len * num_heads
        self.o = torch.empty((max_batch * q_len, num_heads, 512), dtype=torch.bfloat16, device=device)
        self.lse = torch.empty((max_batch * q_len, num_heads), dtype=torch.float32, device=device)
        self.rows_max = rows

    def run(self, d: dict, batch: int, sm_scale: float, stream=None):
        """One call; with d["qo_indptr"] present, the varlen entry point, with d["group_indptr"] present (a plan with
        MLA_VERIFY_SHARED) the one for shared prefixes.  Returns the output buffers' first batch*q_len token rows (with
        qo_indptr the call's rows come first)."""
        if "group_indptr" in d:
            mla_verify_run_shared(self.plan, d["q_nope"], d["q_rope"], d["kv_pool"], d["group_indptr"],
                                  d["shared_indptr"], d["shared_indices"], d["kv_indptr"], d["kv_indices"],
                                  d.get("qo_indptr"), d["out_cache_loc"], d["custom_mask"], d["mask_indptr"], batch,
                                  d["group_indptr"].numel() - 1, sm_scale, self.workspace, self.o, self.lse, stream=stream)
        elif "qo_indptr" in d:
            mla_verify_run_varlen(self.plan, d["q_nope"], d["q_rope"], d["kv_pool"], d["kv_indptr"],
                                  d["kv_indices"], d["qo_indptr"], d["out_cache_loc"], d["custom_mask"],
                                  d["mask_indptr"], batch, sm_scale, self.plan.nsplit, self.workspace, self.o,
                                  self.lse, stream=stream)
        else:
            mla_verify_run(self.plan, d["q_nope"], d["q_rope"], d["kv_pool"], d["kv_indptr"], d["kv_indices"],
                           d["out_cache_loc"], d["custom_mask"], d["mask_indptr"], batch, sm_scale,
                           self.plan.nsplit, self.workspace, self.o, self.lse, stream=stream)
        n = batch * self.plan.params.q_len
        return self.o[:n], self.lse[:n]

    def status(self, stream=None) -> int:
        return mla_verify_read_status(self.plan, self.workspace, stream)


def verifier_for(wl: dict, flags: int = 0, nsplit: Optional[int] = None, device="cuda") -> Verifier:
    L = int(max(wl["prefix_lens"])) + wl["T"] if len(wl["prefix_lens"]) else wl["T"]  # bounds P_b + T_b too
    return Verifier(wl["B"], wl["H"], wl["T"], L, wl["pool"].shape[0], wl["nsplit"] if nsplit is None else nsplit,
                    flags, device)
