"""The calls around the scorer: batch plan, cache writes and attention.

Marshalling only, like the rest of the binding (``include/qsaidx.h`` has the
contracts).  Each call comes as a function and as a ``Prepared`` class: a call
checked once on fixed tensors, which then only crosses the C ABI.  All tensors of
a call lie on one device; the call is queued on that device's current stream
unless ``stream`` is given, whatever the calling thread's current device (a
prepared call: on the stream that was current when it was made).
"""
from __future__ import annotations

import ctypes
import dataclasses
from typing import Any, Optional

from . import (BF16, E_DTYPE, FP8_E4M3FN, FP16, KV_PAGED, OK, QsaError, _check_rows_i32, _ptr, _raise_on, _require,
               _torch_stream, lib)


class PlanShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("num_reqs", "max_blocks", "block_size", "ratio", "num_rows",
                                              "num_free")] + [("num_blocks", ctypes.c_int64)]


class KvShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("num_rows", "num_kv_heads", "head_dim", "block_size", "dtype",
                                              "reserved")] + \
               [(n, ctypes.c_int64) for n in ("num_blocks", "src_row_stride", "src_head_stride", "kv_block_stride",
                                              "kv_slot_stride", "kv_head_stride")]


class KeysShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("num_rows", "head_dim", "block_size", "src_dtype", "k_dtype",
                                              "kv_layout")] + \
               [("num_blocks", ctypes.c_int64), ("src_stride", ctypes.c_int64)]


class AttnShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("num_rows", "num_heads", "num_kv_heads", "head_dim", "block_size",
                                              "num_reqs", "max_blocks", "dtype")] + \
               [("scale", ctypes.c_float), ("reserved", ctypes.c_int32)] + \
               [(n, ctypes.c_int64) for n in ("num_blocks", "q_row_stride", "q_head_stride", "out_row_stride",
                                              "out_head_stride", "kv_block_stride", "kv_slot_stride",
                                              "kv_head_stride")]


def _declare():
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    p = ctypes.POINTER
    for name, args, res in (
            ("qsa_plan_batch", [vp] * 11 + [p(PlanShape), vp], ctypes.c_int),
            ("qsa_plan_batch_check", [vp] * 8 + [p(PlanShape)], ctypes.c_int),
            ("qsa_write_kv", [vp] * 5 + [p(KvShape), vp], ctypes.c_int),
            ("qsa_write_kv_check", [vp] * 5 + [p(KvShape)], ctypes.c_int),
            ("qsa_write_keys", [vp] * 4 + [p(KeysShape), vp], ctypes.c_int),
            ("qsa_write_keys_check", [vp] * 4 + [p(KeysShape)], ctypes.c_int),
            ("qsa_paged_attention", [vp] * 8 + [p(AttnShape), vp, i64, vp], ctypes.c_int),
            ("qsa_paged_attention_check", [vp] * 7 + [p(AttnShape), vp, i64], ctypes.c_int),
            ("qsa_paged_attention_workspace_bytes", [p(AttnShape)], i64),
            ("qsa_sparse_attention", [vp] * 6 + [i32, i32, vp, vp, vp, p(AttnShape), vp, i64, vp], ctypes.c_int),
            ("qsa_sparse_attention_check", [vp] * 6 + [i32, i32, vp, p(AttnShape), vp, i64], ctypes.c_int),
            ("qsa_sparse_attention_workspace_bytes", [p(AttnShape), i32, i32], i64)):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, res


_declare()


def _one_device(**tensors):
    """The device that every given tensor lies on."""
    dev = None
    for name, t in tensors.items():
        if t is None:
            continue
        _require(t.is_cuda, f"{name} must be a device tensor")
        _require(dev is None or t.device == dev, f"{name} is on {t.device}, others on {dev}")
        dev = t.device
    return dev


def _rows(name, t, n, dtype):
    _require(t.dtype == dtype and t.is_contiguous() and t.dim() == 1 and int(t.numel()) == n,
             f"{name} must be contiguous {dtype} [{n}]")


def _half_code(name, t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float16:
        return FP16
    raise QsaError(E_DTYPE, f"{name} must be bf16 or fp16, not {t.dtype}")


class _Prepared:
    """A checked call: ``fn(*args)`` on ``stream`` of ``device``."""

    def _ready(self, fn, args, device, stream, keep):
        import torch
        self._fn, self._keep, self._device = fn, keep, device
        with torch.cuda.device(device):
            self._stream_of = _torch_stream(stream)
        self._args = (*args, self._stream_of.cuda_stream)
        self._index = device.index

    def _launch(self):
        import torch
        if torch.cuda.current_device() == self._index:
            st = self._fn(*self._args)
        else:  # kernels go to the current device's code objects
            with torch.cuda.device(self._device):
                st = self._fn(*self._args)
        if st != OK:
            _raise_on(st)


# ---------------------------------------------------------------------------
# batch plan
# ---------------------------------------------------------------------------

@dataclasses.dataclass
class BatchPlan:
    """A step's metadata on the device (``qsa_plan_batch``'s outputs)."""

    q_starts: Any                    # int32 [n + 1]
    row_to_req: Any                  # int32 [R]
    ctx_lens: Any                    # int32 [R] visible tokens
    slots: Any                       # int64 [R] token slots, -1: none
    col_lens: Optional[Any] = None   # int32 [R] visible compressed columns
    col_slots: Optional[Any] = None  # int64 [R] slot of the column a row completes, -1: none
    blocks_used: Optional[Any] = None  # int32 [1]

    @staticmethod
    def empty(num_reqs: int, num_rows: int, device) -> "BatchPlan":
        """Uninitialised buffers for ``num_reqs`` requests and ``num_rows`` rows."""
        import torch
        i32 = dict(dtype=torch.int32, device=device)
        i64 = dict(dtype=torch.int64, device=device)
        return BatchPlan(torch.empty(num_reqs + 1, **i32), torch.empty(num_rows, **i32),
                         torch.empty(num_rows, **i32), torch.empty(num_rows, **i64), torch.empty(num_rows, **i32),
                         torch.empty(num_rows, **i64), torch.empty(1, **i32))


class PreparedPlanBatch(_Prepared):
    """A validated ``qsa_plan_batch`` call on fixed tensors."""

    def __init__(self, past_lens, new_lens, free_blocks, block_table, *, block_size: int, num_blocks: int,
                 out: BatchPlan, ratio: int = 1, stream=None):
        import torch
        buffers = {f.name: getattr(out, f.name) for f in dataclasses.fields(out)}
        dev = _one_device(past_lens=past_lens, new_lens=new_lens, free_blocks=free_blocks, block_table=block_table,
                          **buffers)
        _require(block_table.dtype == torch.int32 and block_table.dim() == 2 and block_table.is_contiguous(),
                 "block_table must be contiguous int32 [n, max_blocks]")
        n = int(block_table.shape[0])
        rows = int(out.row_to_req.numel())
        _rows("past_lens", past_lens, n, torch.int32)
        _rows("new_lens", new_lens, n, torch.int32)
        _rows("free_blocks", free_blocks, int(free_blocks.numel()), torch.int32)
        for name, size, dtype in (("q_starts", n + 1, torch.int32), ("row_to_req", rows, torch.int32),
                                  ("ctx_lens", rows, torch.int32), ("slots", rows, torch.int64),
                                  ("col_lens", rows, torch.int32), ("col_slots", rows, torch.int64),
                                  ("blocks_used", 1, torch.int32)):
            t = getattr(out, name)
            if t is not None or name in ("q_starts", "row_to_req", "ctx_lens", "slots"):
                _rows(name, t, size, dtype)
        shape = PlanShape(num_reqs=n, max_blocks=int(block_table.shape[1]), block_size=int(block_size),
                          ratio=int(ratio), num_rows=rows, num_free=int(free_blocks.numel()),
                          num_blocks=int(num_blocks))
        ins = (_ptr(past_lens), _ptr(new_lens), _ptr(free_blocks), _ptr(block_table))
        outs = (_ptr(out.q_starts), _ptr(out.row_to_req), _ptr(out.ctx_lens), _ptr(out.slots))
        _raise_on(lib.qsa_plan_batch_check(*ins, *outs, ctypes.byref(shape)))
        self.out = out
        self._ready(lib.qsa_plan_batch,
                    (*ins, *outs, _ptr(out.col_lens), _ptr(out.col_slots), _ptr(out.blocks_used),
                     ctypes.byref(shape)), dev, stream,
                    (past_lens, new_lens, free_blocks, block_table, buffers, shape))

    def __call__(self) -> BatchPlan:
        self._launch()
        return self.out


def plan_batch(past_lens, new_lens, free_blocks, block_table, *, block_size: int, num_blocks: int, num_rows: int,
               ratio: int = 1, out: Optional[BatchPlan] = None, stream=None) -> BatchPlan:
    """``qsa_plan_batch``: a step's row starts, visible counts and cache slots from
    its requests' lengths; ``block_table`` gets the new entries.  ``num_rows`` is
    the length of the per-row outputs (rows behind the last request's see
    nothing and have no slots)."""
    _one_device(block_table=block_table)
    if out is None:
        with _on(stream, block_table.device):
            out = BatchPlan.empty(int(block_table.shape[0]), int(num_rows), block_table.device)
    _require(int(out.row_to_req.numel()) == int(num_rows), "out holds another number of rows than num_rows")
    return PreparedPlanBatch(past_lens, new_lens, free_blocks, block_table, block_size=block_size,
                             num_blocks=num_blocks, out=out, ratio=ratio, stream=stream)()


def _on(stream, device):
    """Memory made inside is made on the launch stream: first written and first
    reused there."""
    import torch
    with torch.cuda.device(device):
        return torch.cuda.stream(_torch_stream(stream))


# ---------------------------------------------------------------------------
# cache writes
# ---------------------------------------------------------------------------

def _kv_strides(name, c):
    _require(c.dim() == 4 and c.stride(3) == 1, f"{name} must be [num_blocks, block_size, num_kv_heads, head_dim] "
                                                "with a contiguous last dimension")
    # the stride of a dimension of one element has no meaning: any allowed value does
    return [int(c.stride(i)) if int(c.shape[i]) > 1 else int(c.shape[3]) for i in range(3)]


class PreparedWriteKv(_Prepared):
    """A validated ``qsa_write_kv`` call on fixed tensors."""

    def __init__(self, k, v, slots, kcache, vcache, *, stream=None):
        import torch
        dev = _one_device(k=k, v=v, slots=slots, kcache=kcache, vcache=vcache)
        code = _half_code("k", k)
        for name, t in (("v", v), ("kcache", kcache), ("vcache", vcache)):
            _require(t.dtype == k.dtype, f"{name} must have k's type")
        _require(k.dim() == 3 and k.shape == v.shape and k.stride(2) == 1 and v.stride(2) == 1,
                 "k and v must be [R, num_kv_heads, head_dim] with a contiguous last dimension")
        R, hk, d = (int(x) for x in k.shape)
        src = [[int(t.stride(0)) if R > 1 else d, int(t.stride(1)) if hk > 1 else d] for t in (k, v)]
        _require(src[0] == src[1], "k and v must have equal strides")
        strides = _kv_strides("kcache", kcache)
        _require(kcache.shape == vcache.shape and strides == _kv_strides("vcache", vcache),
                 "kcache and vcache must have equal shapes and strides")
        _require((int(kcache.shape[2]), int(kcache.shape[3])) == (hk, d), "the caches' heads must be k's")
        _rows("slots", slots, R, torch.int64)
        shape = KvShape(num_rows=R, num_kv_heads=hk, head_dim=d, block_size=int(kcache.shape[1]), dtype=code,
                        num_blocks=int(kcache.shape[0]), src_row_stride=src[0][0],
                        src_head_stride=src[0][1], kv_block_stride=strides[0],
                        kv_slot_stride=strides[1], kv_head_stride=strides[2])
        args = (_ptr(k), _ptr(v), _ptr(slots), _ptr(kcache), _ptr(vcache), ctypes.byref(shape))
        _raise_on(lib.qsa_write_kv_check(*args))
        self._ready(lib.qsa_write_kv, args, dev, stream, (k, v, slots, kcache, vcache, shape))

    def __call__(self):
        self._launch()


def write_kv(k, v, slots, kcache, vcache, *, stream=None):
    """``qsa_write_kv``: rows of ``k`` and ``v`` [R, num_kv_heads, head_dim] into the
    caches [num_blocks, block_size, num_kv_heads, head_dim] (any strides with a
    contiguous last dimension) at ``slots`` (int64 [R]; -1 writes nothing)."""
    PreparedWriteKv(k, v, slots, kcache, vcache, stream=stream)()


class PreparedWriteKeys(_Prepared):
    """A validated ``qsa_write_keys`` call on fixed tensors."""

    def __init__(self, keys, slots, kcache, *, block_size: int, kscale=None, layout: int = KV_PAGED, stream=None):
        import torch
        dev = _one_device(keys=keys, slots=slots, kcache=kcache, kscale=kscale)
        src = _half_code("keys", keys)
        fp8 = kcache.dtype in (torch.float8_e4m3fn, torch.uint8)
        _require(fp8 or kcache.dtype == keys.dtype, "kcache must be fp8 (or bytes) or have the keys' type")
        _require(keys.dim() == 2 and keys.stride(1) == 1, "keys must be [R, D] with a contiguous last dimension")
        R, D = (int(x) for x in keys.shape)
        _require(kcache.is_contiguous(), "kcache must be contiguous")
        nb, b = int(kcache.shape[0]), int(block_size)
        _require(int(kcache.numel()) == nb * b * (D if layout == KV_PAGED else D + 4),
                 "kcache does not hold block_size keys a block")
        if kscale is not None:
            _require(kscale.dtype == torch.float32 and kscale.is_contiguous() and int(kscale.numel()) == nb * b,
                     "kscale must be contiguous f32 [num_blocks, block_size]")
        _rows("slots", slots, R, torch.int64)
        shape = KeysShape(num_rows=R, head_dim=D, block_size=b, src_dtype=src,
                          k_dtype=FP8_E4M3FN if fp8 else src, kv_layout=int(layout), num_blocks=nb,
                          src_stride=int(keys.stride(0)) if R > 1 else D)
        args = (_ptr(keys), _ptr(slots), _ptr(kcache), _ptr(kscale), ctypes.byref(shape))
        _raise_on(lib.qsa_write_keys_check(*args))
        self._ready(lib.qsa_write_keys, args, dev, stream, (keys, slots, kcache, kscale, shape))

    def __call__(self):
        self._launch()


def write_keys(keys, slots, kcache, *, block_size: int, kscale=None, layout: int = KV_PAGED, stream=None):
    """``qsa_write_keys``: index keys [R, D] into the scorer's key cache (16-bit as
    they are, or fp8 with a scale per key in the cache's layout) at ``slots``."""
    PreparedWriteKeys(keys, slots, kcache, block_size=block_size, kscale=kscale, layout=layout, stream=stream)()


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def make_attn_shape(q, kcache, block_table, *, out=None, scale: Optional[float] = None) -> AttnShape:
    """The ``qsa_attn_shape`` of a call on these tensors (scale default
    head_dim ** -0.5)."""
    R, hq, d = (int(x) for x in q.shape)
    kb, ks, kh = _kv_strides("kcache", kcache)
    out = q if out is None else out

    def strides(t):
        return (int(t.stride(0)) if R > 1 else d, int(t.stride(1)) if hq > 1 else d)

    qr, qh = strides(q)
    o_row, o_head = strides(out)
    return AttnShape(num_rows=R, num_heads=hq, num_kv_heads=int(kcache.shape[2]), head_dim=d,
                     block_size=int(kcache.shape[1]), num_reqs=int(block_table.shape[0]),
                     max_blocks=int(block_table.shape[1]), dtype=_half_code("q", q),
                     scale=float(d ** -0.5 if scale is None else scale), num_blocks=int(kcache.shape[0]),
                     q_row_stride=qr, q_head_stride=qh, out_row_stride=o_row, out_head_stride=o_head,
                     kv_block_stride=kb, kv_slot_stride=ks, kv_head_stride=kh)


def _attn_checks(q, kcache, vcache, block_table, out, lse):
    import torch
    _half_code("q", q)
    for name, t in (("kcache", kcache), ("vcache", vcache), ("out", out)):
        _require(t.dtype == q.dtype, f"{name} must have q's type")
    _require(q.dim() == 3 and q.stride(2) == 1, "q must be [R, num_heads, head_dim], its last dimension contiguous")
    _require(out.shape == q.shape and out.stride(2) == 1, "out must have q's shape, its last dimension contiguous")
    _require(kcache.shape == vcache.shape and _kv_strides("kcache", kcache) == _kv_strides("vcache", vcache),
             "kcache and vcache must have equal shapes and strides")
    _require(int(kcache.shape[3]) == int(q.shape[2]), "q and the caches must have one head_dim")
    _require(block_table.dtype == torch.int32 and block_table.dim() == 2 and block_table.is_contiguous(),
             "block_table must be contiguous int32 [num_reqs, max_blocks]")
    if lse is not None:
        _require(lse.dtype == torch.float32 and lse.is_contiguous() and tuple(lse.shape) == tuple(q.shape[:2]),
                 "lse must be contiguous f32 [R, num_heads]")


def _scratch(workspace, nbytes: int, device):
    """The workspace tensor of a call: allocated for "auto", given, or None."""
    import torch
    if isinstance(workspace, str):
        _require(workspace == "auto", 'workspace must be "auto", None or a device tensor')
        return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes > 0 else None
    if workspace is not None:
        _require(workspace.is_cuda and workspace.is_contiguous() and workspace.device == device,
                 "workspace must be a contiguous tensor on the call's device")
    return workspace


def _nbytes(t) -> int:
    return 0 if t is None else int(t.numel() * t.element_size())


class PreparedPagedAttention(_Prepared):
    """A validated ``qsa_paged_attention`` call on fixed tensors; the workspace
    ("auto": allocated once here) is part of it.  Two captured or overlapping
    calls need a workspace each."""

    def __init__(self, q, kcache, vcache, block_table, ctx_lens, q_starts, out, *, lse=None,
                 scale: Optional[float] = None, workspace="auto", stream=None):
        import torch
        dev = _one_device(q=q, kcache=kcache, vcache=vcache, block_table=block_table, ctx_lens=ctx_lens,
                          q_starts=q_starts, out=out, lse=lse)
        _attn_checks(q, kcache, vcache, block_table, out, lse)
        _check_rows_i32("ctx_lens", ctx_lens, int(q.shape[0]))
        _rows("q_starts", q_starts, int(block_table.shape[0]) + 1, torch.int32)
        self.shape = make_attn_shape(q, kcache, block_table, out=out, scale=scale)
        shape = ctypes.byref(self.shape)
        args = (_ptr(q), _ptr(kcache), _ptr(vcache), _ptr(block_table), _ptr(ctx_lens), _ptr(q_starts), _ptr(out))
        _raise_on(lib.qsa_paged_attention_check(*args, shape, None, 0))
        with _on(stream, dev):
            ws = self.workspace = _scratch(workspace, int(lib.qsa_paged_attention_workspace_bytes(shape)), dev)
        _raise_on(lib.qsa_paged_attention_check(*args, shape, _ptr(ws), _nbytes(ws)))
        self.out, self.lse = out, lse
        self._ready(lib.qsa_paged_attention, (*args, _ptr(lse), shape, _ptr(ws), _nbytes(ws)), dev, stream,
                    (q, kcache, vcache, block_table, ctx_lens, q_starts, out, lse, ws))

    def __call__(self):
        self._launch()
        return self.out


class PreparedSparseAttention(_Prepared):
    """A validated ``qsa_sparse_attention`` call on fixed tensors (see
    PreparedPagedAttention)."""

    def __init__(self, q, kcache, vcache, block_table, row_to_req, idx, out, *, ratio: int = 1, token_lens=None,
                 lse=None, scale: Optional[float] = None, workspace="auto", stream=None):
        import torch
        dev = _one_device(q=q, kcache=kcache, vcache=vcache, block_table=block_table, row_to_req=row_to_req, idx=idx,
                          token_lens=token_lens, out=out, lse=lse)
        _attn_checks(q, kcache, vcache, block_table, out, lse)
        R = int(q.shape[0])
        _check_rows_i32("row_to_req", row_to_req, R)
        if token_lens is not None:
            _check_rows_i32("token_lens", token_lens, R)
        _require(idx.dtype == torch.int32 and idx.dim() == 2 and idx.is_contiguous() and int(idx.shape[0]) == R,
                 "idx must be contiguous int32 [R, k]")
        k, ratio = int(idx.shape[1]), int(ratio)
        self.shape = make_attn_shape(q, kcache, block_table, out=out, scale=scale)
        shape = ctypes.byref(self.shape)
        args = (_ptr(q), _ptr(kcache), _ptr(vcache), _ptr(block_table), _ptr(row_to_req), _ptr(idx), k, ratio)
        _raise_on(lib.qsa_sparse_attention_check(*args, _ptr(out), shape, None, 0))
        with _on(stream, dev):
            ws = self.workspace = _scratch(workspace,
                                           int(lib.qsa_sparse_attention_workspace_bytes(shape, k, ratio)), dev)
        _raise_on(lib.qsa_sparse_attention_check(*args, _ptr(out), shape, _ptr(ws), _nbytes(ws)))
        self.out, self.lse = out, lse
        self._ready(lib.qsa_sparse_attention,
                    (*args, _ptr(token_lens), _ptr(out), _ptr(lse), shape, _ptr(ws), _nbytes(ws)), dev, stream,
                    (q, kcache, vcache, block_table, row_to_req, idx, token_lens, out, lse, ws))

    def __call__(self):
        self._launch()
        return self.out


def paged_attention(q, kcache, vcache, block_table, ctx_lens, q_starts, *, scale: Optional[float] = None, out=None,
                    lse=None, workspace="auto", stream=None):
    """``qsa_paged_attention``: attention of q [R, num_heads, head_dim] over the
    paged caches [num_blocks, block_size, num_kv_heads, head_dim]; row r sees the
    first ``ctx_lens[r]`` tokens of its request, whose rows ``q_starts`` gives.
    ``lse``: f32 [R, num_heads] to fill, or None.  Returns out."""
    import torch
    _one_device(q=q)
    with _on(stream, q.device):
        if out is None:  # rows outside all requests are not written
            out = torch.zeros(tuple(q.shape), dtype=q.dtype, device=q.device)
        return PreparedPagedAttention(q, kcache, vcache, block_table, ctx_lens, q_starts, out, lse=lse, scale=scale,
                                      workspace=workspace)()


def sparse_attention(q, kcache, vcache, block_table, row_to_req, idx, *, ratio: int = 1, token_lens=None,
                     scale: Optional[float] = None, out=None, lse=None, workspace="auto", stream=None):
    """``qsa_sparse_attention``: the same over the tokens of the selected columns
    ``idx`` [R, k] (``topk``'s output with the cache's compression ``ratio``, or
    ``expand``'s with 1), left out at and behind ``token_lens``.  Returns out."""
    import torch
    _one_device(q=q)
    with _on(stream, q.device):
        if out is None:
            out = torch.empty(tuple(q.shape), dtype=q.dtype, device=q.device)
        return PreparedSparseAttention(q, kcache, vcache, block_table, row_to_req, idx, out, ratio=ratio,
                                       token_lens=token_lens, lse=lse, scale=scale, workspace=workspace)()


def paged_attention_workspace_bytes(shape: AttnShape) -> int:
    """``qsa_paged_attention_workspace_bytes`` (see ``make_attn_shape``)."""
    return int(lib.qsa_paged_attention_workspace_bytes(ctypes.byref(shape)))


def sparse_attention_workspace_bytes(shape: AttnShape, k: int, ratio: int = 1) -> int:
    """``qsa_sparse_attention_workspace_bytes`` (see ``make_attn_shape``)."""
    return int(lib.qsa_sparse_attention_workspace_bytes(ctypes.byref(shape), int(k), int(ratio)))
