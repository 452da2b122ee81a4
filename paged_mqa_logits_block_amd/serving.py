"""The calls around the scorer: batch plan, cache writes, head norms with rotary
positions, attention, and the verification of drafted tokens.

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
import math
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


class RopeShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("num_rows", "num_heads", "num_kv_heads", "head_dim", "rot_dim",
                                              "rot_offset", "layout", "dtype", "position_offset", "block_size")] + \
               [("eps", ctypes.c_float), ("factor", ctypes.c_float)] + \
               [(n, ctypes.c_int64) for n in ("num_blocks", "q_row_stride", "q_head_stride", "k_row_stride",
                                              "k_head_stride", "v_row_stride", "v_head_stride", "q_out_row_stride",
                                              "q_out_head_stride", "k_out_row_stride", "k_out_head_stride",
                                              "kv_block_stride", "kv_slot_stride", "kv_head_stride")]


class VerifyShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("num_rows", "num_reqs", "vocab", "max_tokens")] + \
               [("prob_stride", ctypes.c_int64), ("draft_stride", ctypes.c_int64)]


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
            ("qsa_norm_rope", [vp] * 12 + [p(RopeShape), vp], ctypes.c_int),
            ("qsa_norm_rope_check", [vp] * 10 + [p(RopeShape)], ctypes.c_int),
            ("qsa_verify_drafts", [vp] * 8 + [p(VerifyShape), vp, i64, vp], ctypes.c_int),
            ("qsa_verify_drafts_check", [vp] * 8 + [p(VerifyShape), vp, i64], ctypes.c_int),
            ("qsa_verify_drafts_workspace_bytes", [p(VerifyShape)], i64),
            ("qsa_paged_attention", [vp] * 8 + [p(AttnShape), vp, i64, vp], ctypes.c_int),
            ("qsa_paged_attention_check", [vp] * 7 + [p(AttnShape), vp, i64], ctypes.c_int),
            ("qsa_paged_attention_workspace_bytes", [p(AttnShape)], i64),
            ("qsa_window_attention", [vp] * 6 + [i32, i32, vp, vp, p(AttnShape), vp, i64, vp], ctypes.c_int),
            ("qsa_window_attention_check", [vp] * 6 + [i32, i32, vp, p(AttnShape), vp, i64], ctypes.c_int),
            ("qsa_window_attention_workspace_bytes", [p(AttnShape), i32, i32], i64),
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


def _int32(name, x) -> int:
    """x as an integer that the call takes unchanged (ctypes drops higher bits)."""
    _require(-2 ** 31 <= int(x) < 2 ** 31, f"{name} = {x} does not fit 32 bits")
    return int(x)


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
        shape = PlanShape(num_reqs=n, max_blocks=int(block_table.shape[1]), block_size=_int32("block_size", block_size),
                          ratio=_int32("ratio", ratio), num_rows=rows, num_free=int(free_blocks.numel()),
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
                          k_dtype=FP8_E4M3FN if fp8 else src, kv_layout=_int32("layout", layout), num_blocks=nb,
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
# head norms and rotary positions
# ---------------------------------------------------------------------------

ROPE_HALF, ROPE_INTERLEAVED = 0, 1


def rope_frequencies(rot_dim: int, base: float = 10000.0, *, scaling: str = "none", factor: float = 1.0,
                     original_len: Optional[int] = None, beta_fast: float = 32.0, beta_slow: float = 1.0,
                     device=None):
    """(inv_freq, rope_scale) for ``norm_rope``: f64 [rot_dim / 2] radians per position,
    base ** (-2 i / rot_dim), and the factor on cosines and sines.  For contexts
    ``factor`` times longer:

    - ``"linear"``: all positions stretched by the factor.
    - ``"ntk"``: the base raised so that the slowest pair is stretched by the factor
      and the fastest is not.
    - ``"yarn"``: pairs that turn less than ``beta_slow`` times in ``original_len``
      positions stretched, those that turn more than ``beta_fast`` times kept, a ramp over the pairs
      between; rope_scale = 0.1 ln(factor) + 1."""
    import torch
    _require(rot_dim >= 0 and rot_dim % 2 == 0, f"rot_dim = {rot_dim} must be even and >= 0")
    _require(base > 1.0 and factor >= 1.0, "base must be > 1 and factor >= 1")
    _require(scaling in ("none", "linear", "ntk", "yarn"), f"unknown scaling {scaling!r}")
    i = torch.arange(0, rot_dim, 2, dtype=torch.float64)
    if scaling == "ntk":
        _require(rot_dim > 2, "ntk needs rot_dim > 2")
        base = base * factor ** (rot_dim / (rot_dim - 2))
    freq = float(base) ** (-i / max(rot_dim, 1))
    scale = 1.0
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "yarn":
        _require(original_len is not None and original_len > 0 and beta_fast > beta_slow > 0,
                 "yarn needs original_len and beta_fast > beta_slow > 0")

        def pair(turns):  # the pair that turns so often in original_len positions
            return rot_dim * math.log(original_len / (turns * 2 * math.pi)) / (2 * math.log(base))

        low = max(math.floor(pair(beta_fast)), 0)
        high = min(math.ceil(pair(beta_slow)), rot_dim - 1)
        # (below 0: not even the first pair turns so often)
        ramp = ((i / 2 - low) / max(high - low, 0.001)).clamp(0.0, 1.0) if pair(beta_slow) >= 0 else torch.ones_like(i)
        freq = freq / factor * ramp + freq * (1.0 - ramp)
        scale = 0.1 * math.log(factor) + 1.0
    return freq.to(device), scale


def _heads(name, t, rows, dim, dtype):
    """(row stride, head stride) of a [R, heads, head_dim] tensor."""
    _require(t.dtype == dtype, f"{name} must have the heads' type {dtype}")
    _require(t.dim() == 3 and int(t.shape[0]) == rows and int(t.shape[2]) == dim and (t.stride(2) == 1 or dim == 1),
             f"{name} must be [R, heads, head_dim] with a contiguous last dimension")
    # the stride of a dimension of one element has no meaning: any allowed value does
    return int(t.stride(0)) if rows > 1 else dim, int(t.stride(1)) if int(t.shape[1]) > 1 else dim


class PreparedNormRope(_Prepared):
    """A validated ``qsa_norm_rope`` call on fixed tensors."""

    def __init__(self, q, k, positions, inv_freq, q_out=None, *, k_out=None, v=None, slots=None, kcache=None,
                 vcache=None, q_weight=None, k_weight=None, eps: float = 1e-6, rot_offset: int = 0,
                 layout: int = ROPE_HALF, rope_scale: float = 1.0, position_offset: int = 0, stream=None):
        import torch
        dev = _one_device(positions=positions, inv_freq=inv_freq, q=q, k=k, v=v, slots=slots, q_out=q_out, k_out=k_out,
                          kcache=kcache, vcache=vcache, q_weight=q_weight, k_weight=k_weight)
        some = q if q is not None else k
        _require(some is not None and some.dim() == 3, "q and k must be [R, heads, head_dim]; one of them may be None")
        code = _half_code("q" if q is not None else "k", some)
        R, d, dt = int(some.shape[0]), int(some.shape[2]), some.dtype
        _require((q is None) == (q_out is None), "q and q_out belong together")
        _require((v is None) == (vcache is None), "v and vcache belong together")
        _require(k is not None or (k_out is None and kcache is None and v is None), "outputs of keys without k")
        for name, x in (("rot_offset", rot_offset), ("layout", layout), ("position_offset", position_offset)):
            _int32(name, x)
        strides = {}
        for name, t, like in (("q", q, q), ("k", k, k), ("v", v, k), ("q_out", q_out, q), ("k_out", k_out, k)):
            strides[name] = (0, 0)
            if t is not None:
                strides[name] = _heads(name, t, R, d, dt)
                _require(t.shape == like.shape, f"{name} must have the shape of its heads")
        cache = dict(block_size=0, num_blocks=0, kv_block_stride=0, kv_slot_stride=0, kv_head_stride=0)
        if kcache is not None:
            kv = _kv_strides("kcache", kcache)
            _require(kcache.dtype == dt and (int(kcache.shape[2]), int(kcache.shape[3])) == (int(k.shape[1]), d),
                     "kcache must have k's type and heads")
            if vcache is not None:
                _require(vcache.dtype == dt and vcache.shape == kcache.shape and _kv_strides("vcache", vcache) == kv,
                         "kcache and vcache must have equal types, shapes and strides")
            _require(slots is not None, "kcache needs slots")
            _rows("slots", slots, R, torch.int64)
            cache = dict(block_size=int(kcache.shape[1]), num_blocks=int(kcache.shape[0]), kv_block_stride=kv[0],
                         kv_slot_stride=kv[1], kv_head_stride=kv[2])
        else:
            _require(slots is None and vcache is None, "slots and vcache go with kcache")
        _rows("positions", positions, R, torch.int32)
        _rows("inv_freq", inv_freq, int(inv_freq.numel()), torch.float64)
        for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
            if w is not None:
                _rows(name, w, d, torch.float32)
        _require(q_weight is None or q is not None, "q_weight without q")
        _require(k_weight is None or k is not None, "k_weight without k")
        self.shape = RopeShape(
            num_rows=R, num_heads=0 if q is None else int(q.shape[1]), num_kv_heads=0 if k is None else int(k.shape[1]),
            head_dim=d, rot_dim=2 * int(inv_freq.numel()), rot_offset=int(rot_offset), layout=int(layout), dtype=code,
            position_offset=int(position_offset), eps=float(eps), factor=float(rope_scale),
            **{f"{n}_{w}_stride": strides[n][i] for n in strides for i, w in enumerate(("row", "head"))}, **cache)
        shape = ctypes.byref(self.shape)
        ins = (_ptr(q), _ptr(k), _ptr(v))
        at = (_ptr(positions), _ptr(inv_freq), _ptr(slots))
        outs = (_ptr(q_out), _ptr(k_out), _ptr(kcache), _ptr(vcache))
        _raise_on(lib.qsa_norm_rope_check(*ins, *at, *outs, shape))
        self.q_out, self.k_out = q_out, k_out
        self._ready(lib.qsa_norm_rope, (*ins, _ptr(q_weight), _ptr(k_weight), *at, *outs, shape), dev, stream,
                    (q, k, v, q_weight, k_weight, positions, inv_freq, slots, q_out, k_out, kcache, vcache))

    def __call__(self):
        self._launch()
        return self.q_out, self.k_out


def norm_rope(q, k, positions, inv_freq, *, q_out=None, k_out=None, v=None, slots=None, kcache=None, vcache=None,
              q_weight=None, k_weight=None, eps: float = 1e-6, rot_offset: int = 0, layout: int = ROPE_HALF,
              rope_scale: float = 1.0, position_offset: int = 0, stream=None):
    """``qsa_norm_rope``: heads of q and k [R, heads, head_dim] (either may be None) normed
    where they have a weight (f32 [head_dim]) and rotated by ``positions`` (int32 [R], plus
    ``position_offset``: -1 with a plan's ``ctx_lens``) in elements [rot_offset,
    rot_offset + 2 len(inv_freq)); ``rope_frequencies`` makes inv_freq and rope_scale.
    With ``kcache`` and ``slots`` the keys go to the paged cache, and v to ``vcache``.
    Returns (q_out, k_out); k_out is None where only the cache takes the keys.  Rows with a
    negative position are not written (0 in outputs made here)."""
    import torch
    _one_device(positions=positions)
    with _on(stream, positions.device):
        if q is not None and q_out is None:
            q_out = torch.zeros(tuple(q.shape), dtype=q.dtype, device=q.device)
        if k is not None and k_out is None and kcache is None:
            k_out = torch.zeros(tuple(k.shape), dtype=k.dtype, device=k.device)
        return PreparedNormRope(q, k, positions, inv_freq, q_out, k_out=k_out, v=v, slots=slots, kcache=kcache,
                                vcache=vcache, q_weight=q_weight, k_weight=k_weight, eps=eps, rot_offset=rot_offset,
                                layout=layout, rope_scale=rope_scale, position_offset=position_offset)()


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


class PreparedWindowAttention(_Prepared):
    """A validated ``qsa_window_attention`` call on fixed tensors (see
    PreparedPagedAttention)."""

    def __init__(self, q, kcache, vcache, block_table, ctx_lens, q_starts, out, *, window: int, sinks: int = 0, lse=None,
                 scale: Optional[float] = None, workspace="auto", stream=None):
        import torch
        dev = _one_device(q=q, kcache=kcache, vcache=vcache, block_table=block_table, ctx_lens=ctx_lens,
                          q_starts=q_starts, out=out, lse=lse)
        _attn_checks(q, kcache, vcache, block_table, out, lse)
        _check_rows_i32("ctx_lens", ctx_lens, int(q.shape[0]))
        _rows("q_starts", q_starts, int(block_table.shape[0]) + 1, torch.int32)
        window, sinks = _int32("window", window), _int32("sinks", sinks)
        self.shape = make_attn_shape(q, kcache, block_table, out=out, scale=scale)
        shape = ctypes.byref(self.shape)
        args = (_ptr(q), _ptr(kcache), _ptr(vcache), _ptr(block_table), _ptr(ctx_lens), _ptr(q_starts), window, sinks,
                _ptr(out))
        _raise_on(lib.qsa_window_attention_check(*args, shape, None, 0))
        with _on(stream, dev):
            ws = self.workspace = _scratch(workspace,
                                           int(lib.qsa_window_attention_workspace_bytes(shape, window, sinks)), dev)
        _raise_on(lib.qsa_window_attention_check(*args, shape, _ptr(ws), _nbytes(ws)))
        self.out, self.lse = out, lse
        self._ready(lib.qsa_window_attention, (*args, _ptr(lse), shape, _ptr(ws), _nbytes(ws)), dev, stream,
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
        k, ratio = int(idx.shape[1]), _int32("ratio", ratio)
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


def window_attention(q, kcache, vcache, block_table, ctx_lens, q_starts, *, window: int, sinks: int = 0,
                     scale: Optional[float] = None, out=None, lse=None, workspace="auto", stream=None):
    """``qsa_window_attention``: ``paged_attention`` in which row r sees the newest ``window`` of
    its ``ctx_lens[r]`` tokens and the first ``sinks``; blocks that no row of a request sees any
    more may have been freed.  Returns out."""
    import torch
    _one_device(q=q)
    with _on(stream, q.device):
        if out is None:  # rows outside all requests are not written
            out = torch.zeros(tuple(q.shape), dtype=q.dtype, device=q.device)
        return PreparedWindowAttention(q, kcache, vcache, block_table, ctx_lens, q_starts, out, window=window,
                                       sinks=sinks, lse=lse, scale=scale, workspace=workspace)()


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


def window_attention_workspace_bytes(shape: AttnShape, window: int, sinks: int = 0) -> int:
    """``qsa_window_attention_workspace_bytes`` (see ``make_attn_shape``)."""
    return int(lib.qsa_window_attention_workspace_bytes(ctypes.byref(shape), _int32("window", window),
                                                        _int32("sinks", sinks)))


def sparse_attention_workspace_bytes(shape: AttnShape, k: int, ratio: int = 1) -> int:
    """``qsa_sparse_attention_workspace_bytes`` (see ``make_attn_shape``)."""
    return int(lib.qsa_sparse_attention_workspace_bytes(ctypes.byref(shape), _int32("k", k), _int32("ratio", ratio)))


# ---------------------------------------------------------------------------
# verification of drafted tokens
# ---------------------------------------------------------------------------

class PreparedVerifyDrafts(_Prepared):
    """A validated ``qsa_verify_drafts`` call on fixed tensors (workspace as in
    PreparedPagedAttention)."""

    def __init__(self, probs, tokens, q_starts, uniforms, sample_uniforms, out_tokens, num_tokens, *, draft_probs=None,
                 workspace="auto", stream=None):
        import torch
        dev = _one_device(probs=probs, draft_probs=draft_probs, tokens=tokens, q_starts=q_starts, uniforms=uniforms,
                          sample_uniforms=sample_uniforms, out_tokens=out_tokens, num_tokens=num_tokens)
        for name, t in (("probs", probs), ("draft_probs", draft_probs)):
            if t is not None:
                _require(t.dtype == torch.float32 and t.dim() == 2 and t.shape == probs.shape and
                         (t.stride(1) == 1 or int(t.shape[1]) == 1), f"{name} must be f32 [R, V], its rows contiguous")
        R, v = (int(x) for x in probs.shape)
        _require(out_tokens.dtype == torch.int32 and out_tokens.dim() == 2 and out_tokens.is_contiguous(),
                 "out_tokens must be contiguous int32 [n, max_tokens]")
        n, most = (int(x) for x in out_tokens.shape)
        _rows("tokens", tokens, R, torch.int32)
        _rows("uniforms", uniforms, R, torch.float32)
        _rows("q_starts", q_starts, n + 1, torch.int32)
        _rows("sample_uniforms", sample_uniforms, n, torch.float32)
        _rows("num_tokens", num_tokens, n, torch.int32)

        def stride(t):
            return v if t is None or R <= 1 else int(t.stride(0))

        self.shape = VerifyShape(num_rows=R, num_reqs=n, vocab=v, max_tokens=most, prob_stride=stride(probs),
                                 draft_stride=stride(draft_probs))
        shape = ctypes.byref(self.shape)
        args = (_ptr(probs), _ptr(draft_probs), _ptr(tokens), _ptr(q_starts), _ptr(uniforms), _ptr(sample_uniforms),
                _ptr(out_tokens), _ptr(num_tokens))
        _raise_on(lib.qsa_verify_drafts_check(*args, shape, None, 0))
        with _on(stream, dev):
            ws = self.workspace = _scratch(workspace, int(lib.qsa_verify_drafts_workspace_bytes(shape)), dev)
        _raise_on(lib.qsa_verify_drafts_check(*args, shape, _ptr(ws), _nbytes(ws)))
        self.out_tokens, self.num_tokens = out_tokens, num_tokens
        self._ready(lib.qsa_verify_drafts, (*args, shape, _ptr(ws), _nbytes(ws)), dev, stream,
                    (probs, draft_probs, tokens, q_starts, uniforms, sample_uniforms, out_tokens, num_tokens, ws))

    def __call__(self):
        self._launch()
        return self.out_tokens, self.num_tokens


def verify_drafts(probs, tokens, q_starts, uniforms, sample_uniforms, *, max_tokens: int, draft_probs=None,
                  out_tokens=None, num_tokens=None, workspace="auto", stream=None):
    """``qsa_verify_drafts``: which drafts of a verify step's requests are kept, and the token
    after them.  ``probs`` f32 [R, V] are the target's distributions of the step's rows,
    ``tokens`` int32 [R] the rows' inputs (a request's last token, then its drafts),
    ``draft_probs`` the distributions the drafts came from, row by row with ``probs`` (None:
    each was certain); ``uniforms`` f32 [R] and ``sample_uniforms`` f32 [n] in [0, 1).
    Returns (int32 [n, max_tokens] tokens, -1 behind the last, int32 [n] their number)."""
    import torch
    _one_device(probs=probs, q_starts=q_starts)
    n = int(q_starts.numel()) - 1
    _require(n >= 0, "q_starts must have an entry more than there are requests")
    with _on(stream, probs.device):
        if out_tokens is None:
            out_tokens = torch.empty((n, int(max_tokens)), dtype=torch.int32, device=probs.device)
        if num_tokens is None:
            num_tokens = torch.empty(n, dtype=torch.int32, device=probs.device)
        _require(out_tokens.dim() == 2 and int(out_tokens.shape[1]) == int(max_tokens),
                 "out_tokens must be [n, max_tokens]")
        return PreparedVerifyDrafts(probs, tokens, q_starts, uniforms, sample_uniforms, out_tokens, num_tokens,
                                    draft_probs=draft_probs, workspace=workspace)()


def verify_drafts_workspace_bytes(shape: VerifyShape) -> int:
    """``qsa_verify_drafts_workspace_bytes``."""
    return int(lib.qsa_verify_drafts_workspace_bytes(ctypes.byref(shape)))
