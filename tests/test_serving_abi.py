"""Host-side checks of the batch plan, cache write and attention calls, through
the *_check entry points (no HIP call), and their workspace queries."""
from __future__ import annotations

import ctypes

import pytest

m = pytest.importorskip("paged_mqa_logits_block_amd")

A = 0x10000


def plan_check(p=A, n=A, f=A, bt=A, qs=A, rr=A, cl=A, sl=A, **kw):
    base = dict(num_reqs=9, max_blocks=100, block_size=16, ratio=4, num_rows=36, num_free=10, num_blocks=500)
    base.update(kw)
    return m.lib.qsa_plan_batch_check(p, n, f, bt, qs, rr, cl, sl, m.PlanShape(**base))


@pytest.mark.parametrize("kw,status", [
    ({}, "OK"), (dict(num_rows=0, rr=None, cl=None, sl=None), "OK"), (dict(num_free=0, f=None), "OK"),
    (dict(ratio=1, block_size=100), "OK"), (dict(num_reqs=4096), "OK"),
    (dict(num_reqs=4097), "E_UNSUPPORTED"), (dict(num_reqs=0), "E_INVALID"), (dict(num_rows=-1), "E_INVALID"),
    (dict(num_free=-1), "E_INVALID"), (dict(ratio=3), "E_INVALID"), (dict(ratio=0), "E_INVALID"),
    (dict(block_size=0), "E_INVALID"), (dict(num_blocks=0), "E_INVALID"), (dict(p=None), "E_INVALID"),
    (dict(bt=None), "E_INVALID"), (dict(qs=None), "E_INVALID"), (dict(sl=None), "E_INVALID"),
    (dict(f=None), "E_INVALID"), (dict(max_blocks=1 << 27), "E_RANGE"), (dict(num_rows=(1 << 30) + 1), "E_RANGE"),
])
def test_plan_check(kw, status):
    assert plan_check(**kw) == getattr(m, status), m.last_error()


def kv_check(k=A, v=A, s=A, kc=A, vc=A, **kw):
    base = dict(num_rows=36, num_kv_heads=4, head_dim=128, block_size=16, dtype=m.BF16, num_blocks=100,
                src_row_stride=512, src_head_stride=128, kv_block_stride=16 * 512, kv_slot_stride=512,
                kv_head_stride=128)
    base.update(kw)
    return m.lib.qsa_write_kv_check(k, v, s, kc, vc, m.KvShape(**base))


@pytest.mark.parametrize("kw,status", [
    ({}, "OK"), (dict(dtype=m.FP16, head_dim=64), "OK"), (dict(num_rows=0, k=None, s=None), "OK"),
    (dict(src_row_stride=0), "OK"),
    (dict(dtype=m.FP8_E4M3FN), "E_DTYPE"), (dict(head_dim=96), "E_UNSUPPORTED"), (dict(block_size=1025), "E_UNSUPPORTED"),
    (dict(num_kv_heads=1025), "E_UNSUPPORTED"), (dict(num_kv_heads=0), "E_INVALID"), (dict(s=None), "E_INVALID"),
    (dict(vc=None), "E_INVALID"), (dict(kv_head_stride=64), "E_INVALID"), (dict(kv_slot_stride=0), "E_INVALID"),
    (dict(src_row_stride=-512), "E_INVALID"), (dict(k=A + 8), "E_ALIGN"), (dict(kv_block_stride=16 * 512 + 4), "E_ALIGN"),
    (dict(num_blocks=1 << 49), "E_RANGE"),
])
def test_write_kv_check(kw, status):
    assert kv_check(**kw) == getattr(m, status), m.last_error()


def keys_check(k=A, s=A, kc=A, ks=None, **kw):
    base = dict(num_rows=36, head_dim=128, block_size=64, src_dtype=m.BF16, k_dtype=m.FP8_E4M3FN,
                kv_layout=m.KV_COPACKED, num_blocks=100, src_stride=128)
    base.update(kw)
    return m.lib.qsa_write_keys_check(k, s, kc, ks, m.KeysShape(**base))


@pytest.mark.parametrize("kw,status", [
    ({}, "OK"), (dict(kv_layout=m.KV_COPACKED_SHUFFLED, block_size=48), "OK"), (dict(kv_layout=m.KV_PAGED, ks=A), "OK"),
    (dict(kv_layout=m.KV_PAGED, k_dtype=m.BF16), "OK"), (dict(src_dtype=m.FP16, head_dim=64), "OK"),
    (dict(kv_layout=m.KV_COPACKED_SHUFFLED, block_size=40), "E_UNSUPPORTED"), (dict(k_dtype=m.BF16), "E_UNSUPPORTED"),
    (dict(ks=A), "E_INVALID"), (dict(k_dtype=m.BF16, kv_layout=m.KV_PAGED, ks=A), "E_INVALID"),
    (dict(src_dtype=m.FP8_E4M3FN), "E_DTYPE"), (dict(k_dtype=m.FP16, kv_layout=m.KV_PAGED), "E_DTYPE"),
    (dict(kv_layout=3), "E_INVALID"), (dict(head_dim=96), "E_UNSUPPORTED"), (dict(src_stride=64), "E_INVALID"),
    (dict(src_stride=132), "E_ALIGN"), (dict(kc=A + 4), "E_ALIGN"), (dict(s=None), "E_INVALID"),
    (dict(block_size=0), "E_INVALID"), (dict(num_blocks=1 << 41), "E_RANGE"),
])
def test_write_keys_check(kw, status):
    assert keys_check(**kw) == getattr(m, status), m.last_error()


def attn_shape(**kw):
    base = dict(num_rows=36, num_heads=32, num_kv_heads=4, head_dim=128, block_size=16, num_reqs=9, max_blocks=1000,
                dtype=m.BF16, scale=0.1, num_blocks=9000, q_row_stride=4096, q_head_stride=128, out_row_stride=4096,
                out_head_stride=128, kv_block_stride=16 * 512, kv_slot_stride=512, kv_head_stride=128)
    base.update(kw)
    return m.AttnShape(**base)


ATTN = [
    ({}, "OK"), (dict(dtype=m.FP16), "OK"), (dict(head_dim=64), "OK"), (dict(num_heads=4), "OK"),
    (dict(num_heads=512, q_row_stride=65536, out_row_stride=65536), "OK"), (dict(q_row_stride=0), "OK"),
    (dict(num_rows=0), "OK"), (dict(block_size=1), "OK"),
    (dict(num_heads=30), "E_INVALID"), (dict(scale=0.0), "E_INVALID"), (dict(scale=-1.0), "E_INVALID"),
    (dict(scale=float("nan")), "E_INVALID"), (dict(scale=float("inf")), "E_INVALID"), (dict(scale=3e38), "E_INVALID"), (dict(num_rows=-1), "E_INVALID"),
    (dict(out_row_stride=0), "E_INVALID"), (dict(out_head_stride=64), "E_INVALID"), (dict(kv_slot_stride=-8), "E_INVALID"),
    (dict(num_reqs=0), "E_INVALID"), (dict(dtype=m.FP8_E4M3FN), "E_DTYPE"), (dict(head_dim=96), "E_UNSUPPORTED"),
    (dict(num_heads=516), "E_UNSUPPORTED"), (dict(block_size=2048), "E_UNSUPPORTED"),
    (dict(num_rows=(1 << 22) + 1), "E_RANGE"), (dict(max_blocks=1 << 27), "E_RANGE"),
    (dict(num_blocks=1 << 48), "E_RANGE"), (dict(q_head_stride=132), "E_ALIGN"), (dict(kv_block_stride=8196), "E_ALIGN"),
]


@pytest.mark.parametrize("kw,status", ATTN)
def test_attention_checks(kw, status):
    s = attn_shape(**kw)
    assert m.lib.qsa_paged_attention_check(A, A, A, A, A, A, A, s, None, 0) == getattr(m, status), m.last_error()
    assert m.lib.qsa_sparse_attention_check(A, A, A, A, A, A, 2048, 4, A, s, None, 0) == getattr(m, status)


def test_attention_pointers_and_sizes():
    s = attn_shape()
    for i in range(7):
        ptrs = [A] * 7
        ptrs[i] = None
        assert m.lib.qsa_paged_attention_check(*ptrs, s, None, 0) == m.E_INVALID
        assert m.lib.qsa_sparse_attention_check(*ptrs[:6], 64, 1, ptrs[6], s, None, 0) == m.E_INVALID
    assert m.lib.qsa_paged_attention_check(A + 2, A, A, A, A, A, A, s, None, 0) == m.E_ALIGN
    assert m.lib.qsa_paged_attention_check(A, A, A, A, A, A, A, None, None, 0) == m.E_INVALID
    for k, ratio, st in ((0, 1, m.E_INVALID), (1, 0, m.E_INVALID), (1 << 20, 17, m.E_RANGE), (1 << 20, 16, m.OK)):
        assert m.lib.qsa_sparse_attention_check(A, A, A, A, A, A, k, ratio, A, s, None, 0) == st


@pytest.mark.parametrize("kw,status", [
    (dict(num_rows=1 << 21), "OK"), (dict(num_rows=(1 << 21) + 1), "E_RANGE"),
    (dict(num_reqs=1 << 21, num_heads=8, num_kv_heads=1), "OK"), (dict(num_reqs=(1 << 21) + 1, num_heads=8, num_kv_heads=1), "E_RANGE"),
    (dict(max_blocks=1 << 20, block_size=1024), "OK"), (dict(max_blocks=(1 << 20) + 1, block_size=1024), "E_RANGE"),
])
def test_attention_limits(kw, status):
    s = attn_shape(**kw)
    assert m.lib.qsa_paged_attention_check(A, A, A, A, A, A, A, s, None, 0) == getattr(m, status), m.last_error()
    assert m.lib.qsa_sparse_attention_check(A, A, A, A, A, A, 2048, 4, A, s, None, 0) == getattr(m, status)


def test_attention_workspace():
    """A workspace is wanted only where few rows meet long tables; one that is
    given must hold it."""
    s = attn_shape()
    need = m.paged_attention_workspace_bytes(s)
    assert need > 0
    check = m.lib.qsa_paged_attention_check
    assert check(A, A, A, A, A, A, A, s, A, need) == m.OK
    assert check(A, A, A, A, A, A, A, s, A, need - 1) == m.E_INVALID
    assert check(A, A, A, A, A, A, A, s, A + 4, need) == m.E_ALIGN
    assert m.paged_attention_workspace_bytes(attn_shape(max_blocks=4)) == 0
    assert m.paged_attention_workspace_bytes(attn_shape(num_rows=0)) == 0
    assert m.sparse_attention_workspace_bytes(s, 2048, 4) > 0
    assert m.sparse_attention_workspace_bytes(attn_shape(num_rows=4096), 2048, 4) == 0
    assert m.sparse_attention_workspace_bytes(s, 0, 4) == 0
    # tables whose steps do not add up in 32 bits are not cut
    big = dict(num_rows=500, num_reqs=500, block_size=1024, num_heads=8, num_kv_heads=1)
    assert m.paged_attention_workspace_bytes(attn_shape(max_blocks=1 << 17, **big)) > 0
    assert m.paged_attention_workspace_bytes(attn_shape(max_blocks=1 << 19, **big)) == 0
    # shapes that the calls refuse need none, and the queries do not fail on them
    for kw in (dict(num_heads=4096), dict(num_heads=2, num_kv_heads=4), dict(num_kv_heads=0), dict(head_dim=0),
               dict(num_rows=-5), dict(num_rows=2 ** 31 - 1), dict(num_reqs=2 ** 31 - 1), dict(block_size=2 ** 31 - 1)):
        assert m.paged_attention_workspace_bytes(attn_shape(**kw)) == 0, kw
        assert m.sparse_attention_workspace_bytes(attn_shape(**kw), 64, 4) == 0, kw
    assert check(A, A, A, A, A, A, A, attn_shape(num_rows=1 << 21, num_reqs=1 << 21, num_kv_heads=32), None,
                 0) == m.E_RANGE


@pytest.mark.parametrize("rows,reqs,kv_heads", [(20, 20, 32), (20, 1000, 32), (1, 1000, 1024), (1, 1023, 1), (600, 600, 1),
                                                (4, 500, 250)])
def test_attention_workspace_is_bounded(rows, reqs, kv_heads):
    """Requests without rows cost no workspace: a state of 32 pairs (and a note) for
    each of 256 workgroups and for each of at most 2 x 1,024 tiles with rows is all
    that a cut launch of the streaming kernel leaves."""
    def need(n):
        s = attn_shape(num_rows=rows, num_reqs=n, num_heads=8 * kv_heads, num_kv_heads=kv_heads,
                       q_row_stride=1024 * kv_heads, out_row_stride=1024 * kv_heads)
        return m.paged_attention_workspace_bytes(s)
    state = 32 * 130 * 4 + 16
    assert 0 < need(reqs) <= (256 + 2 * 1024) * state
    assert need(reqs) == need(min(rows, reqs))


def test_host_tensors_are_refused():
    import torch
    q = torch.zeros(4, 8, 64, dtype=torch.bfloat16)
    kc = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    for call in (lambda: m.paged_attention(q, kc, kc, i.view(1, 4), i, i[:2]),
                 lambda: m.sparse_attention(q, kc, kc, i.view(1, 4), i, i.view(4, 1)),
                 lambda: m.write_kv(q, q, i.long(), kc, kc),
                 lambda: m.write_keys(q[:, 0], i.long(), kc[:, :, 0], block_size=16),
                 lambda: m.plan_batch(i, i, i, i.view(4, 1), block_size=16, num_blocks=4, num_rows=8)):
        with pytest.raises(m.QsaError) as e:
            call()
        assert e.value.status == m.E_INVALID
