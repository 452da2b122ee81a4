"""Host-side checks of the head norm, windowed attention and draft verification
calls, through the *_check entry points (no HIP call), their workspace queries,
and the frequencies of scaled rotary positions."""
from __future__ import annotations

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
m = pytest.importorskip("paged_mqa_logits_block_amd")

A = 0x10000


def rope_check(q=A, k=A, v=A, pos=A, f=A, s=A, qo=A, ko=None, kc=A, vc=A, **kw):
    base = dict(num_rows=36, num_heads=32, num_kv_heads=4, head_dim=128, rot_dim=64, rot_offset=32, layout=m.ROPE_HALF,
                dtype=m.BF16, position_offset=-1, block_size=16, eps=1e-6, factor=1.0, num_blocks=100,
                q_row_stride=4096, q_head_stride=128, k_row_stride=512, k_head_stride=128, v_row_stride=512,
                v_head_stride=128, q_out_row_stride=4096, q_out_head_stride=128, k_out_row_stride=512,
                k_out_head_stride=128, kv_block_stride=16 * 512, kv_slot_stride=512, kv_head_stride=128)
    base.update(kw)
    return m.lib.qsa_norm_rope_check(q, k, v, pos, f, s, qo, ko, kc, vc, m.RopeShape(**base))


NO_K = dict(k=None, v=None, s=None, kc=None, vc=None, num_kv_heads=0)


@pytest.mark.parametrize("kw,status", [
    ({}, "OK"), (dict(dtype=m.FP16, head_dim=64, rot_dim=32), "OK"), (dict(layout=m.ROPE_INTERLEAVED), "OK"), (dict(ko=A), "OK"),
    (dict(kc=None, vc=None, v=None, s=None, ko=A), "OK"), (dict(v=None, vc=None), "OK"), (NO_K, "OK"),
    (dict(num_heads=0, q=None, qo=None), "OK"), (dict(rot_dim=0, rot_offset=0, f=None), "OK"),
    (dict(rot_dim=128, rot_offset=0), "OK"), (dict(rot_dim=16, rot_offset=112), "OK"), (dict(eps=0.0), "OK"),
    (dict(num_rows=0, q=None, qo=None, k=None, pos=None, f=None, s=None), "OK"), (dict(q_row_stride=0), "OK"),
    (dict(factor=-1.0), "OK"), (dict(position_offset=2 ** 31 - 1), "OK"),
    (dict(num_rows=-1), "E_INVALID"), (dict(num_heads=-1), "E_INVALID"), (dict(layout=2), "E_INVALID"),
    (dict(NO_K, num_heads=0, q=None, qo=None), "E_INVALID"), (dict(eps=-1e-6), "E_INVALID"),
    (dict(eps=float("nan")), "E_INVALID"), (dict(factor=float("inf")), "E_INVALID"), (dict(factor=float("nan")), "E_INVALID"),
    (dict(rot_dim=128), "E_INVALID"), (dict(rot_offset=-8), "E_INVALID"), (dict(rot_dim=-16), "E_INVALID"),
    (dict(rot_offset=2 ** 31 - 8), "E_INVALID"), (dict(rot_dim=2 ** 31 - 16), "E_INVALID"),
    (dict(rot_dim=40), "E_UNSUPPORTED"), (dict(rot_offset=4), "E_UNSUPPORTED"), (dict(head_dim=96), "E_UNSUPPORTED"),
    (dict(num_heads=8193), "E_UNSUPPORTED"), (dict(num_kv_heads=1025), "E_UNSUPPORTED"), (dict(block_size=1025), "E_UNSUPPORTED"),
    (dict(dtype=m.FP8_E4M3FN), "E_DTYPE"), (dict(num_rows=1 << 21), "OK"), (dict(num_rows=(1 << 21) + 1), "E_RANGE"),
    (dict(q_row_stride=(1 << 30) + 8), "E_RANGE"), (dict(num_blocks=1 << 49), "E_RANGE"),
    (dict(q=None), "E_INVALID"), (dict(qo=None), "E_INVALID"), (dict(k=None), "E_INVALID"), (dict(pos=None), "E_INVALID"),
    (dict(f=None), "E_INVALID"), (dict(s=None), "E_INVALID"), (dict(v=None), "E_INVALID"), (dict(vc=None), "E_INVALID"),
    (dict(kc=None), "E_INVALID"), (dict(kc=None, vc=None, v=None), "E_INVALID"), (dict(NO_K, ko=A), "E_INVALID"),
    (dict(NO_K, v=A, vc=A, kc=A), "E_INVALID"), (dict(num_heads=0), "E_INVALID"), (dict(block_size=0), "E_INVALID"),
    (dict(num_blocks=0), "E_INVALID"), (dict(q_out_row_stride=0), "E_INVALID"), (dict(q_out_head_stride=64), "E_INVALID"),
    (dict(ko=A, k_out_head_stride=0), "E_INVALID"), (dict(kv_slot_stride=64), "E_INVALID"), (dict(k_row_stride=-8), "E_INVALID"),
    (dict(q=A + 8), "E_ALIGN"), (dict(v=A + 2), "E_ALIGN"), (dict(ko=A + 4), "E_ALIGN"), (dict(k_head_stride=132), "E_ALIGN"),
    (dict(kv_block_stride=16 * 512 + 4), "E_ALIGN"),
])
def test_norm_rope_check(kw, status):
    assert rope_check(**kw) == getattr(m, status), m.last_error()


def test_norm_rope_null_shape():
    assert m.lib.qsa_norm_rope_check(A, A, A, A, A, A, A, A, A, A, None) == m.E_INVALID


def verify_shape(**kw):
    base = dict(num_rows=36, num_reqs=9, vocab=131072, max_tokens=4, prob_stride=131072, draft_stride=131072)
    base.update(kw)
    return m.VerifyShape(**base)


def verify_check(p=A, d=A, t=A, s=A, u=A, us=A, o=A, c=A, ws=None, nbytes=0, **kw):
    return m.lib.qsa_verify_drafts_check(p, d, t, s, u, us, o, c, verify_shape(**kw), ws, nbytes)


@pytest.mark.parametrize("kw,status", [
    ({}, "OK"), (dict(d=None, draft_stride=0), "OK"), (dict(num_rows=0, p=None, t=None, u=None), "OK"),
    (dict(num_reqs=0, s=None, us=None, o=None, c=None), "OK"), (dict(vocab=1), "OK"), (dict(vocab=1 << 20, prob_stride=1 << 20,
                                                                                           draft_stride=1 << 20), "OK"),
    (dict(p=A + 4, d=A + 8), "OK"), (dict(num_rows=1, prob_stride=0, draft_stride=0), "OK"), (dict(max_tokens=1), "OK"),
    (dict(num_rows=-1), "E_INVALID"), (dict(num_reqs=-1), "E_INVALID"), (dict(vocab=0), "E_INVALID"),
    (dict(max_tokens=0), "E_INVALID"), (dict(prob_stride=131071), "E_INVALID"), (dict(draft_stride=131071), "E_INVALID"),
    (dict(p=None), "E_INVALID"), (dict(t=None), "E_INVALID"), (dict(s=None), "E_INVALID"), (dict(u=None), "E_INVALID"),
    (dict(us=None), "E_INVALID"), (dict(o=None), "E_INVALID"), (dict(c=None), "E_INVALID"), (dict(p=A + 2), "E_ALIGN"),
    (dict(vocab=(1 << 20) + 1, prob_stride=1 << 21, draft_stride=1 << 21), "E_UNSUPPORTED"),
    (dict(num_rows=(1 << 24) + 1), "E_RANGE"), (dict(num_reqs=1 << 22), "OK"), (dict(num_reqs=(1 << 22) + 1), "E_RANGE"),
    (dict(num_reqs=1 << 22, max_tokens=257), "E_RANGE"), (dict(prob_stride=(1 << 36) + 1), "E_RANGE"),
])
def test_verify_check(kw, status):
    assert verify_check(**kw) == getattr(m, status), m.last_error()


def test_verify_workspace():
    need = m.verify_drafts_workspace_bytes(verify_shape())
    assert verify_check(ws=A, nbytes=need) == m.OK
    if need:
        assert verify_check(ws=A, nbytes=need - 1) == m.E_INVALID
        assert verify_check(ws=A + 8, nbytes=need) == m.E_ALIGN
    for kw in (dict(vocab=0), dict(num_reqs=-1), dict(num_reqs=0), dict(max_tokens=0), dict(vocab=2 ** 31 - 1)):
        assert m.verify_drafts_workspace_bytes(verify_shape(**kw)) == 0
    assert m.lib.qsa_verify_drafts_workspace_bytes(None) == 0


def attn_shape(**kw):
    base = dict(num_rows=36, num_heads=32, num_kv_heads=4, head_dim=128, block_size=16, num_reqs=9, max_blocks=1000,
                dtype=m.BF16, scale=0.1, num_blocks=9000, q_row_stride=4096, q_head_stride=128, out_row_stride=4096,
                out_head_stride=128, kv_block_stride=16 * 512, kv_slot_stride=512, kv_head_stride=128)
    base.update(kw)
    return m.AttnShape(**base)


@pytest.mark.parametrize("window,sinks,kw,status", [
    (4096, 4, {}, "OK"), (1, 0, {}, "OK"), (2 ** 31 - 1, 2 ** 31 - 1, {}, "OK"), (100, 4, dict(num_rows=0), "OK"),
    (0, 4, {}, "E_INVALID"), (-5, 4, {}, "E_INVALID"), (100, -1, {}, "E_INVALID"), (100, 4, dict(num_heads=30), "E_INVALID"),
    (100, 4, dict(scale=0.0), "E_INVALID"), (100, 4, dict(head_dim=96), "E_UNSUPPORTED"),
    (100, 4, dict(dtype=m.FP8_E4M3FN), "E_DTYPE"), (100, 4, dict(max_blocks=1 << 27), "E_RANGE"),
    (100, 4, dict(q_head_stride=132), "E_ALIGN"),
])
def test_window_check(window, sinks, kw, status):
    s = attn_shape(**kw)
    assert m.lib.qsa_window_attention_check(A, A, A, A, A, A, window, sinks, A, s, None, 0) == getattr(m, status)


def test_window_pointers_and_workspace():
    s = attn_shape()
    check = m.lib.qsa_window_attention_check
    for i in range(7):
        ptrs = [A] * 7
        ptrs[i] = None
        assert check(*ptrs[:6], 100, 4, ptrs[6], s, None, 0) == m.E_INVALID
    assert check(A, A, A, A, A, A, 100, 4, A, None, None, 0) == m.E_INVALID
    need = m.window_attention_workspace_bytes(s, 4096, 4)
    assert need > 0
    assert check(A, A, A, A, A, A, 4096, 4, A, s, A, need) == m.OK
    assert check(A, A, A, A, A, A, 4096, 4, A, s, A, need - 1) == m.E_INVALID
    assert check(A, A, A, A, A, A, 4096, 4, A, s, A + 4, need) == m.E_ALIGN
    assert m.window_attention_workspace_bytes(s, 100, 4) == 0       # a short window is not cut
    assert m.window_attention_workspace_bytes(s, 0, 4) == m.window_attention_workspace_bytes(s, 100, -1) == 0
    assert m.window_attention_workspace_bytes(attn_shape(num_rows=0), 4096, 4) == 0
    # of more tiles than CUs those left over from whole rounds, where that pays
    for rows, window, cut in ((64, 4096, False), (65, 4096, True), (65, 1024, False), (96, 4096, True), (97, 4096, False),
                              (129, 4096, True), (193, 4096, False)):
        rest = attn_shape(num_rows=rows, num_reqs=rows)
        assert (m.window_attention_workspace_bytes(rest, window, 4) > 0) == cut
    # what the parts of the tiles take is bounded, whatever the batch
    for rows, reqs, kv in ((1, 1, 1), (40, 40, 8), (500, 500, 1), (3000, 2, 4), (300, 200, 8), (20, 1000, 32)):
        for window in (1, 300, 4096, 100000, 2 ** 31 - 1):
            big = attn_shape(num_rows=rows, num_reqs=reqs, num_heads=8 * kv, num_kv_heads=kv, max_blocks=1 << 16)
            assert 0 <= m.window_attention_workspace_bytes(big, window, 4) <= 70 << 20
            assert check(A, A, A, A, A, A, window, 4, A, big, None, 0) == m.OK


def test_host_tensors_are_refused():
    q = torch.zeros(4, 8, 64, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    p = torch.zeros(4, 10)
    kc = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    for call in (lambda: m.window_attention(q, kc, kc, i.view(1, 4), i, i[:2], window=4),
                 lambda: m.norm_rope(q, q, i, torch.zeros(8, dtype=torch.float64)),
                 lambda: m.verify_drafts(p, i, i[:3], p[:, 0].contiguous(), p[0, :2], max_tokens=2)):
        with pytest.raises(m.QsaError) as e:
            call()
        assert e.value.status == m.E_INVALID


def test_rope_frequencies():
    f, s = m.rope_frequencies(64, 500.0)
    assert f.dtype == torch.float64 and s == 1.0
    want = 500.0 ** (-np.arange(0, 64, 2) / 64)
    assert np.allclose(f.numpy(), want, rtol=1e-14)
    f2, s = m.rope_frequencies(64, 500.0, scaling="linear", factor=4.0)
    assert np.allclose(f2.numpy(), want / 4, rtol=1e-14) and s == 1.0
    # ntk: the fastest pair as it was, the slowest stretched by the factor
    f2, s = m.rope_frequencies(64, 500.0, scaling="ntk", factor=4.0)
    assert f2[0] == 1.0 and np.isclose(f2[-1], want[-1] / 4, rtol=1e-12) and s == 1.0
    # yarn: by the turns that a pair makes in the original length
    n = 4096
    f2, s = m.rope_frequencies(64, 10000.0, scaling="yarn", factor=8.0, original_len=n)
    want = 10000.0 ** (-np.arange(0, 64, 2) / 64)
    turns = n * want / (2 * math.pi)
    share = (f2.numpy() / want - 1 / 8) / (1 - 1 / 8)
    assert np.allclose(share[turns > 32 * 1.4], 1.0) and np.allclose(share[turns < 1 / 1.4], 0.0, atol=1e-12)
    assert np.all(np.diff(share) <= 1e-12) and 0.05 < share[(turns < 16) & (turns > 2)].mean() < 0.95
    assert np.isclose(s, 0.1 * math.log(8.0) + 1.0)
    f0, _ = m.rope_frequencies(0)
    assert f0.numel() == 0
    for kw in (dict(scaling="other"), dict(scaling="yarn"), dict(factor=0.5), dict(base=1.0),
               dict(scaling="yarn", original_len=0), dict(scaling="yarn", original_len=64, beta_fast=1.0)):
        with pytest.raises(m.QsaError):
            m.rope_frequencies(64, **kw)
    with pytest.raises(m.QsaError):
        m.rope_frequencies(63)
