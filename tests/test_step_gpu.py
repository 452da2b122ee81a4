"""Head norms with rotary positions and draft verification on the GPU, against the
plain 64-bit implementations in step_ref.py."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
m = pytest.importorskip("paged_mqa_logits_block_amd")

import step_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
TINY = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25}  # half a step of the subnormals


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


# ---------------------------------------------------------------------------
# head norms and rotary positions
# ---------------------------------------------------------------------------

def rope_close(got, want, err, dtype, what):
    half = torch.finfo(DT[dtype]).eps / 2
    d = np.abs(got.double().cpu().numpy() - want)
    tol = ref.rope_bounds(want, err, half, TINY[dtype])
    assert np.all(d <= tol), (what, float((d / tol).max()))


ROPE = [
    # dtype, D, rot, offset, interleaved, norms, rows, Hq, Hk, block, order, outputs
    ("bf16", 128, 128, 0, False, "qk", 1, 32, 4, 16, "slot", "cache"),
    ("bf16", 128, 64, 64, True, "qk", 40, 32, 4, 16, "slot", "cache"),
    ("fp16", 64, 32, 0, False, "", 37, 14, 2, 100, "head", "tensors"),
    ("fp16", 128, 48, 24, False, "q", 5, 3, 1, 1, "head", "both"),
    ("bf16", 64, 64, 0, True, "k", 129, 7, 7, 48, "slot", "both"),
    ("fp16", 64, 16, 48, True, "qk", 600, 1, 1, 64, "head", "keys"),
    ("bf16", 64, 0, 0, False, "qk", 9, 5, 2, 16, "slot", "cache"),      # norms alone
    ("bf16", 128, 16, 40, False, "", 2, 40, 8, 16, "slot", "tensors"),
    ("fp16", 128, 112, 8, True, "qk", 3, 2, 2, 3, "slot", "queries"),
    ("bf16", 128, 128, 0, False, "qk", 2500, 8, 2, 64, "head", "cache"),
    ("fp16", 64, 48, 16, False, "qk", 2049, 4, 1, 16, "slot", "both"),
    ("bf16", 128, 96, 16, True, "k", 8193, 1, 1, 16, "slot", "both"),
    # more than 1,024 lanes of a row's heads; more bytes than the L2s hold
    ("bf16", 128, 128, 0, False, "qk", 3, 130, 10, 16, "slot", "both"),
    ("fp16", 64, 32, 8, True, "qk", 2, 256, 3, 16, "slot", "cache"),
    ("bf16", 128, 64, 0, False, "qk", 9000, 6, 2, 64, "head", "both"),
    ("fp16", 64, 64, 0, True, "q", 20000, 5, 1, 16, "slot", "cache"),
]


@pytest.mark.parametrize("case", ROPE, ids=["-".join(str(x) for x in c) for c in ROPE])
def test_norm_rope(case):
    dtype, D, rot, off, inter, norms, rows, Hq, Hk, block, order, outputs = case
    rng = np.random.default_rng(rows * 100 + D + rot)
    g = torch.Generator().manual_seed(rows + rot)
    # one projection's rows, each part a view
    qkv = (torch.randn(rows, Hq + 2 * Hk, D, generator=g) * torch.exp(torch.randn(rows, 1, 1, generator=g))).to(DT[dtype])
    gpu = qkv.cuda()
    q, k, v = gpu[:, :Hq], gpu[:, Hq:Hq + Hk], gpu[:, Hq + Hk:]
    pos = rng.integers(0, 200000, rows).astype(np.int32)
    pos[0] = 0
    if rows > 4:
        pos[1], pos[2], pos[3] = 2 ** 30 - 1, -1, -(2 ** 31) + 5   # far ones, and rows without a position
    freq, factor = m.rope_frequencies(rot, 10000.0)
    if rows % 2:
        factor = 1.375
    wq, wk = (1.0 + 0.3 * torch.randn(D, generator=g) for _ in range(2))
    use_q, use_k = outputs != "keys", outputs != "queries"
    kw = dict(rot_offset=off, layout=m.ROPE_INTERLEAVED if inter else m.ROPE_HALF, rope_scale=factor, eps=1e-5,
              position_offset=5)
    shifted = dev(pos - np.int32(5))
    if "q" in norms and use_q:
        kw["q_weight"] = wq.cuda()
    if "k" in norms and use_k:
        kw["k_weight"] = wk.cuda()
    live = pos >= 0
    fill = 3.0
    if use_q:
        kw["q_out"] = torch.full((rows, Hq, D), fill, dtype=DT[dtype], device="cuda")
    if use_k and outputs != "cache":
        kw["k_out"] = torch.full((rows, Hk, D), fill, dtype=DT[dtype], device="cuda")
    if outputs in ("cache", "both"):
        pool = -(-rows // block) + 4
        shape = (pool, block, Hk, D) if order == "slot" else (pool, Hk, block, D)
        kc, vc = (torch.full(shape, fill, dtype=DT[dtype], device="cuda") for _ in range(2))
        if order == "head":
            kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
        slots = torch.randperm(pool * block, generator=g)[:rows]
        if rows > 8:
            slots[6], slots[7] = -1, pool * block
        kw.update(slots=slots.cuda(), kcache=kc, vcache=vc, v=v)
    qo, ko = m.norm_rope(q if use_q else None, k if use_k else None, shifted, freq.cuda(), **kw)
    assert (qo is None) == (not use_q) and (ko is None) == (not use_k or outputs == "cache")

    def want(x, w):
        return ref.norm_rope(x.double().numpy(), None if w is None else w.double().numpy(), float(np.float32(1e-5)),
                             np.where(live, pos, 0), freq.numpy(), float(np.float32(factor)), off, inter)

    if use_q:
        y, err = want(qkv[:, :Hq], wq if "q" in norms else None)
        rope_close(qo[dev(live)], y[live], err[live], dtype, "q")
        assert torch.all(qo[dev(~live)] == fill)
    if use_k:
        y, err = want(qkv[:, Hq:Hq + Hk], wk if "k" in norms else None)
        if ko is not None:
            rope_close(ko[dev(live)], y[live], err[live], dtype, "k")
            assert torch.all(ko[dev(~live)] == fill)
        if outputs in ("cache", "both"):
            at = slots.numpy()
            ok = live & (at >= 0) & (at < pool * block)
            flat_k, flat_v = (c.contiguous().view(pool * block, Hk, D) for c in (kc, vc))
            rope_close(flat_k[dev(at[ok])], y[ok], err[ok], dtype, "cached k")
            assert torch.equal(flat_v[dev(at[ok])].cpu(), qkv[:, Hq + Hk:][torch.from_numpy(ok)])
            others = np.setdiff1d(np.arange(pool * block), at[ok])
            assert torch.all(flat_k[dev(others)] == fill) and torch.all(flat_v[dev(others)] == fill)


@pytest.mark.parametrize("inter", [False, True])
def test_norm_rope_in_place_and_values(inter):
    """In place; heads of zeros; an infinity or a NaN spoils its own head only, in v
    nothing; a row whose queries are one broadcast head."""
    g = torch.Generator().manual_seed(3)
    x = torch.randn(21, 6, 128, generator=g).to(torch.bfloat16)
    x[4] = 0
    bad = x.clone()
    bad[5, 2, 17], bad[6, 0, 127], bad[7, 5, 64] = float("inf"), float("nan"), float("-inf")
    pos = torch.arange(21, dtype=torch.int32).cuda() * 977
    freq, _ = m.rope_frequencies(64)
    kw = dict(rot_offset=32, layout=int(inter), q_weight=torch.ones(128).cuda(), k_weight=torch.ones(128).cuda())
    clean, clean_k = m.norm_rope(x.cuda(), x.cuda(), pos, freq.cuda(), **kw)
    assert torch.all(clean[4] == 0)
    y = bad.cuda()
    qo, ko = m.norm_rope(y, y.clone(), pos, freq.cuda(), q_out=y, **kw)
    assert qo is y and torch.equal(clean, clean_k)
    spoilt = torch.zeros(21, 6, dtype=torch.bool)
    spoilt[5, 2] = spoilt[6, 0] = spoilt[7, 5] = True
    for out in (qo, ko):
        assert torch.equal(out.cpu()[~spoilt], clean.cpu()[~spoilt])
        assert torch.all(torch.isnan(out.cpu()[spoilt]).any(dim=1))
    # values are stored as they are, whatever they are
    kc, vc = (torch.zeros(3, 8, 6, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    m.norm_rope(None, x.cuda(), pos, freq.cuda(), v=bad.cuda(), slots=torch.arange(21).cuda(), kcache=kc, vcache=vc)
    assert torch.equal(vc.view(24, 6, 128)[:21].cpu().view(torch.int16), bad.view(torch.int16))
    one = x[:1, :1].cuda().expand(21, 6, 128)
    qo, _ = m.norm_rope(one, None, pos, freq.cuda(), rot_offset=32, layout=int(inter))
    qe, _ = m.norm_rope(one.contiguous(), None, pos, freq.cuda(), rot_offset=32, layout=int(inter))
    assert torch.equal(qo, qe)


def test_norm_rope_far_slots():
    """Cache offsets past 2^31 bytes."""
    D, block = 128, 64
    pool = (2 ** 31 // (block * 2 * D)) + 70
    kc, vc = (torch.zeros(pool, block, 1, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k = torch.randn(4, 1, D, device="cuda").to(torch.bfloat16)
    slots = torch.tensor([0, pool * block - 1, pool * block - 65, 2 ** 31 // (2 * D)], device="cuda")
    freq, _ = m.rope_frequencies(D, device="cuda")
    _, ko = m.norm_rope(None, k, torch.arange(4, dtype=torch.int32, device="cuda"), freq,
                        k_out=torch.empty_like(k), v=k, slots=slots, kcache=kc, vcache=vc)
    assert torch.equal(kc.view(-1, 1, D)[slots], ko) and torch.equal(vc.view(-1, 1, D)[slots], k)
    assert int((kc != 0).any(dim=3).sum()) == 4 and int((vc != 0).any(dim=3).sum()) == 4


def test_norm_rope_refusals():
    q = torch.zeros(4, 8, 64, dtype=torch.bfloat16, device="cuda")
    i = torch.zeros(4, dtype=torch.int32, device="cuda")
    f, _ = m.rope_frequencies(32, device="cuda")
    kc = torch.zeros(2, 16, 8, 64, dtype=torch.bfloat16, device="cuda")
    s = torch.zeros(4, dtype=torch.int64, device="cuda")
    good = dict(slots=s, kcache=kc, vcache=kc.clone(), v=q)
    for kw, status in ((dict(q_weight=torch.ones(64, dtype=torch.bfloat16, device="cuda")), m.E_INVALID),
                       (dict(q_out=q.to(torch.float16)), m.E_INVALID), (dict(k_out=q[:, :4]), m.E_INVALID),
                       (dict(good, slots=s.int()), m.E_INVALID), (dict(good, slots=None), m.E_INVALID),
                       (dict(good, v=None), m.E_INVALID), (dict(good, vcache=None), m.E_INVALID),
                       (dict(good, vcache=kc[:, :8]), m.E_INVALID), (dict(good, kcache=kc[:, :, :4]), m.E_INVALID),
                       (dict(slots=s), m.E_INVALID), (dict(rot_offset=12), m.E_UNSUPPORTED),
                       (dict(rot_offset=40), m.E_INVALID), (dict(layout=2), m.E_INVALID), (dict(eps=-1.0), m.E_INVALID)):
        with pytest.raises(m.QsaError) as e:
            m.norm_rope(q, q, i, f, **kw)
        assert e.value.status == status, kw
    for args in ((None, None, i, f), (q, q, i[:3], f), (q, q, i, f.float()), (q.float(), q.float(), i, f),
                 (q, q.to(torch.float16), i, f), (q, q[:3], i, f)):
        with pytest.raises(m.QsaError):
            m.norm_rope(*args)
    for kw in (dict(rot_offset=2 ** 32), dict(layout=2 ** 32), dict(position_offset=2 ** 32), dict(position_offset=2 ** 31)):
        with pytest.raises(m.QsaError) as e:  # not taken for 0 or a negative number
            m.norm_rope(q, q, i, f, **kw)
        assert e.value.status == m.E_INVALID, kw
    out, _ = m.norm_rope(q[:0], q[:0], i[:0], f)  # no rows
    assert out.shape == (0, 8, 64)


# ---------------------------------------------------------------------------
# verification of drafted tokens
# ---------------------------------------------------------------------------

def distributions(rng, R, V, peak=2.0):
    z = rng.normal(size=(R, V)) * peak
    p = np.exp(z - z.max(axis=1, keepdims=True))
    zq = z + rng.normal(size=(R, V)) * 0.7
    q = np.exp(zq - zq.max(axis=1, keepdims=True))
    return (p / p.sum(axis=1, keepdims=True)).astype(np.float32), (q / q.sum(axis=1, keepdims=True)).astype(np.float32)


def run_verify(p, q, tokens, starts, u, us, most, **kw):
    out, count = m.verify_drafts(dev(p), dev(tokens.astype(np.int32)), dev(np.asarray(starts, np.int32)),
                                 dev(u.astype(np.float32)), dev(us.astype(np.float32)), max_tokens=most,
                                 draft_probs=None if q is None else dev(q), **kw)
    return out.cpu().numpy(), count.cpu().numpy()


@pytest.mark.parametrize("V", [1, 2, 3, 63, 2047, 2048, 2049, 5000, 50021, 131072])
@pytest.mark.parametrize("certain", [False, True])
def test_verify_drafts(V, certain):
    rng = np.random.default_rng(V)
    rows = [4, 1, 0, 7, 2, 5, 1, 3]
    starts = np.concatenate([[0], np.cumsum(rows)])
    R, n = int(starts[-1]) + 3, len(rows)   # rows behind the last request's
    p, q = distributions(rng, R, V)
    for trial in range(4):
        tokens = np.array([rng.choice(V, p=q[max(r - 1, 0)].astype(np.float64) / q[max(r - 1, 0)].astype(np.float64).sum())
                           for r in range(R)])
        u, us = rng.random(R).astype(np.float32) * (1.0, 0.3, 0.01, 1e-6)[trial], rng.random(n).astype(np.float32)
        us[0] = (0.0, np.float32(1 - 2.0 ** -24), 0.5, 1.0)[trial]
        want = ref.verify(p, None if certain else q, tokens, starts, u, us, 7)
        for ws in ("auto", None):
            got = run_verify(p, None if certain else q, tokens, starts, u, us, 7, workspace=ws)
            assert np.array_equal(got[1], want[1]) and np.array_equal(got[0], want[0]), (trial, ws)


def test_verify_ties_and_borders():
    """Weights whose sums are exact: a cumulative weight equal to u * total does not pass
    it, the next entry with weight does; a draft with u q equal to p is not kept."""
    V = 8192
    p = np.zeros((4, V), np.float32)
    p[:, [5, 2047, 2048, 8000]] = [0.25, 0.25, 0.125, 0.375]
    q = np.zeros((4, V), np.float32)
    q[:, 5], q[:, 7] = 0.5, 0.5
    for u0, first in ((0.5, 0), (np.float32(0.5) - np.float32(2.0 ** -25), 1)):
        for us, token_p, token_rest in ((0.0, 5, 2047), (0.25, 2047, 2047), (0.5, 2048, 8000), (0.625, 8000, 8000),
                                        (np.float32(1 - 2.0 ** -24), 8000, 8000), (1.0, 8000, 8000)):
            out, count = run_verify(p, q, np.array([0, 5, 0, 0]), [0, 2], np.array([u0, 0, 0, 0]), np.array([us]), 3)
            if first:
                assert count[0] == 2 and list(out[0]) == [5, token_p, -1], (u0, us)
            else:  # rest: 2047 0.25, 2048 0.125, 8000 0.375 of 0.75
                assert count[0] == 1 and out[0, 0] == token_rest and list(out[0, 1:]) == [-1, -1], (u0, us)


def test_verify_odd_inputs():
    """Drafts outside the vocabulary, rows without weight, a target that is nowhere above
    the drafter, entries that are not numbers, starts outside the rows, more rows than
    max_tokens, 100 drafts, strided rows."""
    rng = np.random.default_rng(0)
    V, R = 1500, 110
    p, q = distributions(rng, R, V)
    tokens = rng.integers(0, V, R)
    u, us = rng.random(R).astype(np.float32), rng.random(6).astype(np.float32)

    def check(p, q, tokens, starts, u, us, most, **kw):
        want = ref.verify(p, q, tokens, starts, u, us, most)
        got = run_verify(p, q, tokens, starts, u, us, most, **kw)
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1]), (got, want)
        return got

    for bad in (-1, V, 2 ** 31 - 1, -(2 ** 31)):
        t = tokens.copy()
        t[1] = bad
        for d in (q, None):
            assert check(p, d, t, [0, 3], np.zeros(R), us[:1], 3)[1][0] == 1
    zero = p.copy()
    zero[0] = 0
    out, count = check(zero, q, tokens, [0, 2], u, us[:1], 2)
    assert out[0, 0] == -1 and count[0] == 1
    # the drafter's own distribution, a draft rejected by rounding or an outer u
    out, count = check(p, p, tokens, [0, 2], np.ones(R), us[:1], 2)
    assert count[0] == 1 and out[0, 0] >= 0
    odd = p.copy()
    odd[0, 5], odd[0, 6], odd[0, 7], odd[0, 8] = np.nan, np.inf, -np.inf, -1.0
    for d in (q, None, odd[:, ::-1].copy()):
        for s in (0.0, 0.3, 0.999999):
            check(odd, d, tokens, [0, 1], u, np.array([s]), 2)
            check(odd, d, tokens, [0, 2], np.ones(R), np.array([s]), 2)
    check(p, q, tokens, [-5, 3, 200, 400], u, us[:3], 4)
    check(p, q, tokens, [0, 9, 9, 4, 12, 500, 600], u, us, 4)          # starts that decrease
    out, count = check(p, None, tokens, [0, 101], np.zeros(R), us[:1], 101)  # every draft kept
    assert count[0] == 101
    for at in (63, 64, 65, 99):
        t = tokens.copy()
        t[at + 1] = -1
        assert check(p, q, t, [0, 101], np.zeros(R), us[:1], 101)[1][0] == at + 1
    check(p, None, tokens, [0, 101], np.zeros(R), us[:1], 50)           # cut to the columns there are
    wide = rng.random((R, 2 * V + 3)).astype(np.float32)
    wide[:, 1:1 + V] = p
    pt, st = dev(wide)[:, 1:1 + V], [0, 4, 9]
    want = ref.verify(p, None, tokens, st, u, us[:2], 5)
    out, count = m.verify_drafts(pt, dev(tokens.astype(np.int32)), dev(np.array(st, np.int32)), dev(u), dev(us[:2]), max_tokens=5)
    assert np.array_equal(out.cpu().numpy(), want[0]) and np.array_equal(count.cpu().numpy(), want[1])


def test_verify_largest_vocabulary():
    """As many entries as are built, and tokens among the last ones; rows that start at
    any element."""
    V, R = 1 << 20, 3
    rng = np.random.default_rng(9)
    p, q = (rng.random((R, V)).astype(np.float32) for _ in range(2))
    wide = rng.random((R, V + 1)).astype(np.float32)
    wide[:, 1:] = p
    tokens, u = np.array([0, V - 1, V - 2]), np.array([0.0, 0.0, 0.0], np.float32)
    for kept in (2, 0):
        if kept == 0:
            u[:] = 1.0
            q[0, V - 1] = p[0, V - 1] + 0.5
        for us in (0.0, 0.37, np.float32(1 - 2.0 ** -24)):
            want = ref.verify(p, q, tokens, [0, R], u, [us], 3)
            assert want[1][0] == kept + 1
            for ws in ("auto", None):
                out, count = m.verify_drafts(dev(wide)[:, 1:], dev(tokens.astype(np.int32)), dev(np.array([0, R], np.int32)),
                                             dev(u), dev(np.array([us], np.float32)), max_tokens=3, draft_probs=dev(q),
                                             workspace=ws)
                assert np.array_equal(out.cpu().numpy(), want[0]) and np.array_equal(count.cpu().numpy(), want[1])


@pytest.mark.parametrize("n", [768, 769, 65535, 65536])
def test_verify_many_requests(n):
    """Batches on either side of the numbers of requests where the launch changes, of 0 to 3
    rows each."""
    rng = np.random.default_rng(n)
    starts = np.concatenate([[0], np.cumsum(rng.integers(0, 4, n))])
    R, V = int(starts[-1]), 9
    p, q = distributions(rng, R, V)
    tokens, u, us = rng.integers(0, V, R), rng.random(R).astype(np.float32), rng.random(n).astype(np.float32)
    want = ref.verify(p, q, tokens, starts, u, us, 3)
    got = run_verify(p, q, tokens, starts, u, us, 3)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


def test_verify_rows_far_apart():
    """Rows more than 2^31 elements behind the first one."""
    rng = np.random.default_rng(3)
    R, V, stride = 5, 5000, 600_000_001
    p, q = distributions(rng, R, V)
    far = torch.empty(2, (R - 1) * stride + V, device="cuda")
    pt, qt = (x.as_strided((R, V), (stride, 1)) for x in far)
    pt.copy_(dev(p))
    qt.copy_(dev(q))
    tokens, u, us = rng.integers(0, V, R), rng.random(R).astype(np.float32), rng.random(1).astype(np.float32)
    for u in (u, np.zeros(R, np.float32), np.array([0, 0, 0, 1e9, 0], np.float32)):
        want = ref.verify(p, q, tokens, [0, R], u, us, R)
        out, count = m.verify_drafts(pt, dev(tokens.astype(np.int32)), dev(np.array([0, R], np.int32)), dev(u), dev(us),
                                     max_tokens=R, draft_probs=qt)
        assert np.array_equal(out.cpu().numpy(), want[0]) and np.array_equal(count.cpu().numpy(), want[1])


def test_verify_distribution():
    """A kept draft or the token in its place is distributed as the target: 49,152 requests
    of one draft, each token's share within 5 standard deviations."""
    rng = np.random.default_rng(1)
    V, n = 5, 4096
    p = np.array([0.5, 0.2, 0.15, 0.1, 0.05], np.float32)
    q = np.array([0.1, 0.3, 0.2, 0.1, 0.3], np.float32)
    starts = np.arange(0, 2 * n + 1, 2)
    P, Q = (np.broadcast_to(x, (2 * n, V)).copy() for x in (p, q))
    first = np.zeros(V)
    for _ in range(12):
        tokens = rng.choice(V, size=2 * n, p=q.astype(np.float64) / q.astype(np.float64).sum())
        u, us = rng.random(2 * n).astype(np.float32), rng.random(n).astype(np.float32)
        out, _ = run_verify(P, Q, tokens, starts, u, us, 2)
        first += np.bincount(out[:, 0], minlength=V)
    total = 12 * n
    share, dev_ = first / total, np.sqrt(p * (1 - p) / total)
    assert np.all(np.abs(share - p) < 5 * dev_), (share, p)


def test_verify_refusals():
    p = torch.zeros(4, 10, device="cuda")
    i, u = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(4, device="cuda")
    for args, kw in (((p, i, i[:2], u, u[:1]), dict(max_tokens=0)), ((p.half(), i, i[:2], u, u[:1]), {}),
                     ((p, i.long(), i[:2], u, u[:1]), {}), ((p, i, i[:2], u[:3], u[:1]), {}),
                     ((p, i, i[:2], u, u[:2]), {}), ((p.t(), i, i[:2], u, u[:1]), {}),
                     ((p, i, i[:2], u, u[:1]), dict(draft_probs=p[:, :9])), ((p, i, i[:0], u, u[:0]), {}),
                     ((p, i, i[:2], u, u[:1]), dict(out_tokens=torch.zeros(1, 3, dtype=torch.int32, device="cuda"))),
                     ((p, i, i[:2], u, u[:1]), dict(workspace="none"))):
        with pytest.raises(m.QsaError):
            m.verify_drafts(*args, **{"max_tokens": 2, **kw})
    out, count = m.verify_drafts(p, i, i[:1], u, u[:0], max_tokens=2)  # no requests
    assert out.shape == (0, 2) and count.shape == (0,)
    out, count = m.verify_drafts(p[:0], i[:0], i[:3], u[:0], u[:2], max_tokens=2)  # no rows
    assert out.tolist() == [[-1, -1]] * 2 and count.tolist() == [0, 0]
