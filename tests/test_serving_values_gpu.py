"""Paged and selected attention on the GPU at values where a softmax can go wrong:
scores far apart, very large scores, infinities among a row's own values."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
m = pytest.importorskip("paged_mqa_logits_block_amd")

import serving_ref as ref  # noqa: E402
from test_serving_gpu import Batch, DT, dev, run_paged  # noqa: E402

pytestmark = pytest.mark.gpu


def device_cache(k, v, dtype, block=64):
    """Caches of one request with keys and values [n, hk, d] in scattered blocks, and
    its table; places behind the last token are NaN."""
    n, hk, d = k.shape
    blocks = -(-n // block)
    ids = np.random.default_rng(n).permutation(blocks + 2)[:blocks]
    kv = torch.full((2, blocks + 2, block, hk, d), float("nan"), dtype=DT[dtype])
    pos = np.arange(n)
    for c, x in zip(kv, (k, v)):
        c[torch.from_numpy(ids[pos // block]), torch.from_numpy(pos % block)] = x.to(DT[dtype])
    kv = kv.cuda()
    return kv[0], kv[1], dev(ids[None].astype(np.int32))


def attend_all(kernel, q, kc, vc, table, counts, scale=None):
    """(out, lse) of rows q [R, H, d] over the first counts[r] tokens by one of the
    ways through the kernels."""
    R = q.shape[0]
    lse = torch.empty(q.shape[:2], device="cuda")
    counts = np.asarray(counts, np.int32)
    if kernel.startswith("sparse"):
        width = table.shape[1] * kc.shape[1]  # padded to the whole table, not packed
        idx = np.where(np.arange(width)[None, :] < counts[:, None], np.arange(width), -1).astype(np.int32)
        out = m.sparse_attention(q, kc, vc, table, dev(np.zeros(R, np.int32)), dev(idx), lse=lse, scale=scale,
                                 workspace="auto" if kernel.endswith("cut") else None)
    else:
        out = m.paged_attention(q, kc, vc, table, dev(counts), dev(np.array([0, R], np.int32)), lse=lse, scale=scale,
                                workspace="auto" if kernel.endswith("cut") else None)
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


# kernel: rows, heads per kv head that take it (few rows stream, many take the tile kernel)
KERNELS = {"stream": (1, 8), "stream_cut": (1, 8), "tile": (65, 8), "tile_cut": (65, 8), "sparse": (2, 8),
           "sparse_cut": (2, 8), "sparse_wide": (2, 24), "sparse_wide_cut": (2, 24)}


# ---------------------------------------------------------------------------
# scores far apart
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("gap", [10.0, 14.0, 16.0, 17.5, 19.0, 24.0])
def test_one_dominant_key(kernel, dtype, gap):
    """One early key `gap` above n others of one score, its value 0: what the others
    hold together is the output, though each one's weight is small."""
    rows, group = KERNELS[kernel]
    n, d = 40_000, 64
    g = torch.Generator().manual_seed(int(gap))
    k, v = torch.zeros(n, 1, d), torch.randn(n, 1, d, generator=g) + 1.0
    k[0, 0, 0], v[0] = gap, 0.0
    q = torch.zeros(rows, group, d)
    q[..., 0] = d ** 0.5
    q = q.to(DT[dtype])
    kc, vc, table = device_cache(k, v, dtype)
    out, lse = attend_all(kernel, q.cuda(), kc, vc, table, [n] * rows)
    kk, vv = (x.to(DT[dtype]).double().numpy()[:, 0] for x in (k, v))
    # sums: a product's 16 keys, then one addition per 16 keys of the longest range
    o, l, spread, size = ref.attend(q[0].double().numpy(), kk, vv, d ** -0.5)
    to, tl = ref.bounds(o, l, spread, size, n // 16 + 64, d, torch.finfo(DT[dtype]).eps / 2)
    if dtype == "fp16":
        to = to + ref.fp16_tail(vv)
    for r in range(rows):
        assert np.all(np.abs(out[r] - o) <= to), (r, float((np.abs(out[r] - o) / to).max()))
        assert np.all(np.abs(lse[r] - l) <= tl), r


# ---------------------------------------------------------------------------
# large scores
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("dtype,size", [("fp16", 2.0 ** 12), ("fp16", 1.375 * 2.0 ** 14), ("fp16", 1.75 * 2.0 ** 14),
                                        ("bf16", 1.25 * 2.0 ** 14), ("bf16", 1.375 * 2.0 ** 50)])
@pytest.mark.parametrize("sign", [1, -1])
def test_large_scores(kernel, dtype, size, sign):
    """Scores of +-size^2 d / 8, and 0 for the keys of the other sign: the softmax is
    the mean of the values of the keys with the largest score, the log-sum-exp that
    score and the log of their number.  Rows see 1, 2 or all keys."""
    rows, group = KERNELS[kernel]
    n, d = 700, 64
    g = torch.Generator().manual_seed(3)
    v = torch.randn(n, 1, d, generator=g).to(DT[dtype])
    k = torch.zeros(n, 1, d)
    top = [0, 1, 600] if sign > 0 else list(range(n))  # keys of the largest score
    k[top] = sign * size
    q = torch.full((rows, group, d), size).to(DT[dtype])
    kc, vc, table = device_cache(k, v, dtype)
    score = sign * size * size * d ** 0.5  # exact in 32 bits
    u = torch.finfo(DT[dtype]).eps / 2
    for count in (1, 2, n):
        out, lse = attend_all(kernel, q.cuda(), kc, vc, table, [count] * rows)
        mine = [t for t in top if t < count]
        want = v[mine, 0].double().numpy().mean(axis=0)
        # equal weights, a sum of len(mine) products, a division, two roundings to the type
        tol = (2 * u + (len(mine) + 8) * 2.0 ** -24) * np.abs(v[mine, 0].double().numpy()).mean(axis=0)
        assert np.all(np.abs(out - want) <= tol), count
        assert np.all(np.abs(lse - (score + np.log(len(mine)))) <= 2.0 ** -21 * abs(score) + 1e-6), count


# ---------------------------------------------------------------------------
# infinities that a row sees itself
# ---------------------------------------------------------------------------

def check_values(out, lse, q, k, v, counts, dtype):
    """Against the 64-bit result where that is finite; infinities and NaN are equal."""
    k, v = (x.to(DT[dtype]).double().numpy() for x in (k, v))
    for r, c in enumerate(counts):
        if c == 0:
            assert np.all(out[r] == 0) and np.all(lse[r] == -np.inf), r
            continue
        o, l, spread, size = ref.attend(q[r].double().numpy(), k[:c, 0], v[:c, 0], q.shape[2] ** -0.5)
        finite = np.isfinite(o)
        to, tl = ref.bounds(np.where(finite, o, 0), l, np.where(finite, spread, 0), size, c, q.shape[2],
                            torch.finfo(DT[dtype]).eps / 2)
        assert np.array_equal(out[r][~finite], o[~finite], equal_nan=True), r
        assert np.all(np.abs(out[r][finite] - o[finite]) <= to[finite]), r
        assert np.all(np.abs(lse[r] - l) <= tl), r


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("count", [1, 31, 33, 100, 128, 2000])
def test_own_infinities(kernel, count):
    """Infinite values at the first and the last token, and at the last multiple of 32,
    of rows that all see the same tokens, whatever the count is a multiple of; and of
    both signs in one element."""
    rows, group = KERNELS[kernel]
    d = 64
    g = torch.Generator().manual_seed(count)
    k, v = torch.randn(count, 1, d, generator=g), torch.randn(count, 1, d, generator=g)
    v[0, 0, 3], v[-1, 0, 5], v[-1, 0, 40] = float("inf"), float("inf"), -float("inf")
    v[0, 0, 60], v[-1, 0, 60], v[(count - 1) // 32 * 32, 0, 20] = float("inf"), -float("inf"), float("inf")
    q = torch.randn(rows, group, d, generator=g).to(torch.bfloat16)
    kc, vc, table = device_cache(k, v, "bf16")
    with np.errstate(invalid="ignore"):
        check_values(*attend_all(kernel, q.cuda(), kc, vc, table, [count] * rows), q, k, v, [count] * rows, "bf16")


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_infinity_of_a_small_weight(kernel, dtype):
    """An infinite value whose weight (e^-31) the type holds or not is infinite in the
    output."""
    rows, group = KERNELS[kernel]
    n, d = 300, 64
    g = torch.Generator().manual_seed(7)
    k, v = torch.zeros(n, 1, d), torch.randn(n, 1, d, generator=g)
    k[5, 0, 0], v[250, 0, 9] = 31.0, float("inf")
    q = torch.zeros(rows, group, d)
    q[..., 0] = d ** 0.5
    q = q.to(DT[dtype])
    kc, vc, table = device_cache(k, v, dtype)
    out, lse = attend_all(kernel, q.cuda(), kc, vc, table, [n] * rows)
    assert np.all(out[:, :, 9] == np.inf)
    check_values(out, lse, q, k, v, [n] * rows, dtype)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("dtype,seed", [("bf16", 1), ("fp16", 2), ("bf16", 3)])
def test_values_not_finite_anywhere(kernel, dtype, seed):
    """NaN and infinities of both signs at a tenth of the tokens, one element each, and
    rows of different counts: every element of every row is what its own tokens make
    it."""
    rows, group = KERNELS[kernel]
    rows = max(rows, 3)
    n, d = 900, 64
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    k, v = torch.randn(n, 1, d, generator=g), torch.randn(n, 1, d, generator=g)
    at = rng.choice(n, n // 10, replace=False)
    v[at, 0, rng.integers(0, d, len(at))] = torch.from_numpy(rng.choice([np.nan, np.inf, -np.inf], len(at))).float()
    q = torch.randn(rows, group, d, generator=g).to(DT[dtype])
    counts = rng.integers(0, n + 1, rows)
    counts[:3] = n, 1, 40
    kc, vc, table = device_cache(k, v, dtype)
    with np.errstate(invalid="ignore"):
        check_values(*attend_all(kernel, q.cuda(), kc, vc, table, counts), q, k, v, counts, dtype)


# ---------------------------------------------------------------------------
# entries outside the pool, values of others, in launches whose tiles are not cut too
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("workspace", ["auto", None])
@pytest.mark.parametrize("past,new", [([206], [3]), ([206, 333], [4, 2]), ([206], [80]), ([206, 333], [70, 60])])
def test_bad_entries_cut_and_whole(past, new, workspace):
    b = Batch(12, past, new, group=4)
    b.table = b.table.clone()
    first = (past[0] + 2) // b.block  # the entry of the request's third new row on
    b.table[0, first] = b.kc.shape[0]
    out, lse = run_paged(b, workspace=workspace)
    clean = [r for r in range(b.rows) if b.req[r] == 1 or b.ctx[r] <= first * b.block]
    assert 0 < len(clean) < b.rows
    b.check(out, lse, lambda r: range(b.ctx[r]), rows=clean)
    for r in set(range(b.rows)) - set(clean):
        assert torch.all(torch.isnan(out[r])) and torch.all(torch.isnan(lse[r])), r


@pytest.mark.parametrize("workspace", ["auto", None])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("past,new", [([200], [4]), ([200, 333], [4, 2]), ([200], [80]), ([200, 333], [70, 60])])
def test_values_others_see_cut_and_whole(past, new, value, workspace):
    b = Batch(11, past, new, group=4)
    bad = past[0] + new[0] // 2  # seen by the later rows of request 0 only
    b.vc[int(b.table[0, bad // b.block]), bad % b.block] = value
    out, lse = run_paged(b, workspace=workspace)
    clean = [r for r in range(b.rows) if b.req[r] == 1 or b.ctx[r] <= bad]
    b.check(out, lse, lambda r: range(b.ctx[r]), rows=clean)
    for r in set(range(b.rows)) - set(clean):
        assert torch.all(torch.isnan(out[r]) if np.isnan(value) else out[r] == value), r


# ---------------------------------------------------------------------------
# the two attentions, and keys that are not finite
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,group", [("bf16", 8), ("fp16", 20)])
def test_selection_of_everything(dtype, group):
    """With every token selected both attentions give the 64-bit result, and so are
    within both bounds of each other."""
    b = Batch(90, [250, 90], [4, 4], group=group, dtype=dtype)
    idx = np.where(np.arange(256)[None, :] < b.ctx[:, None], np.arange(256), -1).astype(np.int32)
    lse = torch.empty(b.q.shape[:2], device="cuda")
    out = m.sparse_attention(b.q.cuda(), b.kc, b.vc, b.table, dev(b.req.astype(np.int32)), dev(idx), lse=lse)
    b.check(out, lse, lambda r: range(b.ctx[r]))
    b.check(*run_paged(b), lambda r: range(b.ctx[r]))


@pytest.mark.parametrize("layout", [m.KV_PAGED, m.KV_COPACKED, m.KV_COPACKED_SHUFFLED])
def test_keys_not_finite_stay_so(layout):
    """A key with an infinity or a NaN is stored as one that is not finite: the element
    itself, and with an infinity (whose scale is infinite) all of them."""
    x = torch.ones(5, 64, dtype=torch.bfloat16)
    x[1, 3], x[2, 7], x[4, 63] = float("inf"), float("nan"), -float("inf")
    kc = torch.zeros(1, 16 * (64 if layout == m.KV_PAGED else 68), dtype=torch.uint8, device="cuda")
    ks = torch.zeros(1, 16, device="cuda") if layout == m.KV_PAGED else None
    m.write_keys(x.cuda(), torch.arange(5).cuda(), kc, block_size=16, kscale=ks, layout=layout)
    codes = kc.cpu()[0, :16 * 64].view(torch.float8_e4m3fn).float()
    codes = codes.view(4, 16, 16).transpose(0, 1).reshape(16, 64) if layout == m.KV_COPACKED_SHUFFLED else codes.view(16, 64)
    scale = ks.cpu()[0] if ks is not None else kc.cpu()[0, 16 * 64:].view(torch.float32)
    back = codes * scale[:, None]
    assert torch.all(~torch.isfinite(back[1])) and torch.all(~torch.isfinite(back[4]))
    assert torch.isnan(back[2, 7]) and torch.all(torch.isfinite(back[2, :7])) and torch.all(torch.isfinite(back[2, 8:]))
    for r in (0, 3):
        assert torch.all(back[r] == 448.0 * (torch.tensor(1.0) / 448.0)), r
