"""Attention over a sliding window and the first tokens on the GPU, against the plain
64-bit implementation in serving_ref.py.  Tokens that no row sees are NaN in the caches,
and blocks without a token that is seen have garbage in the table, as after a free."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
m = pytest.importorskip("paged_mqa_logits_block_amd")

from test_serving_gpu import Batch, dev  # noqa: E402
from test_serving_values_gpu import check_values, device_cache  # noqa: E402

pytestmark = pytest.mark.gpu


def seen(ctx, window, sinks):
    """The tokens that a row with ctx visible ones sees."""
    first = min(sinks, ctx)
    return list(range(first)) + list(range(max(ctx - window, first), ctx))


def free_unseen(b, window, sinks, keep=()):
    """Spoils what no row of a request sees: NaN in both caches, garbage for whole
    blocks' entries (but for the requests in `keep`)."""
    table = b.table.cpu().numpy()
    kc, vc = b.kc, b.vc
    for i in range(b.n):
        if i in keep:
            continue
        total = len(b.k[i])
        used = np.zeros(total, bool)
        for r in range(b.starts[i], b.starts[i + 1]):
            used[seen(min(max(int(b.ctx[r]), 0), total), window, sinks)] = True
        pos = np.nonzero(~used)[0]
        if len(pos):
            blk, at = torch.from_numpy(table[i, pos // b.block]).long().cuda(), torch.from_numpy(pos % b.block).cuda()
            kc[blk, at] = float("nan")
            vc[blk, at] = float("nan")
        for e in range(-(-total // b.block)):
            if not used[e * b.block:(e + 1) * b.block].any():
                table[i, e] = b.rng.choice([-1, 2 ** 31 - 1, -2 ** 31, kc.shape[0]])
    b.table = dev(table)


def run_window(b, window, sinks, workspace="auto", q=None, out=None, **kw):
    lse = torch.full((b.q.shape[0], b.q.shape[1]), 7.0, device="cuda")
    out = torch.full(tuple(b.q.shape), 3.0, dtype=b.q.dtype, device="cuda") if out is None else out
    got = m.window_attention(b.q.cuda() if q is None else q, b.kc, b.vc, b.table, dev(b.ctx), dev(b.starts),
                             window=window, sinks=sinks, out=out, lse=lse, workspace=workspace, **kw)
    assert got.data_ptr() == out.data_ptr()
    return out, lse


def check_window(b, window, sinks, rows=None):
    for workspace in ("auto", None):
        out, lse = run_window(b, window, sinks, workspace)
        b.check(out, lse, lambda r: seen(int(b.ctx[r]), window, sinks), rows=rows)
        # rows behind the last request are left as they were
        assert torch.all(out[b.rows:] == 3.0) and torch.all(lse[b.rows:] == 7.0)


CASES = [
    # past, new, window, sinks, kwargs: decode rows, verify rows, chunks and mixtures
    ([0], [1], 1, 0, {}),
    ([0, 1, 5, 40], [1] * 4, 1, 1, {}),
    ([1, 30, 31, 32, 33, 127, 128, 129], [1] * 8, 32, 4, {}),
    ([700, 3000, 0, 64, 5], [4] * 5, 100, 4, dict(group=8, hk=4)),
    ([5000], [1], 1000, 33, dict(group=8, hk=1, dtype="fp16")),
    ([5000], [1], 4096, 0, dict(group=8, hk=1)),
    ([4090, 2], [8, 3], 257, 64, dict(dim=64, group=4, block=64, order="head")),
    ([100, 200], [3, 5], 31, 100, dict(group=7, block=100, order="interleaved")),
    ([100, 200], [2, 2], 65, 3, dict(group=1, hk=8, block=1)),
    ([300], [3], 64, 32, dict(group=32, hk=1)),
    ([300, 20], [2, 1], 63, 31, dict(group=33, hk=1)),
    ([900, 400], [2, 1], 200, 65, dict(group=128, hk=1, dim=64)),
    ([500], [1], 2 ** 31 - 1, 0, dict(group=3, hk=3, block=48, dtype="fp16")),
    ([500], [2], 7, 2 ** 31 - 1, dict(group=3, hk=3, block=48)),
    ([0], [200], 64, 0, dict(group=8, hk=1)),
    ([0], [200], 1, 0, dict(group=4)),
    ([0], [333], 50, 70, dict(group=4)),
    ([1000], [130], 129, 5, dict(group=8, hk=1, block=64)),
    ([1000], [130], 128, 64, dict(group=8, hk=1, block=8)),
    ([630], [257], 300, 1, dict(group=1, hk=2, dim=64, dtype="fp16")),
    ([2000], [300], 513, 63, dict(group=2, hk=1, block=24, dtype="fp16")),
    ([0, 900, 10, 0, 77], [150, 1, 33, 0, 300], 100, 4, dict(group=4, pad=3)),
    ([10, 1500, 0], [1, 100, 17], 777, 5, dict(group=7, hk=1, dim=64, dtype="fp16", block=100, order="head", pad=5)),
    ([400, 0], [70, 65], 33, 100, dict(group=33, hk=1)),
    ([170], [9], 20, 20, dict(group=128, hk=1, dim=64)),
    # few tiles over many keys, cut
    ([9000], [20], 4000, 16, dict(group=4, hk=1)),
    ([9000], [20], 6000, 100, dict(group=4, hk=1, dim=64, dtype="fp16", block=1, order="head")),
    ([9000, 30, 4000], [3, 1, 40], 1500, 40, dict(group=16, hk=1, block=100)),
    ([9000, 4000], [2, 3], 2000, 1000, dict(group=8, hk=2)),
    # requests without rows between others, more tiles than workgroups, all rows in one request
    ([0, 5, 900, 100] * 20, [0, 1, 0, 2] * 20, 60, 2, dict(group=8, hk=8)),
    ([300] * 40, [1, 20] * 20, 90, 10, dict(group=8, hk=4, dim=64)),
    ([500] * 20, [0] * 19 + [70], 77, 3, dict(group=8, hk=2)),
    # as many requests as a wave has lanes, some more, and more than are counted
    ([200, 90] * 32, [1, 3] * 32, 60, 2, dict(group=8, hk=1, dim=64)),
    ([200] * 65, [4] * 65, 33, 0, dict(group=8, hk=1)),
    ([130, 5, 70] * 50, [1, 0, 6] * 50, 40, 4, dict(group=16, hk=2, dim=64, pad=2)),
    ([60] * 1024, [1, 0, 2, 0] * 256, 33, 1, dict(group=4, hk=1, dim=64)),
    ([60] * 1030, [1] * 1030, 33, 1, dict(group=4, hk=1, dim=64, block=48)),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_window_attention(i):
    past, new, window, sinks, kw = CASES[i]
    b = Batch(200 + i, past, new, **kw)
    free_unseen(b, window, sinks)
    check_window(b, window, sinks)


@pytest.mark.parametrize("window", [1, 31, 32, 33, 63, 64, 65, 96, 500])
@pytest.mark.parametrize("sinks", [0, 1, 8, 31, 33, 64, 130])
def test_window_borders(window, sinks):
    """Windows and first tokens on either side of a step's border, in few rows and in a
    chunk."""
    for past, new, kw in (([0, 63, 64, 400, 130], [2, 1, 1, 3, 2], dict(group=8)),
                          ([190, 0], [66, 70], dict(group=4, hk=1, block=8, dtype="fp16"))):
        b = Batch(window * 10 + sinks, past, new, **kw)
        free_unseen(b, window, sinks)
        check_window(b, window, sinks)


@pytest.mark.parametrize("new", [[6, 5], [100, 90]], ids=["few", "chunk"])
@pytest.mark.parametrize("block", [1, 8, 16])
def test_window_any_counts(new, block):
    """Visible counts of any order, rows that see nothing, negative counts: rows far
    apart in a request, with what lies between their windows freed."""
    rng = np.random.default_rng(5)
    past = [400, 313]
    total = [p + a for p, a in zip(past, new)]
    ctx = np.concatenate([rng.integers(0, t + 1, a) for t, a in zip(total, new)])
    ctx[0], ctx[2], ctx[4] = 0, -3, 1
    for window, sinks in ((20, 3), (1, 0), (5, 100)):
        b = Batch(3, past, new, ctx=ctx, block=block)
        free_unseen(b, window, sinks)
        lim = np.maximum(b.ctx, 0)
        for workspace in ("auto", None):
            out, lse = run_window(b, window, sinks, workspace)
            b.check(out, lse, lambda r: seen(int(lim[r]), window, sinks))


LEFT_OVER = [
    # past, new, window, sinks, kwargs: more tiles of long windows than CUs, of which the ones left
    # over from whole rounds are cut: a few, many more than rows and requests tell (two tiles
    # of a request), fewer (requests and rows of padding), half a round
    ([2090] * 65, [1] * 65, 2000, 4, {}),
    ([1000] * 40 + [2300] * 30, [1] * 40 + [5] * 30, 2000, 40, dict(dtype="fp16")),
    ([1900] * 70, [1] * 60 + [0] * 10, 1800, 4, dict(pad=11, block=100)),
    ([200] * 48 + [3250] * 48, [1] * 96, 3150, 33, dict(order="head")),
]


@pytest.mark.parametrize("i", range(len(LEFT_OVER)))
def test_window_left_over_tiles(i):
    past, new, window, sinks, kw = LEFT_OVER[i]
    b = Batch(50 + i, past, new, hk=4, group=8, dim=64, **kw)
    free_unseen(b, window, sinks)
    shape = m.make_attn_shape(b.q.cuda(), b.kc, b.table)
    assert 0 < m.window_attention_workspace_bytes(shape, window, sinks) <= 70 << 20  # they are cut
    check_window(b, window, sinks, rows=sorted({*range(0, b.rows, 7), *range(max(b.rows - 20, 0), b.rows)}))
    # values that are not finite, in tiles that are cut and in others
    bad = {int(b.req[r]): int(b.ctx[r]) - 150 for r in (2, b.rows - 1)}
    for req, tok in bad.items():
        b.vc[int(b.table[req, tok // b.block]), tok % b.block] = float("nan")
    out, _ = run_window(b, window, sinks)
    for r in range(b.rows):
        hit = bad.get(int(b.req[r])) in seen(int(b.ctx[r]), window, sinks)
        assert bool(torch.isnan(out[r]).all()) == hit and bool(torch.isnan(out[r]).any()) == hit, r


def test_window_more_tiles_than_a_row_of_the_grid():
    """1,016 requests of one row with 70 heads over the same tokens: rows with equal queries are
    equal, the first and the last ones right."""
    n, hk, d, window, sinks, total = 1016, 70, 64, 300, 4, 500
    g = torch.Generator().manual_seed(9)
    k, v = torch.randn(total, hk, d, generator=g), torch.randn(total, hk, d, generator=g)
    kc, vc, table = device_cache(k, v, "bf16")
    q = torch.randn(8, hk, d, generator=g).to(torch.bfloat16).repeat(n // 8, 1, 1)
    lse = torch.empty(n, hk, device="cuda")
    args = (q.cuda(), kc, vc, table.repeat(n, 1), torch.full((n,), total, dtype=torch.int32, device="cuda"),
            torch.arange(n + 1, dtype=torch.int32, device="cuda"))
    out = m.window_attention(*args, window=window, sinks=sinks, lse=lse)
    for x in (out, lse):
        x = x.view(n // 8, 8, -1)
        assert torch.equal(x, x[:1].expand_as(x))
    toks = seen(total, window, sinks)
    for r in (0, 3, n - 1):
        for h in range(hk):
            check_values(out[r:r + 1, h:h + 1].double().cpu().numpy(), lse[r:r + 1, h:h + 1].double().cpu().numpy(),
                         q[r:r + 1, h:h + 1], k[toks, h:h + 1], v[toks, h:h + 1], [len(toks)], "bf16")


def test_window_counts_past_the_table():
    """Counts past the table's end are cut to it, and the window is taken from there."""
    for new in ([1], [70]):
        b = Batch(4, [320 - new[0]], new, extra_blocks=0)
        b.ctx[-1] = 2 ** 31 - 1
        out, lse = run_window(b, 50, 3)
        b.ctx[-1] = 320
        b.check(out, lse, lambda r: seen(int(b.ctx[r]), 50, 3))


@pytest.mark.parametrize("new", [[4, 2], [70, 60]], ids=["few", "chunk"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("workspace", ["auto", None])
def test_window_values_others_see(new, value, workspace):
    """Values that are not finite reach the rows that see them and no others: one that
    has left the later rows' window, one among the first tokens, one that the earlier rows do not
    see yet."""
    past, window, sinks = [200, 333], 40, 3
    for bad in (past[0] + new[0] // 2 - window, past[0] + new[0] // 2, 1, sinks, 100):
        b = Batch(11, past, new, group=4)
        entry = int(b.table[0, bad // b.block])
        b.vc[entry, bad % b.block] = value
        out, lse = run_window(b, window, sinks, workspace)
        clean = [r for r in range(b.rows) if b.req[r] == 1 or bad not in seen(int(b.ctx[r]), window, sinks)]
        b.check(out, lse, lambda r: seen(int(b.ctx[r]), window, sinks), rows=clean)
        dirty = sorted(set(range(b.rows)) - set(clean))
        assert (len(dirty) == 0) == (bad in (sinks, 100))
        for r in dirty:
            assert torch.all(torch.isnan(out[r]) if np.isnan(value) else out[r] == value), (bad, r)


@pytest.mark.parametrize("new", [[4, 2], [70, 60]], ids=["few", "chunk"])
@pytest.mark.parametrize("workspace", ["auto", None])
def test_window_bad_entries(new, workspace):
    """Table entries outside the pool under tokens that are seen: rows that see them are
    NaN, others are not touched."""
    past, window, sinks = [206, 333], 40, 3
    for bad in (0, (past[0] - window + 2) // 16, (past[0] + 2) // 16):
        b = Batch(12, past, new, group=4)
        b.table = b.table.clone()
        b.table[0, bad] = b.kc.shape[0]
        out, lse = run_window(b, window, sinks, workspace)
        toks = set(range(bad * 16, bad * 16 + 16))
        clean = [r for r in range(b.rows) if b.req[r] == 1 or not toks & set(seen(int(b.ctx[r]), window, sinks))]
        b.check(out, lse, lambda r: seen(int(b.ctx[r]), window, sinks), rows=clean)
        for r in set(range(b.rows)) - set(clean):
            assert torch.all(torch.isnan(out[r])) and torch.all(torch.isnan(lse[r])), (bad, r)


KERNELS = {"stream": (1, 8), "stream_cut": (1, 8), "tile": (65, 8), "tile_cut": (65, 8)}


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("dtype,seed", [("bf16", 1), ("fp16", 2)])
@pytest.mark.parametrize("window,sinks", [(300, 5), (70, 100), (33, 0)])
def test_window_values_not_finite_anywhere(kernel, dtype, seed, window, sinks):
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
    dt = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
    q = torch.randn(rows, group, d, generator=g).to(dt)
    counts = rng.integers(0, n + 1, rows).astype(np.int32)
    counts[:3] = n, 1, 40
    kc, vc, table = device_cache(k, v, dtype)
    lse = torch.empty(q.shape[:2], device="cuda")
    out = m.window_attention(q.cuda(), kc, vc, table, dev(counts), dev(np.array([0, rows], np.int32)), window=window,
                             sinks=sinks, lse=lse, workspace="auto" if kernel.endswith("cut") else None)
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    with np.errstate(invalid="ignore"):
        for r, c in enumerate(counts):
            toks = seen(int(c), window, sinks)
            check_values(out[r:r + 1], lse[r:r + 1], q[r:r + 1], k[toks], v[toks], [len(toks)], dtype)


def test_window_long_context():
    """A row at the end of 3,000,001 tokens of which the table holds the window's and the
    first tokens' blocks only; and cache offsets past 2^31 elements."""
    n, block, dim, hk, group, window, sinks = 3_000_001, 64, 128, 2, 4, 1000, 70
    g = torch.Generator().manual_seed(1)
    toks = seen(n, window, sinks)
    entries = sorted({t // block for t in toks})
    pool = 2 ** 31 // (block * hk * dim) + 100
    kc = torch.full((pool, block, hk, dim), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    table = np.full((1, n // block + 1), -1, np.int32)
    table[0, entries] = pool - 1 - np.arange(len(entries)) * 3
    rows = torch.randn(2, len(toks), hk, dim, generator=g).to(torch.bfloat16)
    where = torch.from_numpy(table[0, np.array(toks) // block].astype(np.int64)).cuda()
    at = torch.from_numpy(np.array(toks) % block).cuda()
    kc[where, at], vc[where, at] = rows[0].cuda(), rows[1].cuda()
    for R in (1, 80):
        q = torch.randn(R, hk * group, dim, generator=g).to(torch.bfloat16)
        lse = torch.empty(R, hk * group, device="cuda")
        out = m.window_attention(q.cuda(), kc, vc, dev(table), dev(np.full(R, n, np.int32)),
                                 dev(np.array([0, R], np.int32)), window=window, sinks=sinks, lse=lse)
        for h in range(hk):
            hs = slice(h * group, (h + 1) * group)
            check_values(out[:, hs].double().cpu().numpy(), lse[:, hs].double().cpu().numpy(), q[:, hs],
                         rows[0][:, h:h + 1], rows[1][:, h:h + 1], [len(toks)] * R, "bf16")


def test_window_strides_stream_and_repeats():
    """q as a view of a fused projection, out a view of a wider buffer, on a stream of
    its own; equal results from call to call."""
    b = Batch(21, [1000, 60], [3, 40], group=4, hk=2, dim=64)
    free_unseen(b, 500, 9)
    R, hq = b.q.shape[:2]
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        fused = torch.zeros(R, hq + 4, 64, dtype=b.q.dtype, device="cuda")
        fused[:, :hq] = b.q.cuda()
        wide = torch.full((R, hq, 80), 3.0, dtype=b.q.dtype, device="cuda")
    torch.cuda.synchronize()
    out, lse = run_window(b, 500, 9, q=fused[:, :hq], out=wide[:, :, :64], stream=s)
    torch.cuda.synchronize()
    b.check(out, lse, lambda r: seen(int(b.ctx[r]), 500, 9))
    assert torch.all(wide[:, :, 64:] == 3.0)
    for _ in range(3):
        again, lse2 = run_window(b, 500, 9)
        assert torch.equal(again, out) and torch.equal(lse, lse2)


def test_window_graphs_side_by_side():
    """Calls with workspaces of their own, captured in graphs of their own and replayed
    on streams of their own, several times, with other work between."""
    runs = []
    for i, (past, new, kw) in enumerate((([4000, 900], [3, 2], dict(group=8)), ([4000, 900], [40, 33], dict(group=8)),
                                         ([5000], [1], dict(group=4, dim=64)))):
        b = Batch(60 + i, past, new, **kw)
        free_unseen(b, 1500, 20)
        q, ctx, starts = b.q.cuda(), dev(b.ctx), dev(b.starts)
        out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda")
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            call = m.PreparedWindowAttention(q, b.kc, b.vc, b.table, ctx, starts, out, window=1500, sinks=20, lse=lse)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                call()
        runs.append((b, s, graph, call, out, lse, (q, ctx, starts)))
    torch.cuda.synchronize()
    want = None
    for _ in range(4):
        for r in runs:
            r[4].fill_(float("nan"))
            r[5].fill_(float("nan"))
        torch.cuda.synchronize()
        for _, s, graph, *_ in runs:
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for r in runs for t in (r[4], r[5])]
        if want is None:
            for b, _, _, _, out, lse, _ in runs:
                b.check(out, lse, lambda r: seen(int(b.ctx[r]), 1500, 20))
            want = got
        assert all(torch.equal(x, y) for x, y in zip(want, got))
        torch.randn(1000, 1000, device="cuda") @ torch.randn(1000, 1000, device="cuda")


def test_window_refusals():
    b = Batch(80, [40], [2])
    q, ctx, starts = b.q.cuda(), dev(b.ctx), dev(b.starts)
    for kw in (dict(window=0), dict(window=-1), dict(window=2 ** 31), dict(window=4, sinks=-1), dict(window=4, sinks=2 ** 31),
               dict(window=4, scale=0.0), dict(window=4, lse=torch.zeros(2, 8)), dict(window=4, workspace="none")):
        with pytest.raises(m.QsaError):
            m.window_attention(q, b.kc, b.vc, b.table, ctx, starts, **kw)
    for args in ((q.float(), b.kc, b.vc, b.table, ctx, starts), (q, b.kc, b.vc, b.table, ctx[:1], starts),
                 (q, b.kc, b.vc[:, :8], b.table, ctx, starts), (q, b.kc, b.vc, b.table, ctx, starts[:1])):
        with pytest.raises(m.QsaError):
            m.window_attention(*args, window=4)
    assert m.window_attention(q[:0], b.kc, b.vc, b.table, ctx[:0], starts, window=4).shape == (0, 8, 128)
