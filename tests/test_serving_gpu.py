"""The batch plan, the cache writes and paged attention on the GPU, against the
plain 64-bit implementations in serving_ref.py."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
m = pytest.importorskip("paged_mqa_logits_block_amd")

import serving_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


# ---------------------------------------------------------------------------
# batch plan
# ---------------------------------------------------------------------------

def plan_inputs(rng, n, B, past, new, max_blocks, short=0):
    """Lengths, a table whose held entries are distinct pool blocks (other entries
    garbage), and the free list of the rest (``short`` of what is needed)."""
    cap = max_blocks * B
    have = [-(-min(max(p, 0), cap) // B) for p in past]
    pool = sum(have) + sum(max(0, x) // B + 2 for x in new) + 5
    ids = rng.permutation(pool).astype(np.int32)
    table = np.full((n, max_blocks), -7, np.int32)
    at = 0
    for i, h in enumerate(have):
        table[i, :h] = ids[at:at + h]
        at += h
    free = ids[at:]
    if short:
        need = sum(max(0, -(-min(max(p, 0) + max(x, 0), cap) // B) - h) for p, x, h in zip(past, new, have))
        free = free[:max(0, need - short)]
    return table, free, pool


PLAN_CASES = [
    # n, B, ratio, max_blocks, rows, past, new, short
    (1, 16, 4, 10, 1, [0], [1], 0),
    (1, 16, 4, 10, 8, [15], [1], 0),            # padding rows behind
    (9, 16, 4, 400, 36, "lens", [4] * 9, 0),
    (5, 64, 4, 20, 700, [0, 63, 64, 65, 500], [1, 1, 64, 0, 613], 0),
    (4, 48, 3, 9, 100, [0, 1, 47, 400], [10, -5, 30, 60], 0),   # past the table's end, a negative length
    (3, 16, 1, 30, 50, [10, 20, 30], [20, 20, 20], 0),          # rows behind num_rows are dropped
    (3, 16, 2, 30, 50, [10, 20, 30], [2 ** 31 - 1, 5, 5], 0),   # a length past every limit
    (6, 16, 4, 50, 300, [0] * 6, [40] * 6, 7),                  # the free list runs out
    (2, 1, 1, 100, 20, [3, 50], [7, 9], 0),
    (300, 32, 4, 40, 2000, "lens", "mixed", 0),
    (4096, 16, 4, 8, 5000, "lens", "ones", 0),
    (2, 100, 25, 10, 0, [5, 900], [0, 0], 0),                   # no rows at all
]


@pytest.mark.parametrize("case", PLAN_CASES, ids=[f"n{c[0]}_b{c[1]}_r{c[2]}_rows{c[4]}_s{c[7]}" for c in PLAN_CASES])
def test_plan_batch(case):
    n, B, ratio, max_blocks, rows, past, new, short = case
    rng = np.random.default_rng(n * 1000 + B)
    if past == "lens":
        past = [int(x) for x in rng.integers(0, max_blocks * B - 40, n)]
    if new == "mixed":
        new = [int(x) for x in np.where(rng.random(n) < 0.1, rng.integers(1, 100, n), rng.integers(0, 3, n))]
    if new == "ones":
        new = [int(x) for x in rng.integers(0, 3, n)]
    table, free, pool = plan_inputs(rng, n, B, past, [min(x, 4000) for x in new], max_blocks, short)
    want = ref.plan(past, new, free, table, block_size=B, num_blocks=pool, num_rows=rows, ratio=ratio)
    t = dev(table)
    got = m.plan_batch(dev(np.array(past, np.int32)), dev(np.array(new, np.int32)), dev(free), t, block_size=B,
                       num_blocks=pool, num_rows=rows, ratio=ratio)
    for again in range(2):  # a second call on the updated table gives the same
        assert np.array_equal(t.cpu().numpy(), want.table)
        for f in ("q_starts", "row_to_req", "ctx_lens", "slots", "col_lens", "col_slots", "blocks_used"):
            assert np.array_equal(getattr(got, f).cpu().numpy(), getattr(want, f)), f
        got = m.plan_batch(dev(np.array(past, np.int32)), dev(np.array(new, np.int32)), dev(free), t, block_size=B,
                           num_blocks=pool, num_rows=rows, ratio=ratio, out=got)
    if short:
        assert int(got.blocks_used) == len(free) + short


def test_plan_optional_outputs_and_bad_entries():
    """Without the optional outputs; held entries outside the pool give no slot."""
    table = dev(np.array([[3, -1, 9], [99, 2, -1]], np.int32))
    out = m.BatchPlan.empty(2, 6, "cuda")
    out.col_lens = out.col_slots = out.blocks_used = None
    m.plan_batch(dev(np.array([4, 7], np.int32)), dev(np.array([3, 3], np.int32)), dev(np.array([5, 6], np.int32)),
                 table, block_size=4, num_blocks=10, num_rows=6, out=out)
    assert table.cpu().tolist() == [[3, 5, 9], [99, 2, 6]]
    assert out.slots.cpu().tolist() == [20, 21, 22, 11, 24, 25]
    table = dev(np.array([[3, 77, 9]], np.int32))
    m.plan_batch(dev(np.array([6], np.int32)), dev(np.array([6], np.int32)), dev(np.array([5], np.int32)), table,
                 block_size=4, num_blocks=10, num_rows=6, out=m.BatchPlan(*(
                     getattr(out, f)[:2] if f == "q_starts" else getattr(out, f)
                     for f in ("q_starts", "row_to_req", "ctx_lens", "slots"))))
    assert out.slots.cpu().tolist() == [-1, -1, 20, 21, 22, 23]


def test_prepared_plan_keeps_its_buffers():
    """The buffers of a prepared call live as long as it does, whatever becomes of the
    BatchPlan's fields."""
    import gc
    import weakref
    out = m.BatchPlan.empty(2, 6, "cuda")
    fields = ("q_starts", "row_to_req", "ctx_lens", "slots", "col_lens", "col_slots", "blocks_used")
    alive = [weakref.ref(getattr(out, f)) for f in fields]
    call = m.PreparedPlanBatch(dev(np.zeros(2, np.int32)), dev(np.ones(2, np.int32)), dev(np.arange(4, dtype=np.int32)),
                               dev(np.full((2, 3), -1, np.int32)), block_size=4, num_blocks=10, out=out)
    for f in fields:
        setattr(out, f, None)
    gc.collect()
    assert all(r() is not None for r in alive)
    del call
    gc.collect()
    assert all(r() is None for r in alive)


# ---------------------------------------------------------------------------
# cache writes
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,dim,heads,block,rows,order", [
    ("bf16", 128, 4, 16, 36, "slot"), ("fp16", 64, 2, 100, 333, "head"), ("bf16", 128, 1, 1, 7, "slot"),
    ("fp16", 128, 3, 64, 1, "head"), ("bf16", 64, 8, 48, 1000, "interleaved"),
])
def test_write_kv(dtype, dim, heads, block, rows, order):
    g = torch.Generator().manual_seed(rows)
    pool = -(-rows // block) + 5
    # k and v as views of one projection, rows of 3 parts
    qkv = torch.randn(rows, 3 * heads, dim, generator=g).to(DT[dtype]).cuda()
    k, v = qkv[:, heads:2 * heads], qkv[:, 2 * heads:]
    if order == "slot":
        kc, vc = (torch.zeros(pool, block, heads, dim, dtype=DT[dtype], device="cuda") for _ in range(2))
    elif order == "head":
        kc, vc = (torch.zeros(pool, heads, block, dim, dtype=DT[dtype], device="cuda").transpose(1, 2)
                  for _ in range(2))
    else:
        both = torch.zeros(pool, 2, block, heads, dim, dtype=DT[dtype], device="cuda")
        kc, vc = both[:, 0], both[:, 1]
    slots = torch.randperm(pool * block, generator=g)[:rows]
    if rows > 2:
        slots[1], slots[2] = -1, pool * block  # neither is a slot
    m.write_kv(k, v, slots.cuda(), kc, vc)
    for cache, src in ((kc, k), (vc, v)):
        want = torch.zeros(pool * block, heads, dim, dtype=DT[dtype])
        keep = (slots >= 0) & (slots < pool * block)
        want[slots[keep]] = src.cpu()[keep]
        assert torch.equal(cache.cpu().reshape(pool * block, heads, dim), want)


@pytest.mark.parametrize("layout", ["plain", "paged", "noscale", "copacked", "shuffled"])
@pytest.mark.parametrize("dtype,dim,block,rows", [("bf16", 128, 64, 200), ("fp16", 64, 16, 33), ("fp16", 128, 48, 1),
                                                  ("bf16", 64, 3, 50)])
def test_write_keys(layout, dtype, dim, block, rows):
    if layout == "shuffled" and block % 16:
        pytest.skip("the preshuffled layout needs blocks of a multiple of 16")
    g = torch.Generator().manual_seed(rows + dim)
    pool = -(-rows // block) + 4
    x = torch.randn(rows, dim, generator=g) * torch.exp(3 * torch.randn(rows, 1, generator=g))
    if rows > 8:
        x[3] = 0.0
        x[4] = 0.0
        x[4, 5] = -2.0 ** -24 if dtype == "fp16" else 2.0 ** -133  # a single subnormal
        x[5] = torch.sign(x[5]) * 60000.0
    src = torch.zeros(rows, dim + 8, dtype=DT[dtype])
    src[:, :dim] = x.to(DT[dtype])
    keys = src.cuda()[:, :dim]
    slots = torch.randperm(pool * block, generator=g)[:rows]
    if rows > 8:
        slots[7], slots[8] = -1, pool * block
    keep = (slots >= 0) & (slots < pool * block)
    at = slots[keep]
    f = src[keep, :dim].float()
    if layout == "plain":
        kc = torch.zeros(pool, block, dim, dtype=DT[dtype], device="cuda")
        m.write_keys(keys, slots.cuda(), kc, block_size=block)
        want = torch.zeros(pool * block, dim, dtype=DT[dtype])
        want[at] = src[keep, :dim]
        assert torch.equal(kc.cpu().view(-1, dim), want)
        return
    top = f.abs().amax(dim=1)
    scale = torch.where(top > 0, top / 448.0, torch.ones_like(top))
    if layout == "noscale":
        scale = torch.ones_like(top)
    code = (f / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    codes = torch.zeros(pool * block, dim, dtype=torch.uint8)
    scales = torch.zeros(pool * block)
    codes[at], scales[at] = code, scale
    codes = codes.view(pool, block, dim)
    if layout in ("paged", "noscale"):
        kc = torch.zeros(pool, block, dim, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        ks = torch.zeros(pool, block, device="cuda") if layout == "paged" else None
        m.write_keys(keys, slots.cuda(), kc, block_size=block, kscale=ks)
        assert torch.equal(kc.view(torch.uint8).cpu(), codes)
        if ks is not None:
            assert torch.equal(ks.cpu().view(-1), scales)
        return
    kc = torch.zeros(pool, block * (dim + 4), dtype=torch.uint8, device="cuda")
    m.write_keys(keys, slots.cuda(), kc, block_size=block,
                 layout=m.KV_COPACKED if layout == "copacked" else m.KV_COPACKED_SHUFFLED)
    if layout == "shuffled":
        import qsa_inputs
        codes = torch.from_numpy(qsa_inputs.shuffle_keys_16x16(codes.numpy()))
    got = kc.cpu()
    assert torch.equal(got[:, :block * dim], codes.reshape(pool, -1))
    assert torch.equal(got[:, block * dim:].contiguous().view(torch.float32).view(-1), scales)


def test_write_keys_not_finite():
    """A key with an infinity or a NaN spoils its own slot only."""
    x = torch.ones(4, 64, dtype=torch.bfloat16)
    x[1, 3], x[2, 7] = float("inf"), float("nan")
    kc = torch.zeros(1, 16 * 68, dtype=torch.uint8, device="cuda")
    m.write_keys(x.cuda(), torch.arange(4).cuda(), kc, block_size=16, layout=m.KV_COPACKED)
    sc = kc.cpu()[:, 16 * 64:].contiguous().view(torch.float32)[0]
    codes = kc.cpu()[0, :16 * 64].view(16, 64)
    one = torch.tensor([448.0]).to(torch.float8_e4m3fn).view(torch.uint8)
    for r in (0, 3):
        assert torch.all(codes[r] == one) and sc[r] == torch.tensor(1.0) / 448.0
    assert torch.all(codes[4:] == 0) and torch.all(sc[4:] == 0)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

class Batch:
    """Requests with `past` cached and `new` query tokens; caches whose unused
    places are NaN and tables whose unused entries are garbage."""

    def __init__(self, seed, past, new, *, hk=2, group=4, dim=128, dtype="bf16", block=16, order="slot", pad=0,
                 ctx=None, q_gain=2.0, extra_blocks=2):
        self.rng = rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.n, self.hk, self.group, self.dim, self.block = len(past), hk, group, dim, block
        total = [p + a for p, a in zip(past, new)]
        blocks = [-(-t // block) for t in total]
        pool = sum(blocks) + 3
        ids = rng.permutation(pool)
        width = max(max(blocks), 1) + extra_blocks
        table = rng.integers(-2 ** 31, 2 ** 31, (self.n, width)).astype(np.int32)
        kv = torch.full((2, pool * block, hk, dim), float("nan"))
        at = 0
        self.k, self.v = [], []
        for i, (t, b) in enumerate(zip(total, blocks)):
            table[i, :b] = ids[at:at + b]
            at += b
            pos = np.arange(t)
            where = torch.from_numpy(table[i, pos // block].astype(np.int64) * block + pos % block)
            rows = torch.randn(2, t, hk, dim, generator=g).to(DT[dtype])
            kv[:, where] = rows.float()
            self.k.append(rows[0].double().numpy())
            self.v.append(rows[1].double().numpy())
        kv = kv.to(DT[dtype]).view(2, pool, block, hk, dim)
        if order == "head":
            kv = kv.permute(0, 1, 3, 2, 4).contiguous().cuda().permute(0, 1, 3, 2, 4)
        elif order == "interleaved":
            kv = kv.permute(1, 0, 2, 3, 4).contiguous().cuda().permute(1, 0, 2, 3, 4)
        else:
            kv = kv.cuda()
        self.kc, self.vc = kv[0], kv[1]
        self.table = dev(table)
        self.rows = sum(new)
        self.starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.req = np.repeat(np.arange(self.n), new)
        if ctx is None:
            ctx = np.concatenate([np.arange(p + 1, p + a + 1) for p, a in zip(past, new)] + [np.zeros(0)])
        self.ctx = np.concatenate([np.asarray(ctx), np.full(pad, 5)]).astype(np.int32)
        self.q = torch.randn(self.rows + pad, hk * group, dim, generator=g).mul(q_gain).to(DT[dtype])
        self.half_step = torch.finfo(DT[dtype]).eps / 2

    def check(self, out, lse, keys_of, rows=None):
        """Every row against the 64-bit result over the tokens keys_of(row) (a list
        of token numbers of its request), with the bounds derived in serving_ref."""
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        for r in range(self.rows) if rows is None else rows:
            i, toks = self.req[r], np.asarray(keys_of(r), dtype=np.int64)
            for h in range(self.hk):
                hs = slice(h * self.group, (h + 1) * self.group)
                q = self.q[r, hs].double().numpy()
                o, l, spread, size = ref.attend(q, self.k[i][toks, h], self.v[i][toks, h], self.dim ** -0.5)
                if len(toks) == 0:
                    assert np.all(out[r, hs] == 0) and np.all(lse[r, hs] == -np.inf), (r, h)
                    continue
                to, tl = ref.bounds(o, l, spread, size, len(toks), self.dim, self.half_step)
                eo, el = np.abs(out[r, hs] - o), np.abs(lse[r, hs] - l)
                assert np.all(eo <= to), (r, h, float((eo / to).max()), len(toks))
                assert np.all(el <= tl), (r, h, float((el / tl).max()), len(toks))


def run_paged(b, workspace="auto", q=None, out=None, **kw):
    lse = torch.full((b.q.shape[0], b.q.shape[1]), 7.0, device="cuda")
    out = torch.full(tuple(b.q.shape), 3.0, dtype=b.q.dtype, device="cuda") if out is None else out
    got = m.paged_attention(b.q.cuda() if q is None else q, b.kc, b.vc, b.table, dev(b.ctx), dev(b.starts), out=out,
                            lse=lse, workspace=workspace, **kw)
    assert got.data_ptr() == out.data_ptr()
    return out, lse


PAGED = [
    # past, new, kwargs: decode rows, verify rows, chunks and mixtures
    ([0], [1], {}),
    ([1, 30, 31, 32, 33, 127, 128, 129], [1] * 8, {}),
    ([700, 3000, 0, 64, 5], [4] * 5, dict(group=8, hk=4)),
    ([5000], [1], dict(group=8, hk=1, dtype="fp16")),
    ([4090, 2], [8, 3], dict(dim=64, group=4, block=64, order="head")),
    ([100, 200], [3, 5], dict(group=7, block=100, order="interleaved")),
    ([100, 200], [2, 2], dict(group=1, hk=8, block=1)),
    ([300], [3], dict(group=32, hk=1)),
    ([300, 20], [2, 1], dict(group=33, hk=1)),
    ([90, 400], [2, 1], dict(group=128, hk=1, dim=64)),
    ([50], [1], dict(group=3, hk=3, block=48, dtype="fp16")),
    ([0], [64], dict(group=8, hk=1)),
    ([0], [200], dict(group=4)),
    ([1000], [130], dict(group=8, hk=1, block=64)),
    ([63], [257], dict(group=1, hk=2, dim=64, dtype="fp16")),
    ([0, 900, 10, 0, 77], [150, 1, 33, 0, 300], dict(group=4, pad=3)),
    ([10, 500, 0], [1, 100, 17], dict(group=7, hk=1, dim=64, dtype="fp16", block=100, order="head", pad=5)),
    ([40, 0], [70, 65], dict(group=33, hk=1)),
    ([17], [9], dict(group=128, hk=1, dim=64)),
    # few tiles over many keys: parts of one tile from many workgroups
    ([9000], [20], dict(group=4, hk=1)),
    ([9000], [20], dict(group=4, hk=1, dim=64, dtype="fp16", block=1, order="head")),
    ([9000, 30, 4000], [3, 1, 40], dict(group=16, hk=1, block=100)),
    # requests without rows between others, one row each, more tiles than workgroups
    ([0, 5, 9, 100] * 20, [0, 1, 0, 2] * 20, dict(group=8, hk=8)),
    ([300] * 40, [1, 20] * 20, dict(group=8, hk=4, dim=64)),
    # all rows of a batch of few rows per request in one request
    ([500] * 20, [0] * 19 + [70], dict(group=8, hk=2)),
    ([500] * 20, [0] * 3 + [65] + [0] * 16, dict(group=33, hk=1, dim=64)),
]


@pytest.mark.parametrize("i", range(len(PAGED)))
def test_paged_attention(i):
    past, new, kw = PAGED[i]
    b = Batch(i, past, new, **kw)
    out, lse = run_paged(b)
    b.check(out, lse, lambda r: range(b.ctx[r]))
    # rows behind the last request are left as they were
    assert torch.all(out[b.rows:] == 3.0) and torch.all(lse[b.rows:] == 7.0)
    # without a workspace the keys of a tile are not cut
    out, lse = run_paged(b, workspace=None)
    b.check(out, lse, lambda r: range(b.ctx[r]))
    assert torch.all(out[b.rows:] == 3.0) and torch.all(lse[b.rows:] == 7.0)


@pytest.mark.parametrize("rows,group", [(1, 4), (5, 16)])
def test_paged_attention_many_requests(rows, group):
    """More requests than a cut launch takes, in both kernels."""
    n = 1100
    rng = np.random.default_rng(rows)
    b = Batch(14, [int(x) for x in rng.integers(0, 40, n)], [rows] * n, hk=1, group=group, dim=64)
    assert m.paged_attention_workspace_bytes(m.make_attn_shape(b.q.cuda(), b.kc, b.table)) == 0
    out, lse = run_paged(b)
    b.check(out, lse, lambda r: range(b.ctx[r]), rows=range(0, b.rows, 7))
    assert not torch.any(torch.isnan(out))


@pytest.mark.parametrize("kw", [dict(group=8, hk=4), dict(group=40, hk=2, dim=64, dtype="fp16")])
def test_paged_attention_few_of_many_requests(kw):
    """A table of 1,000 requests of which five have rows, some over long contexts whose
    tiles are cut, some that see nothing."""
    past, new = [0] * 1000, [0] * 1000
    for i, p, a in ((0, 3000, 1), (17, 9, 3), (500, 12_000, 2), (501, 0, 1), (999, 700, 4)):
        past[i], new[i] = p, a
    b = Batch(16, past, new, pad=2, **kw)
    b.ctx[4] = 0
    assert m.paged_attention_workspace_bytes(m.make_attn_shape(b.q.cuda(), b.kc, b.table)) > 0
    for workspace in ("auto", None):
        out, lse = run_paged(b, workspace=workspace)
        b.check(out, lse, lambda r: range(b.ctx[r]))
        assert torch.all(out[b.rows:] == 3.0) and torch.all(lse[b.rows:] == 7.0)


def test_paged_attention_many_rows():
    """More rows than a cut launch takes: every tile whole."""
    b = Batch(15, [10, 5], [8000, 300], hk=1, group=1, dim=64)
    out, lse = run_paged(b)
    b.check(out, lse, lambda r: range(b.ctx[r]), rows=[*range(0, b.rows, 211), 7999, 8000, b.rows - 1])
    assert not torch.any(torch.isnan(out))


@pytest.mark.parametrize("new", [[6, 5], [100, 90]], ids=["few", "chunk"])
def test_paged_attention_any_counts(new):
    """Visible counts of any order, rows that see nothing, negative counts and
    counts past the table's end."""
    rng = np.random.default_rng(5)
    past = [400, 313]
    total = [p + a for p, a in zip(past, new)]
    ctx = np.concatenate([rng.integers(0, t + 1, a) for t, a in zip(total, new)])
    ctx[0], ctx[2], ctx[4] = 0, -3, 1
    b = Batch(3, past, new, ctx=ctx, extra_blocks=0, block=1)
    b.ctx[1] = 2 ** 31 - 1  # clamped to the table's columns
    lim = np.minimum(np.maximum(b.ctx, 0), b.table.shape[1])
    lim[1] = total[0]
    b.ctx[1] = total[0] if b.table.shape[1] > total[0] else b.ctx[1]
    out, lse = run_paged(b)
    b.check(out, lse, lambda r: range(lim[r]))


@pytest.mark.parametrize("new", [[4, 2], [70, 60]], ids=["few", "chunk"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_paged_attention_values_others_see(new, value):
    """Values that are not finite reach the rows that see them and no others,
    though rows of one tile share the steps."""
    past = [200, 333]
    b = Batch(11, past, new, group=4)
    bad = past[0] + new[0] // 2  # seen by the later rows of request 0 only
    entry = int(b.table[0, bad // b.block])
    b.vc[entry, bad % b.block] = value
    b.kc[entry, bad % b.block] = value
    out, lse = run_paged(b)
    clean = [r for r in range(b.rows) if b.req[r] == 1 or b.ctx[r] <= bad]
    b.check(out, lse, lambda r: range(b.ctx[r]), rows=clean)
    for r in set(range(b.rows)) - set(clean):
        assert torch.all(torch.isnan(out[r])), r


@pytest.mark.parametrize("rows,reqs", [(64, 1), (64, 2), (8, 2)])
def test_paged_attention_values_other_waves_see(rows, reqs):
    """The same where whole waves of a tile see one count: the first half of the rows
    sees 100 tokens, the second half 200, and token 150's value is not finite."""
    ctx = np.concatenate([np.where(np.arange(rows) < rows // 2, 100, 200) for _ in range(reqs)])
    b = Batch(13, [200] * reqs, [rows] * reqs, group=4, ctx=ctx)
    for i in range(reqs):
        b.vc[int(b.table[i, 150 // b.block]), 150 % b.block] = float("inf")
    for workspace in ("auto", None):
        out, lse = run_paged(b, workspace=workspace)
        clean = [r for r in range(b.rows) if b.ctx[r] == 100]
        b.check(out, lse, lambda r: range(b.ctx[r]), rows=clean)
        assert torch.all(torch.isinf(out[[r for r in range(b.rows) if b.ctx[r] == 200]]))


@pytest.mark.parametrize("new", [[4, 2], [70, 60]], ids=["few", "chunk"])
def test_paged_attention_bad_entries(new):
    """Table entries outside the pool: rows that see their columns are NaN, others
    are not touched by them."""
    past = [206, 333]
    b = Batch(12, past, new, group=4)
    table = b.table.clone()
    first = (past[0] + 2) // b.block  # the entry of the request's second new row on
    table[0, first] = b.kc.shape[0]
    b.table = table
    out, lse = run_paged(b)
    clean = [r for r in range(b.rows) if b.req[r] == 1 or b.ctx[r] <= first * b.block]
    b.check(out, lse, lambda r: range(b.ctx[r]), rows=clean)
    for r in set(range(b.rows)) - set(clean):
        assert torch.all(torch.isnan(out[r])) and torch.all(torch.isnan(lse[r])), r


def test_paged_attention_strides_and_stream():
    """q as a view of a fused projection, out a view of a wider buffer, on a
    stream of its own."""
    b = Batch(21, [100, 60], [3, 40], group=4, hk=2, dim=64)
    R, hq = b.q.shape[:2]
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        fused = torch.zeros(R, hq + 4, 64, dtype=b.q.dtype, device="cuda")
        fused[:, :hq] = b.q.cuda()
        wide = torch.full((R, hq, 80), 3.0, dtype=b.q.dtype, device="cuda")
    torch.cuda.synchronize()
    out, lse = run_paged(b, q=fused[:, :hq], out=wide[:, :, :64], stream=s)
    torch.cuda.synchronize()
    b.check(out, lse, lambda r: range(b.ctx[r]))
    assert torch.all(wide[:, :, 64:] == 3.0)
    got = m.paged_attention(b.q.cuda(), b.kc, b.vc, b.table, dev(b.ctx), dev(b.starts), scale=64 ** -0.5)
    assert torch.equal(got, out)


def test_paged_attention_long_context():
    """3,000,001 tokens in blocks of 1,000, all entries of the table pointing at 7
    blocks: the result is that of 7,000 keys with multiplicities."""
    n, block, dim, group = 3_000_001, 1000, 64, 4
    rng = np.random.default_rng(9)
    kv = torch.from_numpy(rng.standard_normal((2, 7, block, 1, dim))).to(torch.bfloat16)
    table = rng.integers(0, 7, (1, n // block + 1)).astype(np.int32)
    q = torch.from_numpy(rng.standard_normal((1, group, dim))).to(torch.bfloat16)
    lse = torch.empty(1, group, device="cuda")
    out = m.paged_attention(q.cuda(), kv[0].cuda(), kv[1].cuda(), dev(table), dev(np.array([n], np.int32)),
                            dev(np.array([0, 1], np.int32)), lse=lse)
    count = np.zeros((7, block))
    np.add.at(count, table[0, :n // block], 1)
    count[table[0, -1], :n % block] += 1
    k, v = (x.double().numpy().reshape(7 * block, dim) for x in kv)
    z = q[0].double().numpy() @ k.T * dim ** -0.5
    w = np.exp(z) * count.reshape(-1)
    p = w / w.sum(axis=1, keepdims=True)
    want = p @ v
    # the longest chain of additions: the keys of one wave (n / (256 workgroups of 8
    # waves)), the 8 waves and the 256 parts
    size = dim ** -0.5 * (np.abs(q[0].double().numpy()) @ np.abs(k).T).max(axis=1)
    u = torch.finfo(torch.bfloat16).eps / 2
    lse_want = np.log(w.sum(axis=1))
    to, tl = ref.bounds(want, lse_want, p @ np.abs(v), size, n // 2048 + 512, dim, u)
    assert np.all(np.abs(out[0].double().cpu().numpy() - want) <= to)
    assert np.all(np.abs(lse[0].double().cpu().numpy() - lse_want) <= tl)


def test_paged_attention_far_blocks():
    """Pool offsets past 2^31 elements, in both kernels and the writes."""
    hk, dim, block = 4, 128, 64
    per = hk * dim * block
    pool = (2 ** 31) // per + 40
    kc = torch.empty(pool, block, hk, dim, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    new, past = [2, 80], [190, 48]
    b = Batch(31, past, new, hk=hk, group=4, dim=dim, block=block)
    table = b.table.cpu().numpy()
    far = table.copy()
    slots, rows = [], []
    for i in range(2):
        total = past[i] + new[i]
        nb = -(-total // block)
        far[i, :nb] = pool - 1 - table[i, :nb]
        pos = np.arange(total)
        slots.append(far[i, pos // block].astype(np.int64) * block + pos % block)
    kk, vv = (torch.from_numpy(np.concatenate(x)).to(torch.bfloat16).cuda() for x in (b.k, b.v))
    m.write_kv(kk, vv, dev(np.concatenate(slots)), kc, vc)
    b.kc, b.vc, b.table = kc, vc, dev(far)
    out, lse = run_paged(b)
    b.check(out, lse, lambda r: range(b.ctx[r]))


SPARSE = [
    # past, new, k, ratio, kwargs
    ([500], [1], 64, 1, {}),
    ([3000, 700, 20], [4, 4, 2], 256, 4, dict(group=8, hk=2)),
    ([1000], [40], 100, 2, dict(group=7, hk=1, block=100, order="head")),
    ([5000], [2], 2048, 1, dict(group=4, hk=2, dim=64, dtype="fp16")),
    ([400, 50], [2, 1], 33, 3, dict(group=33, hk=1, order="interleaved")),
    ([100], [1], 7, 5, dict(group=128, hk=1, dim=64, block=1)),
    ([20000], [1], 2048, 8, dict(group=8, hk=1)),
    ([300], [1], 1, 1, dict(group=1, hk=4)),
    ([600, 40], [58, 2], 96, 4, dict(group=8, hk=4, dim=64)),   # as many tiles as workgroups, about
    ([600, 40], [70, 2], 96, 4, dict(group=8, hk=4, dim=64)),   # some more
]


def sparse_idx(b, k, ratio):
    """Distinct columns per row, unsorted, padding mixed in, some rows short and
    one without any."""
    rng = b.rng
    idx = np.full((b.rows, k), -1, np.int32)
    for r in range(b.rows):
        cols = -(-int(b.ctx[r]) // ratio)
        n = min(k, cols, k if r % 3 else max(1, k // 2))
        if r == 5 or r == 20:
            n = 0
        place = rng.permutation(k)[:n]
        idx[r, place] = rng.permutation(cols)[:n]
        idx[r, idx[r] < 0] = rng.choice([-1, -5, -2 ** 31], int((idx[r] < 0).sum()))
    return idx


def tokens_of(idx_row, ratio, lim):
    t = [c * ratio + j for c in idx_row.tolist() if c >= 0 for j in range(ratio)]
    return [x for x in t if x < lim]


@pytest.mark.parametrize("i", range(len(SPARSE)))
def test_sparse_attention(i):
    past, new, k, ratio, kw = SPARSE[i]
    b = Batch(50 + i, past, new, **kw)
    idx = sparse_idx(b, k, ratio)
    for workspace in ("auto", None):
        lse = torch.empty(b.q.shape[:2], device="cuda")
        out = m.sparse_attention(b.q.cuda(), b.kc, b.vc, b.table, dev(b.req.astype(np.int32)), dev(idx), ratio=ratio,
                                 token_lens=dev(b.ctx), lse=lse, workspace=workspace)
        b.check(out, lse, lambda r: tokens_of(idx[r], ratio, b.ctx[r]))


def test_sparse_attention_edges():
    """Columns past the table and requests outside it, an index given twice, no
    token limit, and a bad table entry among the selected ones."""
    b = Batch(70, [320 - 3], [3], group=4, extra_blocks=0, block=16)
    req = np.zeros(3, np.int32)
    idx = np.array([[5, 5, 17, 10 ** 9, 2 ** 31 - 1], [0, 1, 2, 79, 80], [3, -1, -1, -1, 9]], np.int32)
    q = b.q.cuda()
    lse = torch.empty(b.q.shape[:2], device="cuda")
    out = m.sparse_attention(q, b.kc, b.vc, b.table, dev(req), dev(idx), ratio=4, lse=lse)
    b.check(out, lse, lambda r: tokens_of(idx[r], 4, 320))
    bad = req.copy()
    bad[1] = 7
    table = b.table.clone()
    table[0, 0] = -1  # tokens 0..15: columns 0..3
    out2 = m.sparse_attention(q, b.kc, b.vc, table, dev(bad), dev(idx), ratio=4)
    assert torch.equal(out2[0], out[0])
    assert torch.all(torch.isnan(out2[1])) and torch.all(torch.isnan(out2[2]))
    none = m.sparse_attention(q, b.kc, b.vc, b.table, dev(bad), dev(np.full((3, 4), -1, np.int32)), ratio=4, lse=lse)
    assert torch.all(none == 0) and torch.all(lse == -float("inf"))


def test_attention_refusals():
    """Tensors that do not fit are refused before anything runs."""
    b = Batch(80, [40], [2])
    q, ctx, starts = b.q.cuda(), dev(b.ctx), dev(b.starts)
    idx, req = dev(np.zeros((2, 4), np.int32)), dev(b.req.astype(np.int32))
    call = m.paged_attention
    for bad in (lambda: call(q.float(), b.kc, b.vc, b.table, ctx, starts),
                lambda: call(q, b.kc.half(), b.vc, b.table, ctx, starts),
                lambda: call(q, b.kc, b.vc, b.table, ctx.long(), starts),
                lambda: call(q, b.kc, b.vc, b.table, ctx[:1], starts),
                lambda: call(q, b.kc, b.vc, b.table, ctx, starts[:1]),
                lambda: call(q, b.kc, b.vc[:, :8], b.table, ctx, starts),
                lambda: call(q, b.kc, b.vc, b.table.t(), ctx, starts),
                lambda: call(q[:, :, ::2], b.kc, b.vc, b.table, ctx, starts),
                lambda: call(q[:, :, :64], b.kc, b.vc, b.table, ctx, starts),
                lambda: call(q[:, :3], b.kc, b.vc, b.table, ctx, starts),
                lambda: call(q, b.kc, b.vc, b.table, ctx, starts, scale=0.0),
                lambda: call(q, b.kc, b.vc, b.table, ctx, starts, lse=torch.zeros(2, 8)),
                lambda: call(q, b.kc, b.vc, b.table, ctx, starts, out=torch.zeros_like(q)[:1]),
                lambda: m.sparse_attention(q, b.kc, b.vc, b.table, req, idx.long()),
                lambda: m.sparse_attention(q, b.kc, b.vc, b.table, req, idx, ratio=0),
                lambda: m.sparse_attention(q, b.kc, b.vc, b.table, req[:1], idx)):
        with pytest.raises(m.QsaError):
            bad()


# ---------------------------------------------------------------------------
# a step as a server runs it
# ---------------------------------------------------------------------------

class Step:
    """Plan, cache writes, scoring, selection and attention of one step on fixed
    buffers; index keys are compressed by taking the completing token's key."""

    B, RATIO, HK, GROUP, D, TOPK = 64, 4, 2, 8, 128, 16

    def __init__(self, n=3, rows=14, max_blocks=12, pool=40):
        dt, c = torch.bfloat16, dict(device="cuda")
        self.rows, self.max_blocks, self.pool = rows, max_blocks, pool
        self.past, self.new = (torch.zeros(n, dtype=torch.int32, **c) for _ in range(2))
        self.free = torch.zeros(pool, dtype=torch.int32, **c)
        self.table = torch.full((n, max_blocks), -1, dtype=torch.int32, **c)
        self.kc, self.vc = (torch.full((pool, self.B, self.HK, self.D), float("nan"), dtype=dt, **c)
                            for _ in range(2))
        cols = self.B // self.RATIO
        self.ic = torch.zeros(pool, cols * (self.D + 4), dtype=torch.uint8, **c)
        self.q = torch.zeros(rows, self.HK * self.GROUP, self.D, dtype=dt, **c)
        self.k, self.v = (torch.zeros(rows, self.HK, self.D, dtype=dt, **c) for _ in range(2))
        self.iq = torch.zeros(rows, 32, self.D, dtype=dt, **c)
        self.iq8 = torch.zeros(rows, 32, self.D, dtype=torch.float8_e4m3fn, **c)
        self.plan = m.BatchPlan.empty(n, rows, "cuda")
        self.dense, self.sparse = torch.zeros_like(self.q), torch.zeros_like(self.q)
        self.width = max_blocks * cols
        self.logits = torch.zeros(rows, self.width, **c)
        self.idx = torch.zeros(rows, self.TOPK, dtype=torch.int32, **c)
        self.calls = [
            m.PreparedPlanBatch(self.past, self.new, self.free, self.table, block_size=self.B, num_blocks=pool,
                                out=self.plan, ratio=self.RATIO),
            m.PreparedWriteKv(self.k, self.v, self.plan.slots, self.kc, self.vc),
            m.PreparedWriteKeys(self.k[:, 0], self.plan.col_slots, self.ic, block_size=cols,
                                layout=m.KV_COPACKED_SHUFFLED),
        ]

    def run(self):
        for call in self.calls:
            call()
        cols = self.B // self.RATIO
        m.paged_logits_topk(self.iq8, self.ic, self.table, self.plan.col_lens, self.plan.row_to_req, k=self.TOPK,
                            width=self.width, block_size=cols, layout=m.KV_COPACKED_SHUFFLED, out=self.logits,
                            idx=self.idx)
        m.paged_attention(self.q, self.kc, self.vc, self.table, self.plan.ctx_lens, self.plan.q_starts, out=self.dense)
        m.sparse_attention(self.q, self.kc, self.vc, self.table, self.plan.row_to_req, self.idx, ratio=self.RATIO,
                           token_lens=self.plan.ctx_lens, out=self.sparse)


class Server:
    """Host side of a run of steps: lengths and the free list."""

    def __init__(self, step, seed):
        self.s, self.g = step, torch.Generator().manual_seed(seed)
        self.n = step.table.shape[0]
        self.lens = [0] * self.n
        self.free = torch.randperm(step.pool, generator=self.g).to(torch.int32).tolist()
        self.k, self.v = ([torch.zeros(0, step.HK, step.D, dtype=torch.float64) for _ in range(self.n)]
                          for _ in range(2))

    def load(self, new):
        """Fills the step's buffers for `new` tokens per request."""
        s = self.s
        s.past.copy_(torch.tensor(self.lens, dtype=torch.int32))
        s.new.copy_(torch.tensor(new, dtype=torch.int32))
        s.free[:len(self.free)].copy_(torch.tensor(self.free, dtype=torch.int32))
        for t, gain in ((s.q, 2.0), (s.k, 1.0), (s.v, 1.0)):
            t.copy_(torch.randn(t.shape, generator=self.g).mul(gain))
        s.iq.copy_(torch.randn(s.iq.shape, generator=self.g))
        s.iq8.copy_(s.iq.to(torch.float8_e4m3fn))

    def commit(self, new):
        s, at = self.s, 0
        used = int(s.plan.blocks_used)
        self.free = self.free[used:]
        for i, a in enumerate(new):
            for mine, src in ((self.k, s.k), (self.v, s.v)):
                mine[i] = torch.cat([mine[i], src[at:at + a].double().cpu()])
            self.lens[i] += a
            at += a

    def check(self, new):
        """Both attentions of every row against the definitions, from the host's
        own copy of the keys; the selection is read from the step."""
        s, at, u = self.s, 0, torch.finfo(torch.bfloat16).eps / 2
        idx = s.idx.cpu().numpy()
        assert torch.all(s.plan.ctx_lens[sum(new):] == 0)
        for i, a in enumerate(new):
            for j in range(a):
                r, ctx = at + j, self.lens[i] - a + j + 1
                cols = ctx // s.RATIO
                assert (idx[r] >= 0).sum() == min(s.TOPK, cols) and idx[r].max() < max(cols, 1)
                toks = tokens_of(idx[r], s.RATIO, ctx)
                for h in range(s.HK):
                    hs = slice(h * s.GROUP, (h + 1) * s.GROUP)
                    q = s.q[r, hs].double().cpu().numpy()
                    for got, t in ((s.dense, list(range(ctx))), (s.sparse, toks)):
                        o, l, spread, size = ref.attend(q, self.k[i][t, h].numpy(), self.v[i][t, h].numpy(),
                                                        s.D ** -0.5)
                        tol, _ = ref.bounds(o, l, spread, size, len(t), s.D, u)
                        err = np.abs(got[r, hs].double().cpu().numpy() - o)
                        assert np.all(err <= tol), (i, j, h, len(t))
            at += a


STEPS = [[14, 0, 0], [0, 9, 5], [4, 4, 4], [1, 1, 1], [4, 4, 6], [2, 0, 3], [0, 0, 0], [4, 5, 5]]


def test_serving_steps():
    """A run of steps: prefill, verify and decode rows, requests that pause, a
    step without rows; every step's outputs against the host's own keys."""
    step = Step()
    server = Server(step, 1)
    for new in STEPS * 3:
        server.load(new)
        step.run()
        server.commit(new)
        server.check(new)


def test_selection_with_the_newest_tokens():
    """Selected columns are whole ones; with the column that a row stands in as one
    index more, each row sees its own token, and all tokens while they fit."""
    step = Step()
    server = Server(step, 3)
    for new in STEPS:
        server.load(new)
        step.run()
        ratio, plan = step.RATIO, step.plan
        tail = torch.where(plan.ctx_lens % ratio > 0, plan.col_lens, -1)
        idx = torch.cat([step.idx, tail[:, None]], dim=1)
        out = m.sparse_attention(step.q, step.kc, step.vc, step.table, plan.row_to_req, idx, ratio=ratio,
                                 token_lens=plan.ctx_lens)
        server.commit(new)
        at = 0
        for i, a in enumerate(new):
            for r in range(at, at + a):
                ctx = server.lens[i] - a + r - at + 1
                toks = tokens_of(idx[r], ratio, ctx)
                assert ctx - 1 in toks and len(set(toks)) == len(toks)
                if ctx <= step.TOPK * ratio:
                    assert sorted(toks) == list(range(ctx))
                for h in range(step.HK):
                    hs = slice(h * step.GROUP, (h + 1) * step.GROUP)
                    o, l, spread, size = ref.attend(step.q[r, hs].double().cpu().numpy(), server.k[i][toks, h].numpy(),
                                                    server.v[i][toks, h].numpy(), step.D ** -0.5)
                    tol, _ = ref.bounds(o, l, spread, size, len(toks), step.D, torch.finfo(torch.bfloat16).eps / 2)
                    assert np.all(np.abs(out[r, hs].double().cpu().numpy() - o) <= tol), (i, r, h)
            at += a


def test_serving_steps_captured():
    """The same from one captured graph, replayed with the program's own work
    between the replays."""
    step = Step()
    server = Server(step, 2)
    server.load([1, 1, 1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step.calls = [type(c)(*args, **kw) for c, args, kw in (
            (step.calls[0], (step.past, step.new, step.free, step.table),
             dict(block_size=step.B, num_blocks=step.pool, out=step.plan, ratio=step.RATIO)),
            (step.calls[1], (step.k, step.v, step.plan.slots, step.kc, step.vc), {}),
            (step.calls[2], (step.k[:, 0], step.plan.col_slots, step.ic),
             dict(block_size=step.B // step.RATIO, layout=m.KV_COPACKED_SHUFFLED)))]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step.run()
    torch.cuda.current_stream().wait_stream(side)
    for new in STEPS * 2:
        server.load(new)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        server.commit(new)
        server.check(new)


def test_attention_graphs_side_by_side():
    """Calls with workspaces of their own, captured in graphs of their own and
    replayed on streams of their own, several times, with other work between."""
    batches = [Batch(60, [4000, 900], [3, 2], group=8), Batch(61, [4000, 900], [40, 33], group=8),
               Batch(62, [5000], [1], group=4, dim=64)]
    idx = [sparse_idx(b, 256, 4) for b in batches]
    runs = []
    for b, ix in zip(batches, idx):
        q, ctx, starts, req, sel = b.q.cuda(), dev(b.ctx), dev(b.starts), dev(b.req.astype(np.int32)), dev(ix)
        outs = [torch.zeros_like(q) for _ in range(2)]
        lses = [torch.zeros(q.shape[:2], device="cuda") for _ in range(2)]
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            calls = [m.PreparedPagedAttention(q, b.kc, b.vc, b.table, ctx, starts, outs[0], lse=lses[0]),
                     m.PreparedSparseAttention(q, b.kc, b.vc, b.table, req, sel, outs[1], ratio=4, token_lens=ctx,
                                               lse=lses[1])]
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                for call in calls:
                    call()
        runs.append((b, ix, s, graph, calls, outs, lses, (q, ctx, starts, req, sel)))
    torch.cuda.synchronize()
    want = None
    for _ in range(4):
        for r in runs:
            for t in (*r[5], *r[6]):
                t.fill_(float("nan"))
        torch.cuda.synchronize()
        for _, _, s, graph, *_ in runs:
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for r in runs for t in (*r[5], *r[6])]
        if want is None:
            for b, ix, _, _, _, outs, lses, _ in runs:
                b.check(outs[0], lses[0], lambda r: range(b.ctx[r]))
                b.check(outs[1], lses[1], lambda r: tokens_of(ix[r], 4, b.ctx[r]))
            want = got
        assert all(torch.equal(x, y) for x, y in zip(want, got))
        torch.randn(1000, 1000, device="cuda") @ torch.randn(1000, 1000, device="cuda")


def test_sparse_attention_of_everything_is_dense():
    """With every column selected the two attentions agree to the rounding of
    their weights and outputs."""
    b = Batch(90, [250, 90], [4, 4], group=8)
    idx = np.stack([np.where(np.arange(256) * 1 < b.ctx[r], np.arange(256), -1) for r in range(b.rows)]).astype(np.int32)
    lse_d, lse_s = (torch.empty(b.q.shape[:2], device="cuda") for _ in range(2))
    q, req = b.q.cuda(), dev(b.req.astype(np.int32))
    m.paged_attention(q, b.kc, b.vc, b.table, dev(b.ctx), dev(b.starts), lse=lse_d)
    m.sparse_attention(q, b.kc, b.vc, b.table, req, dev(idx), lse=lse_s)
    assert torch.allclose(lse_d, lse_s, rtol=0, atol=1e-4)


def test_attention_repeats_bit_for_bit():
    b = Batch(91, [3000, 10, 800], [4, 100, 1], group=8)
    first = run_paged(b)
    for _ in range(5):
        again = run_paged(b)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
