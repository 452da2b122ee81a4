"""Measured cases of the serving operators that stand around the indexer.

Four operators, as a decode or prefill step of a sparse-attention server runs
them: the batch plan (block tables, slot maps and visible counts from request
lengths), the cache writes (keys and values, and the indexer's keys), attention
of a chunk of new tokens over the paged cache, and attention of each row over
the tokens that the indexer selected for it.

``run`` computes them in plain torch operations; where ``own`` is true it makes
the library's calls instead.
"""
import math
import random
import zlib

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
DEV = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # MTP verify step: 9 requests with 4 new rows each; a 262,400-token
        # table of 16-token blocks, index columns of 4 tokens
        dict(name="plan_verify", op="plan", reqs=9, rows=36, pad=4, chunked=False, block=16, ratio=4,
             len_lo=64000, len_hi=128000, table=16400),
        # a mixed step: prefill chunks and decode rows share a 16,384-row budget
        dict(name="plan_mixed", op="plan", reqs=257, rows=16384, pad=0, chunked=True, block=64, ratio=4,
             len_lo=1, len_hi=98304, table=1792),
        # the verify step's keys and values enter the cache
        dict(name="write_kv_verify", op="write_kv", rows=36, skipped=4, kv_heads=4, dim=128, dtype="bf16", block=16,
             pool=2048, order="slot"),
        # a prefill chunk's keys and values, head-major cache
        dict(name="write_kv_chunk", op="write_kv", rows=16384, skipped=0, kv_heads=4, dim=128, dtype="fp16", block=64,
             pool=448, order="head"),
        # a prefill chunk's index keys, quantised into preshuffled co-packed blocks
        dict(name="write_keys_chunk", op="write_keys", rows=16384, skipped=0, dim=128, dtype="bf16", block=64,
             pool=512, layout="shuffled"),
        # one decode row of one request: latency
        dict(name="attn_single", op="attn", reqs=1, q_lo=1, q_hi=1, len_lo=4000, len_hi=4000, kv_heads=4, group=8,
             dim=128, dtype="bf16", block=16, order="slot"),
        # the verify step over long caches of mixed lengths: bound by the cache's bytes
        dict(name="attn_verify", op="attn", reqs=9, q_lo=4, q_hi=4, len_lo=16000, len_hi=65600, kv_heads=4, group=8,
             dim=128, dtype="bf16", block=16, order="slot"),
        # a prefill chunk behind a cached prefix: bound by the products
        dict(name="attn_chunk", op="attn", reqs=1, q_lo=2048, q_hi=2048, len_lo=16384, len_hi=16384, kv_heads=4,
             group=8, dim=128, dtype="bf16", block=64, order="slot"),
        # chunks and single rows in one batch, odd sizes throughout
        dict(name="attn_mixed", op="attn", reqs=17, q_lo=1, q_hi=333, len_lo=1, len_hi=5003, kv_heads=2, group=7,
             dim=64, dtype="fp16", block=100, order="head"),
        # one decode row over its selected tokens: latency
        dict(name="sparse_single", op="sparse", reqs=1, q_lo=1, q_hi=1, len_lo=30001, len_hi=30001, kv_heads=8,
             group=4, dim=64, dtype="fp16", block=16, order="slot", k=2048, ratio=1),
        # the verify step over 2,048 selected columns of 4 tokens
        dict(name="sparse_verify", op="sparse", reqs=9, q_lo=4, q_hi=4, len_lo=64000, len_hi=128000, kv_heads=4,
             group=8, dim=128, dtype="bf16", block=16, order="slot", k=2048, ratio=4),
        # a prefill chunk, every row with a selection of its own
        dict(name="sparse_chunk", op="sparse", reqs=1, q_lo=1000, q_hi=1000, len_lo=24000, len_hi=24000, kv_heads=4,
             group=8, dim=128, dtype="bf16", block=64, order="head", k=512, ratio=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "write_kv", "write_keys", "attn", "attn", "attn", "sparse", "sparse"])
    dtype = rng.choice(["bf16", "fp16"])
    order = rng.choice(["slot", "head"])
    block = rng.choice([1, 16, 16, 48, 64, 100, 128])
    dim = rng.choice([64, 128])
    if op == "plan":
        block = rng.choice([16, 32, 64, 128])
        reqs = _log(rng, 1, 257)
        chunked = rng.random() < 0.5
        rows = max(reqs, _log(rng, reqs, 16384)) if chunked else reqs * rng.randint(1, 8)
        hi = _log(rng, 100, 98304)
        return dict(op=op, reqs=reqs, rows=rows, pad=rng.randint(0, 8), chunked=chunked, block=block,
                    ratio=rng.choice([1, 2, 4]), len_lo=1, len_hi=hi, table=-(-(hi + rows) // block))
    if op == "write_kv":
        rows = _log(rng, 1, 16384)
        return dict(op=op, rows=rows, skipped=rng.randint(0, 4), kv_heads=rng.choice([1, 2, 4]), dim=dim, dtype=dtype,
                    block=block, pool=-(-rows // block) + rng.randint(8, 256), order=order)
    if op == "write_keys":
        rows = _log(rng, 1, 16384)
        block = rng.choice([16, 48, 64, 128])
        return dict(op=op, rows=rows, skipped=rng.randint(0, 4), dim=dim, dtype=dtype, block=block,
                    pool=-(-rows // block) + rng.randint(8, 128),
                    layout=rng.choice(["plain", "paged", "copacked", "shuffled"]))
    kv_heads = rng.choice([1, 2, 4])
    group = rng.choice([1, 3, 4, 7, 8])
    if op == "attn":
        shape = rng.choice(["decode", "chunk", "mixed"])
        if shape == "decode":
            reqs, q = _log(rng, 1, 32), rng.randint(1, 8)
            hi = _log(rng, 100, 65600 if reqs <= 9 else 16000)
            return dict(op=op, reqs=reqs, q_lo=1, q_hi=q, len_lo=max(q, hi // 4), len_hi=hi, kv_heads=kv_heads,
                        group=group, dim=dim, dtype=dtype, block=block, order=order)
        if shape == "chunk":
            q = _log(rng, 64, 2048)
            n = q + _log(rng, 1, 14000)
            return dict(op=op, reqs=1, q_lo=q, q_hi=q, len_lo=n, len_hi=n, kv_heads=kv_heads, group=group, dim=dim,
                        dtype=dtype, block=block, order=order)
        q = _log(rng, 16, 333)
        return dict(op=op, reqs=rng.randint(2, 17), q_lo=1, q_hi=q, len_lo=1, len_hi=q + _log(rng, 100, 5000),
                    kv_heads=kv_heads, group=group, dim=dim, dtype=dtype, block=block, order=order)
    reqs, q = rng.choice([(1, _log(rng, 1, 1000)), (_log(rng, 1, 16), rng.randint(1, 4))])
    k, ratio = rng.choice([64, 511, 512, 1024]), rng.choice([1, 2, 4])
    if reqs * q <= 64:
        k = rng.choice([k, 2048])
    elif k * ratio > 2048:
        ratio = 1
    n = max(q, _log(rng, 200, 64000))
    return dict(op=op, reqs=reqs, q_lo=1 if reqs > 1 else q, q_hi=q, len_lo=max(q, n // 2), len_hi=n,
                kv_heads=kv_heads, group=group, dim=dim, dtype=dtype, block=block, order=order, k=k, ratio=ratio)


def _lengths(case):
    """(past, new) tokens of each request: fixed by the case alone."""
    rng = random.Random(zlib.crc32(repr(sorted((k, v) for k, v in case.items() if k != "name")).encode()))
    n = case["reqs"]
    if case["op"] == "plan":
        total = [_log(rng, case["len_lo"], case["len_hi"]) for _ in range(n)]
        if not case["chunked"]:
            return total, [case["rows"] // n] * n
        # a few chunks take most of the budget, the other requests one row each
        left, new = case["rows"] - n, [1] * n
        chunks = max(1, n // 16)
        for i in rng.sample(range(n), chunks):
            new[i] += left // chunks
        return total, new
    new = [rng.randint(case["q_lo"], case["q_hi"]) for _ in range(n)]
    total = [max(a, _log(rng, case["len_lo"], case["len_hi"])) for a in new]
    return [t - a for t, a in zip(total, new)], new


def _starts(new):
    s = [0]
    for a in new:
        s.append(s[-1] + a)
    return s


def work(case):
    op = case["op"]
    if op == "plan":
        past, new = _lengths(case)
        rows = case["rows"] + case["pad"]
        fresh = sum(-(-(p + a) // case["block"]) - -(-p // case["block"]) for p, a in zip(past, new))
        # lengths and starts of a request; a row's table entry and its five
        # outputs; a new block's list entry and table entry
        return dict(bytes=12 * case["reqs"] + 32 * rows + 8 * fresh, flops=0)
    if op == "write_kv":
        return dict(bytes=case["rows"] * (8 + 2 * 2 * 2 * case["kv_heads"] * case["dim"]), flops=0)
    if op == "write_keys":
        out = 2 * case["dim"] if case["layout"] == "plain" else case["dim"] + 4
        return dict(bytes=case["rows"] * (8 + 2 * case["dim"] + out), flops=0)
    past, new = _lengths(case)
    heads, d = case["kv_heads"] * case["group"], case["dim"]
    rows = sum(new)
    qo = 2 * 2 * rows * heads * d + 4 * rows * heads
    if op == "attn":
        keys = sum(p + a for p, a in zip(past, new))
        pairs = sum(a * p + a * (a + 1) // 2 for p, a in zip(past, new))
        return dict(bytes=qo + 2 * 2 * keys * case["kv_heads"] * d, flops=4 * pairs * heads * d)
    tokens, seen = 0, 0
    for p, a in zip(past, new):
        per = [min(case["k"] * case["ratio"], p + j + 1) for j in range(a)]
        tokens += sum(per)
        seen += min(p + a, sum(per))  # a request's cache is read once at most
    return dict(bytes=qo + 4 * rows * case["k"] + 2 * 2 * seen * case["kv_heads"] * d, flops=4 * tokens * heads * d)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _cache(pool, case, g):
    """A [pool, block, kv_heads, dim] cache, stored slot-major or head-major."""
    b, h, d = case["block"], case["kv_heads"], case["dim"]
    shape = (pool, b, h, d) if case["order"] == "slot" else (pool, h, b, d)
    c = torch.randn(shape, generator=g, device=DEV, dtype=DTYPES[case["dtype"]])
    return c if case["order"] == "slot" else c.transpose(1, 2)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    if op == "plan":
        past, new = _lengths(case)
        n, b = case["reqs"], case["block"]
        have = [-(-p // b) for p in past]
        fresh = sum(-(-(p + a) // b) for p, a in zip(past, new)) - sum(have)
        pool = sum(have) + fresh + 64
        ids = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)
        e = torch.arange(case["table"], device=DEV)
        base = torch.tensor(_starts(have)[:-1], device=DEV)
        held = e[None, :] < torch.tensor(have, device=DEV)[:, None]
        table = torch.where(held, ids[(base[:, None] + e[None, :]).clamp(max=pool - 1)], -1).contiguous()
        rows = case["rows"] + case["pad"]
        empty = lambda m, t: torch.empty(m, dtype=t, device=DEV)  # noqa: E731
        return dict(case=case, past=_i32(past), new=_i32(new), free=ids[sum(have):].contiguous(), table=table,
                    pool=pool, rows=rows, q_starts=empty(n + 1, torch.int32), row_to_req=empty(rows, torch.int32),
                    ctx_lens=empty(rows, torch.int32), slots=empty(rows, torch.int64),
                    col_lens=empty(rows, torch.int32), col_slots=empty(rows, torch.int64),
                    used=empty(1, torch.int32))
    if op in ("write_kv", "write_keys"):
        rows, b, pool = case["rows"], case["block"], case["pool"]
        slots = torch.randperm(pool * b, generator=g, device=DEV)[:rows].clone()
        if case["skipped"]:  # rows of a padded batch that write nothing
            slots[max(0, rows - case["skipped"]):] = -1
        if op == "write_kv":
            src = torch.randn((2, rows, case["kv_heads"], case["dim"]), generator=g, device=DEV,
                              dtype=DTYPES[case["dtype"]])
            # one block more than the operator is told of: the plain form's place for skipped rows
            kc, vc = (_cache(pool + 1, case, g) for _ in range(2))
            return dict(case=case, k=src[0], v=src[1], slots=slots, kc=kc, vc=vc)
        keys = torch.randn((rows, case["dim"]), generator=g, device=DEV, dtype=DTYPES[case["dtype"]])
        if case["layout"] == "plain":
            store = torch.zeros((pool + 1, b, case["dim"]), device=DEV, dtype=DTYPES[case["dtype"]])
            return dict(case=case, keys=keys, slots=slots, store=store)
        if case["layout"] == "paged":
            store = torch.zeros((pool + 1, b, case["dim"]), device=DEV, dtype=torch.uint8)
            return dict(case=case, keys=keys, slots=slots, store=store,
                        scale=torch.zeros((pool + 1, b), device=DEV))
        store = torch.zeros((pool + 1, b * (case["dim"] + 4)), device=DEV, dtype=torch.uint8)
        return dict(case=case, keys=keys, slots=slots, store=store)
    past, new = _lengths(case)
    n, b = case["reqs"], case["block"]
    total = [p + a for p, a in zip(past, new)]
    blocks = [-(-t // b) for t in total]
    pool, width = sum(blocks) + 3, max(blocks) + 2
    ids = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)
    e = torch.arange(width, device=DEV)
    base = torch.tensor(_starts(blocks)[:-1], device=DEV)
    held = e[None, :] < torch.tensor(blocks, device=DEV)[:, None]
    table = torch.where(held, ids[(base[:, None] + e[None, :]).clamp(max=pool - 1)], -1).contiguous()
    rows, heads = sum(new), case["kv_heads"] * case["group"]
    starts = _i32(_starts(new))
    r = torch.arange(rows, device=DEV)
    req = torch.searchsorted(starts[1:].long(), r, right=True)
    ctx = (torch.tensor(past, device=DEV)[req] + r - starts[req] + 1).to(torch.int32)
    q = torch.randn((rows, heads, case["dim"]), generator=g, device=DEV) * 2.0
    state = dict(case=case, q=q.to(DTYPES[case["dtype"]]), kc=_cache(pool, case, g), vc=_cache(pool, case, g),
                 table=table, starts=starts, row_to_req=req.to(torch.int32), ctx=ctx, most=max(total),
                 most_q=max(new), out=torch.zeros((rows, heads, case["dim"]), device=DEV, dtype=DTYPES[case["dtype"]]),
                 lse=torch.zeros((rows, heads), device=DEV))
    if op == "sparse":
        # neighbouring rows select alike: scores of their request plus their own
        ratio, k = case["ratio"], case["k"]
        cols = -(-max(total) // ratio)
        score = torch.randn((n, cols), generator=g, device=DEV)[req]
        score = score + torch.randn((rows, cols), generator=g, device=DEV)
        vis = (ctx.long() + ratio - 1) // ratio
        score.masked_fill_(torch.arange(cols, device=DEV)[None, :] >= vis[:, None], -math.inf)
        top = torch.topk(score, min(k, cols), dim=1)
        idx = torch.where(top.values > -math.inf, top.indices, cols).sort(dim=1).values
        idx = torch.where(idx < cols, idx, -1).to(torch.int32)
        state["idx"] = torch.nn.functional.pad(idx, (0, k - idx.shape[1]), value=-1).contiguous()
    return state


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _plan_plain(s):
    c = s["case"]
    b, ratio, table = c["block"], c["ratio"], s["table"]
    n, width = table.shape
    past, new = s["past"].long(), s["new"].long()
    ends = torch.cumsum(new, 0)
    starts = torch.cat([torch.zeros_like(ends[:1]), ends])
    have, want = (past + b - 1) // b, (past + new + b - 1) // b
    taken = torch.cumsum(want - have, 0)
    base = taken - (want - have)
    e = torch.arange(width, device=DEV)[None, :]
    at = (base[:, None] + e - have[:, None]).clamp(0, s["free"].numel() - 1)
    table.copy_(torch.where((e >= have[:, None]) & (e < want[:, None]), s["free"][at], table))
    r = torch.arange(s["rows"], device=DEV)
    live = r < ends[-1]
    req = torch.searchsorted(ends, r, right=True).clamp(max=n - 1)
    pos = past[req] + r - starts[req]
    block = table[req, (pos // b).clamp(0, width - 1)].long()
    slot = block * b + pos % b
    col = block * (b // ratio) + pos % b // ratio
    last = live & ((pos + 1) % ratio == 0)
    return dict(table=table, q_starts=starts.to(torch.int32),
                row_to_req=torch.where(live, req, 0).to(torch.int32),
                ctx_lens=torch.where(live, pos + 1, 0).to(torch.int32), slots=torch.where(live, slot, -1),
                col_lens=torch.where(live, (pos + 1) // ratio, 0).to(torch.int32),
                col_slots=torch.where(last, col, -1), used=taken[-1:].to(torch.int32))


def _write_kv_plain(s):
    b, pool = s["case"]["block"], s["case"]["pool"]
    at = torch.where(s["slots"] >= 0, s["slots"], pool * b)
    s["kc"][at // b, at % b] = s["k"]
    s["vc"][at // b, at % b] = s["v"]
    return s["kc"][:pool], s["vc"][:pool]


def _keys_views(s):
    """The stored keys as [pool, block, dim] e4m3 values in the layout's own
    order, and their scales [pool, block]."""
    c, store = s["case"], s["store"]
    b, d = c["block"], c["dim"]
    if c["layout"] == "paged":
        return store.view(torch.float8_e4m3fn), s["scale"]
    keys = store[:, :b * d].view(torch.float8_e4m3fn)
    if c["layout"] == "copacked":
        keys = keys.unflatten(1, (b, d))
    else:  # 16 slots as dim / 16 chunks of 16 slots x 16 bytes
        keys = keys.unflatten(1, (b // 16, d // 16, 16, 16))
    return keys, store[:, b * d:].view(torch.float32)


def _write_keys_plain(s):
    c = s["case"]
    b, d, pool = c["block"], c["dim"], c["pool"]
    at = torch.where(s["slots"] >= 0, s["slots"], pool * b)
    if c["layout"] == "plain":
        s["store"][at // b, at % b] = s["keys"]
        return s["store"][:pool]
    x = s["keys"].float()
    top = x.abs().amax(dim=1)
    scale = torch.where(top > 0, top / 448.0, 1.0)
    code = (x / scale[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    keys, scales = _keys_views(s)
    raw = keys.view(torch.uint8)
    if c["layout"] == "shuffled":
        raw[at // b, at % b // 16, :, at % 16] = code.view(-1, d // 16, 16)
    else:
        raw[at // b, at % b] = code
    scales[at // b, at % b] = scale
    return keys[:pool], scales[:pool]


def _softmax(score, seen):
    """Weights and log-sum-exp of each row's seen scores; a row that sees
    nothing has zero weights."""
    score = torch.where(seen, score, -math.inf)
    top = score.amax(dim=-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    p = torch.exp(score - top)
    total = p.sum(dim=-1, keepdim=True)
    return p / total.clamp(min=1e-37), (top + torch.log(total)).squeeze(-1)


def _attn_plain(s):
    c = s["case"]
    n, hk, grp, d, b = c["reqs"], c["kv_heads"], c["group"], c["dim"], c["block"]
    rows, most, mq = s["q"].shape[0], s["most"], s["most_q"]
    t = torch.arange(most, device=DEV)
    block = s["table"][:, t // b].long().clamp(min=0)  # a request's places behind its end are masked
    k = s["kc"][block, t % b].float().permute(0, 2, 3, 1).reshape(n * hk, d, most)
    v = s["vc"][block, t % b].float().permute(0, 2, 1, 3).reshape(n * hk, most, d)
    starts = s["starts"].long()
    j = torch.arange(mq, device=DEV)[None, :]
    row = (starts[:-1, None] + j).clamp(max=rows - 1)
    live = starts[:-1, None] + j < starts[1:, None]
    ctx = torch.where(live, s["ctx"][row].long(), 0)
    q = s["q"][row].float().view(n, mq, hk, grp, d).permute(0, 2, 1, 3, 4).reshape(n * hk, mq * grp, d)
    score = torch.bmm(q, k).mul_(d ** -0.5).view(n, hk, mq, grp, most)
    p, lse = _softmax(score, t < ctx[:, None, :, None, None])
    o = torch.bmm(p.view(n * hk, mq * grp, most), v).view(n, hk, mq, grp, d)
    r = torch.arange(rows, device=DEV)
    req = s["row_to_req"].long()
    at = r - starts[req]
    out = o.permute(0, 2, 1, 3, 4)[req, at].reshape(rows, hk * grp, d)
    return out.to(s["q"].dtype), lse.permute(0, 2, 1, 3)[req, at].reshape(rows, hk * grp)


def _sparse_plain(s):
    c = s["case"]
    hk, grp, d, b, ratio = c["kv_heads"], c["group"], c["dim"], c["block"], c["ratio"]
    rows = s["q"].shape[0]
    idx = s["idx"].long()
    tok = (idx[:, :, None] * ratio + torch.arange(ratio, device=DEV)).flatten(1)
    seen = (tok >= 0) & (tok < s["ctx"][:, None])
    tok = torch.where(seen, tok, 0)
    block = s["table"][s["row_to_req"].long()[:, None], tok // b].long()
    k = s["kc"][block, tok % b].float().permute(0, 2, 3, 1).reshape(rows * hk, d, -1)
    v = s["vc"][block, tok % b].float().permute(0, 2, 1, 3).reshape(rows * hk, -1, d)
    q = s["q"].float().view(rows * hk, grp, d)
    score = torch.bmm(q, k).mul_(d ** -0.5).view(rows, hk, grp, -1)
    p, lse = _softmax(score, seen[:, None, None, :])
    o = torch.bmm(p.view(rows * hk, grp, -1), v)
    return o.reshape(rows, hk * grp, d).to(s["q"].dtype), lse.reshape(rows, hk * grp)


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------

def _prepared(s):
    """The checked call that a serving loop keeps for its buffers."""
    import paged_mqa_logits_block_amd as m

    c = s["case"]
    if c["op"] == "plan":
        return m.PreparedPlanBatch(
            s["past"], s["new"], s["free"], s["table"], block_size=c["block"], num_blocks=s["pool"], ratio=c["ratio"],
            out=m.BatchPlan(q_starts=s["q_starts"], row_to_req=s["row_to_req"], ctx_lens=s["ctx_lens"],
                            slots=s["slots"], col_lens=s["col_lens"], col_slots=s["col_slots"],
                            blocks_used=s["used"]))
    if c["op"] == "write_kv":
        return m.PreparedWriteKv(s["k"], s["v"], s["slots"], s["kc"][:c["pool"]], s["vc"][:c["pool"]])
    if c["op"] == "write_keys":
        layout = {"plain": m.KV_PAGED, "paged": m.KV_PAGED, "copacked": m.KV_COPACKED,
                  "shuffled": m.KV_COPACKED_SHUFFLED}[c["layout"]]
        return m.PreparedWriteKeys(s["keys"], s["slots"], s["store"][:c["pool"]], block_size=c["block"],
                                   kscale=s["scale"][:c["pool"]] if "scale" in s else None, layout=layout)
    if c["op"] == "attn":
        return m.PreparedPagedAttention(s["q"], s["kc"], s["vc"], s["table"], s["ctx"], s["starts"], s["out"],
                                        lse=s["lse"])
    return m.PreparedSparseAttention(s["q"], s["kc"], s["vc"], s["table"], s["row_to_req"], s["idx"], s["out"],
                                     ratio=c["ratio"], token_lens=s["ctx"], lse=s["lse"])


def _run_own(s):
    call = s.get("call")
    if call is None:
        call = s["call"] = _prepared(s)
    call()
    c = s["case"]
    if c["op"] == "plan":
        return {k: s[k] for k in ("table", "q_starts", "row_to_req", "ctx_lens", "slots", "col_lens", "col_slots",
                                  "used")}
    if c["op"] == "write_kv":
        return s["kc"][:c["pool"]], s["vc"][:c["pool"]]
    if c["op"] == "write_keys":
        if c["layout"] == "plain":
            return s["store"][:c["pool"]]
        keys, scales = _keys_views(s)
        return keys[:c["pool"]], scales[:c["pool"]]
    return s["out"], s["lse"]


def run(state):
    if own:
        return _run_own(state)
    return {"plan": _plan_plain, "write_kv": _write_kv_plain, "write_keys": _write_keys_plain, "attn": _attn_plain,
            "sparse": _sparse_plain}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# in 64 bits, from the definitions
# ---------------------------------------------------------------------------

def _attend(q, k, v, counts):
    """softmax(q k^T / sqrt(d)) v of [rows, group, d] queries over [keys, d], row
    r over its first counts[r] keys, in float64."""
    rows, grp, d = q.shape
    z = torch.matmul(q.reshape(rows * grp, d), k.t()).view(rows, grp, -1) / math.sqrt(d)
    z.masked_fill_((torch.arange(k.shape[0], device=DEV)[None, :] >= counts[:, None])[:, None, :], -math.inf)
    lse = torch.logsumexp(z, dim=-1)
    return torch.matmul(torch.exp(z - lse[..., None]).view(rows * grp, -1), v).view(rows, grp, d), lse


def exact(case, seed):
    op = case["op"]
    if op == "plan":
        return None  # whole numbers only
    s = prepare(case, seed)
    if op == "write_kv":
        keep = s["slots"] >= 0
        at = s["slots"][keep]
        both = []
        for cache, rows in ((s["kc"], s["k"]), (s["vc"], s["v"])):
            flat = cache[:case["pool"]].double().reshape(-1, case["kv_heads"], case["dim"])
            flat[at] = rows.double()[keep]
            both.append(flat.view(case["pool"], case["block"], case["kv_heads"], case["dim"]))
        return tuple(both)
    if op == "write_keys":
        if case["layout"] == "plain":
            return None
        b, d, pool = case["block"], case["dim"], case["pool"]
        keys = torch.zeros((pool, b, d), dtype=torch.float64, device=DEV)
        scales = torch.zeros((pool, b), dtype=torch.float64, device=DEV)
        keep = s["slots"] >= 0
        x, at = s["keys"].double()[keep], s["slots"][keep]
        unit = x.abs().max(dim=1).values / 448.0
        unit = torch.where(unit > 0, unit, torch.ones_like(unit))
        keys.view(-1, d)[at] = x / unit[:, None]
        scales.view(-1)[at] = unit
        if case["layout"] == "shuffled":
            keys = keys.view(pool, b // 16, 16, d // 16, 16).transpose(2, 3).contiguous()
        return keys, scales
    past, new = _lengths(case)
    hk, grp, d, b = case["kv_heads"], case["group"], case["dim"], case["block"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    r0 = 0
    for i, (p, a) in enumerate(zip(past, new)):
        pos = torch.arange(p + a, device=DEV)
        where = s["table"][i].long()[pos // b]
        for h in range(hk):
            at = slice(h * grp, h * grp + grp)
            k, v = (s[x][where, pos % b, h].double() for x in ("kc", "vc"))
            q = s["q"][r0:r0 + a, at].double()
            if op == "attn":
                for j in range(0, a, 256):
                    e = min(a, j + 256)
                    counts = torch.arange(p + j + 1, p + e + 1, device=DEV)
                    out[r0 + j:r0 + e, at], lse[r0 + j:r0 + e, at] = _attend(q[j:e], k, v, counts)
                continue
            for j in range(a):
                cols = s["idx"][r0 + j].long()
                cols = cols[cols >= 0]
                toks = (cols[:, None] * case["ratio"] + torch.arange(case["ratio"], device=DEV)).reshape(-1)
                toks = toks[toks <= p + j]
                out[r0 + j, at], lse[r0 + j, at] = (
                    y[0] for y in _attend(q[j:j + 1], k[toks], v[toks], torch.tensor([toks.numel()], device=DEV)))
        r0 += a
    return out, lse
