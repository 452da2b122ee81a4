"""Measured cases of further serving operators, around attention and drafts.

Three operators, as one step of a server with windowed layers and drafted tokens
runs them: the norm of queries and keys with their rotary positions (keys and
values going straight into the paged cache), attention over a sliding window and
the first tokens, and the verification of drafted tokens from given random
numbers.

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
        # one decode row on its way into the cache: latency
        dict(name="rope_single", op="rope", rows=1, pad=0, kv_heads=4, group=8, dim=128, rot=128, offset=0,
             style="half", norm=True, dtype="bf16", block=16, order="slot", cache=True, scaling="none", last=30001),
        # a verify step's 36 rows and 4 rows of padding, far positions with stretched frequencies
        dict(name="rope_verify", op="rope", rows=36, pad=4, kv_heads=4, group=8, dim=128, rot=64, offset=64,
             style="interleaved", norm=True, dtype="bf16", block=16, order="slot", cache=True, scaling="bands",
             last=128000),
        # heads of an odd number of rows rotated out of one projection, without a norm or a cache
        dict(name="rope_odd", op="rope", rows=1001, pad=0, kv_heads=2, group=7, dim=64, rot=32, offset=0,
             style="half", norm=False, dtype="fp16", block=100, order="head", cache=False, scaling="linear",
             last=5003),
        # a prefill chunk: bound by bytes
        dict(name="rope_chunk", op="rope", rows=16384, pad=0, kv_heads=4, group=8, dim=128, rot=128, offset=0,
             style="half", norm=True, dtype="bf16", block=64, order="head", cache=True, scaling="none", last=98304),
        # one decode row of one request: latency
        dict(name="window_single", op="window", reqs=1, q_lo=1, q_hi=1, len_lo=30001, len_hi=30001, window=4096,
             sinks=4, kv_heads=4, group=8, dim=128, dtype="bf16", block=16, order="slot"),
        # a verify step at the end of long requests
        dict(name="window_verify", op="window", reqs=9, q_lo=4, q_hi=4, len_lo=64000, len_hi=128000, window=4096,
             sinks=4, kv_heads=4, group=8, dim=128, dtype="bf16", block=16, order="slot"),
        # many decode rows over short windows: bound by the cache's bytes
        dict(name="window_decode", op="window", reqs=257, q_lo=1, q_hi=1, len_lo=100, len_hi=16000, window=1024,
             sinks=16, kv_heads=4, group=8, dim=128, dtype="fp16", block=64, order="head"),
        # chunks and single rows in one batch, odd sizes throughout
        dict(name="window_mixed", op="window", reqs=17, q_lo=1, q_hi=333, len_lo=1, len_hi=5003, window=777, sinks=5,
             kv_heads=2, group=7, dim=64, dtype="fp16", block=100, order="head"),
        # a prefill chunk behind a cached prefix: bound by the products
        dict(name="window_chunk", op="window", reqs=1, q_lo=2048, q_hi=2048, len_lo=16384, len_hi=16384, window=4096,
             sinks=64, kv_heads=4, group=8, dim=128, dtype="bf16", block=64, order="slot"),
        # one request's drafts of a drafter without probabilities (a lookup), an odd vocabulary: latency
        dict(name="verify_single", op="verify", reqs=1, r_lo=5, r_hi=5, vocab=50021, probs=False),
        # a verify step: 9 requests of 3 drafts
        dict(name="verify_step", op="verify", reqs=9, r_lo=4, r_hi=4, vocab=131072, probs=True),
        # a full batch with 0 to 7 drafts each, rows that start off 16-byte boundaries
        dict(name="verify_many", op="verify", reqs=257, r_lo=1, r_hi=8, vocab=100003, probs=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "window", "window", "window", "verify", "verify"])
    if op == "verify":
        # up to as much probability as the largest listed case holds
        reqs, hi = _log(rng, 1, 257), rng.randint(1, 8)
        vocab = min(_log(rng, 1000, 131072), 115_000_000 // (reqs * hi))
        return dict(op=op, reqs=reqs, r_lo=rng.randint(1, hi), r_hi=hi, vocab=vocab, probs=rng.random() < 0.7)
    dtype, order = rng.choice(["bf16", "fp16"]), rng.choice(["slot", "head"])
    block = rng.choice([1, 16, 16, 48, 64, 100, 128])
    dim, kv_heads, group = rng.choice([64, 128]), rng.choice([1, 2, 4]), rng.choice([1, 3, 4, 7, 8])
    if op == "rope":
        rot = 16 * rng.randint(1, dim // 16)
        rows = _log(rng, 1, 16384)
        return dict(op=op, rows=rows, pad=rng.randint(0, 8), kv_heads=kv_heads, group=group, dim=dim, rot=rot,
                    offset=8 * rng.randint(0, (dim - rot) // 8), style=rng.choice(["half", "interleaved"]),
                    norm=rng.random() < 0.6, dtype=dtype, block=block, order=order, cache=rng.random() < 0.7,
                    scaling=rng.choice(["none", "linear", "bands"]), last=rows + _log(rng, 1, 1_000_000))
    sinks = rng.choice([0, 1, 4, 5, 16, 64, 100])
    shape = rng.choice(["decode", "chunk", "mixed"])
    if shape == "decode":
        reqs, q = _log(rng, 1, 257), rng.randint(1, 8)
        window = _log(rng, 16, max(16, min(8192, 200_000 // (reqs * max(1, q // 4)))))
        hi = _log(rng, 100, 128000)
        return dict(op=op, reqs=reqs, q_lo=1, q_hi=q, len_lo=max(q, hi // 4), len_hi=max(q, hi), window=window,
                    sinks=sinks, kv_heads=kv_heads, group=group, dim=dim, dtype=dtype, block=block, order=order)
    window = _log(rng, 16, 4096)
    if shape == "chunk":
        q = _log(rng, 64, 2048)
        n = q + _log(rng, 1, 14000)
        return dict(op=op, reqs=1, q_lo=q, q_hi=q, len_lo=n, len_hi=n, window=window, sinks=min(sinks, 64),
                    kv_heads=kv_heads, group=group, dim=dim, dtype=dtype, block=block, order=order)
    q = _log(rng, 16, 333)
    return dict(op=op, reqs=rng.randint(2, 17), q_lo=1, q_hi=q, len_lo=1, len_hi=q + _log(rng, 100, 5000),
                window=window, sinks=sinks, kv_heads=kv_heads, group=group, dim=dim, dtype=dtype, block=block,
                order=order)


def _case_rng(case):
    """Random numbers fixed by the case alone."""
    return random.Random(zlib.crc32(repr(sorted((k, v) for k, v in case.items() if k != "name")).encode()))


def _lengths(case):
    """(past, new) tokens of each request of a window case."""
    rng = _case_rng(case)
    new = [rng.randint(case["q_lo"], case["q_hi"]) for _ in range(case["reqs"])]
    total = [max(a, _log(rng, case["len_lo"], case["len_hi"])) for a in new]
    return [t - a for t, a in zip(total, new)], new


def _kept(case):
    """(rows, accepted drafts) of each request of a verify case: a draft is kept
    with probability 0.7 where all before it are."""
    rng = _case_rng(case)
    rows = [rng.randint(case["r_lo"], case["r_hi"]) for _ in range(case["reqs"])]
    kept = []
    for m in rows:
        a = 0
        while a < m - 1 and rng.random() < 0.7:
            a += 1
        kept.append(a)
    return rows, kept


def _starts(new):
    s = [0]
    for a in new:
        s.append(s[-1] + a)
    return s


def work(case):
    op = case["op"]
    if op == "rope":
        heads, elt = case["kv_heads"] * case["group"], 2
        # q in and out, keys in and out, with a cache values too; position and slot; frequencies, weights
        per = 2 * heads + 2 * case["kv_heads"] * (2 if case["cache"] else 1)
        extra = 4 + (8 if case["cache"] else 0)
        return dict(bytes=case["rows"] * (per * case["dim"] * elt + extra) + 4 * case["rot"] +
                    (8 * case["dim"] if case["norm"] else 0),
                    flops=case["rows"] * (heads + case["kv_heads"]) * (3 * case["rot"] + (4 * case["dim"] if case["norm"] else 0)))
    if op == "verify":
        rows, kept = _kept(case)
        v = case["vocab"]
        total = 0
        for m, a in zip(rows, kept):
            total += 4 * v + 20 * min(m - 1, a + 1) + 4 * (a + 2)
            if case["probs"] and a < m - 1:  # the drafter's row is needed where a draft is rejected
                total += 4 * v
        return dict(bytes=total, flops=0)
    past, new = _lengths(case)
    heads, d, w, s = case["kv_heads"] * case["group"], case["dim"], case["window"], case["sinks"]
    rows, keys, pairs = sum(new), 0, 0
    for p, a in zip(past, new):
        first = max(0, p + 1 - w)  # the oldest token of the first row's window
        keys += p + a - first + min(s, first)
        for c in range(p + 1, p + a + 1):
            pairs += min(c, w) + min(s, max(0, c - w))
    return dict(bytes=2 * 2 * rows * heads * d + 4 * rows * heads + 2 * 2 * keys * case["kv_heads"] * d,
                flops=4 * pairs * heads * d)


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


def _frequencies(case):
    """Radians per position of each rotated pair (64 bits), and the factor on cos and
    sin.  "linear": positions stretched by 8; "bands": pairs that turn less than once in
    4,096 positions stretched by 8, those that turn 32 times kept, a ramp between."""
    rot = case["rot"]
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    if case["scaling"] == "none":
        return f, 1.0
    if case["scaling"] == "linear":
        return f / 8.0, 1.0
    turns = 4096.0 * f / (2.0 * math.pi)
    keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
    return f * keep + f / 8.0 * (1.0 - keep), 0.1 * math.log(8.0) + 1.0


def _rope_inputs(case, g):
    rows, hk, d = case["rows"], case["kv_heads"], case["dim"]
    hq, dt = hk * case["group"], DTYPES[case["dtype"]]
    n = rows + case["pad"]
    qkv = (torch.randn((n, hq + 2 * hk, d), generator=g, device=DEV) * 1.5).to(dt)
    # several requests' runs of neighbouring positions; visible counts, one more than the position
    rng = _case_rng(case)
    ctx, left = [], rows
    while left:
        run = min(left, rng.choice([1, 4, rows]))
        end = rng.randint(run, max(run, case["last"]))
        ctx += range(end - run + 1, end + 1)
        left -= run
    ctx += [0] * case["pad"]  # rows of a padded batch have no position
    freq, factor = _frequencies(case)
    s = dict(case=case, q=qkv[:, :hq], k=qkv[:, hq:hq + hk], v=qkv[:, hq + hk:], ctx=_i32(ctx), freq=freq,
             factor=factor, q_weight=None, k_weight=None, eps=1e-6,
             q_out=torch.zeros((n, hq, d), device=DEV, dtype=dt), k_out=None)
    if case["norm"]:
        s["q_weight"], s["k_weight"] = (1.0 + 0.2 * torch.randn(d, generator=g, device=DEV) for _ in range(2))
    if case["cache"]:
        pool = -(-rows // case["block"]) + 8
        # one block more than the operator is told of: the plain form's place for padded rows
        s["kc"], s["vc"] = (_cache(pool + 1, case, g) for _ in range(2))
        slots = torch.randperm(pool * case["block"], generator=g, device=DEV)[:n].clone()
        slots = torch.nn.functional.pad(slots, (0, n - slots.numel()), value=-1)
        slots[rows:] = -1
        s["slots"], s["pool"] = slots, pool
    else:
        s["k_out"] = torch.zeros((n, hk, d), device=DEV, dtype=dt)
    return s


def _window_inputs(case, g):
    past, new = _lengths(case)
    n, b = case["reqs"], case["block"]
    total = [p + a for p, a in zip(past, new)]
    width = -(-max(total) // b) + 2
    # blocks that no row sees any more have been freed: entries of -1
    held = torch.zeros((n, width), dtype=torch.bool)
    for i, (p, a) in enumerate(zip(past, new)):
        first = max(0, p + 1 - case["window"])
        held[i, first // b:-(-(p + a) // b)] = True
        if case["sinks"]:
            held[i, :-(-min(case["sinks"], p + a) // b)] = True
    held = held.to(DEV)
    pool = int(held.sum()) + 3
    ids = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)
    at = torch.cumsum(held.flatten().long(), 0).view(n, width) - 1
    table = torch.where(held, ids[at.clamp(min=0)], -1).contiguous()
    rows, heads = sum(new), case["kv_heads"] * case["group"]
    starts = _i32(_starts(new))
    r = torch.arange(rows, device=DEV)
    req = torch.searchsorted(starts[1:].long(), r, right=True)
    ctx = (torch.tensor(past, device=DEV)[req] + r - starts[req] + 1).to(torch.int32)
    q = torch.randn((rows, heads, case["dim"]), generator=g, device=DEV) * 2.0
    dt = DTYPES[case["dtype"]]
    return dict(case=case, q=q.to(dt), kc=_cache(pool, case, g), vc=_cache(pool, case, g), table=table, starts=starts,
                req=req, ctx=ctx, most_q=max(new), out=torch.zeros((rows, heads, case["dim"]), device=DEV, dtype=dt),
                lse=torch.zeros((rows, heads), device=DEV))


def _verify_inputs(case, g):
    rows, kept = _kept(case)
    starts, v = _starts(rows), case["vocab"]
    R = starts[-1]
    z = torch.randn((R, v), generator=g, device=DEV) * 2.0
    p = torch.softmax(z, dim=1)
    q = None
    if case["probs"]:  # the drafter is the target with noise
        q = torch.softmax(z.add_(torch.randn((R, v), generator=g, device=DEV)), dim=1)
    del z
    # Row r's draft is the input of row r + 1.  Given that a draft is kept, it follows
    # min(p, q) and its random number lies below p / q; given that it is rejected,
    # max(q - p, 0) and above.
    u = torch.rand(R, generator=g, device=DEV)
    tokens = torch.randint(0, v, (R,), generator=g, device=DEV)
    r = torch.arange(R, device=DEV)
    req = torch.searchsorted(torch.tensor(starts[1:], device=DEV), r, right=True)
    place = r - torch.tensor(starts, device=DEV)[req]
    draft = place < torch.tensor(rows, device=DEV)[req] - 1
    keep = draft & (place < torch.tensor(kept, device=DEV)[req])
    for i in range(0, R, 64):
        pi = p[i:i + 64]
        if q is None:
            w = pi
        else:
            qi = q[i:i + 64]
            w = torch.where(keep[i:i + 64, None], torch.minimum(pi, qi), (qi - pi).clamp_(min=0.0))
        x = torch.multinomial(w, 1, generator=g)[:, 0]
        px = pi.gather(1, x[:, None])[:, 0]
        share = px if q is None else (px / qi.gather(1, x[:, None])[:, 0]).clamp(max=1.0)
        ui = u[i:i + 64]
        u[i:i + 64] = torch.where(keep[i:i + 64], 0.999 * ui * share, share + (1.0 - share) * (0.001 + 0.998 * ui))
        nxt = torch.arange(i + 1, i + 1 + x.numel(), device=DEV)
        ok = draft[i:i + 64]
        tokens[nxt[ok]] = x[ok]
    return dict(case=case, p=p, q=q, tokens=tokens.to(torch.int32), starts=_i32(starts), u=u,
                us=torch.rand(case["reqs"], generator=g, device=DEV), most=case["r_hi"],
                out=torch.empty((case["reqs"], case["r_hi"]), dtype=torch.int32, device=DEV),
                count=torch.empty(case["reqs"], dtype=torch.int32, device=DEV))


def prepare(case, seed):
    return {"rope": _rope_inputs, "window": _window_inputs, "verify": _verify_inputs}[case["op"]](case, _gen(seed))


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _turned(x, weight, s, cos, sin):
    """Heads x [rows, heads, dim] normed and rotated, in 32 bits."""
    c = s["case"]
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + s["eps"]) * weight
    o, rot = c["offset"], c["rot"]
    part = x[..., o:o + rot]
    if c["style"] == "half":
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        part = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        part = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    return torch.cat([x[..., :o], part, x[..., o + rot:]], dim=-1)


def _rope_plain(s):
    c = s["case"]
    pos = s["ctx"].long() - 1
    angle = pos[:, None].double() * s["freq"]
    cos, sin = ((f(angle) * s["factor"]).float()[:, None, :] for f in (torch.cos, torch.sin))
    live = (pos >= 0)[:, None, None]
    dt = s["q"].dtype
    q = torch.where(live, _turned(s["q"], s["q_weight"], s, cos, sin).to(dt), s["q_out"])
    k = _turned(s["k"], s["k_weight"], s, cos, sin).to(dt)
    if not c["cache"]:
        return q, torch.where(live, k, s["k_out"])
    b, pool = c["block"], s["pool"]
    at = torch.where(s["slots"] >= 0, s["slots"], pool * b)
    s["kc"][at // b, at % b] = k
    s["vc"][at // b, at % b] = s["v"]
    return q, s["kc"][:pool], s["vc"][:pool]


def _softmax(score, seen):
    """Weights and log-sum-exp of each row's seen scores; a row that sees
    nothing has zero weights."""
    score = torch.where(seen, score, -math.inf)
    top = score.amax(dim=-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    p = torch.exp(score - top)
    total = p.sum(dim=-1, keepdim=True)
    return p / total.clamp(min=1e-37), (top + torch.log(total)).squeeze(-1)


def _window_plain(s):
    c = s["case"]
    n, hk, grp, d, b = c["reqs"], c["kv_heads"], c["group"], c["dim"], c["block"]
    w, sinks, mq = c["window"], c["sinks"], s["most_q"]
    rows = s["q"].shape[0]
    starts = s["starts"].long()
    j = torch.arange(mq, device=DEV)[None, :]
    row = (starts[:-1, None] + j).clamp(max=rows - 1)
    live = starts[:-1, None] + j < starts[1:, None]
    ctx = torch.where(live, s["ctx"][row].long(), 0)
    # a request's tokens: the first ones, then those from the oldest window on
    first = (ctx.amax(dim=1) - (mq - 1) - w).clamp(min=sinks)
    t = torch.cat([torch.arange(sinks, device=DEV).expand(n, sinks),
                   first[:, None] + torch.arange(w + mq - 1, device=DEV)], dim=1)
    most = t.shape[1]
    block = s["table"].gather(1, (t // b).clamp(max=s["table"].shape[1] - 1)).long().clamp(min=0)
    k = s["kc"][block, t % b].float().permute(0, 2, 3, 1).reshape(n * hk, d, most)
    v = s["vc"][block, t % b].float().permute(0, 2, 1, 3).reshape(n * hk, most, d)
    q = s["q"][row].float().view(n, mq, hk, grp, d).permute(0, 2, 1, 3, 4).reshape(n * hk, mq * grp, d)
    score = torch.bmm(q, k).mul_(d ** -0.5).view(n, hk, mq, grp, most)
    ti, ci = t[:, None, :], ctx[:, :, None]
    seen = (ti < ci) & ((ti >= ci - w) | (ti < sinks))
    p, lse = _softmax(score, seen[:, None, :, None, :])
    o = torch.bmm(p.view(n * hk, mq * grp, most), v).view(n, hk, mq, grp, d)
    req = s["req"]
    at = torch.arange(rows, device=DEV) - starts[req]
    out = o.permute(0, 2, 1, 3, 4)[req, at].reshape(rows, hk * grp, d)
    return out.to(s["q"].dtype), lse.permute(0, 2, 1, 3)[req, at].reshape(rows, hk * grp)


def _verify_plain(s):
    n, most, v = s["case"]["reqs"], s["most"], s["case"]["vocab"]
    starts = s["starts"].long()
    p, q = s["p"], s["q"]
    R = p.shape[0]
    j = torch.arange(most, device=DEV)[None, :]
    row = (starts[:-1, None] + j).clamp(max=R - 1)
    drafts = starts[1:] - starts[:-1] - 1
    x = s["tokens"][(row + 1).clamp(max=R - 1)].long()
    px = p[row, x].double()
    qx = torch.ones_like(px) if q is None else q[row, x].double()
    good = (j < drafts[:, None]) & (s["u"][row].double() * qx < px)
    kept = torch.cumprod(good.long(), dim=1).sum(dim=1)
    # what the next token is taken from: the target where every draft was kept, else
    # what it has over the drafter
    i = torch.arange(n, device=DEV)
    last = starts[:-1] + kept
    every = (kept == drafts)[:, None]
    target = p[last]
    if q is None:
        rest = target.clone()
        rest[i, x[i, kept]] = 0.0
    else:
        rest = (target - q[last]).clamp_(min=0.0)
    rest = torch.where(every, target, rest)
    rest = torch.where(rest.sum(dim=1, keepdim=True) > 0, rest, target)
    total = torch.cumsum(rest.double(), dim=1)
    token = torch.searchsorted(total, s["us"].double()[:, None] * total[:, -1:], right=True)[:, 0].clamp(max=v - 1)
    out = torch.where(j < kept[:, None], x, torch.where(j == kept[:, None], token[:, None], -1))
    return out.to(torch.int32), (kept + 1).to(torch.int32)


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------

def _prepared(s):
    """The checked call that a serving loop keeps for its buffers."""
    import paged_mqa_logits_block_amd as m

    c = s["case"]
    if c["op"] == "rope":
        kw = {}
        if c["cache"]:
            kw = dict(v=s["v"], slots=s["slots"], kcache=s["kc"][:s["pool"]], vcache=s["vc"][:s["pool"]])
        return m.PreparedNormRope(
            s["q"], s["k"], s["ctx"], s["freq"], s["q_out"], k_out=s["k_out"], q_weight=s["q_weight"],
            k_weight=s["k_weight"], eps=s["eps"], rot_offset=c["offset"], rope_scale=s["factor"], position_offset=-1,
            layout=m.ROPE_HALF if c["style"] == "half" else m.ROPE_INTERLEAVED, **kw)
    if c["op"] == "window":
        return m.PreparedWindowAttention(s["q"], s["kc"], s["vc"], s["table"], s["ctx"], s["starts"], s["out"],
                                         window=c["window"], sinks=c["sinks"], lse=s["lse"])
    return m.PreparedVerifyDrafts(s["p"], s["tokens"], s["starts"], s["u"], s["us"], s["out"], s["count"],
                                  draft_probs=s["q"])


def _run_own(s):
    call = s.get("call")
    if call is None:
        call = s["call"] = _prepared(s)
    call()
    c = s["case"]
    if c["op"] == "rope":
        return (s["q_out"], s["kc"][:s["pool"]], s["vc"][:s["pool"]]) if c["cache"] else (s["q_out"], s["k_out"])
    return (s["out"], s["lse"]) if c["op"] == "window" else (s["out"], s["count"])


def run(state):
    if own:
        return _run_own(state)
    return {"rope": _rope_plain, "window": _window_plain, "verify": _verify_plain}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# in 64 bits, from the definitions
# ---------------------------------------------------------------------------

def _turn_exact(x, weight, eps, case, freq, factor, pos):
    y = x.double()
    d, rot, o = case["dim"], case["rot"], case["offset"]
    if weight is not None:
        norm = torch.sqrt(y.pow(2).sum(dim=-1) / d + eps)
        y = y / norm[..., None] * weight.double()
    y = y.clone()
    for i in range(rot // 2):
        a, b = (o + i, o + rot // 2 + i) if case["style"] == "half" else (o + 2 * i, o + 2 * i + 1)
        turn = torch.polar(torch.full(pos.shape, float(factor), dtype=torch.float64, device=DEV), pos * freq[i])
        pair = torch.complex(y[..., a], y[..., b]) * turn[:, None]
        y[..., a], y[..., b] = pair.real, pair.imag
    return y


def _attend(q, k, v, seen):
    """softmax(q k^T / sqrt(d)) v of [rows, group, d] queries over [keys, d] where
    seen [rows, keys], in float64."""
    rows, grp, d = q.shape
    z = torch.matmul(q.reshape(rows * grp, d), k.t()).view(rows, grp, -1) / math.sqrt(d)
    z.masked_fill_(~seen[:, None, :], -math.inf)
    lse = torch.logsumexp(z, dim=-1)
    return torch.matmul(torch.exp(z - lse[..., None]).view(rows * grp, -1), v).view(rows, grp, d), lse


def exact(case, seed):
    if case["op"] == "verify":
        return None  # whole numbers only
    s = prepare(case, seed)
    if case["op"] == "rope":
        rows = case["rows"]
        pos = s["ctx"][:rows].double() - 1.0
        q, k = (torch.zeros(s[x].shape, dtype=torch.float64, device=DEV) for x in ("q", "k"))
        for y, x, weight in ((q, s["q"], s["q_weight"]), (k, s["k"], s["k_weight"])):
            y[:rows] = _turn_exact(x[:rows], weight, s["eps"], case, s["freq"], s["factor"], pos)
        if not case["cache"]:
            return q, k
        b, hk, d = case["block"], case["kv_heads"], case["dim"]
        at = s["slots"][:rows]
        both = []
        for cache, values in ((s["kc"], k[:rows]), (s["vc"], s["v"][:rows].double())):
            flat = cache[:s["pool"]].double().reshape(-1, hk, d)
            flat[at] = values
            both.append(flat.view(s["pool"], b, hk, d))
        return q, both[0], both[1]
    past, new = _lengths(case)
    hk, grp, b, w = case["kv_heads"], case["group"], case["block"], case["window"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    r0 = 0
    for i, (p, a) in enumerate(zip(past, new)):
        old = max(0, p + 1 - w)
        pos = torch.tensor(sorted(set(range(min(case["sinks"], p + a))) | set(range(old, p + a))), device=DEV)
        where = s["table"][i].long()[pos // b]
        for h in range(hk):
            at = slice(h * grp, h * grp + grp)
            k, v = (s[x][where, pos % b, h].double() for x in ("kc", "vc"))
            q = s["q"][r0:r0 + a, at].double()
            for j in range(0, a, 256):
                e = min(a, j + 256)
                own_pos = torch.arange(p + j, p + e, device=DEV)[:, None]
                seen = (pos <= own_pos) & ((pos > own_pos - w) | (pos < case["sinks"]))
                out[r0 + j:r0 + e, at], lse[r0 + j:r0 + e, at] = _attend(q[j:e], k, v, seen)
        r0 += a
    return out, lse
