"""Steps of a server with windowed layers and drafted tokens on the GPU: plan, head norms
and rotary positions into the paged cache, windowed attention, verification; what
the verification keeps decides the next plan, and blocks of rejected tokens and those behind
the window go back to the free list.  Every step against the 64-bit definitions."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
m = pytest.importorskip("paged_mqa_logits_block_amd")

import serving_ref  # noqa: E402
import step_ref  # noqa: E402
from test_window_gpu import seen  # noqa: E402

pytestmark = pytest.mark.gpu

B, HK, GROUP, D, W, SINKS, V = 16, 2, 4, 128, 50, 5, 3001
DTYPE = torch.bfloat16
HALF_STEP = torch.finfo(DTYPE).eps / 2


class Step:
    """The step's buffers and calls."""

    def __init__(self, n=4, rows=60, max_blocks=40, pool=60, most=8, stream=None):
        c = dict(device="cuda")
        self.n, self.rows, self.pool, self.most = n, rows, pool, most
        self.past, self.new = (torch.zeros(n, dtype=torch.int32, **c) for _ in range(2))
        self.free = torch.zeros(pool, dtype=torch.int32, **c)
        self.table = torch.full((n, max_blocks), -1, dtype=torch.int32, **c)
        self.kc, self.vc = (torch.full((pool, B, HK, D), float("nan"), dtype=DTYPE, **c) for _ in range(2))
        self.qkv = torch.zeros(rows, (GROUP + 2) * HK, D, dtype=DTYPE, **c)
        self.q, self.k, self.v = self.qkv[:, :GROUP * HK], self.qkv[:, GROUP * HK:-HK], self.qkv[:, -HK:]
        self.q_out, self.out = (torch.zeros(rows, GROUP * HK, D, dtype=DTYPE, **c) for _ in range(2))
        self.qw, self.kw = (1.0 + 0.2 * torch.randn(D, **c) for _ in range(2))
        self.freq, self.scale = m.rope_frequencies(96, scaling="yarn", factor=4.0, original_len=64, device="cuda")
        self.probs, self.drafts = (torch.zeros(rows, V, **c) for _ in range(2))
        self.tokens = torch.zeros(rows, dtype=torch.int32, **c)
        self.u, self.us = torch.zeros(rows, **c), torch.zeros(n, **c)
        self.plan = m.BatchPlan.empty(n, rows, "cuda")
        self.out_tokens = torch.zeros(n, most, dtype=torch.int32, **c)
        self.count = torch.zeros(n, dtype=torch.int32, **c)
        self.calls = [
            m.PreparedPlanBatch(self.past, self.new, self.free, self.table, block_size=B, num_blocks=pool, out=self.plan,
                                stream=stream),
            m.PreparedNormRope(self.q, self.k, self.plan.ctx_lens, self.freq, self.q_out, v=self.v, slots=self.plan.slots,
                               kcache=self.kc, vcache=self.vc, q_weight=self.qw, k_weight=self.kw, rot_offset=16,
                               rope_scale=self.scale, position_offset=-1, stream=stream),
            m.PreparedWindowAttention(self.q_out, self.kc, self.vc, self.table, self.plan.ctx_lens, self.plan.q_starts,
                                      self.out, window=W, sinks=SINKS, stream=stream),
            m.PreparedVerifyDrafts(self.probs, self.tokens, self.plan.q_starts, self.u, self.us, self.out_tokens,
                                   self.count, draft_probs=self.drafts, stream=stream)]

    def run(self):
        for call in self.calls:
            call()


class Server:
    """Host side: lengths, the free list, and what was written of every token."""

    def __init__(self, step, seed):
        self.s, self.rng, self.g = step, np.random.default_rng(seed), torch.Generator().manual_seed(seed)
        self.lens = [0] * step.n
        self.free = self.rng.permutation(step.pool).tolist()
        self.k, self.v = [{} for _ in range(step.n)], [{} for _ in range(step.n)]
        self.gone = set()  # (request, table entry) behind the window

    def load(self, new):
        s = self.s
        s.past.copy_(torch.tensor(self.lens, dtype=torch.int32))
        s.new.copy_(torch.tensor(new, dtype=torch.int32))
        s.free.fill_(-1)
        s.free[:len(self.free)].copy_(torch.tensor(self.free, dtype=torch.int32))
        s.qkv.copy_(torch.randn(s.qkv.shape, generator=self.g) * 1.5)
        z = torch.randn(s.probs.shape, generator=self.g) * 2
        s.probs.copy_(torch.softmax(z, 1))
        s.drafts.copy_(torch.softmax(z + 0.7 * torch.randn(z.shape, generator=self.g), 1))
        x = torch.multinomial(s.drafts.cpu(), 1, generator=self.g)[:, 0]  # row r's draft is row r + 1's input
        s.tokens.copy_(torch.cat([torch.zeros(1, dtype=torch.int64), x[:-1]]).to(torch.int32))
        s.u.copy_(torch.rand(s.rows, generator=self.g))
        s.us.copy_(torch.rand(s.n, generator=self.g))
        s.out.fill_(3.0)

    def check(self, new, prompt):
        s = self.s
        starts = np.concatenate([[0], np.cumsum(new)])
        assert s.plan.q_starts.tolist() == starts.tolist()
        used = int(s.plan.blocks_used)
        self.free = self.free[used:]
        table, kc, vc = s.table.cpu().numpy(), s.kc.cpu(), s.vc.cpu()
        qkv, freq, eps = s.qkv.cpu().double().numpy(), s.freq.cpu().numpy(), float(np.float32(1e-6))
        R = starts[-1]
        pos = np.concatenate([np.arange(p, p + a) for p, a in zip(self.lens, new)] + [np.zeros(0)]).astype(np.int64)
        heads = {}
        for name, at, w in (("q", slice(0, GROUP * HK), s.qw), ("k", slice(GROUP * HK, GROUP * HK + HK), s.kw)):
            y, err = step_ref.norm_rope(qkv[:R, at], w.cpu().double().numpy(), eps, pos, freq, float(np.float32(s.scale)), 16,
                                        False)
            heads[name] = y, step_ref.rope_bounds(y, err, HALF_STEP, 2.0 ** -134)
        y, tol = heads["q"]
        q_out = s.q_out.cpu().double().numpy()
        assert np.all(np.abs(q_out[:R] - y) <= tol)
        out = s.out.cpu().double().numpy()
        assert np.all(out[R:] == 3.0)
        req = np.repeat(np.arange(s.n), new)
        for r in range(R):  # the new tokens in the cache
            i, t = req[r], int(pos[r])
            e = table[i, t // B]
            self.k[i][t], self.v[i][t] = kc[e, t % B].clone(), vc[e, t % B].clone()
            assert np.all(np.abs(self.k[i][t].double().numpy() - heads["k"][0][r]) <= heads["k"][1][r])
            assert torch.equal(self.v[i][t].double(), torch.from_numpy(qkv[r, GROUP * HK + HK:]))
        for r in range(R):  # attention over what was written of the tokens that the row sees
            i, toks = req[r], seen(int(pos[r]) + 1, W, SINKS)
            for t in toks:
                assert torch.equal(kc[table[i, t // B], t % B], self.k[i][t])
            for h in range(HK):
                kk, vv = (np.stack([x[i][t][h].double().numpy() for t in toks]) for x in (self.k, self.v))
                hs = slice(h * GROUP, (h + 1) * GROUP)
                o, l, spread, size = serving_ref.attend(q_out[r, hs], kk, vv, D ** -0.5)
                tol, _ = serving_ref.bounds(o, l, spread, size, len(toks), D, HALF_STEP)
                assert np.all(np.abs(out[r, hs] - o) <= tol), (r, h)
        want = step_ref.verify(s.probs.cpu().numpy(), s.drafts.cpu().numpy(), s.tokens.cpu().numpy(), starts,
                               s.u.cpu().numpy(), s.us.cpu().numpy(), s.most)
        assert np.array_equal(s.out_tokens.cpu().numpy(), want[0]) and np.array_equal(s.count.cpu().numpy(), want[1])
        # the next lengths, and the blocks that are not needed any more
        for i in range(s.n):
            old = self.lens[i] + new[i]
            self.lens[i] += new[i] if prompt else int(want[1][i])
            for e in range(-(-old // B)):
                behind = e * B >= SINKS and (e + 1) * B <= self.lens[i] + 1 - W
                if (e >= -(-self.lens[i] // B) or behind) and (i, e) not in self.gone:
                    self.free.append(int(table[i, e]))
                    s.table[i, e] = -1
                    if behind:
                        self.gone.add((i, e))
        held = [int(x) for x in s.table.cpu().flatten() if x >= 0]
        assert sorted(held + self.free) == list(range(s.pool))


# prompts, then verify steps of 0 to 7 drafts, pauses among them
STEPS = [([40, 0, 13, 1], True), ([0, 55, 0, 3], True)] + [([4, 4, 1, 8], False), ([1, 0, 5, 2], False), ([8, 8, 8, 8], False),
                                                           ([4, 4, 4, 4], False)] * 5


def test_verify_steps():
    step = Step()
    server = Server(step, 1)
    for new, prompt in STEPS:
        server.load(new)
        step.run()
        server.check(new, prompt)
    assert max(server.lens) > W + 2 * B and server.gone


def test_verify_steps_captured():
    """The same from one captured graph, replayed with the program's own work between."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step = Step()
        server = Server(step, 2)
        server.load([1, 1, 1, 1])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step.run()
    torch.cuda.current_stream().wait_stream(side)
    for new, prompt in STEPS:
        server.load(new)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        server.check(new, prompt)


def test_calls_side_by_side():
    """Norms and verifications (with workspaces of their own) on streams of their own, eager
    and captured, several times: equal to what one call alone gives."""
    g = torch.Generator(device="cuda").manual_seed(3)
    runs = []
    for i, (n, v) in enumerate(((3, 50021), (5, 40000), (2, 1000))):
        R = 4 * n
        p, q = (torch.rand(R, v, generator=g, device="cuda") / v for _ in range(2))
        tokens = torch.randint(0, v, (R,), generator=g, device="cuda", dtype=torch.int32)
        starts = torch.arange(0, R + 1, 4, dtype=torch.int32, device="cuda")
        u, us = torch.rand(R, generator=g, device="cuda"), torch.rand(n, generator=g, device="cuda")
        out, count = torch.zeros(n, 4, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
        x = torch.randn(3000 * (i + 1), 6, 64, generator=g, device="cuda").to(torch.float16)
        y, pos = torch.zeros_like(x), torch.arange(x.shape[0], dtype=torch.int32, device="cuda") * 31
        freq, _ = m.rope_frequencies(64, device="cuda")
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            calls = [m.PreparedVerifyDrafts(p, tokens, starts, u, us, out, count, draft_probs=q),
                     m.PreparedNormRope(x, None, pos, freq, y)]
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                for call in calls:
                    call()
        runs.append((s, graph, calls, (out, count, y), (p, q, tokens, starts, u, us, x, pos, freq)))
    torch.cuda.synchronize()
    want = []
    for s, _, calls, outs, _ in runs:
        for call in calls:
            call()
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs])
    for trial in range(6):
        for r in runs:
            for t in r[3]:
                t.zero_()
        torch.cuda.synchronize()
        for s, graph, calls, *_ in runs:
            with torch.cuda.stream(s):
                if trial % 2:
                    graph.replay()
                else:
                    for call in calls:
                        call()
        torch.cuda.synchronize()
        for r, w in zip(runs, want):
            assert all(torch.equal(a, b) for a, b in zip(r[3], w))
        torch.randn(1000, 1000, device="cuda") @ torch.randn(1000, 1000, device="cuda")


def test_own_stream():
    """The functions' stream argument: outputs and workspaces made there."""
    s = torch.cuda.Stream()
    x = torch.randn(50, 4, 64, device="cuda").to(torch.bfloat16)
    pos, (freq, _) = torch.arange(50, dtype=torch.int32, device="cuda"), m.rope_frequencies(64, device="cuda")
    p = torch.rand(8, 50000, device="cuda")
    tokens, starts = torch.arange(8, dtype=torch.int32, device="cuda"), torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    u, us = torch.rand(8, device="cuda"), torch.rand(2, device="cuda")
    torch.cuda.synchronize()
    got = m.norm_rope(x, x, pos, freq, stream=s) + m.verify_drafts(p, tokens, starts, u, us, max_tokens=4, stream=s)
    s.synchronize()
    want = m.norm_rope(x, x, pos, freq) + m.verify_drafts(p, tokens, starts, u, us, max_tokens=4)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
