"""Windowed attention of few rows in tables of many requests, most of them without rows, on
the GPU: against the plain 64-bit implementation in serving_ref.py, and bit for bit against the
same rows in the smallest table."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
m = pytest.importorskip("paged_mqa_logits_block_amd")

from test_serving_gpu import Batch  # noqa: E402
from test_window_gpu import check_window, free_unseen, run_window  # noqa: E402

pytestmark = pytest.mark.gpu

TABLES = [
    # requests, {request: (past, new)}, window, sinks, kwargs: rows first, last, in between, one by
    # one; requests of 4 and 5 rows, whose tiles take every place that there is; a request whose
    # rows are more than a tile's; heads in two parts; windows that are not cut
    (256, {0: (2300, 1), 1: (700, 1), 2: (2300, 1), 3: (1990, 1)}, 2000, 4, dict(hk=8, group=8)),
    (256, {252: (2300, 1), 253: (5, 1), 254: (2300, 1), 255: (1990, 1)}, 2000, 4, dict(hk=8, group=8)),
    (1000, {3: (2300, 1), 64: (0, 1), 65: (2300, 2), 999: (1990, 1)}, 2000, 33, dict(hk=4, group=8)),
    (1024, {i: (1500 + 9 * i, 4) for i in (15, 16, 31, 500, 1008, 1023)}, 1400, 0, dict(group=8, dim=64, dtype="fp16")),
    (3, {0: (1700, 5), 1: (900, 5), 2: (1700, 5)}, 1600, 4, dict(group=8)),
    (700, {10: (1700, 5), 11: (900, 5), 600: (1700, 5)}, 1600, 4, dict(group=8, pad=3)),
    (128, {5: (2000, 40), 90: (3, 1)}, 1800, 70, dict(hk=1, group=1, block=100, order="head")),
    (200, {0: (1500, 2), 199: (1500, 1)}, 1400, 4, dict(hk=1, group=33)),
    (1000, {0: (300, 3), 500: (40, 1), 998: (300, 5)}, 60, 2, dict(group=8, dim=64)),
    # as many rows as make more tiles than CUs, the ones left over cut
    (300, {i: (2090, 1) for i in range(0, 130, 2)}, 2000, 4, dict(hk=4, group=8, dim=64)),
]


@pytest.mark.parametrize("i", range(len(TABLES)))
def test_few_rows_in_a_large_table(i):
    n, live, window, sinks, kw = TABLES[i]
    past, new = ([live.get(r, (0, 0))[x] for r in range(n)] for x in (0, 1))
    b = Batch(300 + i, past, new, **kw)
    # a table without room for more requests with rows than there may be rows
    more = [0] * (min(n, len(b.q)) - len(live))
    alone = Batch(300 + i, [live[r][0] for r in sorted(live)] + more, [live[r][1] for r in sorted(live)] + more, **kw)
    need = [m.window_attention_workspace_bytes(m.make_attn_shape(x.q.cuda(), x.kc, x.table), window, sinks)
            for x in (b, alone)]
    assert need[0] == need[1] and (need[0] > 0) == (window > 100)
    for x in (b, alone):
        free_unseen(x, window, sinks)
    rows = range(b.rows) if b.rows <= 30 else sorted({*range(0, b.rows, 9), *range(b.rows - 3, b.rows)})
    check_window(b, window, sinks, rows=rows)
    out, lse = run_window(b, window, sinks)
    want, want_lse = run_window(alone, window, sinks)
    assert torch.equal(b.q, alone.q) and torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("live", [range(6), range(1024, 1030), (0, 7, 8, 515, 1023, 1029)], ids=["first", "last", "spread"])
@pytest.mark.parametrize("new", [1, 6])
def test_few_rows_among_more_requests_than_are_counted(live, new):
    """Above 1,024 requests tiles are numbered as slots, most of them without rows, in rounds of 8 that
    are rotated; they are cut, and parts without rows are not joined."""
    n, window, sinks = 1030, 3000, 70
    past, a = [0] * n, [0] * n
    for j, r in enumerate(live):
        past[r], a[r] = (3700, 0, 3100, 40, 3700, 2999)[j], new
    b = Batch(330 + new, past, a, hk=1, group=8, dim=64, pad=3)
    free_unseen(b, window, sinks)
    assert m.window_attention_workspace_bytes(m.make_attn_shape(b.q.cuda(), b.kc, b.table), window, sinks) > 0
    check_window(b, window, sinks)
