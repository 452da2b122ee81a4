"""Windowed attention's workspace query: sizes that ctypes would cut to 32 bits, and few
rows in tables of many requests."""
from __future__ import annotations

import pytest

pytest.importorskip("torch")
m = pytest.importorskip("paged_mqa_logits_block_amd")


def attn_shape(rows, reqs, kv=4, group=8, dim=128, max_blocks=1000):
    hq = kv * group
    return m.AttnShape(num_rows=rows, num_heads=hq, num_kv_heads=kv, head_dim=dim, block_size=16, num_reqs=reqs,
                       max_blocks=max_blocks, dtype=m.BF16, scale=0.1, num_blocks=9000, q_row_stride=hq * dim,
                       q_head_stride=dim, out_row_stride=hq * dim, out_head_stride=dim, kv_block_stride=16 * kv * dim,
                       kv_slot_stride=kv * dim, kv_head_stride=dim)


@pytest.mark.parametrize("window,sinks", [(2 ** 32 + 4096, 4), (2 ** 32 + 1, 4), (2 ** 31, 4), (4096, 2 ** 32), (4096, 2 ** 31),
                                          (-2 ** 32 + 4096, 4), (4096, -2 ** 32)])
def test_query_refuses_what_the_call_refuses(window, sinks):
    """A window of 2^32 + 4,096 was answered as one of 4,096."""
    with pytest.raises(m.QsaError) as e:
        m.window_attention_workspace_bytes(attn_shape(36, 9), window, sinks)
    assert e.value.status == m.E_INVALID


def test_query_of_the_largest_sizes():
    s = attn_shape(36, 9)
    assert m.window_attention_workspace_bytes(s, 2 ** 31 - 1, 0) == m.window_attention_workspace_bytes(s, 16000, 0) > 0
    assert m.window_attention_workspace_bytes(s, 4096, 2 ** 31 - 1) > 0


@pytest.mark.parametrize("rows,kv,group", [(1, 4, 8), (4, 8, 8), (9, 8, 8), (20, 4, 8), (5, 1, 8), (3, 2, 33), (2, 1, 1)])
def test_few_rows_are_cut_whatever_the_table(rows, kv, group):
    """What the parts take is bounded by the tiles that can have rows: the table's empty requests
    neither keep a call from being cut nor ask for more."""
    subs = -(-group // 32)
    per_tile = 32 // -(-group // subs)
    alone = m.window_attention_workspace_bytes(attn_shape(rows, rows, kv, group), 4096, 4)
    assert alone > 0
    for reqs in (rows + 1, 64, 128, 256, 512, 1000, 1024):
        assert m.window_attention_workspace_bytes(attn_shape(rows, reqs, kv, group), 4096, 4) == alone, reqs
    state, record = 32 * (128 + 2) * 4, 8
    tiles = rows * kv * subs
    parts, left = divmod(alone - tiles * record, tiles * state)
    assert left == 0 and 2 <= parts <= max(256 // tiles, 2)
    if rows * group <= 64:  # one request's rows, streamed too, share tiles
        one = -(-rows // per_tile) * kv * subs
        size = m.window_attention_workspace_bytes(attn_shape(rows, 1, kv, group), 4096, 4)
        parts, left = divmod(size - one * record, one * state)
        assert left == 0 and parts >= 2


def test_rows_of_many_requests_take_a_place_each():
    """Above 1,024 requests each slot has a place, and a call of few heads is still cut."""
    assert m.window_attention_workspace_bytes(attn_shape(8, 1030, 1), 4096, 4) > 0
    assert m.window_attention_workspace_bytes(attn_shape(8, 1030, 8), 4096, 4) == 0
