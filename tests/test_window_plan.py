"""Windowed attention's workspace query: sizes that ctypes would cut to 32 bits."""
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
