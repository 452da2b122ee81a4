"""Integer arguments that do not fit the C interface's 32 bits are refused, not cut to them."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
m = pytest.importorskip("paged_mqa_logits_block_amd")

WIDE = 2 ** 32


@pytest.mark.parametrize("k,ratio", [(512, WIDE + 4), (WIDE + 512, 4), (512, 2 ** 31), (-WIDE + 512, 4)])
def test_sparse_query(k, ratio):
    s = m.AttnShape(num_rows=36, num_heads=32, num_kv_heads=4, head_dim=128, block_size=16, num_reqs=9, max_blocks=1000,
                    dtype=m.BF16, scale=0.1, num_blocks=9000, q_row_stride=4096, q_head_stride=128, out_row_stride=4096,
                    out_head_stride=128, kv_block_stride=16 * 512, kv_slot_stride=512, kv_head_stride=128)
    assert m.sparse_attention_workspace_bytes(s, 512, 4) > 0
    with pytest.raises(m.QsaError) as e:
        m.sparse_attention_workspace_bytes(s, k, ratio)
    assert e.value.status == m.E_INVALID


@pytest.mark.gpu
def test_calls():
    def i32(*v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    q = torch.zeros(2, 8, 64, dtype=torch.bfloat16, device="cuda")
    kc = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    keys, slots = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda"), torch.tensor([0, 1], device="cuda")
    # the interleaved layout's size
    packed = torch.zeros(4, 16 * 68, dtype=torch.uint8, device="cuda")
    table = i32(0, 1).view(1, 2)
    for call in (lambda: m.sparse_attention(q, kc, kc, table, i32(0, 0), i32(0, 1).view(2, 1), ratio=WIDE + 4),
                 lambda: m.plan_batch(i32(3), i32(2), i32(0, 1, 2, 3), table, block_size=WIDE + 16, num_blocks=4, num_rows=2),
                 lambda: m.plan_batch(i32(3), i32(2), i32(0, 1, 2, 3), table, block_size=16, ratio=WIDE + 4, num_blocks=4,
                                      num_rows=2),
                 lambda: m.write_keys(keys, slots, packed, block_size=16, layout=WIDE + m.KV_PAGED),
                 lambda: m.window_attention(q, kc, kc, table, i32(5, 5), i32(0, 2), window=WIDE + 4),
                 lambda: m.norm_rope(q, None, i32(1, 2), torch.zeros(8, dtype=torch.float64, device="cuda"),
                                     layout=WIDE + m.ROPE_HALF)):
        with pytest.raises(m.QsaError) as e:
            call()
        assert e.value.status == m.E_INVALID and "32 bits" in str(e.value)
