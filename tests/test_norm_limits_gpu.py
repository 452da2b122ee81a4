"""Head norms at the ends of the range of sums of squares that the call's contract gives, against
the plain 64-bit implementation in step_ref.py."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
m = pytest.importorskip("paged_mqa_logits_block_amd")

import step_ref as ref  # noqa: E402
from test_step_gpu import rope_close  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 128])
def test_sums_of_squares_at_both_ends(dim):
    """Without eps, sums of squares of 2^-118 and more and of less than 2^127.  (The squares
    below 2^-126 are rounded to multiples of 2^-149: dim of them put a sum off by at most
    dim 2^-150, 2^-143, or 2^-25 of it, and the root halves that: within the steps that
    the bound of step_ref leaves.)"""
    g = torch.Generator().manual_seed(dim)
    x = torch.randn(64, 1, dim, generator=g).double()
    x[1::4, :, 1:] = 0  # all in one element
    x[1::4, :, 0] = 1.0
    x[2::4, :, :] = 1.0
    x = x.to(torch.bfloat16).double()
    e = torch.floor(torch.log2(x.pow(2).sum(2, keepdim=True)))
    low = torch.arange(64).view(-1, 1, 1) < 32
    # sums of [2^-118, 2^-116) and of [2^125, 2^127)
    target = torch.where(low, -118.0, 126.0)
    x = x * 2.0 ** torch.where(low, torch.ceil((target - e) / 2), torch.floor((target - e) / 2))
    total = x.pow(2).sum(2).flatten().numpy()
    assert total[:32].min() >= 2.0 ** -118 and total[:32].max() < 2.0 ** -116
    assert total[32:].min() >= 2.0 ** 125 and total[32:].max() < 2.0 ** 127
    q = x.to(torch.bfloat16)
    assert torch.equal(q.double(), x)
    w = 1.0 + 0.3 * torch.randn(dim, generator=g)
    pos = np.arange(64, dtype=np.int32)
    freq, _ = m.rope_frequencies(32)
    y, _ = m.norm_rope(q.cuda(), None, torch.from_numpy(pos).cuda(), freq.cuda(), q_weight=w.cuda(), eps=0.0)
    want, err = ref.norm_rope(x.numpy(), w.double().numpy(), 0.0, pos, freq.numpy(), 1.0, 0, False)
    rope_close(y, want, err, "bf16", "q")
