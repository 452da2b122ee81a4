"""Scaled rotary frequencies by parts, at original lengths in which few pairs or none turn often."""
from __future__ import annotations

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
m = pytest.importorskip("paged_mqa_logits_block_amd")


@pytest.mark.parametrize("rot", [2, 16, 64, 128])
@pytest.mark.parametrize("original_len,fast,slow", [(4, 32.0, 1.0), (6, 32.0, 1.0), (7, 32.0, 1.0), (512, 200.0, 100.0),
                                                    (40, 32.0, 1.0), (4096, 32.0, 1.0), (1 << 20, 32.0, 1.0)])
def test_pairs_that_turn_seldom_are_stretched(rot, original_len, fast, slow):
    """The first pair was kept where none turns beta_slow times in the original length."""
    base, factor = 10000.0, 8.0
    plain = base ** (-np.arange(0, rot, 2) / rot)
    turns = original_len * plain / (2 * math.pi)
    got = m.rope_frequencies(rot, base, scaling="yarn", factor=factor, original_len=original_len, beta_fast=fast,
                             beta_slow=slow)[0].numpy()
    assert np.allclose(got[turns < slow], plain[turns < slow] / factor, rtol=1e-13)
    assert np.allclose(got[turns > fast], plain[turns > fast], rtol=1e-13)
    assert np.all((got >= plain / factor * (1 - 1e-13)) & (got <= plain * (1 + 1e-13)))
