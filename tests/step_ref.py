"""Plain 64-bit implementations of head norms with rotary positions, of windowed
attention's visible tokens and of draft verification, for their tests.  Host code
only: numpy loops in the order of the definitions."""
from __future__ import annotations

import numpy as np


def norm_rope(x, weight, eps, pos, freq, factor, offset, interleaved):
    """(y, bound parts) of heads x [rows, heads, D] at positions pos [rows] (float64).
    The second value is an upper bound of each element's error in 32 bits (see
    rope_bounds)."""
    x = x.astype(np.float64)
    rows, heads, d = x.shape
    y, size = x.copy(), np.abs(x)
    rel = 0.0
    if weight is not None:
        inv = 1.0 / np.sqrt((x * x).sum(axis=2, keepdims=True) / d + eps)
        y = x * inv * weight
        size = np.abs(y)
        # the sum of d squares (their rounding and d additions, halved by the root), the
        # mean, eps, root, quotient (2 steps), and two products
        rel = ((d + 3) / 2 + 8) * 2.0 ** -24
    err = rel * size
    n = len(freq)
    for i in range(n):
        a, b = (offset + 2 * i, offset + 2 * i + 1) if interleaved else (offset + i, offset + n + i)
        t = pos.astype(np.float64) * freq[i]
        c, s = factor * np.cos(t)[:, None], factor * np.sin(t)[:, None]
        ya, yb = y[:, :, a].copy(), y[:, :, b].copy()
        y[:, :, a], y[:, :, b] = ya * c - yb * s, yb * c + ya * s
        # the angle: a 64-bit product, in turns rounded to 32 bits (half a step of
        # at most 1/2), the functions' own error (2 steps of at most 1), the factor and
        # its product; then two products and a sum
        angle = 2 * np.pi * 2.0 ** -26 + np.abs(t)[:, None] * 2.0 ** -50 + 2.0 ** -23 + 2.0 ** -23
        both = (size[:, :, a] + size[:, :, b]) * abs(factor) * (rel + angle + 4 * 2.0 ** -24)
        err[:, :, a], err[:, :, b] = both, both
    return y, err


def rope_bounds(y, err, half_step, tiny):
    """Allowed errors of the rounded outputs; tiny: half a step of the type's
    subnormals."""
    return err * 1.01 + half_step * (np.abs(y) + err) + tiny


def weights_of(x):
    """What is not a positive number has no weight."""
    with np.errstate(invalid="ignore"):
        return np.where((x > 0) & (x < np.inf), x, np.float32(0))


def choose(w, u):
    c = np.cumsum(w.astype(np.float64))
    if not c[-1] > 0:
        return None
    past = np.nonzero((c > np.float64(np.float32(u)) * c[-1]) & (w > 0))[0]
    return int(past[0]) if len(past) else int(np.nonzero(w > 0)[0][-1])


def verify(probs, draft, tokens, starts, u, us, max_tokens):
    """Draft verification of float32 probs [R, V] (draft: [R, V] or None)."""
    R, V = probs.shape
    n = len(starts) - 1
    out, count = np.full((n, max_tokens), -1, np.int32), np.zeros(n, np.int32)
    for i in range(n):
        s, e = min(max(int(starts[i]), 0), R), min(max(int(starts[i + 1]), 0), R)
        rows = min(e - s, max_tokens)
        if rows <= 0:
            continue
        kept = 0
        while kept < rows - 1:
            x = int(tokens[s + kept + 1])
            if not 0 <= x < V:
                break
            q = 1.0 if draft is None else np.float64(draft[s + kept, x])
            if not np.float64(u[s + kept]) * q < np.float64(probs[s + kept, x]):
                break
            kept += 1
        p = probs[s + kept]
        if kept == rows - 1:
            rest = p
        elif draft is None:
            rest = p.copy()
            x = int(tokens[s + kept + 1])
            if 0 <= x < V:
                rest[x] = 0
        else:
            with np.errstate(invalid="ignore"):
                rest = p - draft[s + kept]
        token = choose(weights_of(rest), us[i])
        if token is None:
            token = choose(weights_of(p), us[i])
        out[i, :kept] = tokens[s + 1:s + 1 + kept]
        out[i, kept] = -1 if token is None else token
        count[i] = kept + 1
    return out, count
