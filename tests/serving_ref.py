"""Plain 64-bit implementations of the batch plan, the cache writes and paged
attention, and input makers for their tests.  Host code only: numpy loops in the
order of the definitions."""
from __future__ import annotations

import types

import numpy as np


def plan(past, new, free, table, *, block_size, num_blocks, num_rows, ratio):
    n, max_blocks = table.shape
    B, cap = block_size, table.shape[1] * block_size
    table = table.copy()
    p = [min(max(int(x), 0), cap) for x in past]
    starts = [0]
    for x in new:
        starts.append(min(starts[-1] + max(int(x), 0), num_rows))
    used = 0
    for i in range(n):
        end = min(p[i] + starts[i + 1] - starts[i], cap)
        for e in range(-(-p[i] // B), -(-end // B)):
            table[i, e] = free[used] if used < len(free) else -1
            used += 1
    r2r, ctx = np.zeros(num_rows, np.int32), np.zeros(num_rows, np.int32)
    slots, cols = np.full(num_rows, -1, np.int64), np.full(num_rows, -1, np.int64)
    for i in range(n):
        for r in range(starts[i], starts[i + 1]):
            t = p[i] + r - starts[i]
            r2r[r], ctx[r] = i, min(t + 1, cap)
            if t < cap and 0 <= table[i, t // B] < num_blocks:
                b = int(table[i, t // B])
                slots[r] = b * B + t % B
                if (t + 1) % ratio == 0:
                    cols[r] = b * (B // ratio) + t % B // ratio
    return types.SimpleNamespace(table=table, q_starts=np.array(starts, np.int32), row_to_req=r2r, ctx_lens=ctx,
                                 slots=slots, col_lens=(ctx // ratio).astype(np.int32), col_slots=cols,
                                 blocks_used=np.array([used], np.int32))


def attend(q, k, v, scale):
    """(out [H, D], lse [H], bound parts) of queries q [H, D] over keys k, v [n, D]
    (float64).  ``spread`` = sum p |v| and ``delta``: an upper bound of
    sum |q k| * scale and of the scores' size, for error bounds."""
    if k.shape[0] == 0:
        h, d = q.shape
        return np.zeros((h, d)), np.full(h, -np.inf), np.zeros((h, d)), np.zeros(h)
    with np.errstate(all="ignore"):
        z = scale * (q @ k.T)
        top = z.max(axis=1)
        e = np.exp(z - top[:, None])
        lse = top + np.log(e.sum(axis=1))
        p = e / e.sum(axis=1, keepdims=True)
        return p @ v, lse, p @ np.abs(v), scale * (np.abs(q) @ np.abs(k).T).max(axis=1)


def bounds(out, lse, spread, size, n, d, half_step):
    """Allowed errors of a row's outputs and lse against the 64-bit ones.

    Scores are 32-bit sums of d products: off by at most (d + 2) 2^-24 size, with
    the product by the scale and the subtraction of the maximum each rounding a
    number of at most 2 size once more, and exp2 by 2^-22 relative; so a weight is
    off by at most w = (d + 8) 2^-24 size + 2^-22 relative.  Weights are then
    rounded to the type (half a step u), summed with n 32-bit additions (n
    2^-24), normalised by a sum with the errors of the weights before the rounding
    and one division, and the output is rounded once (u)."""
    w = (d + 8) * 2.0 ** -24 * size + 2.0 ** -22
    s = (n + 8) * 2.0 ** -24
    rel = 2 * w + 2 * s + half_step
    tol_o = half_step * np.abs(out) + (1 + half_step) * rel[:, None] * spread * 1.01 + 1e-30
    tol_l = (w + s) * 1.01 + 2.0 ** -22 * np.abs(lse)
    return tol_o, tol_l


def fp16_tail(v):
    """What fp16 weights add to a row's allowed error over values v [n, D].

    `bounds` takes each weight as rounded by half a step relative to itself, which
    fp16 does down to 2^-14 only; below, it is off by up to 2^-25.  The weights are
    taken relative to a reference that lies at least 13 (in log2) below the row's
    largest score, so that the largest weight is 2^13 or more: a probability is off by
    2^-38 at most.  An output below 2^-14 is itself off by up to 2^-25."""
    return 2.0 ** -38 * np.abs(v).sum(axis=0) + 2.0 ** -25
