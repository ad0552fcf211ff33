"""Bounds for long caches that a key left out or counted twice breaks, and what they need (numpy, no library calls)."""
from __future__ import annotations

import numpy as np

RUN = 128  # keys of a run: a key tile of either kernel, or several


def marks(n, D):
    """The value element that is 1 for each of n keys: one per run."""
    return (np.arange(n) // RUN) % D


def marked_rows(q_len, kv_len, window, D):
    """(out, lse) of every row under equal scores and the marks as values: counts over the number of visible keys."""
    out, lse = [], []
    for n, kv in zip(q_len, kv_len):
        for i in range(n):
            pos = kv - n + i
            j = np.arange(max(0, pos - window + 1) if window else 0, pos + 1)
            count = np.bincount(marks(kv, D)[j], minlength=D) if j.size else np.zeros(D)
            out.append(count / max(j.size, 1))
            lse.append(np.log(j.size) if j.size else -np.inf)
    return np.array(out), np.array(lse)


def marked_limits(out, lse):
    """Sums of whole numbers are exact: out is off by its rounding to bf16, half a step of 2^-8, and the quotient's
    2^-24; lse by a few roundings of a logarithm below 12."""
    return 1.01 * 2.0 ** -8 * out, np.full(lse.shape, 16 * 2.0 ** -24 * 12)


def noise_rows(q, keys, values, scale, e4m3, left_out=()):
    """(out, bound of the 2-norm of a row's error) of the rows q [n, D], the newest of the keys [kv, D], in fp64.

    The error is the sum of roundings that do not depend on one another: out's to bf16 (2^-8 of it at most) and, key by
    key, the numerator's (2^-8, or 2^-11 for e4m3 caches) and the score's, (D + 16) 2^-23 of sum |q||k| scale. Its mean
    square is at most the sum of the squares of their bounds, and with uniform errors a third of it, which is the room
    that a row's 128 elements need to stay within it. e4m3 caches: a numerator below fp16's normal steps is off by up to
    2^-31 of its reference instead, which meets values that do not depend on the scores here."""
    n, kv, D = q.shape[0], keys.shape[0], q.shape[1]
    s = q @ keys.T * scale
    see = np.arange(kv)[None] <= (kv - n + np.arange(n))[:, None]
    see[:, list(left_out)] = False
    s = np.where(see, s, -np.inf)
    w = np.exp(s - s.max(1, keepdims=True))
    w /= w.sum(1, keepdims=True)
    ds = (D + 16) * 2.0 ** -23 * (np.abs(q) @ np.abs(keys).T * scale).max(1) + 2.0 ** -21
    out = w @ values
    each = (2.0 ** -11 if e4m3 else 2.0 ** -8) + 2 * ds
    square = 2.0 ** -16 * (out ** 2).sum(1) + each ** 2 * (w ** 2 @ (values ** 2).sum(1))
    return out, np.sqrt(square + (2.0 ** -62 * (values ** 2).sum() if e4m3 else 0.0))
