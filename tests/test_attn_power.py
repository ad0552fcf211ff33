"""The bounds that the GPU tests of long caches use fail when a run of keys is left out or counted twice (CPU)."""
import numpy as np
import pytest

from attn_power import RUN, marked_limits, marked_rows, marks, noise_rows
from attn_ref import bf16, e4m3


@pytest.mark.parametrize("q_len,kv_len,window", [([1], [131072], 0), ([5], [131072], 0), ([2, 3], [40000, 20001], 5000)])
def test_a_run_left_out_or_doubled_breaks_the_marked_bound(q_len, kv_len, window):
    D = 128
    out, lse = marked_rows(q_len, kv_len, window, D)
    lim, lse_lim = marked_limits(out, lse)
    t = q_len[0] - 1  # the first request's last row, its runs one after another
    lo = max(0, kv_len[0] - window) if window else 0
    for run in range(lo // RUN + 1, kv_len[0] // RUN - 1, 7):
        for sign in (-1, 1):
            n = kv_len[0] - lo
            count = out[t] * n
            count[marks(kv_len[0], D)[run * RUN]] += sign * RUN
            assert np.any(np.abs(count / (n + sign * RUN) - out[t]) > lim[t]), run
            assert abs(np.log(n + sign * RUN) - lse[t]) > lse_lim[t], run


@pytest.mark.parametrize("f8", [False, True])
def test_a_run_left_out_breaks_the_norm_bound(f8):
    rng = np.random.default_rng(3)
    n, kv, D = 5, 131072, 128
    q = bf16(rng.standard_normal((n, D)) * 1.5)
    k = (e4m3(rng.standard_normal((kv, D)) * 3) * 0.3 if f8 else bf16(rng.standard_normal((kv, D)))).astype(np.float64)
    v = (e4m3(rng.standard_normal((kv, D)) * 3) * 0.3 if f8 else bf16(rng.standard_normal((kv, D)))).astype(np.float64)
    out, bound = noise_rows(q, k, v, D ** -0.5, f8)
    assert np.all(bound < 0.02 * np.linalg.norm(out, axis=1))
    for first in (0, 4096, 70000, kv - 5 * RUN):
        other, _ = noise_rows(q, k, v, D ** -0.5, f8, left_out=range(first, first + RUN))
        assert np.all(np.linalg.norm(other - out, axis=1) > bound), first
