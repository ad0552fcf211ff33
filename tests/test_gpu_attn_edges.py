"""Calls at the edges of what the attention half takes: each test holds one
property of the row kernels and, with a block table wide enough that the call
counts as a large one, of the chunk kernel."""
import numpy as np
import pytest

import quantized_expert_ffn_top10_b200 as M
from attn_power import marked_limits, marked_rows, marks, noise_rows
from attn_ref import attn_limits, bf16
from test_gpu_attn import Case

pytestmark = pytest.mark.gpu


def wide(c, keys=1 << 16):
    """The case's table with room for so many keys (the columns behind its pages hold no page)."""
    import torch
    t = c.cache.table_dev
    cols = max(t.shape[1], -(-keys // c.cache.page))
    out = torch.full((t.shape[0], cols), -1, dtype=torch.int32, device="cuda")
    out[:, :t.shape[1]] = t
    return out


def check_rows(c, rows, ref=None):
    """The rows [rows] of the step against the reference."""
    import torch
    torch.cuda.synchronize()
    ref = ref or c.ref()
    lim, lse_lim = attn_limits(ref, c.D, max(c.kv_len), c.f8)
    got, lse = c.out.double().cpu().numpy(), c.lse.double().cpu().numpy()
    assert np.all(np.abs(got - ref[0])[rows] <= lim[rows])
    with np.errstate(invalid="ignore"):
        off = np.abs(lse - ref[1])
    assert np.all((off <= lse_lim)[rows] | np.isneginf(ref[1])[rows])
    assert np.array_equal(np.isneginf(lse)[rows], np.isneginf(ref[1])[rows])


@pytest.mark.parametrize("window", [(1 << 31) - 1, 1 << 30, (1 << 30) - 1])
@pytest.mark.parametrize("which,page", [("decode", 16), ("prefill", 16), ("prefill", 24)])
def test_widest_windows(cuda_ok, which, page, window):
    """The largest window there is means no window, also for rows before the
    first key (requests with fewer keys than new rows)."""
    c = Case([5, 5, 5, 5], [0, 2, 40, 3], Hq=8, Hk=1, page=page, window=window, seed=50)
    c.run(which)
    c.check()
    c.out.fill_(7.0)
    c.run(which, table=wide(c))
    c.check()


@pytest.mark.parametrize("extra", [dict(), dict(window=7), dict(slopes=True)])
@pytest.mark.parametrize("tables", ["tight", "wide"])
def test_rows_of_a_wider_request_keep_their_positions(cuda_ok, tables, extra):
    """A request that brings more rows than max_q: the first max_q rows are
    those of the whole request, the others stay as they were."""
    c = Case([3, 1, 6], [40, 9, 300], Hq=16, Hk=1, page=16, seed=51, **extra)
    c.run("decode", max_q=2, table=wide(c) if tables == "wide" else None)
    rows = [0, 1, 3, 4, 5]
    check_rows(c, rows)
    left = [2, 6, 7, 8, 9]
    assert bool((c.out[left] == 7.0).all()) and bool((c.lse[left] == 7.0).all())
    assert M.moe_last_device_error() == 0


@pytest.mark.parametrize("softcap", [1e3, 1e4, 1e6, 1e8, 1e20, 1e30, 3e38])
@pytest.mark.parametrize("extra", [dict(), dict(f8=True), dict(slopes=True), dict(window=200)])
@pytest.mark.parametrize("which", ["decode", "decode16", "prefill", "chunk"])
def test_large_caps(cuda_ok, which, extra, softcap):
    """A cap far above the scores changes them by less than their rounding: the
    cap's own arithmetic adds a few 2^-24 of the score (the limits' 16 steps)."""
    if which in ("decode", "decode16"):
        c = Case([1, 5], [300, 77], Hq=6 if which == "decode" else 24, Hk=2, page=16, softcap=softcap, seed=52, **extra)
        c.run("decode")
    else:
        c = Case([140, 33], [900, 33], Hq=4, Hk=2, page=16, softcap=softcap, seed=53, **extra)
        c.run("prefill", table=wide(c) if which == "chunk" else None)
    c.check()


@pytest.mark.parametrize("slopes", [False, True])
@pytest.mark.parametrize("q_gain", [0.3, 6.0, 40.0])
@pytest.mark.parametrize("f8", [False, True])
def test_caps_and_slopes_of_the_chunk_kernel(cuda_ok, f8, q_gain, slopes):
    """Scores below, around and above the cap, hidden or not, with slopes and without."""
    c = Case([300, 45], [1500, 45], Hq=4, Hk=1, page=16, softcap=12.0, q_gain=q_gain, slopes=slopes, f8=f8, seed=54)
    c.run("prefill", table=wide(c))
    c.check()


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("which,page,tables", [("decode", 16, "tight"), ("prefill", 16, "wide"), ("prefill", 24, "wide"),
                                               ("prefill", 64, "wide"), ("prefill", 1, "wide"), ("prefill", 256, "wide")])
def test_pages_given_back_behind_a_window(cuda_ok, which, page, tables, f8):
    """Table entries of pages that no row sees may hold anything: they are
    neither read nor reported."""
    import torch
    q, kv, window = ([5, 3], [1000, 333], 100) if which == "decode" else ([70, 3], [1801, 777], 300)
    c = Case(q, kv, Hq=8, Hk=2, page=page, window=window, f8=f8, seed=55)
    table = wide(c) if tables == "wide" else c.cache.table_dev.clone()
    for b in range(2):
        first = kv[b] - q[b] - window + 1  # the first key that a row sees
        gone = torch.tensor([-1, 1 << 30, c.cache.n_pages], dtype=torch.int32, device="cuda")
        table[b, :first // page] = gone.repeat(first // page // 3 + 1)[:first // page]
    c.run(which, table=table)
    c.check()
    table[0, (kv[0] - 1) // page] = -1  # a page that rows see is still reported
    c.run(which, table=table)
    torch.cuda.synchronize()
    assert M.moe_last_device_error() == M.MOE_ERR_SLOT


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("page", [256, 24])
def test_never_written_places_cost_nothing(cuda_ok, page, f8):
    """NaN patterns behind the last token and before the window's first, in
    pages that hold visible tokens: same results and, within 2.5 times, the same
    time as with zeros there (the medians of 20 calls)."""
    import torch
    c = Case([700], [2900], Hq=16, Hk=2, page=page, f8=f8, window=1000, seed=56)
    table = wide(c)

    def median_us():
        ts = []
        for _ in range(20):
            e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
            e[0].record()
            c.run("prefill", table=table)
            e[1].record()
            torch.cuda.synchronize()
            ts.append(e[0].elapsed_time(e[1]))
        return sorted(ts)[10] * 1e3

    first = 2900 - 700 - 1000 + 1  # the first key that a row sees; Paged leaves NaN behind the last
    j = torch.arange(first, device="cuda")
    rows = c.cache.table_dev[0, (j // page).long()].long()
    for x in (c.cache.k, c.cache.v):
        if f8:
            x.view(torch.uint8)[rows, j % page] = 0x7f
        else:
            x[rows, j % page] = float("nan")
    median_us()
    stale = median_us()
    c.check()
    for x in (c.cache.k, c.cache.v):
        x.copy_(x.float().nan_to_num(0.0).to(x.dtype))
    clean = median_us()
    c.check()
    assert stale <= 2.5 * clean, (stale, clean)


@pytest.mark.parametrize("kv", [3000, 60000])
@pytest.mark.parametrize("slope", [0.5, 0.31, 0.0371])
def test_a_far_key_that_outweighs_its_bias(cuda_ok, slope, kv):
    """One key near the start, behind all rows, whose score passes its bias by 50:
    its softmax weight is 1 and lse is the score less the bias, both large. Eight
    roundings to fp32 (half a step, 2^-24, of the larger of the two) is what
    scale, slope, product and sums may add."""
    import torch
    n, at, D = 64, 100, 128
    c = Case([n], [kv], Hq=4, Hk=1, page=16, slopes=True, seed=57)
    c.slopes = np.full(4, slope, np.float32)
    c.t_slopes = torch.as_tensor(c.slopes).cuda()
    # q = 8 everywhere, and a key element that makes q . k scale exceed the largest bias by about 50 (whole eighths: the
    # sum of 128 equal products is exact)
    x = float(bf16(np.round((slope * kv + 50) * D ** 0.5 / (8 * D) * 8) / 8))
    c.t_q.fill_(8.0)
    c.q[:] = 8.0
    c.cache.k.zero_()
    c.cache.k[int(c.cache.table[0, at // 16]), at % 16] = x
    c.run("prefill", table=wide(c))
    torch.cuda.synchronize()
    assert M.moe_last_device_error() == 0
    score = 8.0 * x * D * float(np.float32(c.scale))
    pos = kv - n + np.arange(n)
    want = score - float(np.float32(slope)) * (pos - at)
    near = np.exp(-want) / (1 - np.exp(-slope))  # the other keys, scores of 0, next to the row at most
    assert want.min() > 25 and near.max() < 1e-9
    lse = c.lse.double().cpu().numpy()
    assert np.all(np.abs(lse - want[:, None]) <= 8 * 2.0 ** -24 * score), np.abs(lse - want[:, None]).max() / score * 2 ** 24
    v = c.values[0][at, 0]
    assert np.all(np.abs(c.out.double().cpu().numpy() - v) <= 1.01 * (2.0 ** -8 * np.abs(v) + 1e-8))


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("which,q_len,kv_len,Hq,Hk,page,window,tables", [
    ("decode", [1], [131072], 8, 1, 64, 0, "tight"), ("decode", [5], [131072], 16, 2, 64, 0, "tight"),
    ("decode", [2] * 5, [40000, 129, 77777, 1, 30011], 8, 1, 16, 0, "tight"),
    ("decode", [5, 1, 3], [60000, 20001, 128], 16, 2, 256, 0, "wide"), ("decode", [4], [70001], 8, 1, 16, 33333, "tight"),
    ("prefill", [300, 7], [20000, 33333], 4, 2, 16, 0, "wide"), ("prefill", [129], [40003], 4, 1, 24, 0, "wide"),
    ("prefill", [513, 40], [30000, 9000], 8, 1, 64, 5000, "wide"), ("prefill", [20, 3], [3000, 1111], 4, 1, 16, 0, "tight")])
def test_every_key_counts_once(cuda_ok, which, q_len, kv_len, Hq, Hk, page, window, tables, f8):
    """Equal scores (queries of zeros), and one value element per run of 128
    keys that is 1: every sum is a whole number, so the output is a count over
    the number of visible keys, and a run left out or added twice moves it."""
    import torch
    D = 128
    c = Case(q_len, kv_len, Hq=Hq, Hk=Hk, D=D, page=page, f8=f8, scales=False, window=window, seed=59)
    c.t_q.zero_()
    c.cache.v.zero_()
    for b, n in enumerate(kv_len):
        j = torch.arange(n, device="cuda")
        rows = c.cache.table_dev[b, (j // page).long()].long()
        at = torch.as_tensor(marks(n, D)).cuda()
        if f8:
            c.cache.v.view(torch.uint8)[rows, j % page, :, at] = 0x38  # 1.0
        else:
            c.cache.v[rows, j % page, :, at] = 1.0
    c.run(which, table=wide(c, 1 << 18) if tables == "wide" else None)
    torch.cuda.synchronize()
    assert M.moe_last_device_error() == 0
    out, want = marked_rows(q_len, kv_len, window, D)
    lim, lse_lim = marked_limits(out, want)
    got, lse = c.out.double().cpu().numpy(), c.lse.double().cpu().numpy()
    bad = ~(np.abs(got - out[:, None]) <= lim[:, None])
    assert not bad.any(), np.argwhere(bad)[0]
    empty = np.isneginf(want)
    assert np.isneginf(lse[empty]).all()
    assert np.all(np.abs(lse[~empty] - want[~empty][:, None]) <= lse_lim[~empty][:, None])


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("which,n,kv,Hq,Hk,page", [("decode", 5, 131072, 4, 2, 64), ("decode", 5, 131072, 16, 2, 64),
                                                   ("prefill", 40, 50000, 4, 2, 16)])
def test_long_caches_in_norm(cuda_ok, which, n, kv, Hq, Hk, page, f8):
    """Random keys and values: a bound of each row's error in the 2-norm, tight
    enough that one run of 128 keys left out breaks it (test_attn_power.py)."""
    import torch
    c = Case([n], [kv], Hq=Hq, Hk=Hk, page=page, f8=f8, seed=60)
    c.run(which)
    torch.cuda.synchronize()
    assert M.moe_last_device_error() == 0
    got = c.out.double().cpu().numpy()
    for h in range(0, Hq, Hq // 4):
        K, V = (x[0][:, h // (Hq // Hk)].astype(np.float64) for x in (c.keys, c.values))
        out, bound = noise_rows(c.q[:, h], K, V, c.scale, f8)
        off = np.linalg.norm(got[:, h] - out, axis=1)
        assert np.all(off <= bound), (h, (off / bound).max())


@pytest.mark.parametrize("tables", ["tight", "wide"])
@pytest.mark.parametrize("scale", [2.0 ** -64, 1e-30, 0.1])
def test_queries_of_zeros_and_tiny_ones_with_an_e4m3_cache(cuda_ok, scale, tables):
    """Their scores are zero, or as good as: the mean of the values that they see."""
    import torch
    c = Case([50, 9], [390, 4], Hq=4, Hk=2, page=16, f8=True, seed=86)
    gain = np.resize(2.0 ** np.array([0, -90, -120, 0, -20]), 59)
    c.q = bf16(c.q * gain[:, None, None])
    c.q[0::5] = 0.0
    c.t_q = torch.as_tensor(c.q).to(torch.bfloat16).cuda()
    c.scale = scale
    c.run("prefill", table=wide(c) if tables == "wide" else None)
    c.check()
