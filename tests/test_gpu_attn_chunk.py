"""What test_gpu_attn.py shows of small calls, shown of the tensor-core chunk
kernel: prefixes, infinities that some rows see, bad pages through its tensor
maps and through its gather, replay, repeats, streams, offsets, strides."""
import numpy as np
import pytest

import quantized_expert_ffn_top10_b200 as M
from attn_ref import attn_limits
from test_gpu_attn import Case
from test_gpu_attn_edges import wide

pytestmark = pytest.mark.gpu


def run(c, which="prefill", table=None, max_q=None, stream=None):
    """The case with a table so wide that the call counts as a large one, which the chunk kernel takes."""
    table = wide(c) if table is None else table
    most = min(max_q or (max(c.q_len) if which == "decode" else c.t_q.shape[0]), c.t_q.shape[0])
    group = c.t_q.shape[1] // c.cache.Hk
    assert most * group > 32 and c.t_q.shape[0] * group * table.shape[1] * c.cache.page >= 1 << 19
    c.run(which, table=table, max_q=max_q, stream=stream)


@pytest.mark.parametrize("page", [16, 24])
@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("window", [0, 50])
def test_prefix_rows_see_one_another(cuda_ok, f8, window, page):
    c = Case([90, 400, 30, 5], [90, 600, 30, 3], Hq=4, Hk=2, page=page, window=window, f8=f8, prefix=[33, 570, 1000, 2], seed=70)
    run(c)
    c.check()
    c = Case([5, 8], [300, 9], Hq=16, Hk=2, page=page, window=window, f8=f8, prefix=[298, 0], seed=71)
    run(c, "decode")
    c.check()


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("page,n,kv,window,back", [(16, 40, 100, 0, 2), (16, 300, 1000, 0, 250), (24, 300, 1000, 0, 130),
                                                   (64, 300, 1000, 200, 420), (16, 130, 4000, 0, 100)])
def test_values_that_are_not_finite_reach_only_rows_that_see_them(cuda_ok, page, n, kv, window, back, f8):
    """Finite keys, one value element that is infinite (e4m3 has none: NaN): rows
    that see it get it in that element alone, whatever their numerator."""
    import torch
    c = Case([n], [kv], Hq=4, Hk=2, page=page, window=window, f8=f8, seed=72)
    at = kv - back
    spot = (int(c.cache.table[0, at // page]), at % page, 0, 9)
    if f8:
        c.cache.v.view(torch.uint8)[spot] = 0x7f
    else:
        c.cache.v[spot] = float("-inf")
    run(c)
    torch.cuda.synchronize()
    assert M.moe_last_device_error() == 0
    ref, got = c.ref(), c.out.double().cpu().numpy()
    lim, _ = attn_limits(ref, c.D, kv, f8)
    ok = np.abs(got - ref[0]) <= lim
    pos = kv - n + np.arange(n)
    sees = (pos >= at) & ((pos < at + window) if window else True)
    assert sees.any() and not sees.all()
    hit = got[sees][:, 0:2, 9]
    assert np.isnan(hit).all() if f8 else np.isneginf(hit).all()
    ok[np.ix_(sees, [0, 1], [9])] = True
    assert ok.all(), np.argwhere(~ok)[0]


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("page", [16, 24, 128, 256])
def test_bad_pages_are_reported_and_read_as_zeros(cuda_ok, page, f8):
    import torch
    c = Case([30, 20], [5 * page + 40, 60], Hq=4, Hk=2, page=page, f8=f8, seed=73)
    table = wide(c)
    table[0, 1], table[0, 2] = c.cache.n_pages, -1
    run(c, table=table)
    torch.cuda.synchronize()
    assert M.moe_last_device_error() == M.MOE_ERR_SLOT
    assert M.moe_last_device_error() == 0
    for x in (c.keys, c.values):
        x[0][page:3 * page] = 0.0
    c.check()


def test_rows_behind_the_last_request_stay(cuda_ok):
    import torch
    c = Case([30, 25], [400, 90], Hq=4, Hk=2, page=16, seed=74)
    n, T = 55, 80
    c.t_q = torch.cat([c.t_q, torch.full((T - n, 4, 128), float("nan"), dtype=torch.bfloat16, device="cuda")])
    out = torch.full((T, 4, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, 4), 3.0, device="cuda")
    c.out, c.lse = out, lse
    run(c)
    torch.cuda.synchronize()
    assert bool((out[n:] == 3.0).all()) and bool((lse[n:] == 3.0).all())
    c.out, c.lse = out[:n], lse[:n]
    c.check()


@pytest.mark.parametrize("which", ["decode", "prefill"])
def test_offsets_outside_the_step_touch_nothing(cuda_ok, which):
    import torch
    c = Case([8, 6], [400, 90], Hq=32, Hk=2, page=16, seed=75)
    for cu in ([0, 0, 0], [14, 14, 14], [17, 900, 3], [-4, -2, -1]):
        c.cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        c.out.fill_(7.0)
        run(c, which, max_q=8)
        torch.cuda.synchronize()
        assert M.moe_last_device_error() == 0
        assert bool((c.out == 7.0).all()), cu
    c.cu = torch.tensor([0, 8, 1 << 30], dtype=torch.int32, device="cuda")  # cut to the rows there are
    run(c, which, max_q=8)
    c.check()


def test_strided_queries(cuda_ok):
    import torch
    c = Case([40], [277], Hq=4, Hk=2, page=16, seed=76)
    big = torch.full((40, 8, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    big[:, 2:6] = c.t_q
    c.t_q = big[:, 2:6]
    run(c)
    c.check()


def test_large_and_tiny_queries_with_an_e4m3_cache(cuda_ok):
    """Rows of queries far outside fp16's range, and rows of zeros."""
    import torch
    c = Case([50], [390], Hq=4, Hk=2, page=16, f8=True, seed=77)
    gain = np.resize(2.0 ** np.array([60, -90, 0, 20, -20]), 50)
    c.q *= gain[:, None, None]
    c.q[2::5] = 0.0
    c.t_q = torch.as_tensor(c.q).to(torch.bfloat16).cuda()
    c.scale = 2.0 ** -64 * c.scale
    run(c)
    c.check()


def test_more_requests_than_a_cta_keeps(cuda_ok):
    rng = np.random.default_rng(78)
    q = [int(x) for x in rng.integers(0, 4, 1300)]
    c = Case(q, [x + int(y) for x, y in zip(q, rng.integers(0, 60, 1300))], Hq=16, Hk=1, D=64, page=16, seed=78)
    run(c, table=wide(c, 1 << 10))
    c.check()
    run(c, "decode", table=wide(c, 1 << 10))
    c.check()


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("which", ["decode", "prefill"])
def test_repeated_calls_are_bit_identical(cuda_ok, which, f8):
    """Items cut over many CTAs, and short ones beside them."""
    import torch
    c = Case([5, 3, 8] if which == "decode" else [500, 3, 700], [30000, 17, 9000], Hq=16, Hk=2, page=16, f8=f8, seed=79)
    run(c, which)
    first = (c.out.clone(), c.lse.clone())
    c.check()
    for _ in range(3):
        c.out.fill_(0)
        run(c, which)
        torch.cuda.synchronize()
        assert torch.equal(c.out, first[0]) and torch.equal(c.lse, first[1])


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("which", ["decode", "prefill"])
def test_captured_call_follows_new_lengths(cuda_ok, which, f8):
    """The tensor maps of a captured call stand for the cache, not for its lengths or its table."""
    import torch
    q = ([5, 2], [1, 6]) if which == "decode" else ([130, 7], [37, 100])
    a = Case(q[0], [2700, 30], Hq=16, Hk=2, page=16, f8=f8, scales=False, seed=80)
    b = Case(q[1], [90, 2655], Hq=16, Hk=2, page=16, f8=f8, scales=False, seed=81)
    n_pages = max(a.cache.n_pages, b.cache.n_pages)
    k = torch.zeros((n_pages, 16, 2, 128), dtype=a.cache.k.dtype, device="cuda")
    v = torch.zeros_like(k)
    table = torch.full((2, 1 << 12), -1, dtype=torch.int32, device="cuda")
    hold = Case(q[0], [2700, 30], Hq=16, Hk=2, page=16, f8=f8, scales=False, seed=82)
    hold.desc = M.moe_kv_desc(k, v, 16)
    T = hold.t_q.shape[0]
    run(hold, which, table=table, max_q=8 if which == "decode" else None)
    torch.cuda.synchronize()
    M.moe_last_device_error()  # (no pages yet)
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        run(hold, which, table=table, max_q=8 if which == "decode" else None)
    for c in (a, b, a):
        n = c.t_q.shape[0]
        assert n <= T
        k[:c.cache.n_pages], v[:c.cache.n_pages] = c.cache.k, c.cache.v
        table.fill_(-1)
        table[:, :c.cache.table.shape[1]] = c.cache.table_dev
        hold.t_q[:n] = c.t_q
        hold.kv.copy_(c.kv)
        hold.cu.copy_(c.cu)
        hold.out.fill_(0)
        g.replay()
        torch.cuda.synchronize()
        c.out, c.lse = hold.out[:n].clone(), hold.lse[:n].clone()
        c.check()
        assert bool((hold.out[n:] == 0).all())


def test_two_streams_with_a_workspace_each(cuda_ok):
    import torch
    cs = [Case([200], [4000 + 100 * i], Hq=16, Hk=2, page=16, f8=bool(i), seed=83 + i) for i in range(2)]
    tables = [wide(c) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s, t in zip(cs, streams, tables):
            run(c, stream=s, table=t)
    for c in cs:
        c.check()


@pytest.mark.parametrize("extra", [dict(), dict(f8=True), dict(softcap=20.0, slopes=True), dict(window=300, f8=True)])
def test_negative_and_zero_scales(cuda_ok, extra):
    """Scores of the other sign, and equal ones."""
    for scale in (-0.05, 0.0):
        c = Case([60, 7], [900, 300], Hq=4, Hk=2, page=16, seed=85, **extra)
        c.scale = scale
        run(c)
        c.check()
        c.run("prefill")
        c.check()
