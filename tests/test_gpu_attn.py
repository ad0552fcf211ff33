"""Attention over the paged cache against a 64-bit reference: head layouts,
types, odd lengths and pages, masks that leave rows empty, non-finite values in
hidden places, bad pages, captured calls, streams."""
import numpy as np
import pytest

import quantized_expert_ffn_top10_b200 as M
from attn_ref import Paged, attn_limits, attn_ref, bf16, e4m3

pytestmark = pytest.mark.gpu


class Case:
    """A seeded call: what the library gets, and the reference's inputs."""

    def __init__(self, q_len, kv_len, Hq=16, Hk=2, D=128, f8=False, page=16, softcap=0.0, window=0, slopes=False,
                 prefix=None, seed=1, q_gain=1.5, scales=True, **paged):
        import torch
        rng = np.random.default_rng(seed)
        self.q_len, self.kv_len, self.D, self.f8 = q_len, kv_len, D, f8
        T = sum(q_len)
        rnd = e4m3 if f8 else bf16
        self.q = bf16(rng.standard_normal((T, Hq, D)) * q_gain)
        ks = rng.uniform(0.2, 0.5, Hk).astype(np.float32) if f8 and scales else None
        vs = rng.uniform(0.2, 0.5, Hk).astype(np.float32) if f8 and scales else None
        gain = 3.0 if f8 else 1.0
        raw_k = [rnd(rng.standard_normal((max(n, 0), Hk, D)) * gain) for n in kv_len]
        raw_v = [rnd(rng.standard_normal((max(n, 0), Hk, D)) * gain) for n in kv_len]
        self.cache = Paged(raw_k, raw_v, page, f8, seed=seed, k_scale=ks, v_scale=vs, **paged)
        self.keys = [k if ks is None else k * ks[:, None].astype(np.float64) for k in raw_k]
        self.values = [v if vs is None else v * vs[:, None].astype(np.float64) for v in raw_v]
        self.opt = dict(softcap=softcap, window=window)
        self.slopes = 2.0 ** (-8.0 * np.arange(1, Hq + 1) / Hq) if slopes else None
        self.slopes = None if self.slopes is None else self.slopes.astype(np.float32)
        self.prefix = prefix
        self.scale = D ** -0.5
        self.desc = self.cache.desc(Hq)
        dev = "cuda"
        i32 = dict(dtype=torch.int32, device=dev)
        self.t_q = torch.as_tensor(self.q).to(torch.bfloat16).to(dev)
        self.cu = torch.tensor([0] + list(np.cumsum(q_len)), **i32)
        self.kv = torch.tensor(kv_len, **i32)
        self.t_slopes = None if self.slopes is None else torch.as_tensor(self.slopes).to(dev)
        self.t_prefix = None if prefix is None else torch.tensor(prefix, **i32)
        self.out = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device=dev)
        self.lse = torch.full((T, Hq), 7.0, dtype=torch.float32, device=dev)
        n = M.moe_attn_workspace_bytes(T, len(q_len), Hq, Hk, D)
        self.ws = torch.full((n,), 255, dtype=torch.uint8, device=dev)  # NaN patterns: nothing of it may count

    def run(self, which, stream=None, max_q=None, table=None):
        kw = dict(slopes=self.t_slopes, prefix=self.t_prefix, lse=self.lse, stream=stream, **self.opt)
        table = self.cache.table_dev if table is None else table
        if which == "decode":
            M.moe_attn_decode(self.desc, self.t_q, self.cu, self.kv, table, self.out, max_q or max(self.q_len + [1]), self.ws,
                              self.scale, **kw)
        else:
            M.moe_attn_prefill(self.desc, self.t_q, self.cu, self.kv, table, self.out, self.ws, self.scale, **kw)

    def ref(self):
        return attn_ref(self.q, self.keys, self.values, self.q_len, self.kv_len, self.scale, slopes=self.slopes,
                        prefix=self.prefix, **self.opt)

    def check(self, ref=None):
        import torch
        torch.cuda.synchronize()
        assert M.moe_last_device_error() == 0
        ref = ref or self.ref()
        lim, lse_lim = attn_limits(ref, self.D, max(self.kv_len), self.f8)
        got, lse = self.out.double().cpu().numpy(), self.lse.double().cpu().numpy()
        bad = ~(np.abs(got - ref[0]) <= lim)
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[0], got[bad][:3], ref[0][bad][:3])
        empty = np.isneginf(ref[1])
        assert np.array_equal(np.isneginf(lse), empty)
        with np.errstate(invalid="ignore"):
            off = np.abs(lse - ref[1])
        assert np.all((off <= lse_lim) | empty), np.nanmax(np.where(empty, 0, off))


SHAPES = [
    dict(q_len=[1], kv_len=[1]),
    dict(q_len=[1], kv_len=[2], Hq=1, Hk=1, D=64),
    dict(q_len=[1], kv_len=[997]),
    dict(q_len=[1], kv_len=[64], Hq=8, Hk=8, D=64, page=1),
    dict(q_len=[5], kv_len=[63], Hq=6, Hk=2, page=48),
    dict(q_len=[5], kv_len=[65], Hq=10, Hk=2, page=128, head_major=True),
    dict(q_len=[8], kv_len=[8], Hq=16, Hk=1),
    dict(q_len=[3, 0, 1, 5, 0], kv_len=[700, 40, 1, 5, 0], Hq=12, Hk=4, D=64, page=8),
    dict(q_len=[5, 5, 2], kv_len=[3, 5, 0]),                       # rows before the first key: empty
    dict(q_len=[8] * 3, kv_len=[300, 1025, 64], Hq=32, Hk=2),      # 128 rows share a cached head
    dict(q_len=[1] * 40, kv_len=list(range(1, 400, 10)), Hq=8, Hk=4, D=64, page=16, head_major=True),
    dict(q_len=[2] * 7, kv_len=[2000, 3, 17, 129, 500, 256, 2], Hq=20, Hk=4, page=32, one_buffer=True),
    dict(q_len=[5], kv_len=[6000], Hq=16, Hk=2, page=64),          # one request over every CTA
    # wide windows over long caches: the chunk kernel, its two key streams, items cut over many CTAs
    dict(q_len=[5], kv_len=[20011], Hq=16, Hk=2, page=64),
    dict(q_len=[8], kv_len=[9000], Hq=10, Hk=1, page=24),
    dict(q_len=[5, 4, 0, 5, 1, 5], kv_len=[3000, 129, 7, 2048, 5000, 4], Hq=20, Hk=2, D=64, page=256, head_major=True),
    dict(q_len=[8] * 12, kv_len=[128 * i + i for i in range(1, 13)], Hq=32, Hk=2, page=8, one_buffer=True),
]
EXTRAS = [
    dict(softcap=50.0, q_gain=0.5), dict(softcap=50.0, q_gain=40.0, f8=True),  # far below the cap, and far above
    dict(), dict(f8=True), dict(f8=True, scales=False, softcap=20.0), dict(softcap=15.0, window=37), dict(slopes=True),
    dict(window=1), dict(f8=True, slopes=True, window=100),
]


@pytest.mark.parametrize("extra", range(len(EXTRAS)))
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_decode(cuda_ok, shape, extra):
    c = Case(**{**SHAPES[shape], **EXTRAS[extra]}, seed=100 * shape + extra)
    c.run("decode")
    c.check()


CHUNKS = [
    dict(q_len=[1], kv_len=[1]),
    dict(q_len=[37], kv_len=[37], Hq=4, Hk=2),
    dict(q_len=[129], kv_len=[400], Hq=5, Hk=1, D=64, page=48),
    dict(q_len=[64, 0, 33, 1], kv_len=[64, 9, 500, 77], Hq=6, Hk=2, page=8, head_major=True),
    dict(q_len=[200], kv_len=[90], Hq=3, Hk=3, D=64),              # rows before the first key
    dict(q_len=[300, 17], kv_len=[1300, 17], Hq=8, Hk=1, page=64),
    dict(q_len=[257], kv_len=[257], Hq=16, Hk=2, page=1),
    dict(q_len=[1500], kv_len=[2900], Hq=16, Hk=2, page=64),       # several items, and cut ones, in every CTA
    dict(q_len=[700, 900, 11], kv_len=[700, 2222, 2000], Hq=12, Hk=4, D=64, page=16, head_major=True),
    dict(q_len=[500, 40], kv_len=[1500, 3000], Hq=8, Hk=2, page=24),
]


@pytest.mark.parametrize("extra", range(len(EXTRAS)))
@pytest.mark.parametrize("shape", range(len(CHUNKS)))
def test_prefill(cuda_ok, shape, extra):
    c = Case(**{**CHUNKS[shape], **EXTRAS[extra]}, seed=7000 + 100 * shape + extra)
    c.run("prefill")
    c.check()


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("window", [0, 50])
def test_prefix_rows_see_one_another(cuda_ok, f8, window):
    """Tokens inside the prefix see the whole prefix; those behind it are causal."""
    c = Case([90, 40, 30], [90, 200, 30], Hq=4, Hk=2, page=16, f8=f8, window=window, prefix=[33, 170, 1000], seed=5)
    c.run("prefill")
    c.check()
    c = Case([5, 8], [70, 9], Hq=4, Hk=2, page=16, f8=f8, window=window, prefix=[68, 0], seed=6)
    c.run("decode")
    c.check()


@pytest.mark.parametrize("which", ["decode", "prefill"])
@pytest.mark.parametrize("f8", [False, True])
def test_hidden_values_never_count(cuda_ok, which, f8):
    """NaN and infinite keys and values that the mask hides from a row do not
    reach it (they may reach the rows that see them): the last cached tokens of
    a causal window, and the first ones of a sliding window."""
    import torch
    n, kv = (5, 150) if which == "decode" else (70, 2500)
    for window, at in ((0, kv - 1), (0, kv - 2), (20, 3 if which == "decode" else kv - 65)):
        c = Case([n], [kv], Hq=6, Hk=2, page=16, f8=f8, window=window, seed=11)
        page, off = int(c.cache.table[0, at // 16]), at % 16
        for x, vals in ((c.cache.k, (np.nan,)), (c.cache.v, (np.nan, np.nan) if f8 else (np.inf, np.nan))):
            row = torch.as_tensor(np.resize(np.array(vals, np.float32), c.D))
            x[page, off, 1] = row.to(x.dtype).to(x.device)
        c.run(which)
        torch.cuda.synchronize()
        assert M.moe_last_device_error() == 0
        ref = c.ref()  # built before the poison
        got = c.out.double().cpu().numpy()
        lim, _ = attn_limits(ref, c.D, kv, f8)
        for i in range(n):
            pos = kv - n + i
            sees = at <= pos and (not window or at > pos - window)
            heads = slice(0, 3) if sees else slice(0, 6)  # cached head 1 serves heads 3 to 5
            assert np.all(np.abs(got[i, heads] - ref[0][i, heads]) <= lim[i, heads]), (window, at, i)
            if sees:
                assert np.isnan(got[i, 3:]).all()


@pytest.mark.parametrize("which", ["decode", "prefill"])
def test_hidden_infinite_values_reach_only_rows_that_see_them(cuda_ok, which):
    """Finite keys, one infinite value element in the newest token: rows that
    see it get that infinity in that element alone."""
    import torch
    n, kv = (5, 100) if which == "decode" else (40, 100)
    c = Case([n], [kv], Hq=4, Hk=2, page=16, seed=12)
    at = kv - 2
    c.cache.v[int(c.cache.table[0, at // 16]), at % 16, 0, 9] = float("-inf")
    c.run(which)
    torch.cuda.synchronize()
    ref, got = c.ref(), c.out.double().cpu().numpy()
    lim, _ = attn_limits(ref, c.D, kv, False)
    for i in range(n):
        ok = np.abs(got[i] - ref[0][i]) <= lim[i]
        if kv - n + i >= at:
            assert np.isneginf(got[i, 0:2, 9]).all()
            ok[0:2, 9] = True
        assert ok.all(), i


@pytest.mark.parametrize("which", ["decode", "prefill"])
def test_rows_behind_the_last_request_stay(cuda_ok, which):
    import torch
    c = Case([3, 2], [40, 9], Hq=4, Hk=2, page=16, seed=13)
    T = 9
    c.t_q = torch.cat([c.t_q, torch.full((T - 5, 4, 128), float("nan"), dtype=torch.bfloat16, device="cuda")])
    out = torch.full((T, 4, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, 4), 3.0, device="cuda")
    c.out, c.lse = out, lse
    c.run(which)
    torch.cuda.synchronize()
    assert bool((out[5:] == 3.0).all()) and bool((lse[5:] == 3.0).all())
    c.out, c.lse = out[:5], lse[:5]
    c.check()


@pytest.mark.parametrize("which", ["decode", "prefill"])
def test_bad_pages_are_reported_and_read_as_zeros(cuda_ok, which):
    import torch
    c = Case([2, 2], [50, 40], Hq=4, Hk=2, page=16, seed=14)
    table = c.cache.table_dev.clone()
    table[0, 1] = c.cache.n_pages        # one past the cache
    table[0, 2] = -1
    c.run(which, table=table)
    torch.cuda.synchronize()
    assert M.moe_last_device_error() == M.MOE_ERR_SLOT
    assert M.moe_last_device_error() == 0
    for x in (c.keys, c.values):
        x[0][16:48] = 0.0
    c.check()


@pytest.mark.parametrize("f8", [False, True])
def test_a_window_over_a_128k_cache(cuda_ok, f8):
    """Every CTA holds a piece of one of two heads, some of both."""
    c = Case([5], [131072], Hq=16, Hk=2, page=64, f8=f8, seed=23)
    c.run("decode")
    c.check()


def test_many_requests(cuda_ok):
    """More requests than a CTA keeps the lengths of."""
    rng = np.random.default_rng(24)
    n = 1300
    c = Case([1] * n, [int(x) for x in rng.integers(0, 70, n)], Hq=2, Hk=1, D=64, page=16, seed=24)
    c.run("decode")
    c.check()
    q = [int(x) for x in rng.integers(0, 3, n)]
    c = Case(q, [x + 5 for x in q], Hq=3, Hk=1, D=64, page=16, seed=25)
    c.run("prefill")
    c.check()


@pytest.mark.parametrize("which", ["decode", "prefill"])
def test_offsets_outside_the_step_touch_nothing(cuda_ok, which):
    """Offsets past the rows, falling ones, and requests without rows."""
    import torch
    c = Case([3, 2], [40, 9], Hq=4, Hk=2, page=16, seed=26)
    for cu in ([0, 0, 0], [5, 5, 5], [7, 900, 3], [-4, -2, -1]):
        c.cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        c.out.fill_(7.0)
        c.run(which, max_q=8)
        torch.cuda.synchronize()
        assert M.moe_last_device_error() == 0
        assert bool((c.out == 7.0).all()), cu
    c.cu = torch.tensor([0, 3, 1 << 30], dtype=torch.int32, device="cuda")  # cut to the rows there are
    c.out.fill_(7.0)
    c.run(which, max_q=8)
    c.check()


def test_windows_wider_than_promised_are_cut(cuda_ok):
    """Rows past max_q of a request are left as they were."""
    import torch
    c = Case([3], [40], Hq=4, Hk=2, page=16, seed=27)
    c.run("decode", max_q=2)
    torch.cuda.synchronize()
    assert bool((c.out[2] == 7.0).all()) and not bool((c.out[0] == 7.0).all())


def test_lengths_past_the_table_are_cut(cuda_ok):
    import torch
    c = Case([1], [32], Hq=4, Hk=2, page=16, seed=15)
    c.kv = torch.tensor([1 << 30], dtype=torch.int32, device="cuda")
    c.run("decode", table=c.cache.table_dev[:, :2].contiguous())
    c.check()


def test_strided_queries(cuda_ok):
    """Queries as a slice of a wider row (a fused projection)."""
    import torch
    c = Case([4], [77], Hq=4, Hk=2, page=16, seed=16)
    wide = torch.full((4, 8, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 2:6] = c.t_q
    c.t_q = wide[:, 2:6]
    c.run("decode")
    c.check()


def test_large_and_tiny_queries_with_an_e4m3_cache(cuda_ok):
    """Rows of queries far outside fp16's range, and a row of zeros."""
    import torch
    c = Case([5], [90], Hq=4, Hk=2, page=16, f8=True, seed=17)
    gain = 2.0 ** np.array([60, -90, 0, 20, -20])
    c.q *= gain[:, None, None]
    c.q[2] = 0.0
    c.t_q = torch.as_tensor(c.q).to(torch.bfloat16).cuda()
    c.scale = 2.0 ** -64 * c.scale
    c.run("decode")
    c.check()


@pytest.mark.parametrize("which", ["decode", "prefill"])
def test_repeated_calls_are_bit_identical(cuda_ok, which):
    import torch
    c = Case([5, 3, 8], [3000, 17, 900], Hq=16, Hk=2, page=16, seed=18)
    c.run(which)
    first = (c.out.clone(), c.lse.clone())
    for _ in range(3):
        c.out.fill_(0)
        c.run(which)
        torch.cuda.synchronize()
        assert torch.equal(c.out, first[0]) and torch.equal(c.lse, first[1])


@pytest.mark.parametrize("which", ["decode", "prefill"])
def test_captured_call_follows_new_lengths(cuda_ok, which):
    """A captured call reads lengths, tables and rows at replay."""
    import torch
    a = Case([5, 2], [700, 30], Hq=8, Hk=2, page=16, seed=19)
    b = Case([1, 6], [90, 655], Hq=8, Hk=2, page=16, seed=20)
    a.run(which)
    torch.cuda.synchronize()
    n_pages = max(a.cache.n_pages, b.cache.n_pages)
    k = torch.zeros((n_pages, 16, 2, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    width = max(a.cache.table.shape[1], b.cache.table.shape[1])
    table = torch.full((2, width), -1, dtype=torch.int32, device="cuda")
    hold = Case([5, 2], [700, 30], Hq=8, Hk=2, page=16, seed=21)
    hold.desc = M.moe_kv_desc(k, v, 8)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        hold.run(which, max_q=8, table=table)
    for c in (a, b, a):
        k[:c.cache.n_pages], v[:c.cache.n_pages] = c.cache.k, c.cache.v
        table.fill_(-1)
        table[:, :c.cache.table.shape[1]] = c.cache.table_dev
        hold.t_q.copy_(c.t_q)
        hold.kv.copy_(c.kv)
        hold.cu.copy_(c.cu)
        hold.out.fill_(0)
        g.replay()
        torch.cuda.synchronize()
        c.out, c.lse = hold.out.clone(), hold.lse.clone()
        c.check()


def test_two_streams_with_a_workspace_each(cuda_ok):
    import torch
    cs = [Case([5], [4000 + 100 * i], Hq=16, Hk=2, page=16, seed=30 + i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s in zip(cs, streams):
            c.run("decode", stream=s)
    for c in cs:
        c.check()


def test_wrong_tensors_are_refused(cuda_ok):
    import torch
    c = Case([2], [20], Hq=4, Hk=2, page=16, seed=22)
    for name, bad in (("t_q", c.t_q.float()), ("cu", c.cu.long()), ("kv", c.kv.cpu()), ("out", c.out[:, :2]),
                      ("lse", c.lse.double()), ("ws", c.ws[:256])):
        good = getattr(c, name)
        setattr(c, name, bad)
        with pytest.raises(M.MoeError):
            c.run("decode")
        setattr(c, name, good)
    with pytest.raises(M.MoeError):
        M.moe_kv_desc(c.cache.k, c.cache.v.float(), 4)
    with pytest.raises(M.MoeError):
        M.moe_kv_desc(c.cache.k, c.cache.v[:, :8], 4)
    torch.cuda.synchronize()
    assert bool((c.out == 7.0).all())


@pytest.mark.parametrize("f8", [False, True])
def test_caches_as_plain_bits(cuda_ok, f8):
    """int16 stands for bf16 and uint8 for e4m3, for queries and outputs too."""
    import torch
    c = Case([2], [50], Hq=4, Hk=2, page=16, f8=f8, seed=28)
    bits = torch.uint8 if f8 else torch.int16
    c.desc = M.moe_kv_desc(c.cache.k.view(bits), c.cache.v.view(bits), 4, c.cache.k_scale, c.cache.v_scale)
    out, c.t_q = c.out, c.t_q.view(torch.int16)
    c.out = out.view(torch.int16)
    c.run("decode")
    c.out = out
    c.check()


def test_empty_batches(cuda_ok):
    """A step whose requests all sit out, and one without requests, change nothing."""
    import torch
    c = Case([2, 1], [50, 9], Hq=4, Hk=2, page=16, seed=29)
    c.cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    for which in ("decode", "prefill"):
        c.run(which, max_q=4)
    c.kv, c.cu = c.kv[:0], c.cu[:1]
    for which in ("decode", "prefill"):
        c.run(which, max_q=4, table=c.cache.table_dev[:0])
    torch.cuda.synchronize()
    assert M.moe_last_device_error() == 0 and bool((c.out == 7.0).all()) and bool((c.lse == 7.0).all())
