"""The attention half's C ABI without a GPU: host-side refusals come before any
CUDA call, and the rotation frequencies agree with their formulas."""
import ctypes
import math

import numpy as np
import pytest

import quantized_expert_ffn_top10_b200 as M
from quantized_expert_ffn_top10_b200 import build as B

FAKE = 1 << 24  # aligned addresses that are never dereferenced: every call below fails a host check first


@pytest.fixture(scope="module")
def lib():
    B.build()
    return M.lib()


def _desc(**kw):
    f = dict(k_cache=FAKE, v_cache=2 * FAKE, k_scale=None, v_scale=None, page_stride=16 * 256, token_stride=256,
             head_stride=128, n_pages=10, page_size=16, n_heads=16, n_kv_heads=2, head_dim=128, kv_type=M.MOE_KV_BF16)
    f.update(kw)
    d = M.KvDesc()
    for k, v in f.items():
        setattr(d, k, v)
    return d


def _attn(lib, which="decode", desc=None, q=3 * FAKE, q_stride=2048, T=5, cu=4 * FAKE, kv=5 * FAKE, Bn=1, table=6 * FAKE,
          width=10, max_q=5, scale=0.1, softcap=0.0, window=0, slopes=None, prefix=None, out=7 * FAKE, lse=None,
          ws=8 * FAKE, ws_bytes=1 << 40):
    d = desc if desc is not None else _desc()
    mq = (max_q,) if which == "decode" else ()
    fn = lib.moe_attn_decode if which == "decode" else lib.moe_attn_prefill
    return fn(ctypes.byref(d), q, q_stride, T, cu, kv, Bn, table, width, *mq, scale, softcap, window, slopes, prefix,
              out, lse, ws, ws_bytes, None)


DESC_CASES = [
    (dict(k_cache=None), M.MOE_ERR_ARG), (dict(v_cache=2 * FAKE + 8), M.MOE_ERR_ARG),
    (dict(head_dim=96), M.MOE_ERR_SHAPE), (dict(n_heads=15), M.MOE_ERR_SHAPE), (dict(n_kv_heads=0), M.MOE_ERR_SHAPE),
    (dict(n_heads=1024, n_kv_heads=2), M.MOE_ERR_SHAPE), (dict(kv_type=2), M.MOE_ERR_SHAPE),
    (dict(token_stride=252), M.MOE_ERR_SHAPE), (dict(head_stride=-128), M.MOE_ERR_SHAPE),
    (dict(kv_type=M.MOE_KV_E4M3, token_stride=264), M.MOE_ERR_SHAPE),
    (dict(n_pages=0), M.MOE_ERR_RANGE), (dict(page_size=0), M.MOE_ERR_RANGE),
    (dict(n_pages=1 << 20, page_size=1 << 12), M.MOE_ERR_RANGE),
    (dict(k_scale=FAKE), M.MOE_ERR_ARG),                                  # a bf16 cache has no scales
    (dict(kv_type=M.MOE_KV_E4M3, k_scale=FAKE + 2), M.MOE_ERR_ARG),
]


@pytest.mark.parametrize("change,code", DESC_CASES)
def test_cache_descriptor_refusals(lib, change, code):
    assert _attn(lib, desc=_desc(**change)) == code
    assert _attn(lib, "prefill", desc=_desc(**change)) == code
    assert _rope(lib, desc=_desc(**change)) == code


def test_reserved_fields_must_be_zero(lib):
    d = _desc()
    d.reserved[1] = 1
    assert _attn(lib, desc=d) == M.MOE_ERR_SHAPE


@pytest.mark.parametrize("which", ["decode", "prefill"])
def test_attention_refusals(lib, which):
    a = lambda **kw: _attn(lib, which, **kw)  # noqa: E731
    assert a(T=-1) == M.MOE_ERR_RANGE
    assert a(T=M.MOE_PREFILL_MAX_T + 1 if which == "prefill" else M.MOE_ATTN_MAX_B * 8 + 1) == M.MOE_ERR_RANGE
    assert a(Bn=-1) == M.MOE_ERR_RANGE and a(Bn=M.MOE_ATTN_MAX_B + 1) == M.MOE_ERR_RANGE
    assert a(width=0) == M.MOE_ERR_RANGE
    assert a(window=-1) == M.MOE_ERR_RANGE
    assert a(softcap=-1.0) == M.MOE_ERR_RANGE and a(softcap=math.nan) == M.MOE_ERR_RANGE
    assert a(softcap=math.inf) == M.MOE_ERR_RANGE and a(scale=math.nan) == M.MOE_ERR_RANGE
    assert a(softcap=1e-38) == M.MOE_ERR_RANGE
    assert a(q_stride=2040) == M.MOE_ERR_SHAPE and a(q_stride=2052) == M.MOE_ERR_SHAPE
    for name in ("q", "cu", "kv", "table", "out", "ws"):
        assert a(**{name: None}) == M.MOE_ERR_ARG, name
    assert a(q=3 * FAKE + 8) == M.MOE_ERR_ARG and a(out=7 * FAKE + 2) == M.MOE_ERR_ARG
    assert a(ws=8 * FAKE + 128) == M.MOE_ERR_ARG and a(cu=4 * FAKE + 1) == M.MOE_ERR_ARG
    assert a(slopes=FAKE + 2) == M.MOE_ERR_ARG and a(lse=FAKE + 2) == M.MOE_ERR_ARG
    assert a(out=3 * FAKE + 64) == M.MOE_ERR_ARG                           # overlaps q
    need = M.moe_attn_workspace_bytes(5, 1, 16, 2, 128)
    assert need > 0 and a(ws_bytes=need - 1) == M.MOE_ERR_WS
    assert a(T=0) == M.MOE_OK and a(Bn=0) == M.MOE_OK
    if which == "decode":
        assert a(max_q=0) == M.MOE_ERR_RANGE and a(max_q=M.MOE_DECODE_MAX_T + 1) == M.MOE_ERR_RANGE


def test_attention_workspace(lib):
    assert M.moe_attn_workspace_bytes(1, 1, 16, 2, 128) % 256 == 0
    for bad in ((-1, 1, 16, 2, 128), (1, 1, 15, 2, 128), (1, 1, 16, 2, 80), (1, 1, 0, 1, 64)):
        assert M.moe_attn_workspace_bytes(*bad) == 0


def test_no_workspace_for_sizes_that_no_call_takes(lib):
    most = M.MOE_ATTN_MAX_B * M.MOE_DECODE_MAX_T
    assert M.moe_attn_workspace_bytes(most, M.MOE_ATTN_MAX_B, M.MOE_ATTN_MAX_HEADS, 1, 64) > 0
    for bad in ((most + 1, 1, 16, 2, 128), (5, M.MOE_ATTN_MAX_B + 1, 16, 2, 128), (5, 1, M.MOE_ATTN_MAX_HEADS + 1, 1, 64)):
        assert M.moe_attn_workspace_bytes(*bad) == 0


def _rope(lib, desc=None, q=3 * FAKE, qs=2560, k=3 * FAKE + 4096, ks=2560, v=3 * FAKE + 4608, vs=2560, T=5, pos=4 * FAKE,
          slot=5 * FAKE, qn=None, kn=None, eps=1e-6, inv=6 * FAKE, rot=128, scale=1.0, out=7 * FAKE, os_=2048):
    d = desc if desc is not None else _desc()
    return lib.moe_qk_norm_rope(ctypes.byref(d), q, qs, k, ks, v, vs, T, pos, slot, qn, kn, eps, inv, rot, 0, scale, out,
                                os_, None)


def test_rope_refusals(lib):
    r = lambda **kw: _rope(lib, **kw)  # noqa: E731
    assert r(T=-1) == M.MOE_ERR_RANGE and r(T=M.MOE_KV_MAP_MAX_T + 1) == M.MOE_ERR_RANGE
    assert r(eps=-1.0) == M.MOE_ERR_RANGE and r(eps=math.nan) == M.MOE_ERR_RANGE and r(scale=math.inf) == M.MOE_ERR_RANGE
    assert r(rot=8) == M.MOE_ERR_SHAPE and r(rot=144) == M.MOE_ERR_SHAPE and r(rot=-16) == M.MOE_ERR_SHAPE
    assert r(qs=2040) == M.MOE_ERR_SHAPE and r(ks=2564) == M.MOE_ERR_SHAPE and r(vs=128) == M.MOE_ERR_SHAPE
    assert r(os_=1024) == M.MOE_ERR_SHAPE
    for name in ("q", "k", "v", "pos", "slot", "inv", "out"):
        assert r(**{name: None}) == M.MOE_ERR_ARG, name
    assert r(k=3 * FAKE + 4104) == M.MOE_ERR_ARG and r(pos=4 * FAKE + 2) == M.MOE_ERR_ARG
    assert r(qn=FAKE + 4) == M.MOE_ERR_ARG and r(kn=FAKE + 8) == M.MOE_ERR_ARG
    assert r(out=3 * FAKE + 16) == M.MOE_ERR_ARG            # q_out overlaps q without being q
    assert r(out=3 * FAKE, os_=2048) == M.MOE_ERR_ARG       # q itself, but rows at another stride
    assert r(T=0) == M.MOE_OK
    assert r(T=0, inv=None, rot=0) == M.MOE_OK


def test_rope_outputs_over_its_inputs_are_refused(lib):
    """q_out over keys or values, whole or in part: of a fused buffer with as many
    cached heads as query heads (rows of 256 + 256 + 256), and of their own buffers."""
    d = _desc(n_heads=2)
    fused = dict(desc=d, qs=768, k=3 * FAKE + 512, ks=768, v=3 * FAKE + 1024, vs=768)
    r = lambda **kw: _rope(lib, **{**fused, **kw})  # noqa: E731
    for at in (512, 1024, 512 + 16, 1024 - 16):                # the keys, the values, parts of both
        for token in (0, 1, 4):
            assert r(out=3 * FAKE + at + token * 2 * 768, os_=768) == M.MOE_ERR_ARG, (at, token)
    assert r(out=3 * FAKE + 512, os_=512) == M.MOE_ERR_ARG     # at another stride
    own = dict(desc=d, qs=256, k=5 * FAKE, ks=256, v=6 * FAKE, vs=256, os_=256)
    for out in (5 * FAKE, 6 * FAKE, 5 * FAKE + 512, 6 * FAKE - 16):
        assert _rope(lib, out=out, **own) == M.MOE_ERR_ARG
    assert _rope(lib, out=5 * FAKE + 16, **{**own, "ks": 512, "os_": 512}) == M.MOE_ERR_ARG


def _map(lib, kv=FAKE, q=2 * FAKE, Bn=4, page=16, free=3 * FAKE, n_free=10, table=4 * FAKE, width=8, T=9, kvn=5 * FAKE,
         cu=6 * FAKE, pos=7 * FAKE, slot=8 * FAKE, used=9 * FAKE):
    return lib.moe_kv_map(kv, q, Bn, page, free, n_free, table, width, T, kvn, cu, pos, slot, used, None)


def test_map_refusals(lib):
    m = lambda **kw: _map(lib, **kw)  # noqa: E731
    assert m(Bn=-1) == M.MOE_ERR_RANGE and m(Bn=M.MOE_ATTN_MAX_B + 1) == M.MOE_ERR_RANGE
    assert m(T=-1) == M.MOE_ERR_RANGE and m(T=M.MOE_KV_MAP_MAX_T + 1) == M.MOE_ERR_RANGE
    assert m(page=0) == M.MOE_ERR_RANGE and m(n_free=-1) == M.MOE_ERR_RANGE and m(width=0) == M.MOE_ERR_RANGE
    for name in ("kv", "q", "free", "table", "kvn", "cu", "pos", "slot", "used"):
        assert m(**{name: None}) == M.MOE_ERR_ARG, name
        assert m(**{name: 10 * FAKE + 2}) == M.MOE_ERR_ARG, name
    assert m(kvn=FAKE) == M.MOE_ERR_ARG                     # lengths updated in place
    assert m(kvn=FAKE + 12) == M.MOE_ERR_ARG                # or overlapping by one
    assert m(slot=7 * FAKE + 32) == M.MOE_ERR_ARG           # two outputs overlap
    assert m(free=4 * FAKE + 4) == M.MOE_ERR_ARG            # the free list inside the table


def test_a_single_row_may_have_any_stride():
    """One row out of a buffer whose rows are no multiple of 8 elements apart."""
    import torch
    x = torch.zeros(3, 4 * 64 + 3, dtype=torch.bfloat16)[:, :4 * 64].unflatten(1, (4, 64))
    assert x[:1].stride(0) == 4 * 64 + 3
    assert M._rows16(x[:1], 4, 64, "here", "q", -1) == (x.data_ptr(), 4 * 64)
    assert M._rows16(x[:2], 4, 64, "here", "q", -1)[1] == 4 * 64 + 3  # the library refuses these


def test_strerror_names_the_page_error(lib):
    assert "page" in M.strerror(M.MOE_ERR_PAGES)


# ---------------------------------------------------------------- rotation frequencies (fp32 results of fp64 formulas)

HALF_STEP = 2.0 ** -24


def test_plain_linear_and_base_frequencies(lib):
    for rot, base in ((64, 1e4), (128, 1e6), (2, 500.0)):
        i = np.arange(rot // 2)
        f, s = M.moe_rope_inv_freq(rot, base)
        ref = base ** (-2.0 * i / rot)
        assert s == 1.0 and np.all(np.abs(f - ref) <= 1.01 * HALF_STEP * ref)
        f, s = M.moe_rope_inv_freq(rot, base, M.MOE_ROPE_LINEAR, 8.0)
        assert s == 1.0 and np.all(np.abs(f - ref / 8) <= 1.01 * HALF_STEP * ref / 8)
    f, _ = M.moe_rope_inv_freq(64, 1e4, M.MOE_ROPE_BASE, 4.0)
    p, _ = M.moe_rope_inv_freq(64, 1e4)
    # the rule's two ends: the fastest frequency stays, the slowest is divided by the factor
    assert f[0] == p[0] == 1.0 and abs(f[-1] * 4 / p[-1] - 1) <= 4 * HALF_STEP


def test_frequencies_by_parts(lib):
    rot, base, factor, L = 128, 1e6, 4.0, 32768.0
    f, s = M.moe_rope_inv_freq(rot, base, M.MOE_ROPE_PARTS, factor, L, 32.0, 1.0)
    p = base ** (-2.0 * np.arange(rot // 2) / rot)
    turns = L * p / (2 * math.pi)
    fast, slow = turns >= 32, turns <= 1
    assert fast.any() and slow.any() and (~fast & ~slow).any()
    assert np.all(np.abs(f[fast] - p[fast]) <= 1.01 * HALF_STEP * p[fast])
    assert np.all(np.abs(f[slow] - p[slow] / factor) <= 1.01 * HALF_STEP * p[slow])
    mid = ~fast & ~slow
    assert np.all((f[mid] < p[mid]) & (f[mid] > p[mid] / factor))
    assert abs(s - (0.1 * math.log(factor) + 1)) <= 2 * HALF_STEP
    assert M.moe_rope_inv_freq(rot, base, M.MOE_ROPE_PARTS, 1.0, L)[1] == 1.0


@pytest.mark.parametrize("rot,base,factor,L,fast,slow", [(128, 1e6, 4.0, 32768.0, 32.0, 1.0), (64, 1e4, 16.0, 4096.0, 32.0, 1.0),
                                                         (96, 5e5, 2.5, 8192.0, 7.0, 0.5)])
def test_the_ramp_of_frequencies_by_parts_is_linear_in_the_turns(lib, rot, base, factor, L, fast, slow):
    """Every frequency against the formula, so that another ramp fails (one linear in the index, as in the method's
    published code, is off by far more than a rounding)."""
    f, _ = M.moe_rope_inv_freq(rot, base, M.MOE_ROPE_PARTS, factor, L, fast, slow)
    i = np.arange(rot // 2)
    p = base ** (-2.0 * i / rot)
    turns = L * p / (2 * math.pi)
    keep = np.clip((turns - slow) / (fast - slow), 0, 1)
    ref = p * keep + p / factor * (1 - keep)
    assert np.all(np.abs(f - ref) <= 1.01 * HALF_STEP * ref)
    at = [rot * math.log(L / (n * 2 * math.pi)) / (2 * math.log(base)) for n in (fast, slow)]
    lo, hi = math.floor(at[0]), math.ceil(at[1])
    by_index = 1 - np.clip((i - lo) / (hi - lo), 0, 1)
    other = p * by_index + p / factor * (1 - by_index)
    assert np.max(np.abs(f / other - 1)) > 0.1


@pytest.mark.parametrize("args", [(3, 1e4), (0, 1e4), (64, 1.0), (64, math.nan), (64, 1e4, 4), (64, 1e4, -1),
                                  (64, 1e4, 1, 0.5), (2, 1e4, 2, 2.0), (64, 1e4, 3, 2.0, 0.0), (64, 1e4, 3, 2.0, 4096.0, 1.0, 1.0)])
def test_frequency_refusals(lib, args):
    with pytest.raises(M.MoeError):
        M.moe_rope_inv_freq(*args)
