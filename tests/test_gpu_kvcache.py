"""Block tables and slots, and the norm and rotation that fill the cache,
against 64-bit references; then the operators together, as a step uses them."""
import numpy as np
import pytest

import quantized_expert_ffn_top10_b200 as M
from attn_ref import attn_limits, attn_ref, bf16, map_ref, rope_ref

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- moe_kv_map

def _run_map(kv_len, q_len, page, free, table, T):
    import torch
    i32 = dict(dtype=torch.int32, device="cuda")
    B = len(kv_len)
    t = dict(kv=torch.tensor(kv_len, **i32), q=torch.tensor(q_len, **i32), free=torch.tensor(free, **i32),
             table=torch.tensor(np.asarray(table), **i32), kv_new=torch.full((B,), 77, **i32),
             cu=torch.full((B + 1,), 77, **i32), position=torch.full((T,), 77, **i32), slot=torch.full((T,), 77, **i32),
             used=torch.full((1,), 77, **i32))
    M.moe_kv_map(t["kv"], t["q"], page, t["free"], t["table"], t["kv_new"], t["cu"], t["position"], t["slot"], t["used"])
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in t.items()}, M.moe_last_device_error()


def _case(B, page, max_kv, max_q, seed, pad=0, short=0, width=None):
    rng = np.random.default_rng(seed)
    kv = rng.integers(0, max_kv + 1, B)
    q = rng.integers(0, max_q + 1, B)
    have, want = -(-kv // page), -(-(kv + q) // page)
    width = int(want.max()) + 1 if width is None else width
    ids = rng.permutation(int(want.sum()) + 5)
    table = np.full((B, width), -1, np.int64)
    at = 0
    for b in range(B):
        n = min(int(have[b]), width)
        table[b, :n] = ids[at:at + n]
        at += int(have[b])
    free = ids[at:at + max(0, int((want - have).sum()) - short)]
    return kv, q, page, free, table, int(q.sum()) + pad


@pytest.mark.parametrize("B,page,max_kv,max_q,pad", [
    (1, 16, 0, 1, 0), (1, 1, 5, 3, 2), (1, 64, 4000, 8192, 0), (3, 16, 40, 5, 7), (7, 48, 1000, 300, 1), (33, 8, 100, 9, 64),
    (257, 16, 3000, 8, 0), (700, 128, 5000, 1, 300), (4096, 16, 64, 3, 5)])
def test_map(cuda_ok, B, page, max_kv, max_q, pad):
    args = _case(B, page, max_kv, max_q, seed=B * 31 + page, pad=pad)
    got, st = _run_map(*args)
    ref = map_ref(*args)
    assert st == 0 and not ref["short"]
    for name in ("table", "kv_new", "cu", "position", "slot"):
        assert np.array_equal(got[name], ref[name]), name
    assert got["used"][0] == ref["used"]


def test_map_without_requests(cuda_ok):
    got, st = _run_map([], [], 16, [3], np.zeros((0, 4)), 3)
    assert st == 0 and got["cu"].tolist() == [0] and got["slot"].tolist() == [-1] * 3 and got["used"][0] == 0
    assert got["position"].tolist() == [0] * 3


@pytest.mark.parametrize("short", [1, 3, 1000])
def test_map_runs_out_of_pages(cuda_ok, short):
    """Requests are served in order; the first that does not fit and all later
    ones that ask for a page get none, and the call reports it."""
    args = _case(40, 4, 30, 9, seed=3, pad=4, short=short)
    got, st = _run_map(*args)
    ref = map_ref(*args)
    assert ref["short"] and st == M.MOE_ERR_PAGES
    for name in ("table", "kv_new", "cu", "position", "slot"):
        assert np.array_equal(got[name], ref[name]), name
    assert got["used"][0] == ref["used"]


def test_map_row_without_room(cuda_ok):
    args = _case(20, 4, 30, 9, seed=4, width=7)
    got, st = _run_map(*args)
    ref = map_ref(*args)
    assert ref["short"] and st == M.MOE_ERR_PAGES
    for name in ("table", "kv_new", "cu", "position", "slot"):
        assert np.array_equal(got[name], ref[name]), name


def test_map_odd_inputs_are_reported(cuda_ok):
    args = ([5, -3, 4], [2, 2, -1], 4, [9, 8, 7], [[1, 2, -1], [-1, -1, -1], [3, -1, -1]], 6)
    got, st = _run_map(*args)
    ref = map_ref(*args)
    assert st == M.MOE_ERR_RANGE
    for name in ("table", "kv_new", "cu", "position", "slot"):
        assert np.array_equal(got[name], ref[name]), name
    # fewer rows than tokens: the rest is dropped
    args = ([5, 3], [4, 4], 4, [9, 8, 7], [[1, 2, -1], [6, -1, -1]], 6)
    got, st = _run_map(*args)
    ref = map_ref(*args)
    assert st == M.MOE_ERR_RANGE
    for name in ("table", "kv_new", "cu", "position", "slot"):
        assert np.array_equal(got[name], ref[name]), name
    # a table that lacks a cached token's page
    got, st = _run_map([5], [1], 4, [9], [[1, -1]], 1)
    assert st == M.MOE_ERR_SLOT and got["slot"][0] == -1
    # free page ids that would pass the slot range
    got, st = _run_map([0], [1], 1 << 10, [1 << 22], [[-1]], 1)
    assert st == M.MOE_ERR_SLOT and got["slot"][0] == -1


# ---------------------------------------------------------------- moe_qk_norm_rope

def _rope_case(T, Hq, Hk, D, rot, interleaved, norm, f8, page=16, head_major=False, seed=0, max_pos=1 << 18, in_place=False,
               rot_scale=1.0, scales=True):
    import torch
    rng = np.random.default_rng(seed)
    W = (Hq + 2 * Hk) * D
    raw = bf16(rng.standard_normal((T, W)))
    buf = torch.as_tensor(raw).to(torch.bfloat16).cuda()
    q, k, v = (buf[:, a * D:b * D].view(T, b - a, D) for a, b in ((0, Hq), (Hq, Hq + Hk), (Hq + Hk, Hq + 2 * Hk)))
    n_pages = -(-T // page) + 2
    shape = (n_pages, Hk, page, D) if head_major else (n_pages, page, Hk, D)
    dt = torch.float8_e4m3fn if f8 else torch.bfloat16
    caches = [torch.full(shape, 5.0, dtype=torch.float32, device="cuda").to(dt) for _ in range(2)]
    caches = [c.transpose(1, 2) if head_major else c for c in caches]
    sc = [rng.uniform(0.05, 0.3, Hk).astype(np.float32) if f8 and scales else None for _ in range(2)]
    t_sc = [None if s is None else torch.as_tensor(s).cuda() for s in sc]
    desc = M.moe_kv_desc(caches[0], caches[1], Hq, *t_sc)
    pos = rng.integers(0, max_pos, T).astype(np.int32)
    if T > 1:
        pos[0], pos[-1] = 0, max_pos - 1
    slot = rng.permutation(n_pages * page)[:T].astype(np.int32)
    dead = rng.random(T) < 0.2 if T > 4 else np.zeros(T, bool)
    slot[dead] = -1
    inv = M.moe_rope_inv_freq(rot, 1e6)[0] if rot else None
    qn, kn = (rng.uniform(0.5, 1.5, D).astype(np.float32) if norm else None for _ in range(2))
    up = lambda x: None if x is None else torch.as_tensor(x).cuda()  # noqa: E731
    q_out = q if in_place else torch.full((T, Hq, D), 9.0, dtype=torch.bfloat16, device="cuda")
    M.moe_qk_norm_rope(desc, q, k, v, up(pos), up(slot), q_out, up(inv), q_norm=up(qn), k_norm=up(kn), eps=1e-5,
                       rot_scale=rot_scale, interleaved=interleaved)
    torch.cuda.synchronize()
    assert M.moe_last_device_error() == 0
    h = raw.reshape(T, Hq + 2 * Hk, D)
    live = ~dead
    args = (pos, inv, rot, interleaved, rot_scale)
    rq = rope_ref(h[:, :Hq], *args, qn, 1e-5)
    rk = rope_ref(h[:, Hq:Hq + Hk], *args, kn, 1e-5)
    got_q = q_out.double().cpu().numpy()
    # one rounding to bf16, and the fp32 arithmetic before it: the norm's sum and root, the angle's
    # fp32 sine and cosine (2^-22 each at most) and three products, together within 2^-18 of the pair's size
    size = np.sqrt((rq ** 2).sum(-1, keepdims=True))
    lim = 2.0 ** -8 * np.abs(rq) + 2.0 ** -18 * size
    assert np.all(np.abs(got_q - rq)[live] <= 1.01 * lim[live]), np.max((np.abs(got_q - rq) - lim)[live])
    if in_place:
        assert np.array_equal(got_q[dead], h[:, :Hq][dead])
    else:
        assert np.all(got_q[dead] == 9.0)
    written = np.zeros((n_pages, page), bool)
    written[slot[live] // page, slot[live] % page] = True
    for cache, r, s in ((caches[0], rk, sc[0]), (caches[1], h[:, Hq + Hk:], sc[1])):
        c = cache.double().cpu().numpy()
        assert np.all(c[~written] == 5.0)
        g = c[slot[live] // page, slot[live] % page]
        r = r[live]
        size = np.sqrt((r ** 2).sum(-1, keepdims=True))
        if f8:
            sv = 1.0 if s is None else s.astype(np.float64)[:, None]
            r, size = np.clip(r / sv, -448, 448), size / sv
            lim = np.maximum(2.0 ** -4 * np.abs(r), 2.0 ** -10) + 2.0 ** -18 * size  # e4m3: half a step; 2^-10 below 2^-6
        else:
            lim = 2.0 ** -8 * np.abs(r) + 2.0 ** -18 * size
        assert np.all(np.abs(g - r) <= 1.01 * lim)


@pytest.mark.parametrize("T,Hq,Hk,D,rot,page", [
    (1, 16, 2, 128, 128, 16), (5, 16, 2, 128, 128, 64), (8, 1, 1, 64, 64, 1), (7, 3, 1, 64, 16, 48), (33, 5, 5, 128, 32, 8),
    (130, 32, 8, 64, 48, 16), (3, 20, 4, 128, 0, 16), (64, 40, 8, 128, 96, 32), (1025, 4, 2, 64, 64, 16),
    # several tokens to a CTA: a ragged last one, one head a token, more heads than a CTA has threads for at once
    (2371, 5, 1, 64, 32, 16), (2400, 1, 1, 128, 128, 64), (2369, 64, 8, 128, 112, 32)])
@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_and_rotation(cuda_ok, T, Hq, Hk, D, rot, page, f8, interleaved):
    _rope_case(T, Hq, Hk, D, rot, interleaved, norm=T % 2 == 1, f8=f8, page=page, head_major=T % 3 == 0, seed=T + rot)


def test_norm_and_rotation_in_place(cuda_ok):
    _rope_case(37, 16, 2, 128, 64, False, True, False, in_place=True, seed=1)
    _rope_case(37, 16, 2, 128, 64, True, False, True, in_place=True, seed=2, rot_scale=1.25)


def test_e4m3_without_scales_saturates(cuda_ok):
    import torch
    k = torch.zeros((2, 16, 1, 64), dtype=torch.float8_e4m3fn, device="cuda")
    v = torch.zeros_like(k)
    desc = M.moe_kv_desc(k, v, 1)
    x = torch.tensor([1000.0, -1e30, float("inf"), 448.0, -449.0, 0.3, -0.0, float("nan")] * 8, device="cuda")
    row = x.to(torch.bfloat16).view(1, 1, 64).contiguous()
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = torch.empty_like(row)
    M.moe_qk_norm_rope(desc, row, row, row, z, z + 17, q_out)
    torch.cuda.synchronize()
    got = v[1, 1, 0].float().cpu()
    ref = row.view(-1).float().clamp(-448, 448).to(torch.float8_e4m3fn).float().cpu()
    assert torch.equal(got.nan_to_num(7777.0), ref.nan_to_num(7777.0)) and torch.equal(k[1, 1, 0].float().cpu().nan_to_num(1),
                                                                                     got.nan_to_num(1))
    assert torch.equal(q_out.float().nan_to_num(5), row.float().nan_to_num(5))


def test_e4m3_writes_divide_by_the_scale(cuda_ok):
    """x / scale, rounded once to fp32 and once to e4m3: quotients that are
    exact ties between two codes, and scales whose reciprocal is not finite."""
    import torch
    scales = np.array([3.0, 7.0, 13.0, 15.0, 1e-39, 3.4e38, 0.3, 0.07], np.float32)
    Hk, D, T, page = len(scales), 64, 16, 16
    x = np.zeros((T, Hk, D), np.float32)
    rng = np.random.default_rng(58)
    for h in range(4):  # t * scale is exact in bf16, and t (5 bits) a tie between two codes
        x[:, h] = rng.choice(np.arange(17, 32, 2), (T, D)) * scales[h]
    x[:, 4] = rng.choice([0.0, 1e-38, -1e-38], (T, D))
    x[:, 5] = np.clip(rng.standard_normal((T, D)), -3, 3) * 1e38
    x[:, 6:] = rng.standard_normal((T, 2, D)) * 5
    x = torch.as_tensor(bf16(x)).to(torch.bfloat16).cuda()
    k = torch.zeros((1, page, Hk, D), dtype=torch.float8_e4m3fn, device="cuda")
    v = torch.zeros_like(k)
    sc = torch.as_tensor(scales).cuda()
    desc = M.moe_kv_desc(k, v, Hk, sc, sc)
    at = torch.arange(T, dtype=torch.int32, device="cuda")
    M.moe_qk_norm_rope(desc, x, x, x, at, at, torch.empty_like(x))
    torch.cuda.synchronize()
    want = (x.float() / sc[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).float()
    for cache in (k, v):
        got = cache[0].float()
        assert torch.equal(got, want), [int((got[:, h] != want[:, h]).sum()) for h in range(Hk)]


def test_slot_past_the_cache_is_reported(cuda_ok):
    import torch
    k = torch.full((2, 16, 1, 64), 2.0, dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    desc = M.moe_kv_desc(k, v, 1)
    row = torch.ones((2, 1, 64), dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    slot = torch.tensor([32, 3], dtype=torch.int32, device="cuda")
    out = torch.full_like(row, 4.0)
    M.moe_qk_norm_rope(desc, row, row, row, pos, slot, out)
    torch.cuda.synchronize()
    assert M.moe_last_device_error() == M.MOE_ERR_SLOT
    assert bool((out[0] == 4.0).all()) and bool((out[1] == 1.0).all())
    assert int((k == 1.0).sum()) == 64 and int((v == 1.0).sum()) == 64


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("f8", [False, True])
def test_a_prompt_and_its_windows(cuda_ok, f8):
    """Two requests: a prompt chunk, then windows of 5, 1 and 8 tokens, each step
    through the map, the norm and rotation, and attention; against attention in
    64 bits over what the cache holds after each step, and the cache against the
    64-bit rotation of every token so far."""
    import torch
    rng = np.random.default_rng(40)
    Hq, Hk, D, page, width = 6, 2, 64, 16, 20
    i32 = dict(dtype=torch.int32, device="cuda")
    dt = torch.float8_e4m3fn if f8 else torch.bfloat16
    k = torch.full((60, Hk, page, D), float("nan"), dtype=torch.bfloat16, device="cuda").to(dt).transpose(1, 2)
    v = k.clone(memory_format=torch.preserve_format)
    assert v.stride() == k.stride()
    sc = torch.tensor([0.1, 0.2], device="cuda") if f8 else None
    desc = M.moe_kv_desc(k, v, Hq, sc, sc)
    free = torch.tensor(rng.permutation(60), **i32)
    table = torch.full((2, width), -1, **i32)
    kv = torch.zeros(2, **i32)
    inv, rs = M.moe_rope_inv_freq(D, 1e4, M.MOE_ROPE_PARTS, 4.0, 64.0)
    t_inv = torch.as_tensor(inv).cuda()
    qn, kn = (rng.uniform(0.5, 1.5, D).astype(np.float32) for _ in range(2))
    t_qn, t_kn = torch.as_tensor(qn).cuda(), torch.as_tensor(kn).cuda()
    all_k, all_v = [[], []], [[], []]
    at = 0
    for step, (n0, n1) in enumerate(((70, 41), (5, 5), (1, 0), (8, 3))):
        T = n0 + n1
        raw = bf16(rng.standard_normal((T, (Hq + 2 * Hk) * D)))
        buf = torch.as_tensor(raw).to(torch.bfloat16).cuda()
        q, kk, vv = (buf[:, a * D:b * D].view(T, b - a, D) for a, b in ((0, Hq), (Hq, Hq + Hk), (Hq + Hk, Hq + 2 * Hk)))
        new = torch.tensor([n0, n1], **i32)
        kv_new, cu = torch.empty(2, **i32), torch.empty(3, **i32)
        pos, slot, used = torch.empty(T, **i32), torch.empty(T, **i32), torch.empty(1, **i32)
        M.moe_kv_map(kv, new, page, free[at:].contiguous(), table, kv_new, cu, pos, slot, used)
        M.moe_qk_norm_rope(desc, q, kk, vv, pos, slot, q, t_inv, q_norm=t_qn, k_norm=t_kn, rot_scale=rs)
        out = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(T, Hq, device="cuda")
        ws = torch.empty(M.moe_attn_workspace_bytes(T, 2, Hq, Hk, D), dtype=torch.uint8, device="cuda")
        if step == 0:
            M.moe_attn_prefill(desc, q, cu, kv_new, table, out, ws, D ** -0.5, lse=lse)
        else:
            M.moe_attn_decode(desc, q, cu, kv_new, table, out, 8, ws, D ** -0.5, lse=lse)
        torch.cuda.synchronize()
        assert M.moe_last_device_error() == 0
        at += int(used)
        kv = kv_new
        lens = kv.cpu().tolist()
        # what the cache holds now, token by token
        tb = table.cpu().numpy()
        scn = np.ones(2) if sc is None else sc.double().cpu().numpy()
        K, V = (x.double().cpu().numpy() * scn[:, None] for x in (k, v))
        keys = [np.stack([K[tb[b, j // page], j % page] for j in range(lens[b])]) for b in range(2)]
        vals = [np.stack([V[tb[b, j // page], j % page] for j in range(lens[b])]) for b in range(2)]
        h = raw.reshape(T, Hq + 2 * Hk, D)
        p = pos.cpu().numpy()
        for b, (a, e) in enumerate(((0, n0), (n0, T))):
            all_k[b].append(rope_ref(h[a:e, Hq:Hq + Hk], p[a:e], inv, D, False, rs, kn, 1e-6))
            all_v[b].append(h[a:e, Hq + Hk:])
            for held, made in ((keys[b], np.concatenate(all_k[b])), (vals[b], np.concatenate(all_v[b]))):
                size = np.sqrt((made ** 2).sum(-1, keepdims=True))
                half = np.maximum(2.0 ** -4 * np.abs(made), 2.0 ** -10 * scn[:, None]) if f8 else 2.0 ** -8 * np.abs(made)
                assert np.all(np.abs(held - made) <= 1.01 * (half + 2.0 ** -18 * size))
        ref = attn_ref(q.double().cpu().numpy(), keys, vals, [n0, n1], lens, D ** -0.5)
        lim, lse_lim = attn_limits(ref, D, max(lens), f8)
        assert np.all(np.abs(out.double().cpu().numpy() - ref[0]) <= lim), step
        assert np.all(np.abs(lse.double().cpu().numpy() - ref[1]) <= lse_lim), step
