"""Plain 64-bit references of the attention half (numpy, loops where they are
clearest) and builders of paged caches for its tests.  Nothing here calls the
library."""
from __future__ import annotations

import math

import numpy as np

E4M3_MAX = 448.0


def map_ref(kv_len, q_len, page, free, table, T):
    """moe_kv_map by hand: request after request, token after token."""
    kv_len, q_len, table = [int(x) for x in kv_len], [int(x) for x in q_len], np.array(table, np.int64)
    B, width = table.shape
    kv_new, cu, pos, slot = [], [0], np.zeros(T, np.int64), np.full(T, -1, np.int64)
    asked, used, short = 0, 0, False
    for b in range(B):
        old, new = max(kv_len[b], 0), max(q_len[b], 0)
        have, want = -(-old // page), -(-(old + new) // page)
        fits = want <= width
        need = want - have if fits else 0
        ok = fits and (need == 0 or asked + need <= len(free))
        if ok:
            for i in range(need):
                table[b, have + i] = free[asked + i]
            used = max(used, asked + need) if need else used
        else:
            short = True
        asked += need
        kv_new.append(old + new if ok else old)
        for i in range(new):
            t = cu[-1] + i
            if t < T:
                pos[t] = old + i
                if ok:
                    slot[t] = table[b, (old + i) // page] * page + (old + i) % page
        cu.append(cu[-1] + new)
    return dict(table=table, kv_new=np.array(kv_new), cu=np.minimum(np.array(cu), T), position=pos, slot=slot, used=used,
                short=short)


def rope_ref(x, position, inv_freq, rot, interleaved, rot_scale, norm, eps):
    """Normed and turned heads of x [T, heads, D] in fp64."""
    y = np.asarray(x, np.float64).copy()
    if norm is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(norm, np.float64)
    z = y.copy()
    for p in range(rot // 2):
        a, b = (2 * p, 2 * p + 1) if interleaved else (p, p + rot // 2)
        th = np.asarray(position, np.float64) * float(inv_freq[p])
        c, s = np.cos(th)[:, None] * rot_scale, np.sin(th)[:, None] * rot_scale
        z[..., a], z[..., b] = y[..., a] * c - y[..., b] * s, y[..., b] * c + y[..., a] * s
    return z


def attn_ref(q, keys, values, q_len, kv_len, scale, softcap=0.0, window=0, slopes=None, prefix=None):
    """(out, lse, weight, slack, most) in fp64: q [T, Hq, D]; keys, values: per request
    [kv, Hk, D].  weight = sum_j softmax_j |v_j| (what a relative error of the
    numerators scales with); slack [T, Hq] = the largest sum_d |q_d k_jd| * scale
    over visible keys (what a relative error of the scores scales with); most = the
    largest |v_j| of the request's keys."""
    T, Hq, D = q.shape
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    weight, slack, most = np.zeros((T, Hq, D)), np.zeros((T, Hq)), np.zeros((T, Hq, D))
    t = 0
    for b, n in enumerate(q_len):
        kv = int(kv_len[b])
        K, V = np.asarray(keys[b], np.float64), np.asarray(values[b], np.float64)
        G = Hq // K.shape[1]
        pos, j = kv - n + np.arange(n)[:, None], np.arange(kv)[None]
        hi = np.maximum(pos + 1, 0 if prefix is None else min(int(prefix[b]), kv))
        seen = (j < hi) & ((j > pos - window) if window else True)
        rows = np.flatnonzero(seen.any(1))  # the others keep 0 and -inf
        if rows.size:
            sl = t + rows
            for h in range(Hq):
                k, v, qq = K[:, h // G], V[:, h // G], q[sl, h]
                s = qq @ k.T * scale
                mask = seen[rows]
                slack[sl, h] = np.where(mask, np.abs(qq) @ np.abs(k).T, 0).max(1) * abs(scale)
                if softcap:
                    s = softcap * np.tanh(s / softcap)
                if slopes is not None:
                    s = s - float(slopes[h]) * np.abs(pos[rows] - j)
                s = np.where(mask, s, -np.inf)
                m = s.max(1, keepdims=True)
                e = np.exp(s - m)
                tot = e.sum(1, keepdims=True)
                out[sl, h] = e @ v / tot
                weight[sl, h] = e @ np.abs(v) / tot
                most[sl, h] = np.abs(v).max(0)
                lse[sl, h] = (m + np.log(tot))[:, 0]
        t += n
    return out, lse, weight, slack, most


def attn_limits(ref, D, n_keys, e4m3):
    """Bounds of |out - ref| and |lse - ref|, counted in roundings.

    out: its own rounding to bf16, 2^-8 of the value; the numerators' rounding
    to bf16 2^-8 (fp16, e4m3 caches: 2^-11) of the weight; for e4m3 caches also
    what falls below fp16's normal steps: there a numerator, lifted by 2^6 at
    least, is off by half of fp16's smallest, 2^-25, which is 2^-31 of its
    reference, and meets |v_j|, not the weighted mean of |v| (which is far smaller
    where the keys that matter hold a zero), so the n keys are off by n 2^-31
    max |v| over a sum of at least 1; the fp32 sum over the keys, each
    step cut or rounded to 2^-23; and a score error ds, which moves every
    softmax weight by at most 2 ds.  ds: D products summed in fp32 at 2^-23 a
    step, scaling and base-2 exponent of the score itself (|s| <= slack) at a
    few 2^-24, and the exponential at 2^-22."""
    out, lse, weight, slack, most = ref
    ds = (D + 16) * 2.0 ** -23 * slack + 2.0 ** -21
    p, floor = (2.0 ** -11, n_keys * 2.0 ** -31 * most) if e4m3 else (2.0 ** -8, 0.0)
    lim = 1.01 * (2.0 ** -8 * np.abs(out) + (p + (2 * ds)[..., None] + n_keys * 2.0 ** -22) * weight + floor) + 1e-30
    return lim, ds + n_keys * 2.0 ** -23 + np.where(np.isfinite(lse), np.abs(lse), 0) * 2.0 ** -22


class Paged:
    """A paged cache on the device holding given keys and values per request."""

    def __init__(self, keys, values, page, e4m3, head_major=False, seed=0, stale=float("nan"), spare=3, one_buffer=False,
                 k_scale=None, v_scale=None):
        import torch
        Hk, D = keys[0].shape[1:]
        rng = np.random.default_rng(seed)
        have = [-(-k.shape[0] // page) for k in keys]
        self.n_pages, self.page, self.Hk, self.D = sum(have) + spare, page, Hk, D
        ids = rng.permutation(self.n_pages)
        self.table = np.full((len(keys), max(have) + 2), -1, np.int32)
        dt = torch.float8_e4m3fn if e4m3 else torch.bfloat16
        store = []
        for src in (keys, values):
            x = torch.full((self.n_pages, page, Hk, D), stale, dtype=torch.float32)
            at = 0
            for b, k in enumerate(src):
                n = have[b]
                self.table[b, :n] = ids[at:at + n]
                flat = x[torch.as_tensor(ids[at:at + n].copy())].reshape(n * page, Hk, D)
                flat[:k.shape[0]] = torch.as_tensor(np.asarray(k, np.float32))
                x[torch.as_tensor(ids[at:at + n].copy())] = flat.reshape(n, page, Hk, D)
                at += n
            store.append(x.to(dt))
        if one_buffer:  # keys and values of a page side by side in one allocation
            both = torch.empty((self.n_pages, 2, page, Hk, D), dtype=dt)
            both[:, 0], both[:, 1] = store[0], store[1]
            both = both.cuda()
            self.k, self.v = both[:, 0], both[:, 1]
        elif head_major:
            self.k, self.v = (x.transpose(1, 2).contiguous().cuda().transpose(1, 2) for x in store)
        else:
            self.k, self.v = (x.cuda() for x in store)
        self.table_dev = torch.from_numpy(self.table).cuda()
        self.k_scale = None if k_scale is None else torch.tensor(k_scale, dtype=torch.float32).cuda()
        self.v_scale = None if v_scale is None else torch.tensor(v_scale, dtype=torch.float32).cuda()

    def desc(self, n_heads):
        import quantized_expert_ffn_top10_b200 as M
        return M.moe_kv_desc(self.k, self.v, n_heads, self.k_scale, self.v_scale)


def bf16(x):
    """Values rounded to bf16, as float64."""
    import torch
    return torch.as_tensor(np.asarray(x, np.float32)).to(torch.bfloat16).double().numpy()


def e4m3(x):
    import torch
    return torch.as_tensor(np.asarray(x, np.float32)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).double().numpy()
