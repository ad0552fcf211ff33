"""Python binding of libmoe.so (include/moe.h): argument marshalling only.

Every step of the layer runs in the library's CUDA kernels; this module turns
torch tensors into pointers and sizes and raises on a non-zero return code.
There is no fallback: if libmoe.so is missing or fails to load, import fails.
"""
from __future__ import annotations

import ctypes
import os



class ArenaDesc(ctypes.Structure):
    """moe_arena_desc of include/moe.h."""
    _fields_ = [("H", ctypes.c_int32), ("I", ctypes.c_int32), ("block", ctypes.c_int32),
                ("bits_gate", ctypes.c_int32), ("bits_up", ctypes.c_int32), ("bits_down", ctypes.c_int32),
                ("slot_bytes", ctypes.c_int64), ("off_codes", ctypes.c_int64 * 3),
                ("off_scales", ctypes.c_int64 * 3), ("n_slots", ctypes.c_int32), ("reserved", ctypes.c_int32)]


def as_desc(d) -> ArenaDesc:
    """Copy any object with the descriptor's field names into an ArenaDesc."""
    if isinstance(d, ArenaDesc):
        return d
    o = ArenaDesc()
    for name, _ in ArenaDesc._fields_:
        v = getattr(d, name)
        if name in ("off_codes", "off_scales"):
            for i in range(3):
                getattr(o, name)[i] = v[i]
        else:
            setattr(o, name, v)
    return o

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")

MOE_OK, MOE_ERR_ARG, MOE_ERR_SHAPE, MOE_ERR_RANGE = 0, -1, -2, -3
MOE_ERR_WS, MOE_ERR_CUDA, MOE_ERR_SLOT, MOE_ERR_TIMEOUT = -4, -5, -6, -7
MOE_ERR_STATIC, MOE_ERR_PAGES = -8, -9
MOE_DECODE_MAX_T, MOE_PREFILL_MAX_T, MOE_ROUTER_F64_MAX_T = 8, 8192, 128
MOE_ROUTE_STATIC_MAX_T, MOE_ROUTE_STATIC_BYTES = 8, 128 * 1024

EXPORTS = ("moe_workspace_bytes", "moe_route", "moe_forward_decode", "moe_forward_prefill",
           "moe_route_histogram", "moe_rank_experts", "moe_last_device_error", "moe_strerror",
           "moe_set_stage_events", "moe_launch_count", "moe_timeout_site", "moe_route_static",
           "moe_debug_set", "moe_workspace_offset", "moe_router_gamma", "moe_profile_bytes",
           "moe_profile_write", "moe_profile_read", "moe_profile_hit_rate", "moe_forward_partial",
           "moe_finish_rows", "moe_kv_map", "moe_rope_inv_freq", "moe_qk_norm_rope",
           "moe_attn_workspace_bytes", "moe_attn_decode", "moe_attn_prefill")
MOE_SLOT_REMOTE = -2
MOE_DBG_SPIN_LIMIT, MOE_DBG_BARRIER_EXTRA = 1, 2
MOE_WS_FAST_LOGITS, MOE_WS_PAIR_OUT, MOE_WS_SLOW_COUNT = 1, 2, 3
MOE_KV_BF16, MOE_KV_E4M3 = 0, 1
MOE_ATTN_MAX_HEADS, MOE_ATTN_MAX_B, MOE_ATTN_MAX_KV, MOE_KV_MAP_MAX_T = 512, 4096, 1 << 30, 1048576
MOE_ROPE_PLAIN, MOE_ROPE_LINEAR, MOE_ROPE_BASE, MOE_ROPE_PARTS = 0, 1, 2, 3


class RouteOut(ctypes.Structure):
    _fields_ = [("topk_idx", ctypes.c_void_p), ("topk_w", ctypes.c_void_p),
                ("expert_offsets", ctypes.c_void_p), ("perm", ctypes.c_void_p),
                ("n_rechecked", ctypes.c_void_p)]


class KvDesc(ctypes.Structure):
    """moe_kv_desc of include/moe.h (made by moe_kv_desc below)."""
    _fields_ = [("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("n_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("kv_type", ctypes.c_int32), ("reserved", ctypes.c_int32 * 2)]


class MoeError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {code} ({strerror(code)})")
        self.code = code


_lib = None


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libmoe.so not built at {LIB_PATH}; run quantized_expert_ffn_top10_b200.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        P, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        L.moe_workspace_bytes.restype = sz
        L.moe_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
        L.moe_route.restype = i32
        L.moe_route.argtypes = [P, i32, i32, P, P, i32, i32, P, P, P, P, P, sz, P]
        fwd = [P, P, P, i32, i32, P, i32, P, P, i32, i32, i32, P, P, P, P, P, sz, P]
        L.moe_forward_decode.restype = i32
        L.moe_forward_decode.argtypes = fwd
        L.moe_forward_prefill.restype = i32
        L.moe_forward_prefill.argtypes = fwd
        L.moe_forward_partial.restype = i32
        L.moe_forward_partial.argtypes = [i32, P, P, P, i32, i32, P, i32, P, P, i32, i32, P, P, P, P,
                                          ctypes.c_size_t, P]
        L.moe_finish_rows.restype = i32
        L.moe_finish_rows.argtypes = [P, P, i32, i32, i32, P, P, P]
        L.moe_route_histogram.restype = i32
        L.moe_route_histogram.argtypes = [P, i32, i32, i32, P, P]
        L.moe_rank_experts.restype = i32
        L.moe_rank_experts.argtypes = [P, i32, i32, P]
        L.moe_last_device_error.restype = i32
        L.moe_last_device_error.argtypes = [P]
        L.moe_strerror.restype = ctypes.c_char_p
        L.moe_strerror.argtypes = [i32]
        L.moe_set_stage_events.restype = i32
        L.moe_set_stage_events.argtypes = [P, i32]
        L.moe_launch_count.restype = ctypes.c_uint64
        L.moe_launch_count.argtypes = []
        L.moe_timeout_site.restype = i32
        L.moe_timeout_site.argtypes = [P]
        L.moe_route_static.restype = i32
        L.moe_route_static.argtypes = [P, i32, i32, P, P, i32, i32, P, P, P, P, P]
        L.moe_debug_set.restype = i32
        L.moe_debug_set.argtypes = [i32, i32]
        L.moe_workspace_offset.restype = sz
        L.moe_workspace_offset.argtypes = [i32, i32, i32, i32, i32, i32]
        L.moe_router_gamma.restype = ctypes.c_double
        L.moe_router_gamma.argtypes = [i32, i32, i32]
        L.moe_profile_bytes.restype = ctypes.c_int64
        L.moe_profile_bytes.argtypes = [i32, i32, i32]
        L.moe_profile_write.restype = ctypes.c_int64
        L.moe_profile_write.argtypes = [P, i32, i32, i32, P, sz]
        L.moe_profile_read.restype = i32
        L.moe_profile_read.argtypes = [P, sz, P, P, P, P, P]
        L.moe_profile_hit_rate.restype = ctypes.c_double
        L.moe_profile_hit_rate.argtypes = [P, i32, i32, i32, i32, P]
        i64, f32, f64 = ctypes.c_int64, ctypes.c_float, ctypes.c_double
        L.moe_kv_map.restype = i32
        L.moe_kv_map.argtypes = [P, P, i32, i32, P, i32, P, i32, i32, P, P, P, P, P, P]
        L.moe_rope_inv_freq.restype = i32
        L.moe_rope_inv_freq.argtypes = [i32, i32, f64, f64, f64, f64, f64, P, P]
        L.moe_qk_norm_rope.restype = i32
        L.moe_qk_norm_rope.argtypes = [P, P, i64, P, i64, P, i64, i32, P, P, P, P, f32, P, i32, i32, f32, P, i64, P]
        L.moe_attn_workspace_bytes.restype = sz
        L.moe_attn_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
        L.moe_attn_decode.restype = i32
        L.moe_attn_decode.argtypes = [P, P, i64, i32, P, P, i32, P, i32, i32, f32, f32, i32, P, P, P, P, P, sz, P]
        L.moe_attn_prefill.restype = i32
        L.moe_attn_prefill.argtypes = [P, P, i64, i32, P, P, i32, P, i32, f32, f32, i32, P, P, P, P, P, sz, P]
        _lib = L
    return _lib


def strerror(code: int) -> str:
    return lib().moe_strerror(int(code)).decode()


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _check(rc: int, where: str, raise_on_error: bool):
    if rc != MOE_OK and raise_on_error:
        raise MoeError(rc, where)
    return rc


def moe_workspace_bytes(T: int, E: int, top_k: int, H: int, I: int) -> int:
    return int(lib().moe_workspace_bytes(T, E, top_k, H, I))


def moe_route(x, router_w, router_bias, top_k, topk_idx, topk_w, expert_offsets, perm, ws,
              stream=None, raise_on_error=True) -> int:
    """x [T, H] bf16, router_w [E, H] fp32, router_bias [E] fp32 or None (CUDA tensors)."""
    T, H = x.shape
    E = router_w.shape[0]
    rc = lib().moe_route(_ptr(x), T, H, _ptr(router_w), _ptr(router_bias), E, top_k, _ptr(topk_idx),
                         _ptr(topk_w), _ptr(expert_offsets), _ptr(perm), _ptr(ws), ws.numel() * ws.element_size(),
                         _stream(stream))
    return _check(rc, "moe_route", raise_on_error)


def moe_route_static(x, router_w, router_bias, top_k, topk_idx, topk_w, expert_offsets, perm,
                     stream=None, raise_on_error=True) -> int:
    """moe_route with the library's fixed device scratch instead of a workspace
    (T <= MOE_ROUTE_STATIC_MAX_T).  Calls that overlap on the GPU race."""
    T, H = x.shape
    E = router_w.shape[0]
    rc = lib().moe_route_static(_ptr(x), T, H, _ptr(router_w), _ptr(router_bias), E, top_k, _ptr(topk_idx),
                                _ptr(topk_w), _ptr(expert_offsets), _ptr(perm), _stream(stream))
    return _check(rc, "moe_route_static", raise_on_error)


def _forward(fn, name, desc, arena, slot_table, L, layer, x, router_w, router_bias, top_k, residual, out,
             hist, route_out, ws, stream, raise_on_error, steer=None, T=None, E=None):
    T = x.shape[0] if T is None else T
    E = router_w.shape[0] if E is None else E
    ro = None
    if route_out is not None:
        ro = RouteOut(*[_ptr(route_out.get(k)) for k in ("topk_idx", "topk_w", "expert_offsets", "perm",
                                                          "n_rechecked")])
    rc = fn(ctypes.byref(as_desc(desc)), _ptr(arena), _ptr(slot_table), L, layer, _ptr(x), T, _ptr(router_w),
            _ptr(router_bias), E, top_k, int(bool(residual)), _ptr(steer), _ptr(out), _ptr(hist),
            ctypes.byref(ro) if ro is not None else None, _ptr(ws),
            ws.numel() * ws.element_size() if hasattr(ws, "numel") else 0, _stream(stream))
    return _check(rc, name, raise_on_error)


def moe_forward_decode(desc: ArenaDesc, arena, slot_table, L, layer, x, router_w, router_bias, top_k,
                       residual, out, hist=None, route_out=None, ws=None, stream=None, raise_on_error=True,
                       steer=None):
    """One MoE layer for a decode window (T <= 8).  route_out: optional dict of
    device tensors topk_idx / topk_w / expert_offsets / perm / n_rechecked;
    steer: optional fp32 [H] direction projected out of every output row."""
    return _forward(lib().moe_forward_decode, "moe_forward_decode", desc, arena, slot_table, L, layer, x,
                    router_w, router_bias, top_k, residual, out, hist, route_out, ws, stream, raise_on_error,
                    steer=steer)


def moe_forward_prefill(desc: ArenaDesc, arena, slot_table, L, layer, x, router_w, router_bias, top_k,
                        residual, out, hist=None, route_out=None, ws=None, stream=None, raise_on_error=True,
                        steer=None):
    """One MoE layer for a prefill chunk (T <= 8192), tensor-core grouped GEMMs."""
    return _forward(lib().moe_forward_prefill, "moe_forward_prefill", desc, arena, slot_table, L, layer, x,
                    router_w, router_bias, top_k, residual, out, hist, route_out, ws, stream, raise_on_error,
                    steer=steer)


def moe_forward_partial(prefill, desc: ArenaDesc, arena, slot_table, L, layer, x, router_w, router_bias, top_k,
                        partial, hist=None, route_out=None, ws=None, stream=None, raise_on_error=True):
    """Expert parallelism: partial [T, H] fp32 receives each token's gate-weighted
    sum over the experts held here (slot != MOE_SLOT_REMOTE), no residual."""
    T, E = x.shape[0], router_w.shape[0]
    ro = None
    if route_out is not None:
        ro = RouteOut(*[_ptr(route_out.get(k)) for k in ("topk_idx", "topk_w", "expert_offsets", "perm",
                                                          "n_rechecked")])
    rc = lib().moe_forward_partial(int(bool(prefill)), ctypes.byref(as_desc(desc)), _ptr(arena), _ptr(slot_table),
                                   L, layer, _ptr(x), T, _ptr(router_w), _ptr(router_bias), E, top_k, _ptr(partial),
                                   _ptr(hist), ctypes.byref(ro) if ro is not None else None, _ptr(ws),
                                   ws.numel() * ws.element_size() if hasattr(ws, "numel") else 0, _stream(stream))
    return _check(rc, "moe_forward_partial", raise_on_error)


def moe_finish_rows(x, total, residual, out, steer=None, stream=None, raise_on_error=True) -> int:
    """out = bf16((residual ? x : 0) + total), steering projection first when given."""
    T, H = total.shape
    rc = lib().moe_finish_rows(_ptr(x), _ptr(total), T, H, int(bool(residual)), _ptr(steer), _ptr(out),
                               _stream(stream))
    return _check(rc, "moe_finish_rows", raise_on_error)


def moe_route_histogram(expert_offsets, E, L, layer, hist, stream=None, raise_on_error=True) -> int:
    rc = lib().moe_route_histogram(_ptr(expert_offsets), E, L, layer, _ptr(hist), _stream(stream))
    return _check(rc, "moe_route_histogram", raise_on_error)


def moe_rank_experts(hist_host):
    """hist_host: numpy uint32 [L, E] -> numpy uint16 [L*E, 2] (layer, expert), most routed first."""
    import numpy as np
    h = np.ascontiguousarray(hist_host, dtype=np.uint32)
    L, E = h.shape
    pairs = np.zeros((L * E, 2), np.uint16)
    rc = lib().moe_rank_experts(h.ctypes.data_as(ctypes.c_void_p), L, E, pairs.ctypes.data_as(ctypes.c_void_p))
    _check(rc, "moe_rank_experts", True)
    return pairs


def moe_last_device_error(stream=None) -> int:
    return int(lib().moe_last_device_error(_stream(stream)))


def moe_set_stage_events(events) -> int:
    """events: list of 5 torch.cuda.Event(enable_timing=True) (or [] to turn off);
    later forward calls record them at the stage boundaries."""
    for e in events:
        if e.cuda_event == 0:
            e.record()  # make sure the event exists before its handle is taken
    n = len(events)
    arr = (ctypes.c_void_p * max(n, 1))(*[e.cuda_event for e in events])
    return _check(lib().moe_set_stage_events(arr if n else None, n), "moe_set_stage_events", True)


def moe_launch_count() -> int:
    return int(lib().moe_launch_count())


def moe_timeout_site(stream=None) -> int:
    return int(lib().moe_timeout_site(_stream(stream)))


def moe_debug_set(key: int, value: int) -> int:
    """Test hook: see include/moe.h (MOE_DBG_SPIN_LIMIT, MOE_DBG_BARRIER_EXTRA)."""
    return _check(lib().moe_debug_set(int(key), int(value)), "moe_debug_set", True)


def moe_workspace_offset(T: int, E: int, top_k: int, H: int, I: int, field: int) -> int:
    """Byte offset of a workspace field (MOE_WS_FAST_LOGITS, MOE_WS_PAIR_OUT)."""
    v = int(lib().moe_workspace_offset(T, E, top_k, H, I, field))
    if v == ctypes.c_size_t(-1).value:
        raise MoeError(MOE_ERR_ARG, "moe_workspace_offset")
    return v


def moe_router_gamma(T: int, E: int, H: int) -> float:
    """Bound factor of a chunk router's fast logits (include/moe.h)."""
    return float(lib().moe_router_gamma(T, E, H))


def moe_profile_write(pairs, L: int, E: int) -> bytes:
    """STRP v1 expert profile (include/moe.h) of the ranked (layer, expert)
    pairs (numpy uint16 [n, 2], rank order)."""
    import numpy as np
    pr = np.ascontiguousarray(pairs, dtype=np.uint16).reshape(-1, 2)
    n = pr.shape[0]
    size = int(lib().moe_profile_bytes(n, L, E))
    if size < 0:
        raise MoeError(MOE_ERR_RANGE, "moe_profile_bytes")
    buf = np.zeros(size, np.uint8)
    rc = int(lib().moe_profile_write(pr.ctypes.data_as(ctypes.c_void_p), n, L, E,
                                     buf.ctypes.data_as(ctypes.c_void_p), size))
    if rc < 0:
        raise MoeError(rc, "moe_profile_write")
    return buf.tobytes()


def moe_profile_read(data: bytes):
    """(L, E, pairs uint16 [n, 2], inverse int32 [L, E]) of an STRP v1 file."""
    import numpy as np
    raw = np.frombuffer(data, np.uint8).copy()
    Lc, Ec, nc = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    P = ctypes.c_void_p
    rc = lib().moe_profile_read(raw.ctypes.data_as(P), raw.size, ctypes.byref(Lc), ctypes.byref(Ec),
                                ctypes.byref(nc), None, None)
    _check(rc, "moe_profile_read", True)
    pairs = np.zeros((nc.value, 2), np.uint16)
    inv = np.zeros((Lc.value, Ec.value), np.int32)
    rc = lib().moe_profile_read(raw.ctypes.data_as(P), raw.size, ctypes.byref(Lc), ctypes.byref(Ec),
                                ctypes.byref(nc), pairs.ctypes.data_as(P), inv.ctypes.data_as(P))
    _check(rc, "moe_profile_read", True)
    return Lc.value, Ec.value, pairs, inv


def moe_profile_hit_rate(pairs, L: int, E: int, slots: int, hist) -> float:
    """Fraction of the routed reads in hist [L, E] that land in the first
    `slots` ranked pairs."""
    import numpy as np
    pr = np.ascontiguousarray(pairs, dtype=np.uint16).reshape(-1, 2)
    h = np.ascontiguousarray(hist, dtype=np.uint32)
    v = float(lib().moe_profile_hit_rate(pr.ctypes.data_as(ctypes.c_void_p), pr.shape[0], L, E, slots,
                                         h.ctypes.data_as(ctypes.c_void_p)))
    if v < 0:
        raise MoeError(MOE_ERR_ARG, "moe_profile_hit_rate")
    return v


# ---------------------------------------------------------------- the attention half of a layer

def _refuse(where, what):
    raise MoeError(MOE_ERR_ARG, f"{where}: {what}")


def _need(ok, where, what):
    if not ok:
        _refuse(where, what)


def _flat(t, n, dtype, where, what, dev):
    """Device pointer of n adjacent elements of this type (None stays None)."""
    if t is None:
        return None
    if t.dtype is dtype and t.numel() >= n and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    _refuse(where, f"{what} is a contiguous {dtype} tensor of at least {n} elements on the current device")


def _rows16(t, n, d, where, what, dev):
    """(pointer, elements from row to row) of a bf16 [T, n, d] tensor whose rows are whole."""
    st, shape = t.stride(), t.shape
    if (len(shape) == 3 and shape[1] == n and shape[2] == d and st[2] == 1 and (n == 1 or st[1] == d)
            and t.get_device() == dev):
        import torch
        if t.dtype is torch.bfloat16 or t.dtype in (torch.int16, torch.uint16):
            return t.data_ptr(), st[0] if shape[0] > 1 else n * d  # (a single row's stride means nothing)
    _refuse(where, f"{what} is a bf16 [T, {n}, {d}] tensor with adjacent heads on the current device")


def moe_kv_desc(k_cache, v_cache, n_heads: int, k_scale=None, v_scale=None) -> KvDesc:
    """Descriptor of a paged cache from its two tensors, both [pages, page size,
    kv heads, head dim] in any order of strides (a head-major cache is passed
    transposed); bfloat16 (or int16), or float8_e4m3fn (or uint8) with optional
    fp32 [kv heads] scales.  It holds the tensors it points to."""
    import torch
    where = "moe_kv_desc"
    wide = (torch.bfloat16, torch.int16, torch.uint16)
    _need(k_cache.dim() == 4 and k_cache.shape == v_cache.shape and k_cache.dtype == v_cache.dtype
          and k_cache.device == v_cache.device and k_cache.is_cuda, where, "two equal 4-d device caches")
    _need(k_cache.dtype in wide or k_cache.dtype in (torch.float8_e4m3fn, torch.uint8), where, "bf16 or e4m3 caches")
    pages, size, heads, dim = k_cache.shape
    strides = []
    for i in range(4):  # a dimension of one element may have any stride: 0 serves
        sk, sv = k_cache.stride(i), v_cache.stride(i)
        _need(sk == sv or k_cache.shape[i] == 1, where, "caches of equal strides")
        strides.append(sk if k_cache.shape[i] > 1 else 0)
    _need(strides[3] == 1, where, "adjacent elements of a head")
    d = KvDesc(k_cache.data_ptr(), v_cache.data_ptr(), None, None, strides[0], strides[1], strides[2], pages, size,
               n_heads, heads, dim, MOE_KV_BF16 if k_cache.dtype in wide else MOE_KV_E4M3)
    dev = k_cache.get_device()
    d.k_scale = _flat(k_scale, heads, torch.float32, where, "k_scale", dev)
    d.v_scale = _flat(v_scale, heads, torch.float32, where, "v_scale", dev)
    d.device_index = dev
    d.held = (k_cache, v_cache, k_scale, v_scale)
    return d


_now = None  # (current device, current stream handle of a device), looked up once: they are half a small call's cost


def _here(kv, where, stream):
    """(current device, stream handle); refuses a cache on another device."""
    global _now
    if _now is None:
        import torch
        torch.cuda.init()
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _now = (getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device),
                raw or (lambda dev: torch.cuda.current_stream(dev).cuda_stream))
    dev = _now[0]()
    if kv is not None and getattr(kv, "device_index", dev) != dev:
        _refuse(where, "the cache is on another device than the current one")
    return dev, _now[1](dev) if stream is None else _stream(stream)


def moe_kv_map(kv_len, q_len, page_size, free_pages, block_table, kv_len_new, cu_q, position, slot, n_used,
               stream=None, raise_on_error=True) -> int:
    """Block tables, offsets, positions and cache slots of a step's new tokens
    (all int32 CUDA tensors; position and slot have one entry per row)."""
    import torch
    where, i32 = "moe_kv_map", torch.int32
    dev, st = _here(None, where, stream)
    B, T = kv_len.numel(), position.numel()
    _need(block_table.dim() == 2 and block_table.shape[0] == B, where, "block_table is [B, width]")
    width = block_table.shape[1]
    rc = lib().moe_kv_map(
        _flat(kv_len, B, i32, where, "kv_len", dev), _flat(q_len, B, i32, where, "q_len", dev), B, page_size,
        _flat(free_pages, 0, i32, where, "free_pages", dev), 0 if free_pages is None else free_pages.numel(),
        _flat(block_table, B * width, i32, where, "block_table", dev), width, T,
        _flat(kv_len_new, B, i32, where, "kv_len_new", dev), _flat(cu_q, B + 1, i32, where, "cu_q", dev),
        _flat(position, T, i32, where, "position", dev), _flat(slot, T, i32, where, "slot", dev),
        _flat(n_used, 1, i32, where, "n_used", dev), st)
    return _check(rc, where, raise_on_error)


def moe_qk_norm_rope(kv: KvDesc, q, k, v, position, slot, q_out, inv_freq=None, q_norm=None, k_norm=None, eps=1e-6,
                     rot_scale=1.0, interleaved=False, stream=None, raise_on_error=True) -> int:
    """Per-head norm and rotation of q and k [T, heads, dim] bf16, q to q_out
    (q itself for in place), k and v into the cache at slot [T].  inv_freq fp32
    [rot_dim / 2] or None (no rotation); q_norm, k_norm fp32 [dim] or None."""
    import torch
    where, f32, i32 = "moe_qk_norm_rope", torch.float32, torch.int32
    dev, st = _here(kv, where, stream)
    T, D = q.shape[0], kv.head_dim
    _need(k.shape[0] == T and v.shape[0] == T and q_out.shape[0] == T, where, "q, k, v and q_out have T rows")
    qp, qs = _rows16(q, kv.n_heads, D, where, "q", dev)
    kp, ks = _rows16(k, kv.n_kv_heads, D, where, "k", dev)
    vp, vs = _rows16(v, kv.n_kv_heads, D, where, "v", dev)
    op, os_ = _rows16(q_out, kv.n_heads, D, where, "q_out", dev)
    rot = 0 if inv_freq is None else 2 * inv_freq.numel()
    rc = lib().moe_qk_norm_rope(
        ctypes.byref(kv), qp, qs, kp, ks, vp, vs, T, _flat(position, T, i32, where, "position", dev),
        _flat(slot, T, i32, where, "slot", dev), _flat(q_norm, D, f32, where, "q_norm", dev),
        _flat(k_norm, D, f32, where, "k_norm", dev), eps, _flat(inv_freq, rot // 2, f32, where, "inv_freq", dev), rot,
        int(bool(interleaved)), rot_scale, op, os_, st)
    return _check(rc, where, raise_on_error)


def moe_attn_workspace_bytes(T: int, B: int, n_heads: int, n_kv_heads: int, head_dim: int) -> int:
    return int(lib().moe_attn_workspace_bytes(T, B, n_heads, n_kv_heads, head_dim))


def _attn(fn, where, max_q, kv, q, cu_q, kv_len, block_table, out, ws, scale, softcap, window, slopes, prefix, lse,
          stream, raise_on_error):
    import torch
    f32, i32 = torch.float32, torch.int32
    dev, st = _here(kv, where, stream)
    T, D, B = q.shape[0], kv.head_dim, kv_len.numel()
    qp, qs = _rows16(q, kv.n_heads, D, where, "q", dev)
    _need(block_table.dim() == 2 and block_table.shape[0] == B, where, "block_table is [B, width]")
    width = block_table.shape[1]
    _need(out.shape[0] == T and out.is_contiguous(), where, "out is contiguous with T rows")
    op, _ = _rows16(out, kv.n_heads, D, where, "out", dev)
    _need(ws.get_device() == dev and ws.is_contiguous(), where, "ws is a contiguous tensor on the current device")
    rc = fn(ctypes.byref(kv), qp, qs, T, _flat(cu_q, B + 1, i32, where, "cu_q", dev),
            _flat(kv_len, B, i32, where, "kv_len", dev), B,
            _flat(block_table, B * width, i32, where, "block_table", dev), width, *max_q, scale, softcap, window,
            _flat(slopes, kv.n_heads, f32, where, "slopes", dev), _flat(prefix, B, i32, where, "prefix", dev), op,
            _flat(lse, T * kv.n_heads, f32, where, "lse", dev), ws.data_ptr(), ws.numel() * ws.element_size(),
            st)
    return _check(rc, where, raise_on_error)


def moe_attn_decode(kv: KvDesc, q, cu_q, kv_len, block_table, out, max_q, ws, scale, softcap=0.0, window=0, slopes=None,
                    prefix=None, lse=None, stream=None, raise_on_error=True) -> int:
    """Attention of windows of 1 to max_q <= 8 new tokens a request over the
    paged cache (include/moe.h); q, out [T, heads, dim] bf16, lse [T, heads]."""
    return _attn(lib().moe_attn_decode, "moe_attn_decode", (max_q,), kv, q, cu_q, kv_len, block_table, out, ws, scale,
                 softcap, window, slopes, prefix, lse, stream, raise_on_error)


def moe_attn_prefill(kv: KvDesc, q, cu_q, kv_len, block_table, out, ws, scale, softcap=0.0, window=0, slopes=None,
                     prefix=None, lse=None, stream=None, raise_on_error=True) -> int:
    """Attention of a prompt chunk of T <= 8192 rows over the paged cache."""
    return _attn(lib().moe_attn_prefill, "moe_attn_prefill", (), kv, q, cu_q, kv_len, block_table, out, ws, scale,
                 softcap, window, slopes, prefix, lse, stream, raise_on_error)


def moe_rope_inv_freq(rot_dim: int, base: float, kind: int = MOE_ROPE_PLAIN, factor: float = 1.0,
                      original_len: float = 0.0, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """(numpy fp32 [rot_dim / 2] frequencies, factor on cosine and sine); include/moe.h gives the kinds, and says
    which models' scaling MOE_ROPE_PARTS is not (theirs go to moe_qk_norm_rope as they are)."""
    import numpy as np
    f = np.zeros(max(rot_dim // 2, 1), np.float32)
    s = ctypes.c_float(0.0)
    rc = lib().moe_rope_inv_freq(kind, rot_dim, base, factor, original_len, beta_fast, beta_slow,
                                 f.ctypes.data_as(ctypes.c_void_p), ctypes.byref(s))
    _check(rc, "moe_rope_inv_freq", True)
    return f, s.value
