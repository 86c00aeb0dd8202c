"""Binding of the operators around the NVFP4 KV cache: block tables and slot
maps, head norms with rotation (and their gradient), rows quantised into the
paged cache, and attention over it. Like the package's other entry points these
only check and marshal arguments; ``include/nvfp4.h`` states what each computes.

    cache = alloc_kv_cache(pages, 64, kv_heads, 128, k_amax, v_amax)
    plan = nvfp4_kv_plan(cached, new, block_table, free_pages, 64, tokens)
    r = nvfp4_qk_norm_rope(q, k, plan["positions"], cos_sin, q_weight, k_weight)
    nvfp4_kv_append(cache, r["k"], v, plan["slots"])
    o = nvfp4_kv_attention(r["q"], cache, plan["table"], plan["seq_lens"], plan["q_start"],
                           max_q, workspace=ws)["out"]
"""
from __future__ import annotations

import ctypes as C
import math
import struct

import torch

from . import _check, _i32, _i64, _vp, lib

_BF16 = (torch.bfloat16, torch.int16, torch.uint16)
_I32 = (torch.int32, torch.uint32)


class _Cache(C.Structure):
    _fields_ = [("k_codes", _vp), ("k_scales", _vp), ("v_codes", _vp), ("v_scales", _vp),
                ("k_amax", _vp), ("v_amax", _vp), ("pages", _i64), ("kv_heads", _i32),
                ("page_size", _i32), ("head_dim", _i32), ("four_over_six", _i32)]


class _Rows(C.Structure):
    _fields_ = [("ptr", _vp), ("stride", _i64)]


class _QkConfig(C.Structure):
    _fields_ = [("tokens", _i64), ("q_heads", _i32), ("kv_heads", _i32), ("head_dim", _i32),
                ("rotary_dim", _i32), ("interleaved", _i32), ("eps", C.c_float),
                ("q_weight", _vp), ("k_weight", _vp), ("positions", _vp), ("cos_sin", _vp),
                ("max_pos", _i64)]


class _AttentionConfig(C.Structure):
    _fields_ = [("block_table", _vp), ("seq_len", _vp), ("q_start", _vp), ("requests", _i64),
                ("table_cols", _i64), ("tokens", _i64), ("q_heads", _i32), ("max_q", _i32),
                ("window", _i32), ("scale", C.c_float)]


# the same structs, packed into bytes: several times cheaper than filling a
# ctypes structure field by field
_CACHE, _QK, _ATTENTION = struct.Struct("@6Pq4i"), struct.Struct("@q5if4Pq"), struct.Struct(
    "@3P3q3if")
assert (_CACHE.size, _QK.size, _ATTENTION.size) == tuple(
    map(C.sizeof, (_Cache, _QkConfig, _AttentionConfig)))

_loaded = None


def _lib() -> C.CDLL:
    global _loaded
    if _loaded is None:
        _loaded = lib()
    return _loaded


def declare(L: C.CDLL) -> None:
    """Argument types of the library's entry points of this module."""
    size = C.c_size_t
    L.nvfp4_kv_plan.argtypes = [_vp, _vp, _i64, _vp, _i64, _i32, _vp, _i64, _i64, _vp, _vp, _vp,
                                _vp, _vp, _vp, _vp]
    L.nvfp4_qk_norm_rope.argtypes = [_vp, _Rows, _Rows, _Rows, _Rows, _vp, _vp]
    L.nvfp4_qk_norm_rope_bwd.argtypes = [_vp] + [_Rows] * 6 + [
        _vp, _vp, _vp, size, _vp, _vp]
    L.nvfp4_kv_append.argtypes = [_vp, _Rows, _Rows, _vp, _i64, _vp, _vp, _vp, _vp]
    L.nvfp4_kv_attention.argtypes = [_vp, _vp, _Rows, _vp,
                                     _vp, _vp, size, _vp, _vp]
    for name in ("nvfp4_kv_plan", "nvfp4_qk_norm_rope", "nvfp4_qk_norm_rope_bwd",
                 "nvfp4_kv_append", "nvfp4_kv_attention"):
        getattr(L, name).restype = C.c_int
    for name in ("nvfp4_qk_norm_rope_ws_bytes", "nvfp4_kv_attention_ws_bytes"):
        getattr(L, name).argtypes = []
        getattr(L, name).restype = size


# The library launches on the current device. These calls are short, so an entry
# point compares that with its first tensor's device and only calls itself again
# under torch.cuda.device where they differ.

def _elsewhere(dev: int) -> bool:
    return dev >= 0 and dev != torch._C._cuda_getDevice()


def _stream(dev: int) -> int:
    return torch._C._cuda_getCurrentRawStream(dev)


# A call here lasts a few microseconds on the GPU, so a tensor is checked by one
# short expression and what is wrong with it is looked up only if that fails.

def _refuse(t, name: str, shape, dtypes, dev: int):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor, got {type(t).__name__}")
    if t.dtype not in dtypes:
        kind = "bf16" if dtypes is _BF16 else dtypes[0]
        raise TypeError(f"{name} must hold {kind} data, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (this library has no CPU path)")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device} but the call runs on cuda:{dev}: every buffer "
                         "of a call must be on one device")
    raise ValueError(f"{name} must be contiguous")


def _typed(t: torch.Tensor, name: str, shape, dtype, dev: int) -> int:
    if (t.dtype is dtype and t.shape == shape and t.get_device() == dev >= 0
            and t.is_contiguous()):
        return t.data_ptr()
    return _refuse(t, name, shape, (dtype,), dev)


def _optional(t: torch.Tensor | None, name: str, n: int, dtypes, dev: int) -> int:
    """A buffer of at least n elements, or None."""
    if t is None:
        return 0
    if t.dtype not in dtypes or t.get_device() != dev or dev < 0 or not t.is_contiguous():
        _refuse(t, name, None, dtypes, dev)
    if t.numel() < n:
        raise ValueError(f"{name} holds {t.numel()} elements; the call needs {n}")
    return t.data_ptr()


def _rows(t: torch.Tensor, name: str, tokens: int, heads: int, dim: int,
          dev: int | None = None) -> _Rows:
    """A [tokens, heads, dim] bf16 tensor whose heads are contiguous and whose
    tokens may be apart (a view of a packed projection)."""
    dev = t.get_device() if dev is None else dev
    if t.dtype not in _BF16 or t.shape != (tokens, heads, dim) or t.get_device() != dev or dev < 0:
        st = t.stride()
        if len(st) == 3 and t.shape == (tokens, heads, dim) and t.dtype in _BF16 and (
                (dim > 1 and st[2] != 1) or (heads > 1 and st[1] != dim)):
            raise ValueError(f"{name}: the values of a token's heads must be contiguous")
        _refuse(t, name, (tokens, heads, dim), _BF16, dev)
    if t.is_contiguous():
        return _Rows(t.data_ptr(), heads * dim)
    st = t.stride()
    if (dim > 1 and st[2] != 1) or (heads > 1 and st[1] != dim):
        raise ValueError(f"{name}: the values of a token's heads must be contiguous")
    return _Rows(t.data_ptr(), st[0] if tokens > 1 else max(st[0], heads * dim))


# ------------------------------------------------------------------- cache --

def alloc_kv_cache(pages: int, page_size: int, kv_heads: int, head_dim: int,
                   k_amax: torch.Tensor, v_amax: torch.Tensor, four_over_six: bool = False) -> dict:
    """An empty paged NVFP4 cache on the device of k_amax. k_amax, v_amax: fp32
    [kv_heads], the (calibrated) largest magnitudes of K and V per head."""
    dev, c = k_amax.device, {"k_amax": k_amax, "v_amax": v_amax,
                             "four_over_six": int(four_over_six)}
    for n in ("k", "v"):
        c[n + "_codes"] = torch.zeros((pages, kv_heads, page_size, head_dim // 2),
                                      dtype=torch.uint8, device=dev)
        c[n + "_scales"] = torch.zeros((pages, kv_heads, page_size, head_dim // 16),
                                       dtype=torch.uint8, device=dev)
    return c


def _cache(c: dict, dev: int) -> tuple[bytes, int, int]:
    """The C struct of a cache, its KV heads and head_dim."""
    kc, u8 = c["k_codes"], torch.uint8
    if kc.dim() != 4:
        raise ValueError("k_codes must be [pages, kv_heads, page_size, head_dim/2]")
    pages, heads, page, half = shape = kc.shape
    scales = (pages, heads, page, half // 8)
    return _CACHE.pack(_typed(kc, "k_codes", shape, u8, dev),
                       _typed(c["k_scales"], "k_scales", scales, u8, dev),
                       _typed(c["v_codes"], "v_codes", shape, u8, dev),
                       _typed(c["v_scales"], "v_scales", scales, u8, dev),
                       _typed(c["k_amax"], "k_amax", (heads,), torch.float32, dev),
                       _typed(c["v_amax"], "v_amax", (heads,), torch.float32, dev),
                       pages, heads, page, 2 * half, int(c.get("four_over_six", 0))
                       ), heads, 2 * half


# ----------------------------------------------------------------- entries --

def nvfp4_kv_plan(cached: torch.Tensor, new: torch.Tensor, table: torch.Tensor,
                  free_pages: torch.Tensor, page_size: int, tokens: int,
                  out: dict | None = None, status: torch.Tensor | None = None) -> dict:
    """Block tables and slot maps from request lengths (int32 [requests] each).
    `table` (int32 [requests, columns]) is extended in place with pages from
    the front of `free_pages`. Returns {"table", "seq_lens", "q_start", "slots",
    "positions", "pages_used"}, allocated here unless `out` (an earlier return
    value) is passed."""
    dev = cached.get_device()
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return nvfp4_kv_plan(cached, new, table, free_pages, page_size, tokens, out, status)
    B = cached.shape[0]
    if table.dim() != 2:
        raise ValueError("table must be [requests, columns]")
    if tokens < 0:
        raise ValueError("tokens must not be negative")
    device, i32 = cached.device, torch.int32
    ins = (_typed(cached, "cached", (B,), i32, dev), _typed(new, "new", (B,), i32, dev), B,
           _typed(table, "table", (B, table.shape[1]), i32, dev), table.shape[1], page_size,
           _typed(free_pages, "free_pages", (free_pages.numel(),), i32, dev), free_pages.numel(),
           tokens)
    if out is None:
        empty = torch.empty
        seq, start = empty(B, dtype=i32, device=device), empty(B + 1, dtype=i32, device=device)
        slots = empty(tokens, dtype=torch.int64, device=device)
        pos, used = empty(tokens, dtype=i32, device=device), empty(1, dtype=i32, device=device)
        outs = (seq.data_ptr(), start.data_ptr(), slots.data_ptr(), pos.data_ptr(),
                used.data_ptr())
        out = {"table": table, "seq_lens": seq, "q_start": start, "slots": slots,
               "positions": pos, "pages_used": used}
    else:
        outs = (_typed(out["seq_lens"], "seq_lens", (B,), i32, dev),
                _typed(out["q_start"], "q_start", (B + 1,), i32, dev),
                _typed(out["slots"], "slots", (tokens,), torch.int64, dev),
                _typed(out["positions"], "positions", (tokens,), i32, dev),
                _typed(out["pages_used"], "pages_used", (1,), i32, dev))
        out = dict(out, table=table)
    status_code = _lib().nvfp4_kv_plan(
        *ins, *outs, 0 if status is None else _optional(status, "status", 1, _I32, dev),
        _stream(dev))
    if status_code:
        _check("nvfp4_kv_plan", status_code)
    return out


def _weight(w: torch.Tensor, name: str, dim: int, dev: int) -> int:
    if w.dtype not in _BF16 or w.shape != (dim,):
        raise ValueError(f"{name} must be bf16 [{dim}]")
    if w.get_device() != dev or dev < 0 or not w.is_contiguous():
        _refuse(w, name, None, _BF16, dev)
    return w.data_ptr()


def _qk(q, k, positions, cos_sin, q_weight, k_weight, eps, interleaved, dev) -> bytes:
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k must be [tokens, heads, head_dim]")
    T, hq, D = q.shape
    if cos_sin.dim() != 2:
        raise ValueError("cos_sin must be [positions, rotary_dim]")
    if cos_sin.dtype is not torch.float32:
        raise TypeError(f"cos_sin must be torch.float32, got {cos_sin.dtype}")
    length, rotary = cos_sin.shape
    return _QK.pack(T, hq, k.shape[1], D, rotary, interleaved, eps,
                    0 if q_weight is None else _weight(q_weight, "q_weight", D, dev),
                    0 if k_weight is None else _weight(k_weight, "k_weight", D, dev),
                    _typed(positions, "positions", (T,), torch.int32, dev),
                    _typed(cos_sin, "cos_sin", cos_sin.shape, torch.float32, dev), length)


def nvfp4_qk_norm_rope(q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor,
                       cos_sin: torch.Tensor, q_weight: torch.Tensor | None = None,
                       k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                       interleaved: bool = False, q_out: torch.Tensor | None = None,
                       k_out: torch.Tensor | None = None,
                       status: torch.Tensor | None = None) -> dict:
    """RMS norm of every head (where its weight is given) and rotation of q
    [tokens, q_heads, head_dim] and k [tokens, kv_heads, head_dim] (bf16; tokens
    may be apart) in one launch. cos_sin: fp32 [positions, rotary_dim], cosines
    then sines. Returns {"q", "k"}; q_out, k_out may be q and k themselves. Nothing is
    recorded for autograd: nvfp4_qk_norm_rope_bwd gives the gradient."""
    dev = q.get_device()
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return nvfp4_qk_norm_rope(q, k, positions, cos_sin, q_weight, k_weight, eps,
                                      interleaved, q_out, k_out, status)
    cfg = _qk(q, k, positions, cos_sin, q_weight, k_weight, eps, interleaved, dev)
    (T, hq, D), hk = q.shape, k.shape[1]
    rq, rk = _rows(q, "q", T, hq, D, dev), _rows(k, "k", T, hk, D, dev)
    if q_out is None:
        q_out = torch.empty((T, hq, D), dtype=q.dtype, device=q.device)
        ro = _Rows(q_out.data_ptr(), hq * D)
    else:
        ro = _rows(q_out, "q_out", T, hq, D, dev)
    if k_out is None:
        k_out = torch.empty((T, hk, D), dtype=k.dtype, device=q.device)
        ko = _Rows(k_out.data_ptr(), hk * D)
    else:
        ko = _rows(k_out, "k_out", T, hk, D, dev)
    status_code = _lib().nvfp4_qk_norm_rope(
        cfg, rq, rk, ro, ko, 0 if status is None else _optional(status, "status", 1, _I32, dev),
        _stream(dev))
    if status_code:
        _check("nvfp4_qk_norm_rope", status_code)
    return {"q": q_out, "k": k_out}


def _workspace(nbytes: int, device) -> torch.Tensor:
    return torch.zeros((nbytes + 3) // 4, dtype=torch.int32, device=device)


def qk_norm_rope_workspace(device) -> torch.Tensor:
    """A zeroed workspace for nvfp4_qk_norm_rope_bwd, for calls of any size: it
    serves one call at a time and is allocated and cleared once."""
    return _workspace(_lib().nvfp4_qk_norm_rope_ws_bytes(), device)


def nvfp4_qk_norm_rope_bwd(gq_out: torch.Tensor, gk_out: torch.Tensor, q: torch.Tensor,
                           k: torch.Tensor, positions: torch.Tensor, cos_sin: torch.Tensor,
                           q_weight: torch.Tensor | None = None,
                           k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                           interleaved: bool = False, workspace: torch.Tensor | None = None,
                           gq: torch.Tensor | None = None, gk: torch.Tensor | None = None,
                           status: torch.Tensor | None = None) -> dict:
    """Gradient of nvfp4_qk_norm_rope from the gradients of its outputs and its
    inputs: {"gq", "gk", "gq_weight", "gk_weight"} (weight gradients fp32, None
    without the weight). workspace: from qk_norm_rope_workspace; a fresh one is
    cleared for the call when none is given."""
    dev = q.get_device()
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return nvfp4_qk_norm_rope_bwd(gq_out, gk_out, q, k, positions, cos_sin, q_weight,
                                          k_weight, eps, interleaved, workspace, gq, gk, status)
    device = q.device
    cfg = _qk(q, k, positions, cos_sin, q_weight, k_weight, eps, interleaved, dev)
    (T, hq, D), hk = q.shape, k.shape[1]
    ins = (_rows(gq_out, "gq_out", T, hq, D, dev), _rows(gk_out, "gk_out", T, hk, D, dev),
           _rows(q, "q", T, hq, D, dev), _rows(k, "k", T, hk, D, dev))
    if gq is None:
        gq = torch.empty((T, hq, D), dtype=q.dtype, device=device)
    if gk is None:
        gk = torch.empty((T, hk, D), dtype=k.dtype, device=device)
    f32 = torch.float32
    gqw = gkw = None
    if q_weight is not None:
        gqw = torch.empty(D, dtype=f32, device=device)
    if k_weight is not None:
        gkw = torch.empty(D, dtype=f32, device=device)
    if workspace is None and (gqw is not None or gkw is not None):
        workspace = qk_norm_rope_workspace(device)
    status_code = _lib().nvfp4_qk_norm_rope_bwd(
        cfg, *ins, _rows(gq, "gq", T, hq, D, dev), _rows(gk, "gk", T, hk, D, dev),
        0 if gqw is None else gqw.data_ptr(), 0 if gkw is None else gkw.data_ptr(),
        _optional(workspace, "workspace", 1, _I32, dev),
        0 if workspace is None else 4 * workspace.numel(),
        0 if status is None else _optional(status, "status", 1, _I32, dev), _stream(dev))
    if status_code:
        _check("nvfp4_qk_norm_rope_bwd", status_code)
    return {"gq": gq, "gk": gk, "gq_weight": gqw, "gk_weight": gkw}


def nvfp4_kv_append(cache: dict, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor,
                    dequant: bool = False, status: torch.Tensor | None = None) -> dict:
    """Quantise K and V rows (bf16 [tokens, kv_heads, head_dim]; tokens may be
    apart) into the cache's slots (int64 [tokens], -1 = skip). Returns {"k",
    "v"}: with dequant the values the codes stand for (bf16), else None."""
    dev = cache["k_codes"].get_device()
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return nvfp4_kv_append(cache, k, v, slots, dequant, status)
    c, hk, D = _cache(cache, dev)
    T = k.shape[0]
    rk, rv = _rows(k, "k", T, hk, D, dev), _rows(v, "v", T, hk, D, dev)
    at = _typed(slots, "slots", (T,), torch.int64, dev)
    kd = vd = None
    if dequant:
        kd = torch.empty((T, hk, D), dtype=torch.bfloat16, device=k.device)
        vd = torch.empty((T, hk, D), dtype=torch.bfloat16, device=k.device)
    status_code = _lib().nvfp4_kv_append(
        c, rk, rv, at, T, kd.data_ptr() if dequant else 0, vd.data_ptr() if dequant else 0,
        0 if status is None else _optional(status, "status", 1, _I32, dev), _stream(dev))
    if status_code:
        _check("nvfp4_kv_append", status_code)
    return {"k": kd, "v": vd}


def kv_attention_workspace(device) -> torch.Tensor:
    """A zeroed workspace for nvfp4_kv_attention, for calls of any size: it
    serves one call at a time and is allocated and cleared once."""
    return _workspace(_lib().nvfp4_kv_attention_ws_bytes(), device)


def nvfp4_kv_attention(q: torch.Tensor, cache: dict, table: torch.Tensor, seq_lens: torch.Tensor,
                       q_start: torch.Tensor, max_q: int, scale: float | None = None,
                       window: int = 0, out: torch.Tensor | None = None,
                       lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                       status: torch.Tensor | None = None) -> dict:
    """Causal attention of the new query rows q (bf16 [tokens, q_heads,
    head_dim]) over the cache: request b owns rows q_start[b] .. q_start[b+1]-1
    and the first seq_lens[b] tokens of its block table row. max_q: an upper
    bound of the requests' query rows. scale defaults to head_dim ** -0.5.
    workspace: from kv_attention_workspace; a fresh one is cleared for the call
    when none is given. Returns {"out", "lse"}."""
    dev = q.get_device()
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return nvfp4_kv_attention(q, cache, table, seq_lens, q_start, max_q, scale, window,
                                      out, lse, workspace, status)
    device, i32 = q.device, torch.int32
    if q.dim() != 3 or table.dim() != 2:
        raise ValueError("q must be [tokens, q_heads, head_dim], table [requests, columns]")
    c, _, dim = _cache(cache, dev)
    T, hq, D = q.shape
    if D != dim:
        raise ValueError(f"q has head_dim {D}, the cache {dim}")
    if scale is None:
        scale = D ** -0.5
    elif not math.isfinite(scale):
        raise ValueError("scale must be finite")
    B, cols = seq_lens.shape[0], table.shape[1]
    cfg = _ATTENTION.pack(_typed(table, "table", (B, cols), i32, dev),
                          _typed(seq_lens, "seq_lens", (B,), i32, dev),
                          _typed(q_start, "q_start", (B + 1,), i32, dev), B, cols, T, hq, max_q,
                          window, scale)
    rq = _rows(q, "q", T, hq, D, dev)
    if out is None:
        out = torch.empty((T, hq, D), dtype=torch.bfloat16, device=device)
        out_at = out.data_ptr()
    else:
        out_at = _optional(out, "out", T * hq * D, _BF16, dev)
    if lse is None:
        lse = torch.empty((T, hq), dtype=torch.float32, device=device)
        lse_at = lse.data_ptr()
    else:
        lse_at = _optional(lse, "lse", T * hq, (torch.float32,), dev)
    if workspace is None:
        workspace = kv_attention_workspace(device)
    status_code = _lib().nvfp4_kv_attention(
        c, cfg, rq, out_at, lse_at, _optional(workspace, "workspace", 1, _I32, dev),
        4 * workspace.numel(), 0 if status is None else _optional(status, "status", 1, _I32, dev),
        _stream(dev))
    if status_code:
        _check("nvfp4_kv_attention", status_code)
    return {"out": out, "lse": lse}
