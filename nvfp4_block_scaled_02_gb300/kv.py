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
import functools
import math

import torch

from . import _check, _dev, _i32, _i64, _need, _stream, _vp, lib

_BF16 = (torch.bfloat16, torch.int16, torch.uint16)
_BYTES = (torch.uint8, torch.int8)


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


def declare(L: C.CDLL) -> None:
    """Argument types of the library's entry points of this module."""
    size = C.c_size_t
    L.nvfp4_kv_plan.argtypes = [_vp, _vp, _i64, _vp, _i64, _i32, _vp, _i64, _i64, _vp, _vp, _vp,
                                _vp, _vp, _vp, _vp]
    L.nvfp4_qk_norm_rope.argtypes = [C.POINTER(_QkConfig), _Rows, _Rows, _Rows, _Rows, _vp, _vp]
    L.nvfp4_qk_norm_rope_bwd.argtypes = [C.POINTER(_QkConfig)] + [_Rows] * 6 + [
        _vp, _vp, _vp, size, _vp, _vp]
    L.nvfp4_kv_append.argtypes = [C.POINTER(_Cache), _Rows, _Rows, _vp, _i64, _vp, _vp, _vp, _vp]
    L.nvfp4_kv_attention.argtypes = [C.POINTER(_Cache), C.POINTER(_AttentionConfig), _Rows, _vp,
                                     _vp, _vp, size, _vp, _vp]
    for name in ("nvfp4_kv_plan", "nvfp4_qk_norm_rope", "nvfp4_qk_norm_rope_bwd",
                 "nvfp4_kv_append", "nvfp4_kv_attention"):
        getattr(L, name).restype = C.c_int
    for name in ("nvfp4_qk_norm_rope_ws_bytes", "nvfp4_kv_attention_ws_bytes"):
        getattr(L, name).argtypes = []
        getattr(L, name).restype = size


def _on_device(fn):
    """Run an entry point with the device of its first tensor current (no
    device switch where it is current already: these calls are short)."""
    @functools.wraps(fn)
    def wrapper(*args, **kwargs):
        x = args[0] if not isinstance(args[0], dict) else args[0]["k_codes"]
        if not x.is_cuda or x.device.index == torch.cuda.current_device():
            return fn(*args, **kwargs)
        with torch.cuda.device(x.device):
            return fn(*args, **kwargs)
    return wrapper


def _rows(t: torch.Tensor, name: str, tokens: int, heads: int, dim: int) -> _Rows:
    """A [tokens, heads, dim] bf16 tensor whose heads are contiguous and whose
    tokens may be apart (a view of a packed projection)."""
    if t.dtype not in _BF16:
        raise TypeError(f"{name} must hold bf16 data, got {t.dtype}")
    if t.shape != (tokens, heads, dim):
        raise ValueError(f"{name} must be [{tokens}, {heads}, {dim}], got {list(t.shape)}")
    if t.is_contiguous():
        return _Rows(_dev(t, name), heads * dim)
    st = t.stride()
    if (dim > 1 and st[2] != 1) or (heads > 1 and st[1] != dim):
        raise ValueError(f"{name}: the values of a token's heads must be contiguous")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (this library has no CPU path)")
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device} but the call runs on "
                         f"cuda:{torch.cuda.current_device()}: every buffer of a call must "
                         "be on one device")
    return _Rows(t.data_ptr(), st[0] if tokens > 1 else max(st[0], heads * dim))


def _typed(t: torch.Tensor, name: str, shape, dtype) -> int:
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return _dev(t, name)


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


def _cache(c: dict) -> _Cache:
    kc = c["k_codes"]
    if kc.dim() != 4:
        raise ValueError("k_codes must be [pages, kv_heads, page_size, head_dim/2]")
    pages, heads, page, half = shape = kc.shape
    scales = (pages, heads, page, half // 8)
    return _Cache(_typed(kc, "k_codes", shape, torch.uint8),
                  _typed(c["k_scales"], "k_scales", scales, torch.uint8),
                  _typed(c["v_codes"], "v_codes", shape, torch.uint8),
                  _typed(c["v_scales"], "v_scales", scales, torch.uint8),
                  _typed(c["k_amax"], "k_amax", (heads,), torch.float32),
                  _typed(c["v_amax"], "v_amax", (heads,), torch.float32),
                  pages, heads, page, 2 * half, int(c.get("four_over_six", 0)))


# ----------------------------------------------------------------- entries --

@_on_device
def nvfp4_kv_plan(cached: torch.Tensor, new: torch.Tensor, table: torch.Tensor,
                  free_pages: torch.Tensor, page_size: int, tokens: int,
                  out: dict | None = None, status: torch.Tensor | None = None) -> dict:
    """Block tables and slot maps from request lengths (int32 [requests] each).
    `table` (int32 [requests, columns]) is extended in place with pages from
    the front of `free_pages`. Returns {"table", "seq_lens", "q_start", "slots",
    "positions", "pages_used"}, allocated here unless `out` (an earlier return
    value) is passed."""
    B = cached.shape[0]
    if table.dim() != 2:
        raise ValueError("table must be [requests, columns]")
    dev, i32 = cached.device, torch.int32
    if out is None:
        if tokens < 0:
            raise ValueError("tokens must not be negative")
        out = {"seq_lens": torch.empty(B, dtype=i32, device=dev),
               "q_start": torch.empty(B + 1, dtype=i32, device=dev),
               "slots": torch.empty(tokens, dtype=torch.int64, device=dev),
               "positions": torch.empty(tokens, dtype=i32, device=dev),
               "pages_used": torch.empty(1, dtype=i32, device=dev)}
    _need(status, "status", 1, "i32")
    _check("nvfp4_kv_plan", lib().nvfp4_kv_plan(
        _typed(cached, "cached", (B,), i32), _typed(new, "new", (B,), i32), B,
        _typed(table, "table", (B, table.shape[1]), i32), table.shape[1], page_size,
        _typed(free_pages, "free_pages", (free_pages.numel(),), i32), free_pages.numel(), tokens,
        _typed(out["seq_lens"], "seq_lens", (B,), i32),
        _typed(out["q_start"], "q_start", (B + 1,), i32),
        _typed(out["slots"], "slots", (tokens,), torch.int64),
        _typed(out["positions"], "positions", (tokens,), i32),
        _typed(out["pages_used"], "pages_used", (1,), i32), _dev(status, "status"), _stream(dev)))
    out["table"] = table
    return out


def _qk(q, k, positions, cos_sin, q_weight, k_weight, eps, interleaved) -> _QkConfig:
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k must be [tokens, heads, head_dim]")
    T, hq, D = q.shape
    if cos_sin.dim() != 2:
        raise ValueError("cos_sin must be [positions, rotary_dim]")
    if cos_sin.dtype is not torch.float32:
        raise TypeError(f"cos_sin must be torch.float32, got {cos_sin.dtype}")
    for w, n in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None and (w.dtype not in _BF16 or w.shape != (D,)):
            raise ValueError(f"{n} must be bf16 [{D}]")
    return _QkConfig(T, hq, k.shape[1], D, cos_sin.shape[1], int(interleaved), eps,
                     _dev(q_weight, "q_weight"), _dev(k_weight, "k_weight"),
                     _typed(positions, "positions", (T,), torch.int32),
                     _typed(cos_sin, "cos_sin", tuple(cos_sin.shape), torch.float32),
                     cos_sin.shape[0])


@_on_device
def nvfp4_qk_norm_rope(q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor,
                       cos_sin: torch.Tensor, q_weight: torch.Tensor | None = None,
                       k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                       interleaved: bool = False, q_out: torch.Tensor | None = None,
                       k_out: torch.Tensor | None = None,
                       status: torch.Tensor | None = None) -> dict:
    """RMS norm of every head (where its weight is given) and rotation of q
    [tokens, q_heads, head_dim] and k [tokens, kv_heads, head_dim] (bf16; tokens
    may be apart) in one launch. cos_sin: fp32 [positions, rotary_dim], cosines
    then sines. Returns {"q", "k"}; q_out, k_out may be q and k themselves."""
    cfg = _qk(q, k, positions, cos_sin, q_weight, k_weight, eps, interleaved)
    T, hq, D = q.shape
    hk = k.shape[1]
    if q_out is None:
        q_out = torch.empty((T, hq, D), dtype=q.dtype, device=q.device)
    if k_out is None:
        k_out = torch.empty((T, hk, D), dtype=k.dtype, device=q.device)
    _need(status, "status", 1, "i32")
    _check("nvfp4_qk_norm_rope", lib().nvfp4_qk_norm_rope(
        C.byref(cfg), _rows(q, "q", T, hq, D), _rows(k, "k", T, hk, D),
        _rows(q_out, "q_out", T, hq, D), _rows(k_out, "k_out", T, hk, D),
        _dev(status, "status"), _stream(q.device)))
    return {"q": q_out, "k": k_out}


def _workspace(nbytes: int, device) -> torch.Tensor:
    return torch.zeros((nbytes + 3) // 4, dtype=torch.int32, device=device)


def qk_norm_rope_workspace(device) -> torch.Tensor:
    """A zeroed workspace for nvfp4_qk_norm_rope_bwd, for calls of any size: it
    serves one call at a time and is allocated and cleared once."""
    return _workspace(lib().nvfp4_qk_norm_rope_ws_bytes(), device)


@_on_device
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
    cfg = _qk(q, k, positions, cos_sin, q_weight, k_weight, eps, interleaved)
    T, hq, D = q.shape
    hk, dev = k.shape[1], q.device
    if gq is None:
        gq = torch.empty((T, hq, D), dtype=q.dtype, device=dev)
    if gk is None:
        gk = torch.empty((T, hk, D), dtype=k.dtype, device=dev)
    gqw = None if q_weight is None else torch.empty(D, dtype=torch.float32, device=dev)
    gkw = None if k_weight is None else torch.empty(D, dtype=torch.float32, device=dev)
    if workspace is None and (gqw is not None or gkw is not None):
        workspace = qk_norm_rope_workspace(dev)
    _need(workspace, "workspace", 1, "i32")
    _need(status, "status", 1, "i32")
    _check("nvfp4_qk_norm_rope_bwd", lib().nvfp4_qk_norm_rope_bwd(
        C.byref(cfg), _rows(gq_out, "gq_out", T, hq, D), _rows(gk_out, "gk_out", T, hk, D),
        _rows(q, "q", T, hq, D), _rows(k, "k", T, hk, D), _rows(gq, "gq", T, hq, D),
        _rows(gk, "gk", T, hk, D), _dev(gqw, "gq_weight"), _dev(gkw, "gk_weight"),
        _dev(workspace, "workspace"), 0 if workspace is None else workspace.numel() * 4,
        _dev(status, "status"), _stream(dev)))
    return {"gq": gq, "gk": gk, "gq_weight": gqw, "gk_weight": gkw}


@_on_device
def nvfp4_kv_append(cache: dict, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor,
                    dequant: bool = False, status: torch.Tensor | None = None) -> dict:
    """Quantise K and V rows (bf16 [tokens, kv_heads, head_dim]; tokens may be
    apart) into the cache's slots (int64 [tokens], -1 = skip). Returns {"k",
    "v"}: with dequant the values the codes stand for (bf16), else None."""
    c = _cache(cache)
    T, hk, D = k.shape[0], c.kv_heads, c.head_dim
    kd = vd = None
    if dequant:
        kd = torch.empty((T, hk, D), dtype=torch.bfloat16, device=k.device)
        vd = torch.empty((T, hk, D), dtype=torch.bfloat16, device=k.device)
    _need(status, "status", 1, "i32")
    _check("nvfp4_kv_append", lib().nvfp4_kv_append(
        C.byref(c), _rows(k, "k", T, hk, D), _rows(v, "v", T, hk, D),
        _typed(slots, "slots", (T,), torch.int64), T, _dev(kd, "k dequant"),
        _dev(vd, "v dequant"), _dev(status, "status"), _stream(k.device)))
    return {"k": kd, "v": vd}


def kv_attention_workspace(device) -> torch.Tensor:
    """A zeroed workspace for nvfp4_kv_attention, for calls of any size: it
    serves one call at a time and is allocated and cleared once."""
    return _workspace(lib().nvfp4_kv_attention_ws_bytes(), device)


@_on_device
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
    c = _cache(cache)
    if q.dim() != 3 or table.dim() != 2:
        raise ValueError("q must be [tokens, q_heads, head_dim], table [requests, columns]")
    T, hq, D = q.shape
    B, dev, i32 = seq_lens.shape[0], q.device, torch.int32
    if D != c.head_dim:
        raise ValueError(f"q has head_dim {D}, the cache {c.head_dim}")
    if out is None:
        out = torch.empty((T, hq, D), dtype=torch.bfloat16, device=dev)
    else:
        _need(out, "out", T * hq * D, "bf16")
    if lse is None:
        lse = torch.empty((T, hq), dtype=torch.float32, device=dev)
    else:
        _need(lse, "lse", T * hq, "f32")
    if workspace is None:
        workspace = kv_attention_workspace(dev)
    _need(workspace, "workspace", 1, "i32")
    _need(status, "status", 1, "i32")
    cfg = _AttentionConfig(_typed(table, "table", (B, table.shape[1]), i32),
                           _typed(seq_lens, "seq_lens", (B,), i32),
                           _typed(q_start, "q_start", (B + 1,), i32), B, table.shape[1], T, hq,
                           max_q, window, D ** -0.5 if scale is None else scale)
    if not math.isfinite(cfg.scale):
        raise ValueError("scale must be finite")
    _check("nvfp4_kv_attention", lib().nvfp4_kv_attention(
        C.byref(c), C.byref(cfg), _rows(q, "q", T, hq, D), _dev(out, "out"), _dev(lse, "lse"),
        _dev(workspace, "workspace"), workspace.numel() * 4, _dev(status, "status"),
        _stream(dev)))
    return {"out": out, "lse": lse}
