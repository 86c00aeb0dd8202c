"""Binding of the quantised linear layer's operators: the residual norm that encodes
its input (and its gradient), products of NVFP4 and MXFP8 encodings grouped by
expert. Like the package's other entry points these only
check and marshal arguments; ``include/nvfp4.h`` states what each computes.

    a = nvfp4_add_rms_norm(x, weight, residual)
    y = nvfp4_grouped_matmul(a, a["row_amax"], w, w_amax, group_start, workspace=ws)
"""
from __future__ import annotations

import ctypes as C
import struct

import torch

from . import (Config, SCALE_E4M3, TARGET_MXFP8, TARGET_NVFP4, _check, _i32, _i64, _Out, _vp)
from .kv import _BF16, _I32, _lib, _optional, _refuse, _typed

_F32 = (torch.float32,)
_U8 = (torch.uint8, torch.int8)


class _Operand(C.Structure):
    _fields_ = [("codes", _vp), ("scales", _vp), ("amax", _vp), ("amax_count", _i64),
                ("scale_max", C.c_float)]


# structs packed into bytes, as in kv; the default config is packed once
_OPERAND, _OUT = struct.Struct("@3Pqf4x"), struct.Struct("@4P")
assert _OPERAND.size == C.sizeof(_Operand) and _OUT.size == C.sizeof(_Out)
_DEFAULT = bytes(Config().c())
_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


def declare(L: C.CDLL) -> None:
    """Argument types of the library's entry points of this module."""
    size = C.c_size_t
    L.nvfp4_grouped_matmul.argtypes = [_vp, _vp, _i64, _i64, _i64, _i64, _vp, _vp, _vp, size, _vp,
                                       _vp]
    L.nvfp4_mx_grouped_matmul.argtypes = [_vp] * 4 + [_i64] * 4 + [_vp, _vp, _vp, size, _vp, _vp]
    L.nvfp4_mx_grouped_wgrad.argtypes = [_vp] * 4 + [_i64] * 4 + [_vp, _vp, _i32, _vp, size, _vp,
                                                                  _vp]
    L.nvfp4_add_rms_norm.argtypes = [_vp, _i32, _vp, _vp, _vp, _i64, _i64, C.c_float, _vp, _vp,
                                     _vp, _vp, _vp, _vp, _vp]
    L.nvfp4_add_rms_norm_bwd.argtypes = [_vp] * 4 + [_i64, _i64, C.c_float, _vp, _vp, _vp, size,
                                                     _vp, _vp]
    for name in ("nvfp4_grouped_matmul", "nvfp4_mx_grouped_matmul", "nvfp4_mx_grouped_wgrad",
                 "nvfp4_add_rms_norm", "nvfp4_add_rms_norm_bwd"):
        getattr(L, name).restype = C.c_int
    for name in ("nvfp4_grouped_matmul_ws_bytes", "nvfp4_add_rms_norm_ws_bytes"):
        getattr(L, name).argtypes = []
        getattr(L, name).restype = size


def grouped_matmul_workspace(device) -> torch.Tensor:
    """A workspace (89 MB, its counters cleared) for the three grouped products, for
    calls of any size: it serves one call at a time and is allocated and cleared once."""
    t = torch.empty((_lib().nvfp4_grouped_matmul_ws_bytes() + 3) // 4, dtype=torch.int32,
                    device=device)
    t[:1024].zero_()
    return t


def _bytes(t: torch.Tensor, name: str, n: int, dev: int) -> int:
    """An encoding's array of exactly n bytes."""
    if t.dtype in _U8 and t.numel() == n and t.get_device() == dev >= 0 and t.is_contiguous():
        return t.data_ptr()
    if t.dtype not in _U8 or t.get_device() != dev or dev < 0 or not t.is_contiguous():
        _refuse(t, name, None, _U8, dev)
    raise ValueError(f"{name} holds {t.numel()} bytes; the call needs {n}")


def _rows_of(t: torch.Tensor, name: str) -> tuple[int, int]:
    """Rows and bytes per row of an encoding's codes."""
    shape = t.shape
    if len(shape) == 2:
        return shape
    if len(shape) < 2:
        raise ValueError(f"{name} must be [rows, bytes] or [slices, rows, bytes]")
    width = shape[-1]
    return (t.numel() // width if width else 0), width


def _groups_of(t: torch.Tensor, name: str) -> tuple[int, int, int]:
    """Groups, rows of a group and bytes per row of the weights' codes."""
    shape = t.shape
    if len(shape) == 3:
        return shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be [rows, bytes] or [groups, rows, bytes]")
    return 1, shape[0], shape[1]


def _starts(start: torch.Tensor | None, groups: int, dev: int) -> int:
    if start is None:
        if groups != 1:
            raise ValueError(f"group_start is needed with {groups} groups")
        return 0
    return _typed(start, "group_start", (groups + 1,), torch.int32, dev)


def _result(out, shape, dtypes, dev: int) -> int:
    if out.dtype in dtypes and out.shape == shape and out.get_device() == dev and (
            out.is_contiguous()):
        return out.data_ptr()
    return _refuse(out, "out", shape, dtypes, dev)


def _outer_max(cfg: Config | None, name: str) -> float:
    if cfg is None:
        return 0.0
    if cfg.scale_fmt != SCALE_E4M3:
        raise ValueError(f"{name}: the products take E4M3 block scales only")
    return cfg.scale_max or (256.0 if cfg.four_over_six else 448.0)


def nvfp4_grouped_matmul(a: dict, a_amax: torch.Tensor, b: dict, b_amax: torch.Tensor,
                         group_start: torch.Tensor | None = None, a_cfg: Config | None = None,
                         b_cfg: Config | None = None, out: torch.Tensor | None = None,
                         workspace: torch.Tensor | None = None,
                         status: torch.Tensor | None = None) -> torch.Tensor:
    """bf16 [rows, out_cols]: the NVFP4 rows of `a` (a row encoding: "codes" and
    "scales") times the weights of each row's group, `b` ("codes" [groups, out_cols,
    cols/2], or [out_cols, cols/2] for one group). a_amax: fp32 [1] or [rows] (as
    nvfp4_quantize_per_token's row_amax); b_amax: fp32 [groups]. group_start: int32
    [groups + 1]; rows outside of it are left as they are in `out` (unset in a fresh
    one). a_cfg, b_cfg: how the operands were encoded (Four-Over-Six and scale_max set
    the outer scale). workspace: from grouped_matmul_workspace; a fresh one is cleared
    for the call when none is given."""
    ac, bc = a["codes"], b["codes"]
    dev = ac.get_device()
    if dev >= 0 and dev != _device():
        with torch.cuda.device(dev):
            return nvfp4_grouped_matmul(a, a_amax, b, b_amax, group_start, a_cfg, b_cfg, out,
                                        workspace, status)
    asc, bsc = a["scales"], b["scales"]
    T, half = _rows_of(ac, "a codes")
    E, N, bhalf = _groups_of(bc, "b codes")
    n, f32 = a_amax.numel(), torch.float32
    # one expression for what is usual; what is wrong is looked up only if it fails
    if not (half == bhalf and (n == 1 or n == T) and b_amax.numel() == E
            and asc.numel() * 8 == T * half and bsc.numel() * 8 == E * N * half
            and ac.dtype in _U8 and asc.dtype in _U8 and bc.dtype in _U8 and bsc.dtype in _U8
            and a_amax.dtype is f32 and b_amax.dtype is f32
            and dev == asc.get_device() == bc.get_device() == bsc.get_device() >= 0
            and dev == a_amax.get_device() == b_amax.get_device()
            and ac.is_contiguous() and asc.is_contiguous() and bc.is_contiguous()
            and bsc.is_contiguous() and a_amax.is_contiguous() and b_amax.is_contiguous()):
        if half != bhalf:
            raise ValueError(f"a has rows of {2 * half} values, b of {2 * bhalf}")
        if n != 1 and n != T:
            raise ValueError(f"a_amax holds {n} elements; the call needs 1 or {T}")
        if b_amax.numel() != E:
            raise ValueError(f"b_amax holds {b_amax.numel()} elements; the call needs {E}")
        _bytes(ac, "a codes", T * half, dev)
        _bytes(asc, "a scales", T * half // 8, dev)
        _bytes(bc, "b codes", E * N * half, dev)
        _bytes(bsc, "b scales", E * N * half // 8, dev)
        _optional(a_amax, "a_amax", n, _F32, dev)
        _optional(b_amax, "b_amax", E, _F32, dev)
    pa = _OPERAND.pack(ac.data_ptr(), asc.data_ptr(), a_amax.data_ptr(), n,
                       0.0 if a_cfg is None else _outer_max(a_cfg, "a_cfg"))
    pb = _OPERAND.pack(bc.data_ptr(), bsc.data_ptr(), b_amax.data_ptr(), E,
                       0.0 if b_cfg is None else _outer_max(b_cfg, "b_cfg"))
    start = _starts(group_start, E, dev)
    if out is None:
        out = torch.empty((T, N), dtype=torch.bfloat16, device=ac.device)
        to = out.data_ptr()
    else:
        to = _result(out, (T, N), _BF16, dev)
    if workspace is None:
        workspace = grouped_matmul_workspace(ac.device)
    ws, ws_bytes = _optional(workspace, "workspace", 1, _I32, dev), 4 * workspace.numel()
    code = _lib().nvfp4_grouped_matmul(
        pa, pb, T, E, N, 2 * half, start, to, ws, ws_bytes,
        0 if status is None else _optional(status, "status", 1, _I32, dev), _raw_stream(dev))
    if code:
        _check("nvfp4_grouped_matmul", code)
    return out


def nvfp4_mx_grouped_matmul(a: dict, b: dict, group_start: torch.Tensor | None = None,
                            out: torch.Tensor | None = None,
                            workspace: torch.Tensor | None = None,
                            status: torch.Tensor | None = None) -> torch.Tensor:
    """nvfp4_grouped_matmul with MXFP8 operands (as nvfp4_mx_quantize and
    nvfp4_requant_transpose give them): `a` "codes" [rows, cols], `b` "codes" [groups,
    out_cols, cols]."""
    ac, bc = a["codes"], b["codes"]
    dev = ac.get_device()
    if dev >= 0 and dev != _device():
        with torch.cuda.device(dev):
            return nvfp4_mx_grouped_matmul(a, b, group_start, out, workspace, status)
    T, K = _rows_of(ac, "a codes")
    E, N, bk = _groups_of(bc, "b codes")
    if K != bk:
        raise ValueError(f"a has rows of {K} values, b of {bk}")
    asc, bsc = a["scales"], b["scales"]
    if not (asc.numel() * 32 == T * K and bsc.numel() * 32 == E * N * K
            and ac.dtype in _U8 and asc.dtype in _U8 and bc.dtype in _U8 and bsc.dtype in _U8
            and dev == asc.get_device() == bc.get_device() == bsc.get_device() >= 0
            and ac.is_contiguous() and asc.is_contiguous() and bc.is_contiguous()
            and bsc.is_contiguous()):
        _bytes(ac, "a codes", T * K, dev)
        _bytes(asc, "a scales", T * K // 32, dev)
        _bytes(bc, "b codes", E * N * K, dev)
        _bytes(bsc, "b scales", E * N * K // 32, dev)
    ins = (ac.data_ptr(), asc.data_ptr(), bc.data_ptr(), bsc.data_ptr())
    start = _starts(group_start, E, dev)
    if out is None:
        out = torch.empty((T, N), dtype=torch.bfloat16, device=ac.device)
        to = out.data_ptr()
    else:
        to = _result(out, (T, N), _BF16, dev)
    if workspace is None:
        workspace = grouped_matmul_workspace(ac.device)
    ws, ws_bytes = _optional(workspace, "workspace", 1, _I32, dev), 4 * workspace.numel()
    code = _lib().nvfp4_mx_grouped_matmul(
        *ins, T, E, N, K, start, to, ws, ws_bytes,
        0 if status is None else _optional(status, "status", 1, _I32, dev), _raw_stream(dev))
    if code:
        _check("nvfp4_mx_grouped_matmul", code)
    return out


def nvfp4_mx_grouped_wgrad(g: dict, x: dict, group_start: torch.Tensor | None = None,
                           out: torch.Tensor | None = None,
                           out_dtype: torch.dtype = torch.bfloat16,
                           workspace: torch.Tensor | None = None,
                           status: torch.Tensor | None = None) -> torch.Tensor:
    """Every group's weight gradient [groups, out_rows, out_cols] (bf16 or fp32): the
    sum over the group's rows of g's times x's values, both MXFP8 column encodings
    ("codes" [out_rows, rows] and [out_cols, rows], as nvfp4_mx_quantize's "col").
    Every entry of group_start is a multiple of 32."""
    gc, xc = g["codes"], x["codes"]
    dev = gc.get_device()
    if dev >= 0 and dev != _device():
        with torch.cuda.device(dev):
            return nvfp4_mx_grouped_wgrad(g, x, group_start, out, out_dtype, workspace, status)
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"out_dtype must be bf16 or fp32, got {out_dtype}")
    (sn, N, T), (sk, K, xt) = _groups_of(gc, "g codes"), _groups_of(xc, "x codes")
    if sn != 1 or sk != 1:
        raise ValueError("g and x must be one matrix each")
    if T != xt:
        raise ValueError(f"g has {T} rows, x {xt}")
    E = 1 if group_start is None else group_start.numel() - 1
    if E < 0:
        raise ValueError("group_start must hold groups + 1 entries")
    gsc, xsc = g["scales"], x["scales"]
    if not (gsc.numel() * 32 == N * T and xsc.numel() * 32 == K * T
            and gc.dtype in _U8 and gsc.dtype in _U8 and xc.dtype in _U8 and xsc.dtype in _U8
            and dev == gsc.get_device() == xc.get_device() == xsc.get_device() >= 0
            and gc.is_contiguous() and gsc.is_contiguous() and xc.is_contiguous()
            and xsc.is_contiguous()):
        _bytes(gc, "g codes", N * T, dev)
        _bytes(gsc, "g scales", N * T // 32, dev)
        _bytes(xc, "x codes", K * T, dev)
        _bytes(xsc, "x scales", K * T // 32, dev)
    ins = (gc.data_ptr(), gsc.data_ptr(), xc.data_ptr(), xsc.data_ptr())
    start = _starts(group_start, E, dev)
    if out is None:
        f32 = out_dtype is torch.float32
        out = torch.empty((E, N, K), dtype=out_dtype, device=gc.device)
        to = out.data_ptr()
    else:
        f32 = out.dtype is torch.float32
        to = _result(out, (E, N, K), _F32 if f32 else _BF16, dev)
    if workspace is None:
        workspace = grouped_matmul_workspace(gc.device)
    ws, ws_bytes = _optional(workspace, "workspace", 1, _I32, dev), 4 * workspace.numel()
    code = _lib().nvfp4_mx_grouped_wgrad(
        *ins, T, E, N, K, start, to, f32, ws, ws_bytes,
        0 if status is None else _optional(status, "status", 1, _I32, dev), _raw_stream(dev))
    if code:
        _check("nvfp4_mx_grouped_wgrad", code)
    return out


def _matrix(t: torch.Tensor, name: str, shape, dev: int) -> int:
    if (t.dtype in _BF16 and t.shape == shape and t.get_device() == dev >= 0
            and t.is_contiguous()):
        return t.data_ptr()
    return _refuse(t, name, shape, _BF16, dev)


def nvfp4_add_rms_norm(x: torch.Tensor, weight: torch.Tensor,
                       residual: torch.Tensor | None = None, eps: float = 1e-6,
                       target: int = TARGET_NVFP4, cfg: Config | None = None,
                       global_amax: torch.Tensor | None = None, dequant: bool = False,
                       h: torch.Tensor | None = None, y: torch.Tensor | None = None,
                       out: dict | None = None, row_amax: torch.Tensor | None = None,
                       status: torch.Tensor | None = None) -> dict:
    """h = x + residual, its RMS norm times weight, and the row encoding of that: NVFP4
    with an outer scale for each row ("row_amax") or from global_amax (fp32 [1]), or
    MXFP8 (target). x, residual: bf16 [rows, cols]; weight: bf16 [cols]. Returns {"h",
    "y", "codes", "scales", "choice", "dequant", "row_amax"}: h is x itself without a
    residual, y (bf16) is written where a buffer is passed, dequant (NVFP4) where asked
    for, choice with Four-Over-Six; what a call does not write is None. `out`: an
    encoding of an earlier call, written where it lies (its dequant too, if it has one).
    Nothing is recorded for autograd: nvfp4_add_rms_norm_bwd gives the gradient."""
    dev = x.get_device()
    if dev >= 0 and dev != _device():
        with torch.cuda.device(dev):
            return nvfp4_add_rms_norm(x, weight, residual, eps, target, cfg, global_amax, dequant,
                                      h, y, out, row_amax, status)
    shape = x.shape
    if len(shape) != 2:
        raise ValueError("x must be [rows, cols]")
    R, Cc = shape
    # one expression for what is usual; what is wrong is looked up only if it fails
    if not (x.dtype in _BF16 and x.is_contiguous() and dev >= 0 and weight.dtype in _BF16
            and weight.shape == (Cc,) and weight.get_device() == dev and weight.is_contiguous()
            and (residual is None or (residual.dtype in _BF16 and residual.shape == shape
                                      and residual.get_device() == dev
                                      and residual.is_contiguous()))):
        _matrix(x, "x", shape, dev)
        _matrix(weight, "weight", (Cc,), dev)
        _matrix(residual, "residual", shape, dev)
    fp4 = target == TARGET_NVFP4
    if not fp4 and target != TARGET_MXFP8:
        raise ValueError("target must be TARGET_MXFP8 or TARGET_NVFP4")
    if dequant and not fp4:
        raise ValueError("dequant is of the NVFP4 target")
    if row_amax is not None and (global_amax is not None or not fp4):
        raise ValueError("row_amax is written for the NVFP4 target without global_amax")
    empty, device = torch.empty, x.device
    if residual is None:
        if h is not None and h is not x:
            raise ValueError("h is x itself without a residual")
        h, h_at = x, 0
    elif h is None:
        h = empty(shape, dtype=x.dtype, device=device)
        h_at = h.data_ptr()
    else:
        h_at = _matrix(h, "h", shape, dev)
    fos = fp4 and cfg is not None and bool(cfg.four_over_six)
    per, block = (2, 16) if fp4 else (1, 32)
    if out is None:
        codes = empty((R, Cc // per), dtype=torch.uint8, device=device)
        scales = empty((R, Cc // block), dtype=torch.uint8, device=device)
        choice = dq = None
        if fos:
            choice = empty((R, (Cc + 511) // 512), dtype=torch.int32, device=device)
        if dequant and fp4:
            dq = empty(shape, dtype=torch.bfloat16, device=device)
        o = _OUT.pack(codes.data_ptr(), scales.data_ptr(), choice.data_ptr() if fos else 0,
                      0 if dq is None else dq.data_ptr())
    else:
        codes, scales, dq = out["codes"], out["scales"], out.get("dequant")
        choice = out.get("choice") if fos else None
        if dequant and dq is None:
            raise ValueError("dequant is asked for, but out has no buffer for it")
        if dq is not None and not fp4:
            raise ValueError("out has a dequant buffer, which is of the NVFP4 target")
        o = _OUT.pack(
            _bytes(codes, "out codes", R * Cc // per, dev),
            _bytes(scales, "out scales", R * Cc // block, dev),
            _optional(choice, "out choice", R * ((Cc + 511) // 512), _I32, dev),
            _optional(dq, "out dequant", R * Cc, _BF16, dev))
    amax_at = row_at = 0
    if not fp4:
        row_amax = None
    elif global_amax is not None:
        amax_at, row_amax = _optional(global_amax, "global_amax", 1, _F32, dev), None
    elif row_amax is None:
        row_amax = empty(R, dtype=torch.float32, device=device)
        row_at = row_amax.data_ptr()
    else:
        row_at = _optional(row_amax, "row_amax", R, _F32, dev)
    code = _lib().nvfp4_add_rms_norm(
        _DEFAULT if cfg is None else bytes(cfg.c()), target, x.data_ptr(),
        0 if residual is None else residual.data_ptr(), weight.data_ptr(), R, Cc, eps, h_at,
        0 if y is None else _matrix(y, "y", shape, dev), amax_at, row_at, o,
        0 if status is None else _optional(status, "status", 1, _I32, dev), _raw_stream(dev))
    if code:
        _check("nvfp4_add_rms_norm", code)
    return {"h": h, "y": y, "codes": codes, "scales": scales, "choice": choice, "dequant": dq,
            "row_amax": row_amax}


def add_rms_norm_workspace(device) -> torch.Tensor:
    """A workspace for nvfp4_add_rms_norm_bwd, for calls of any size: it serves one
    call at a time and needs no clearing."""
    return torch.empty((_lib().nvfp4_add_rms_norm_ws_bytes() + 3) // 4, dtype=torch.int32,
                       device=device)


def nvfp4_add_rms_norm_bwd(gy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor,
                           gh: torch.Tensor | None = None, eps: float = 1e-6,
                           workspace: torch.Tensor | None = None, gx: torch.Tensor | None = None,
                           status: torch.Tensor | None = None) -> dict:
    """Gradient of nvfp4_add_rms_norm from the gradient of its normed output (the
    encoding passed straight through), its h and, where the residual stream goes on, the
    gradient gh of h: {"gx" (bf16, of x and of the residual), "gw" (fp32 [cols])}.
    workspace: from add_rms_norm_workspace; a fresh one is taken when none is given."""
    dev = h.get_device()
    if dev >= 0 and dev != _device():
        with torch.cuda.device(dev):
            return nvfp4_add_rms_norm_bwd(gy, h, weight, gh, eps, workspace, gx, status)
    shape = h.shape
    if len(shape) != 2:
        raise ValueError("h must be [rows, cols]")
    R, Cc = shape
    if not (h.dtype in _BF16 and h.is_contiguous() and dev >= 0 and gy.dtype in _BF16
            and gy.shape == shape and gy.get_device() == dev and gy.is_contiguous()
            and weight.dtype in _BF16 and weight.shape == (Cc,) and weight.get_device() == dev
            and weight.is_contiguous()
            and (gh is None or (gh.dtype in _BF16 and gh.shape == shape and gh.get_device() == dev
                                and gh.is_contiguous()))):
        _matrix(gy, "gy", shape, dev)
        _matrix(h, "h", shape, dev)
        _matrix(weight, "weight", (Cc,), dev)
        _matrix(gh, "gh", shape, dev)
    if gx is None:
        gx = torch.empty(shape, dtype=h.dtype, device=h.device)
        gx_at = gx.data_ptr()
    else:
        gx_at = _matrix(gx, "gx", shape, dev)
    gw = torch.empty(Cc, dtype=torch.float32, device=h.device)
    if workspace is None:
        workspace = add_rms_norm_workspace(h.device)
    code = _lib().nvfp4_add_rms_norm_bwd(
        gy.data_ptr(), h.data_ptr(), weight.data_ptr(), 0 if gh is None else gh.data_ptr(), R, Cc,
        eps, gx_at, gw.data_ptr(), _optional(workspace, "workspace", 1, _I32, dev),
        4 * workspace.numel(),
        0 if status is None else _optional(status, "status", 1, _I32, dev), _raw_stream(dev))
    if code:
        _check("nvfp4_add_rms_norm_bwd", code)
    return {"gx": gx, "gw": gw}
