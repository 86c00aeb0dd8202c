"""Refusals of the quantised linear layer's operators, without a GPU: the library's argument
errors (returned before any CUDA call) and the binding's checks of tensors."""
import ctypes as C

import pytest
import torch

import nvfp4_block_scaled_02_gb300 as nv
from nvfp4_block_scaled_02_gb300 import linear

FAKE = 0x100000  # a 16-byte aligned, never dereferenced address
OK, NULL, SHAPE, ALIGN, ENUM = 0, 1, 2, 3, 4
BIG = 1 << 31


@pytest.fixture(scope="module")
def L():
    nv.build()
    return nv.lib()


def operand(**kw):
    d = dict(codes=FAKE, scales=FAKE, amax=FAKE, amax_count=1, scale_max=0.0)
    d.update(kw)
    return linear._Operand(*[d[n] for n, _ in linear._Operand._fields_])


def test_grouped_matmul_argument_errors(L):
    size = L.nvfp4_grouped_matmul_ws_bytes()

    def call(a=None, b=None, rows=8, groups=3, n=16, k=64, start=FAKE, out=FAKE, ws=FAKE, nb=size,
             status=None):
        a, b = a or operand(), b or operand(amax_count=groups)
        return L.nvfp4_grouped_matmul(C.byref(a), C.byref(b), rows, groups, n, k, start, out, ws,
                                      nb, status, None)
    assert L.nvfp4_grouped_matmul(None, C.byref(operand()), 1, 1, 1, 32, None, FAKE, FAKE, size,
                                  None, None) == NULL
    for bad in (dict(rows=-1), dict(groups=-1), dict(n=-1), dict(k=-32), dict(rows=BIG),
                dict(n=BIG), dict(k=BIG), dict(groups=1025), dict(k=48), dict(k=0),
                dict(groups=1024, n=1 << 22), dict(rows=1 << 30, n=1 << 20, groups=1),
                dict(a=operand(amax_count=7)), dict(b=operand(amax_count=2)), dict(nb=size - 1)):
        assert call(**bad) == SHAPE, bad
    for v in (-1.0, float("nan"), float("inf")):
        assert call(a=operand(scale_max=v)) == ENUM
        assert call(b=operand(scale_max=v, amax_count=3)) == ENUM
    for name in ("codes", "scales", "amax"):
        assert call(a=operand(**{name: None})) == NULL
        assert call(b=operand(**{name: None}, amax_count=3)) == NULL
        off = 2 if name == "amax" else 8
        assert call(a=operand(**{name: FAKE + off})) == ALIGN
        assert call(b=operand(**{name: FAKE + off}, amax_count=3)) == ALIGN
    for name in ("start", "out", "ws"):
        assert call(**{name: None}) == NULL
        assert call(**{name: FAKE + 2}) == ALIGN
    assert call(status=FAKE + 2) == ALIGN
    for empty in (dict(rows=0, a=operand(amax_count=0)), dict(n=0), dict(groups=0)):
        assert call(**{**dict(out=None, ws=None, start=None), **empty}) == OK


def test_mx_grouped_matmul_argument_errors(L):
    size = L.nvfp4_grouped_matmul_ws_bytes()

    def call(ac=FAKE, as_=FAKE, bc=FAKE, bs=FAKE, rows=8, groups=3, n=16, k=64, start=FAKE,
             out=FAKE, ws=FAKE, nb=size, status=None):
        return L.nvfp4_mx_grouped_matmul(ac, as_, bc, bs, rows, groups, n, k, start, out, ws, nb,
                                         status, None)
    for bad in (dict(rows=-1), dict(groups=1025), dict(k=40), dict(k=0), dict(rows=BIG),
                dict(nb=4)):
        assert call(**bad) == SHAPE, bad
    for name in ("ac", "as_", "bc", "bs", "start", "out", "ws"):
        assert call(**{name: None}) == NULL, name
        assert call(**{name: FAKE + 2}) == ALIGN, name
    assert call(rows=0, ac=None, out=None, ws=None) == OK
    assert call(status=FAKE + 1) == ALIGN


def test_mx_grouped_wgrad_argument_errors(L):
    size = L.nvfp4_grouped_matmul_ws_bytes()

    def call(gc=FAKE, gs=FAKE, xc=FAKE, xs=FAKE, rows=64, groups=3, n=16, k=24, start=FAKE,
             out=FAKE, f32=0, ws=FAKE, nb=size, status=None):
        return L.nvfp4_mx_grouped_wgrad(gc, gs, xc, xs, rows, groups, n, k, start, out, f32, ws,
                                        nb, status, None)
    for bad in (dict(rows=-32), dict(rows=48), dict(groups=-1), dict(n=BIG), dict(k=BIG),
                dict(nb=size - 1), dict(groups=1000, n=1 << 20, k=1 << 20)):
        assert call(**bad) == SHAPE, bad
    assert call(f32=2) == ENUM and call(f32=-1) == ENUM
    for name in ("gc", "gs", "xc", "xs", "start", "out", "ws"):
        assert call(**{name: None}) == NULL, name
        assert call(**{name: FAKE + 2}) == ALIGN, name
    assert call(status=FAKE + 1) == ALIGN
    for empty in (dict(groups=0), dict(n=0), dict(k=0)):
        assert call(**{**dict(out=None, ws=None), **empty}) == OK


def test_sums_too_long_for_the_waits(L):
    size, most = L.nvfp4_grouped_matmul_ws_bytes(), 1 << 25
    a = operand()
    for k, want in ((most + 32, SHAPE), (most, NULL)):  # (NULL: past the sizes, no workspace)
        assert L.nvfp4_grouped_matmul(C.byref(a), C.byref(a), 1, 1, 16, k, None, FAKE, None, size,
                                      None, None) == want
        assert L.nvfp4_mx_grouped_matmul(FAKE, FAKE, FAKE, FAKE, 1, 1, 16, k, None, FAKE, None,
                                         size, None, None) == want
        assert L.nvfp4_mx_grouped_wgrad(FAKE, FAKE, FAKE, FAKE, k, 1, 16, 16, None, FAKE, 0, None,
                                        size, None, None) == want


def cfg(**kw):
    return nv.Config(**kw).c()


def test_add_rms_norm_argument_errors(L):
    def call(c=None, target=nv.TARGET_NVFP4, x=FAKE, res=FAKE, w=FAKE, rows=4, cols=64, eps=1e-6,
             h=FAKE, y=None, gamax=None, row=FAKE, out=None, status=None):
        c, out = c or cfg(), out or nv._Out(FAKE, FAKE, None, None)
        return L.nvfp4_add_rms_norm(C.addressof(c), target, x, res, w, rows, cols, eps, h, y, gamax,
                                    row, C.addressof(out), status, None)
    assert L.nvfp4_add_rms_norm(None, 1, FAKE, None, FAKE, 4, 64, 1e-6, None, None, None, FAKE,
                                FAKE, None, None) == NULL
    for bad in (dict(target=2), dict(target=-1), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(c=cfg(blocks=nv.BLOCKS_COL)),
                dict(c=cfg(rounding=nv.ROUND_SR)), dict(c=cfg(scale_fmt=nv.SCALE_UE5M3)),
                dict(c=cfg(scale_max=-1.0)), dict(c=cfg(four_over_six=2)),
                dict(c=cfg(four_over_six=1, four_over_six_rule=nv.FOS_MAE)),
                dict(target=nv.TARGET_MXFP8, out=nv._Out(FAKE, FAKE, None, FAKE))):
        assert call(**bad) == ENUM, bad
    for bad in (dict(rows=-1), dict(cols=-16), dict(rows=BIG), dict(cols=16400), dict(cols=24),
                dict(cols=48, target=nv.TARGET_MXFP8)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(x=None), dict(w=None), dict(h=None), dict(row=None),
                dict(out=nv._Out(None, FAKE, None, None)),
                dict(out=nv._Out(FAKE, None, None, None))):
        assert call(**bad) == NULL, bad
    for bad in (dict(x=FAKE + 8), dict(res=FAKE + 2), dict(w=FAKE + 8), dict(h=FAKE + 4),
                dict(y=FAKE + 8), dict(gamax=FAKE + 2), dict(row=FAKE + 2), dict(status=FAKE + 1),
                dict(out=nv._Out(FAKE + 8, FAKE, None, None)),
                dict(out=nv._Out(FAKE, FAKE + 4, None, None)),
                dict(out=nv._Out(FAKE, FAKE, FAKE + 4, None)),
                dict(out=nv._Out(FAKE, FAKE, None, FAKE + 8))):
        assert call(**bad) == ALIGN, bad
    for empty in (dict(rows=0), dict(cols=0)):
        assert call(x=None, w=None, res=None, row=None, **empty) == OK


def test_add_rms_norm_bwd_argument_errors(L):
    size = L.nvfp4_add_rms_norm_ws_bytes()

    def call(gy=FAKE, h=FAKE, w=FAKE, gh=FAKE, rows=4, cols=64, eps=1e-6, gx=FAKE, gw=FAKE,
             ws=FAKE, nb=size, status=None):
        return L.nvfp4_add_rms_norm_bwd(gy, h, w, gh, rows, cols, eps, gx, gw, ws, nb, status, None)
    for bad in (dict(eps=-1.0), dict(eps=float("nan"))):
        assert call(**bad) == ENUM
    for bad in (dict(rows=-1), dict(cols=24), dict(cols=16400), dict(rows=BIG), dict(nb=size - 1)):
        assert call(**bad) == SHAPE, bad
    for name in ("gy", "h", "w", "gx", "gw", "ws"):
        assert call(**{name: None}) == NULL, name
    for name in ("gy", "h", "w", "gh", "gx", "gw", "ws"):
        assert call(**{name: FAKE + 8}) == ALIGN, name
    assert call(status=FAKE + 2) == ALIGN and call(cols=0, gw=None) == OK


def test_the_binding_refuses_tensors_of_the_host():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16)
    enc = {"codes": torch.zeros(4, 32, dtype=torch.uint8),
           "scales": torch.zeros(4, 4, dtype=torch.uint8)}
    one = torch.ones(1)
    ws = torch.zeros(8, dtype=torch.int32)
    for f in (lambda: nv.nvfp4_add_rms_norm(x, w), lambda: nv.nvfp4_add_rms_norm_bwd(x, x, w),
              lambda: nv.nvfp4_grouped_matmul(enc, one, enc, one, workspace=ws),
              lambda: nv.nvfp4_mx_grouped_matmul(enc, enc, workspace=ws),
              lambda: nv.nvfp4_mx_grouped_wgrad(enc, enc, workspace=ws)):
        with pytest.raises(ValueError):
            f()


def test_the_binding_refuses_shapes():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        nv.nvfp4_add_rms_norm(x[None], w)
    with pytest.raises(ValueError):
        nv.nvfp4_add_rms_norm_bwd(x[None], x[None], w)
    flat = {"codes": torch.zeros(64, dtype=torch.uint8),
            "scales": torch.zeros(4, dtype=torch.uint8)}
    enc = {"codes": torch.zeros(4, 32, dtype=torch.uint8),
           "scales": torch.zeros(4, 4, dtype=torch.uint8)}
    with pytest.raises(ValueError):
        nv.nvfp4_mx_grouped_matmul(flat, enc)
    with pytest.raises(ValueError):
        nv.nvfp4_mx_grouped_matmul(enc, flat)
    with pytest.raises(TypeError):
        nv.nvfp4_mx_grouped_wgrad(enc, enc, out_dtype=torch.float16)
