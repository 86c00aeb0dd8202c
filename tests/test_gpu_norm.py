"""The residual norm with its encodings and its gradient against plain forms in 64 bits, byte for
byte where the codes do not depend on how a sum rounds."""
import subprocess
import sys

import pytest
import torch

import nvfp4_block_scaled_02_gb300 as nv
from conftest import ROOT

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
EPS = 1e-6


def randn(seed, *shape, size=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(*shape, generator=g, device="cuda")
    return (x * torch.exp(0.5 * torch.randn(shape[-1], generator=g, device="cuda")) * size).to(BF16)


def weight(seed, cols):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (1 + 0.2 * torch.randn(cols, generator=g, device="cuda")).to(BF16)


def powers(seed, cols):
    """Weights that are powers of two: h w is then a bf16 value."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    k = torch.randint(-3, 4, (cols,), generator=g, device="cuda").float()
    sign = torch.randint(0, 2, (cols,), generator=g, device="cuda") * 2 - 1
    return (torch.exp2(k) * sign).to(BF16)


def divided(x, by):
    """x / by in fp32 (torch divides by a number by multiplying with its reciprocal)."""
    return x / torch.full_like(x, by)


def exact(h, w, eps=EPS):
    v = h.double()
    r = 1 / (v.square().mean(1, keepdim=True) + eps).sqrt()
    return v * r * w.double(), r


# one block and less than a warp, odd numbers of blocks, one, two blocks a thread, the widest
FP4_SIZES = [(1, 16), (3, 48), (5, 32), (7, 1040), (1021, 1056), (4, 4096), (333, 7168), (2, 8208),
             (3, 16384), (2000, 512)]
MX_SIZES = [(1, 32), (3, 96), (1021, 1056), (4, 4096), (333, 7168), (3, 8224), (2, 16384),
            (2000, 512)]


@pytest.mark.parametrize("rows,cols", FP4_SIZES)
@pytest.mark.parametrize("fos", [0, 1])
@pytest.mark.parametrize("residual", [True, False])
def test_per_row_encoding_is_that_of_the_weighted_sum(rows, cols, fos, residual):
    x, w = randn(1, rows, cols), powers(2, cols)
    res = randn(3, rows, cols, size=2.0) if residual else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cfg = nv.Config(four_over_six=fos)
    y = torch.empty_like(x)
    r = nv.nvfp4_add_rms_norm(x, w, res, eps=EPS, cfg=cfg, dequant=True, y=y, status=status)
    h = (x.float() + res.float()).to(BF16) if residual else x
    assert torch.equal(r["h"], h) and (residual or r["h"] is x)
    # h w is exact in bf16 here: the encoder's own bytes
    want = nv.nvfp4_quantize_per_token((h.float() * w.float()).to(BF16), cfg, dequant=False)
    assert torch.equal(r["codes"], want["codes"].view(rows, -1))
    assert torch.equal(r["scales"], want["scales"].view(rows, -1))
    if fos:
        # bits of blocks that a last word does not have are 0 in both
        assert torch.equal(r["choice"], want["choice"].view(rows, -1))
    yv, inv = exact(h, w)
    amax = want["row_amax"].double() * inv[:, 0]
    # r: the sum's roundings (at most cols / 16 in a row, halved by the square root) and rsqrt's
    tol = (cols / 32 + 8) * 2.0 ** -24
    assert ((r["row_amax"].double() - amax).abs() <= amax * tol).all()
    assert ((y.double() - yv).abs() <= yv.abs() * (2.0 ** -8 + 2 * tol)).all()
    # the values that the codes stand for, from the outer scale that was written
    M = 256.0 if fos else 448.0
    amax32 = r["row_amax"]
    g = torch.where(amax32 > 0, divided(amax32, 6 * M), torch.ones_like(amax32))
    d = r["scales"].view(torch.float8_e4m3fn).float() * g[:, None]
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6],
                       device="cuda")
    q = torch.stack([lut[(r["codes"] & 15).int()], lut[(r["codes"] >> 4).int()]], -1).flatten(-2)
    assert torch.equal(r["dequant"], (q * d.repeat_interleave(16, 1)).to(BF16))
    assert status.item() == 0


@pytest.mark.parametrize("rows,cols", FP4_SIZES)
def test_per_row_encoding_with_any_weight(rows, cols):
    """Codes and scales by the format's steps of 32 bits on the exact products h w."""
    x, w, res = randn(1, rows, cols), weight(2, cols), randn(3, rows, cols)
    r = nv.nvfp4_add_rms_norm(x, w, res, eps=EPS)
    v = (r["h"].float() * w.float()).unflatten(1, (-1, 16))
    top = v.abs().amax(2, keepdim=True)
    g = divided(top.amax(1, keepdim=True), 2688)
    s8 = (top * (1 / (6 * g))).clamp(max=448).to(torch.float8_e4m3fn)
    d = s8.float() * g
    y = v * torch.where(d > 0, 1 / d, torch.zeros_like(d))
    a = y.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
            + (a >= 3.5) + (a > 5)) + 8 * torch.signbit(y).to(torch.uint8)
    code = code.flatten(1)
    assert torch.equal(r["scales"], s8.view(torch.uint8).flatten(1))
    assert torch.equal(r["codes"], code[:, 0::2] + 16 * code[:, 1::2])


@pytest.mark.parametrize("rows,cols", FP4_SIZES)
@pytest.mark.parametrize("fos", [0, 1])
def test_encoding_under_a_tensors_scale(rows, cols, fos):
    x, w, res = randn(1, rows, cols), weight(2, cols), randn(3, rows, cols)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    h = (x.float() + res.float()).to(BF16)
    yv, _ = exact(h, w)
    amax = (yv.abs().amax() * 1.01).float().view(1)
    r = nv.nvfp4_add_rms_norm(x, w, res, eps=EPS, cfg=nv.Config(four_over_six=fos),
                              global_amax=amax, dequant=True, status=status)
    assert r["row_amax"] is None and torch.equal(r["h"], h)
    M = 256.0 if fos else 448.0
    g = divided(amax, 6 * M).double()
    sc = r["scales"].view(torch.float8_e4m3fn).double()
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6],
                       dtype=torch.float64, device="cuda")
    q = torch.stack([lut[(r["codes"] & 15).long()], lut[(r["codes"] >> 4).long()]], -1).flatten(-2)
    d = (sc * g).repeat_interleave(16, 1)
    # a value is within half a step of its code (the steps between magnitudes are 1/2, 1 and 2
    # scales), up to the roundings of r and of the products; past 6 scales only by what the
    # scale itself was rounded down (2^-4 of it)
    near = 1 + 2.0 ** -14
    half = torch.where(q.abs() < 2, 0.25, torch.where(q.abs() < 4, 0.5, 1.0)) * d * near
    off = (q * d - yv).abs()
    top = yv.abs().unflatten(1, (-1, 16)).amax(2)
    # scales below E4M3's normal range (2^-6) are spaced by 2^-9
    space = torch.maximum(sc * 2.0 ** -4, torch.full_like(sc, 2.0 ** -10)) * g * 6 * near
    if not fos:
        assert ((6 * sc * g - top).abs() <= space).all()
        assert (off <= half + space.repeat_interleave(16, 1)).all()
    else:
        # the scale is that of max -> 6 or of max -> 4
        assert (((6 * sc * g - top).abs() <= space) | ((4 * sc * g - top).abs() <= space)).all()
        assert (off <= half + space.repeat_interleave(16, 1)).all()
    assert torch.equal(r["dequant"], (q.float() * (sc.float() * divided(amax, 6 * M))
                                      .repeat_interleave(16, 1)).to(BF16))
    assert status.item() == 0


@pytest.mark.parametrize("rows,cols", MX_SIZES)
@pytest.mark.parametrize("residual", [True, False])
def test_mxfp8_encoding(rows, cols, residual):
    x, w = randn(1, rows, cols), weight(2, cols)
    res = randn(3, rows, cols, size=2.0) if residual else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = torch.empty_like(x)
    r = nv.nvfp4_add_rms_norm(x, w, res, eps=EPS, target=nv.TARGET_MXFP8, y=y, status=status)
    h = (x.float() + res.float()).to(BF16) if residual else x
    assert torch.equal(r["h"], h)
    yv, _ = exact(h, w)
    tol = (cols / 32 + 8) * 2.0 ** -23
    assert ((y.double() - yv).abs() <= yv.abs() * (2.0 ** -8 + tol)).all()
    e = r["scales"].double() - 127
    top = yv.unflatten(1, (-1, 32)).abs().amax(2)
    # the smallest power of two that holds the block, up to the roundings of y
    assert (top <= 448 * torch.exp2(e) * (1 + tol)).all()
    assert (top > 448 * torch.exp2(e - 1) * (1 - tol)).all()
    v = yv / torch.exp2(e).repeat_interleave(32, 1)
    c = r["codes"].view(torch.float8_e4m3fn).double()
    half = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 4)
    assert ((c - v).abs() <= half * (1 + tol) + v.abs() * tol).all()
    assert status.item() == 0


def bwd_reference(gy, h, w, gh, eps=EPS):
    gy, h, w = gy.double(), h.double(), w.double()
    r = 1 / (h.square().mean(1, keepdim=True) + eps).sqrt()
    u = gy * w
    m = (u * h).mean(1, keepdim=True)
    gx = r * (u - h * r * r * m)
    size = r * (u.abs() + h.abs() * r * r * (u * h).abs().mean(1, keepdim=True))
    if gh is not None:
        gx, size = gx + gh.double(), size + gh.double().abs()
    terms = gy * h * r
    return gx, size, terms.sum(0), terms.abs().sum(0)


@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 48), (1021, 1056), (4, 4096), (2000, 512),
                                       (333, 7168), (5, 8208), (700, 16384), (3000, 4096)])
@pytest.mark.parametrize("stream", [True, False])
def test_gradient(rows, cols, stream):
    gy, h, w = randn(1, rows, cols, size=1e-2), randn(2, rows, cols), weight(3, cols)
    gh = randn(4, rows, cols, size=1e-2) if stream else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = nv.add_rms_norm_workspace("cuda").fill_(-1)  # of any content
    r = nv.nvfp4_add_rms_norm_bwd(gy, h, w, gh, eps=EPS, workspace=ws, status=status)
    gx, size, gw, gw_size = bwd_reference(gy, h, w, gh)
    # fp32 steps: the two sums (at most cols / 8 roundings in a row), r, the products
    tol = (cols / 8 + 16) * 2.0 ** -24
    assert ((r["gx"].double() - gx).abs() <= gx.abs() * 2.0 ** -8 * 1.001 + size * 2 * tol).all()
    assert ((r["gw"].double() - gw).abs() <= gw_size * ((rows + 16) * 2.0 ** -24 + tol)).all()
    again = nv.nvfp4_add_rms_norm_bwd(gy, h, w, gh, eps=EPS, workspace=ws)
    assert torch.equal(again["gw"], r["gw"]) and torch.equal(again["gx"], r["gx"])
    assert status.item() == 0


def test_gradient_against_differences():
    """gx along random directions and gw against central differences of the forward in 64 bits."""
    rows, cols, step = 3, 64, 1e-4
    gy, h, w, gh = (randn(i, rows, cols) for i in range(3, 7))
    w = w[0].contiguous()
    r = nv.nvfp4_add_rms_norm_bwd(gy, h, w, gh, eps=EPS)

    def loss(hv, wv):
        y = hv / (hv.square().mean(1, keepdim=True) + EPS).sqrt() * wv
        return (y * gy.double()).sum() + (hv * gh.double()).sum()

    for i in range(8):
        d = randn(20 + i, rows, cols).double()
        got = (r["gx"].double() * d).sum()
        want = (loss(h.double() + step * d, w.double()) - loss(h.double() - step * d, w.double())
                ) / (2 * step)
        # bf16 halves a step of each gx; the third derivative's part is step^2
        bound = (r["gx"].double().abs() * d.abs()).sum() * 2.0 ** -8 + 1e-4
        assert (got - want).abs() <= bound
        dw = randn(40 + i, 1, cols)[0].double()
        want = (loss(h.double(), w.double() + step * dw) - loss(h.double(), w.double() - step * dw)
                ) / (2 * step)
        got = (r["gw"].double() * dw).sum()
        assert (got - want).abs() <= 1e-5 * (r["gw"].double().abs() * dw.abs()).sum() + 1e-6


def test_in_place():
    x, res, w = randn(1, 300, 1056), randn(2, 300, 1056), weight(3, 1056)
    want = nv.nvfp4_add_rms_norm(x, w, res, eps=EPS)
    stream = res.clone()
    got = nv.nvfp4_add_rms_norm(x, w, stream, eps=EPS, h=stream)
    assert torch.equal(stream, want["h"]) and torch.equal(got["codes"], want["codes"])
    xs = x.clone()
    nv.nvfp4_add_rms_norm(xs, w, res, eps=EPS, h=xs)
    assert torch.equal(xs, want["h"])
    gy, h = randn(4, 300, 1056), want["h"]
    wantb = nv.nvfp4_add_rms_norm_bwd(gy, h, w, x, eps=EPS)["gx"]
    for i in range(3):
        bufs = [gy.clone(), h.clone(), x.clone()]
        nv.nvfp4_add_rms_norm_bwd(bufs[0], bufs[1], w, bufs[2], eps=EPS, gx=bufs[i])
        assert torch.equal(bufs[i], wantb)


def test_rows_of_zeros_and_small_rows():
    x, w = torch.zeros(4, 64, dtype=BF16, device="cuda"), weight(1, 64)
    x[2] = randn(2, 1, 64, size=1e-20)[0]
    x[3] = randn(2, 1, 64, size=1e-30)[0]
    for eps in (0.0, EPS):
        r = nv.nvfp4_add_rms_norm(x, w, eps=eps, dequant=True, y=torch.empty_like(x))
        assert r["dequant"].isfinite().all() and not r["dequant"][:2].any()
        assert r["y"].isfinite().all() and not r["y"][:2].any()
        assert not r["row_amax"][:2].any()
        m = nv.nvfp4_add_rms_norm(x, w, eps=eps, target=nv.TARGET_MXFP8)
        assert not m["codes"][:2].any()
        b = nv.nvfp4_add_rms_norm_bwd(randn(5, 4, 64), x, w, eps=eps)
        assert b["gx"][:3].isfinite().all() and b["gw"].isfinite().all()
    # without eps a row's size does not matter down to where its squares leave fp32
    a = nv.nvfp4_add_rms_norm(x[2:3], w, eps=0.0, dequant=True)
    big = nv.nvfp4_add_rms_norm((x[2:3].double() * 2.0 ** 64).to(BF16), w, eps=0.0, dequant=True)
    assert torch.equal(a["codes"], big["codes"]) and torch.equal(a["scales"], big["scales"])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 1e30])
def test_values_that_are_no_numbers_are_flagged(bad):
    w = weight(1, 96)
    for at in (0, 95):
        x = randn(2, 5, 96)
        x[3, at] = bad
        for target in (nv.TARGET_NVFP4, nv.TARGET_MXFP8):
            for amax in (None, torch.ones(1, device="cuda")):
                status = torch.zeros(1, dtype=torch.int32, device="cuda")
                nv.nvfp4_add_rms_norm(x, w, target=target, global_amax=amax, status=status)
                assert status.item() & nv.DEV_NONFINITE_INPUT
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        nv.nvfp4_add_rms_norm_bwd(randn(3, 5, 96), x, w, status=status)
        assert status.item() & nv.DEV_NONFINITE_INPUT
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    nv.nvfp4_add_rms_norm(randn(2, 5, 96), w, global_amax=torch.full((1,), -1.0, device="cuda"),
                          status=status)
    assert status.item() == nv.DEV_BAD_AMAX


def test_empty():
    w = weight(1, 64)
    x = torch.empty(0, 64, dtype=BF16, device="cuda")
    r = nv.nvfp4_add_rms_norm(x, w)
    assert r["codes"].shape == (0, 32) and r["row_amax"].shape == (0,)
    b = nv.nvfp4_add_rms_norm_bwd(x, x, w)
    assert b["gx"].shape == (0, 64) and not b["gw"].any()


def test_what_would_not_be_written_is_refused():
    x, w, one = randn(1, 4, 64), weight(2, 64), torch.ones(1, device="cuda")
    rows = torch.zeros(4, device="cuda")
    for kw in (dict(target=nv.TARGET_MXFP8, dequant=True),
               dict(target=nv.TARGET_MXFP8, row_amax=rows), dict(global_amax=one, row_amax=rows)):
        with pytest.raises(ValueError):
            nv.nvfp4_add_rms_norm(x, w, **kw)
    assert nv.nvfp4_add_rms_norm(x, w, row_amax=rows)["row_amax"] is rows and rows.all()


def test_two_streams_at_once():
    """Forward and gradient on two streams, each with its workspace, give the bits of a call
    alone."""
    w = weight(1, 1056)
    cases = [(randn(i, r, 1056), randn(10 + i, r, 1056), randn(20 + i, r, 1056))
             for i, r in enumerate((5, 1021, 3000))]
    spaces = [nv.add_rms_norm_workspace("cuda") for _ in range(2)]

    def step(case, ws):
        x, res, gy = case
        f = nv.nvfp4_add_rms_norm(x, w, res)
        b = nv.nvfp4_add_rms_norm_bwd(gy, f["h"], w, res, workspace=ws)
        return f["h"], f["codes"], f["scales"], f["row_amax"], b["gx"], b["gw"]

    alone = [step(c, spaces[0]) for c in cases]
    side = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for s in (0, 1):
            with torch.cuda.stream(side[s]):
                for c in cases[::1 - 2 * s]:
                    got[s].append(step(c, spaces[s]))
    torch.cuda.synchronize()
    for s in (0, 1):
        for i, r in enumerate(got[s]):
            assert all(torch.equal(a, b) for a, b in zip(r, alone[::1 - 2 * s][i % 3]))


BITS = """
import hashlib, sys, torch
import nvfp4_block_scaled_02_gb300 as nv
for cols in map(int, sys.argv[1:]):
    g = torch.Generator(device="cuda")
    g.manual_seed(cols)
    gy, h = (torch.randn(8192, cols, generator=g, device="cuda").bfloat16() for _ in range(2))
    gw = nv.nvfp4_add_rms_norm_bwd(gy, h, h[0].clone())["gw"]
    print(cols, hashlib.sha256(gw.cpu().numpy().tobytes()).hexdigest())
"""


def test_weight_gradients_bits_do_not_depend_on_earlier_calls():
    """Widths of one number of warps in either order, each order in a process of its own."""
    lines = []
    for order in (["64", "128", "192", "256"], ["256", "192", "128", "64"]):
        r = subprocess.run([sys.executable, "-c", BITS, *order], cwd=ROOT, capture_output=True,
                           text=True, timeout=300)
        assert r.returncode == 0, r.stderr
        lines.append(sorted(r.stdout.splitlines()))
    assert len(lines[0]) == 4 and lines[0] == lines[1]


def is_nan(scales):
    """Of scale bytes: NaN of E4M3."""
    return scales == 0x7F


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 1e30])
@pytest.mark.parametrize("cols", [96, 16384])
def test_rows_that_are_no_numbers_show_it(bad, cols):
    """Such a row's results are NaN throughout (1e30: its squares are past fp32), the other rows'
    as without it; so are the product's rows and the gradients."""
    rows, w = 5, weight(1, cols)
    clean = randn(2, rows, cols)
    rest = [0, 1, 2, 4]
    weights = randn(7, 1, 40, cols, size=cols ** -0.5)
    b_amax = nv.nvfp4_amax(weights)
    b = nv.nvfp4_quantize(weights, b_amax, dequant=False)["row"]
    one = torch.full((1,), 9.0, device="cuda")
    for at in (0, cols - 1):
        x = clean.clone()
        x[3, at] = bad
        for fos in (0, 1):
            cfg = nv.Config(four_over_six=fos)
            for amax in (None, one):
                status = torch.zeros(1, dtype=torch.int32, device="cuda")
                kw = dict(cfg=cfg, global_amax=amax, dequant=True)
                want = nv.nvfp4_add_rms_norm(clean, w, y=torch.empty_like(x), **kw)
                r = nv.nvfp4_add_rms_norm(x, w, y=torch.empty_like(x), status=status, **kw)
                assert status.item() == nv.DEV_NONFINITE_INPUT
                assert r["y"][3].isnan().all() and r["dequant"][3].isnan().all()
                assert is_nan(r["scales"][3]).all()
                for name in ("y", "codes", "scales", "dequant"):
                    assert torch.equal(r[name][rest], want[name][rest])
                if amax is None:
                    assert r["row_amax"][3].isnan()
                    assert torch.equal(r["row_amax"][rest], want["row_amax"][rest])
                a = one if amax is not None else r["row_amax"]
                out = nv.nvfp4_grouped_matmul(r, a, b, b_amax, a_cfg=cfg)
                assert out[3].isnan().all() and out[rest].isfinite().all()
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        want = nv.nvfp4_add_rms_norm(clean, w, target=nv.TARGET_MXFP8)
        r = nv.nvfp4_add_rms_norm(x, w, target=nv.TARGET_MXFP8, status=status)
        assert status.item() == nv.DEV_NONFINITE_INPUT
        assert r["codes"][3].view(torch.float8_e4m3fn).float().isnan().all()
        assert torch.equal(r["codes"][rest], want["codes"][rest])
        assert torch.equal(r["scales"][rest], want["scales"][rest])
        gy, gh = randn(3, rows, cols), randn(4, rows, cols)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        want = nv.nvfp4_add_rms_norm_bwd(gy, clean, w, gh)
        r = nv.nvfp4_add_rms_norm_bwd(gy, x, w, gh, status=status)
        assert status.item() == nv.DEV_NONFINITE_INPUT
        assert r["gx"][3].isnan().all() and torch.equal(r["gx"][rest], want["gx"][rest])
        assert r["gw"].isnan().all()


def test_weights_that_are_no_numbers_show_it():
    """A NaN of the weight reaches its block of every row under a tensor's scale and its value in
    MXFP8, every row with a scale of its own; all of it is flagged."""
    x, w = randn(1, 5, 96), weight(2, 96)
    bad = w.clone()
    bad[37] = float("nan")
    one = torch.full((1,), 9.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = nv.nvfp4_add_rms_norm(x, w, global_amax=one, dequant=True)
    r = nv.nvfp4_add_rms_norm(x, bad, global_amax=one, dequant=True, status=status)
    assert status.item() == nv.DEV_NONFINITE_INPUT
    assert torch.equal(is_nan(r["scales"]), torch.arange(6, device="cuda").eq(2).expand(5, 6))
    nan = torch.arange(96, device="cuda").div(16, rounding_mode="floor").eq(2).expand(5, 96)
    assert torch.equal(r["dequant"].isnan(), nan)
    assert torch.equal(r["dequant"][~nan], want["dequant"][~nan])
    status.zero_()
    r = nv.nvfp4_add_rms_norm(x, bad, status=status)
    assert status.item() == nv.DEV_NONFINITE_INPUT
    assert is_nan(r["scales"]).all() and r["row_amax"].isnan().all()
    status.zero_()
    want = nv.nvfp4_add_rms_norm(x, w, target=nv.TARGET_MXFP8)
    r = nv.nvfp4_add_rms_norm(x, bad, target=nv.TARGET_MXFP8, status=status)
    assert status.item() == nv.DEV_NONFINITE_INPUT
    v = r["codes"].view(torch.float8_e4m3fn).float()
    nan = torch.arange(96, device="cuda").eq(37).expand(5, 96)
    assert torch.equal(v.isnan(), nan)
    keep = torch.tensor([0, 2], device="cuda")  # blocks of 32 without it
    assert torch.equal(r["scales"][:, keep], want["scales"][:, keep])
    assert torch.equal(v.view(5, 3, 32)[:, keep],
                       want["codes"].view(torch.float8_e4m3fn).float().view(5, 3, 32)[:, keep])


def test_an_earlier_calls_encoding_holds_what_this_call_wrote():
    """Into an encoding of an earlier call: nothing of that call is handed on, and what has no
    place is refused."""
    x, w = randn(1, 4, 1056), weight(2, 1056)
    fos = nv.Config(four_over_six=1)
    first = nv.nvfp4_add_rms_norm(randn(3, 4, 1056), w, cfg=fos, dequant=True)
    choice = first["choice"].clone()
    want = nv.nvfp4_add_rms_norm(x, w, dequant=True)
    r = nv.nvfp4_add_rms_norm(x, w, out=first)
    assert r["choice"] is None and torch.equal(first["choice"], choice)
    for name in ("codes", "scales", "dequant"):
        assert r[name] is first[name] and torch.equal(r[name], want[name])
    again = nv.nvfp4_add_rms_norm(x, w, cfg=fos, out=first)
    assert again["choice"] is first["choice"]
    assert torch.equal(again["choice"], nv.nvfp4_add_rms_norm(x, w, cfg=fos)["choice"])
    plain = nv.nvfp4_add_rms_norm(x, w)
    with pytest.raises(ValueError):
        nv.nvfp4_add_rms_norm(x, w, out=plain, dequant=True)
    mx = nv.nvfp4_add_rms_norm(x, w, target=nv.TARGET_MXFP8)
    assert nv.nvfp4_add_rms_norm(x, w, target=nv.TARGET_MXFP8, out=mx)["codes"] is mx["codes"]
    with pytest.raises(ValueError):
        nv.nvfp4_add_rms_norm(x, w, target=nv.TARGET_MXFP8, out={**mx, "dequant": first["dequant"]})


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 1e30])
@pytest.mark.parametrize("fos", [0, 1])
def test_rows_that_are_no_numbers_are_zeros_to_the_transpose(bad, fos):
    """Re-quantised for a weights' gradient such a row is a row of zeros, whatever its blocks'
    scales, and the product has NaN in its row alone."""
    rows, cols, w = 64, 512, weight(1, 512)
    cfg, amax = nv.Config(four_over_six=fos), torch.full((1,), 9.0, device="cuda")
    zero = randn(2, rows, cols)
    zero[37] = 0
    x = zero.clone()
    x[37, 100] = bad
    out = []
    for v in (zero, x):
        r = nv.nvfp4_add_rms_norm(v, w, cfg=cfg, global_amax=amax)
        out.append((r, nv.nvfp4_requant_transpose(r["codes"], r["scales"], amax, cfg, nv.Config())))
    (a, at), (b, bt) = out
    assert is_nan(b["scales"][37]).all() and not b["codes"][37].any()
    assert torch.equal(at["codes"], bt["codes"]) and torch.equal(at["scales"], bt["scales"])
    p = nv.nvfp4_grouped_matmul(b, amax, a, amax, a_cfg=cfg, b_cfg=cfg)
    q = nv.nvfp4_grouped_matmul(a, amax, a, amax, a_cfg=cfg, b_cfg=cfg)
    assert p[37].isnan().all()
    p[37] = q[37]
    assert torch.equal(p, q)
