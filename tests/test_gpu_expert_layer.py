"""The operators of the quantised linear layer together, as examples/expert_layer.py runs them:
every stage against its formula in 64 bits of the operands that it was given."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_02_gb300 as nv
from conftest import ROOT
from linear_ref import fp4_values, mx_values, product_bound, ragged
from test_gpu_matmul import randn, starts
from test_gpu_norm import bwd_reference, exact

sys.path.insert(0, os.path.join(ROOT, "examples"))
from expert_layer import ExpertLayer  # noqa: E402

pytestmark = pytest.mark.gpu


def check_layer(layer, x, res, gy, gh, start, y, n, g):
    at = start.tolist()
    rows, cols = x.shape
    h = (x.float() + res.float()).to(torch.bfloat16)
    assert torch.equal(n["h"], h)
    xv = fp4_values(n["codes"], n["scales"], layer.amax.expand(rows))
    # the encoding stands for the norm's output: within half a step of a code and, past 6
    # scales, within what the scale was rounded by
    yv, _ = exact(h, layer.norm_weight)
    sc = n["scales"].view(torch.float8_e4m3fn).double().repeat_interleave(16, 1) * (
        layer.amax.double() / 2688)
    assert ((xv - yv).abs() <= sc * (1 + 6 * 2.0 ** -4) * 1.001 + 1e-3 * layer.amax.double()).all()
    wv = fp4_values(layer.w["codes"], layer.w["scales"], layer.w_amax[:, None])
    wt = mx_values(layer.wt["codes"], layer.wt["scales"])
    gq, xt, gn = g["encoded"]
    gr = mx_values(gq["row"]["codes"], gq["row"]["scales"])[0]
    gc = mx_values(gq["col"]["codes"], gq["col"]["scales"])[0]
    xtv = mx_values(xt["codes"], xt["scales"])[0]
    for e in range(len(at) - 1):
        i, j = at[e], at[e + 1]
        if j > i:
            ref = xv[i:j] @ wv[e].T
            assert ((y[i:j].double() - ref).abs() <= product_bound(xv[i:j], wv[e], ref)).all()
            ref = gr[i:j] @ wt[e].T
            assert ((gn[i:j].double() - ref).abs() <= product_bound(gr[i:j], wt[e], ref)).all()
        ref = gc[:, i:j] @ xtv[:, i:j].T
        assert ((g["weights"][e].double() - ref).abs()
                <= product_bound(gc[:, i:j], xtv[:, i:j], ref, True)).all()
    gx, size, gw, gw_size = bwd_reference(gn, h, layer.norm_weight, gh)
    tol = (cols / 8 + 16) * 2.0 ** -24
    assert ((g["x"].double() - gx).abs() <= gx.abs() * 2.0 ** -8 * 1.001 + size * 2 * tol).all()
    assert ((g["norm_weight"].double() - gw).abs() <= gw_size * ((rows + 16) * 2.0 ** -24 + tol)).all()
    assert layer.status.item() == 0


def make(E, rows, out, cols, seed=0):
    layer = ExpertLayer(randn(seed, E, out, cols, size=cols ** -0.5), randn(seed + 1, 1, cols)[0])
    layer.amax.fill_(40.0)
    x, res = randn(seed + 2, rows, cols), randn(seed + 3, rows, cols)
    gy, gh = randn(seed + 4, rows, out, size=1e-2), randn(seed + 5, rows, cols, size=1e-2)
    return layer, x, res, gy, gh


@pytest.mark.parametrize("E,rows,out,cols", [(4, 320, 160, 128), (1, 64, 96, 512),
                                             (6, 1024, 512, 1056), (3, 2048, 1024, 768)])
def test_layer(E, rows, out, cols):
    layer, x, res, gy, gh = make(E, rows, out, cols)
    start = starts(ragged(np.random.default_rng(E), E, rows, unit=32))
    y, n = layer.forward(x, res, start)
    check_layer(layer, x, res, gy, gh, start, y, n, layer.backward(gy, n, start, gh))


def test_layer_in_a_graph():
    """Captured once, replayed with other inputs and other groups."""
    E, rows, out, cols = 5, 512, 256, 544
    layer, x, res, gy, gh = make(E, rows, out, cols)
    start = starts(ragged(np.random.default_rng(0), E, rows, unit=32))

    def step():
        y, n = layer.forward(x, res, start)
        return y, n, layer.backward(gy, n, start, gh)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, n, g = step()
    for i in range(1, 4):
        x.copy_(randn(10 * i, rows, cols))
        res.copy_(randn(10 * i + 1, rows, cols))
        gy.copy_(randn(10 * i + 2, rows, out, size=1e-2))
        start.copy_(starts(ragged(np.random.default_rng(i), E, rows, unit=32)))
        graph.replay()
        check_layer(layer, x, res, gy, gh, start, y, n, g)


def test_norm_and_product_of_a_decode_step():
    """Rows with an outer scale each go from the norm to the product; rows that are not there yet
    (a batch's padding) are left alone."""
    T, K, N = 7, 4096, 640
    x, res, w = randn(1, T, K), randn(2, T, K), randn(3, 1, K)[0]
    weights = randn(4, 1, N, K, size=K ** -0.5)
    b_amax = nv.nvfp4_amax(weights)
    b = nv.nvfp4_quantize(weights, b_amax, dequant=False)["row"]
    n = nv.nvfp4_add_rms_norm(x, w, res)
    av = fp4_values(n["codes"], n["scales"], n["row_amax"])
    bv = fp4_values(b["codes"], b["scales"], b_amax[:, None])[0]
    out = nv.nvfp4_grouped_matmul(n, n["row_amax"], b, b_amax)
    ref = av @ bv.T
    assert ((out.double() - ref).abs() <= product_bound(av, bv, ref)).all()
    some = torch.full((T, N), 5.0, dtype=torch.bfloat16, device="cuda")
    nv.nvfp4_grouped_matmul(n, n["row_amax"], b, b_amax,
                            torch.tensor([0, 4], dtype=torch.int32, device="cuda"), out=some)
    assert torch.equal(some[:4], out[:4]) and (some[4:] == 5).all()


def test_example_runs():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "expert_layer.py"),
                        "--experts", "4", "--rows", "512", "--out", "256", "--cols", "512"],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "status 0" in r.stdout, r.stdout + r.stderr
