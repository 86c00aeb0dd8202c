"""The products grouped by expert against plain products in 64 bits of the values that the
codes stand for."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_02_gb300 as nv
from linear_ref import fp4_values, mx_values, product_bound, ragged

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module")
def ws():
    return nv.grouped_matmul_workspace("cuda")


def randn(seed, *shape, size=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(*shape, generator=g, device="cuda")
    return (x * torch.exp(0.5 * torch.randn(shape[-1], generator=g, device="cuda")) * size
            ).to(torch.bfloat16)


def starts(n, first=0):
    return torch.tensor(np.concatenate([[0], np.cumsum(n)]) + first, **I32)


def check_rows(out, before, a, b, start):
    """out against a @ b[e].T group by group; rows outside the groups as they were before."""
    at = start.tolist()
    for e in range(len(at) - 1):
        i, j = at[e], at[e + 1]
        if j > i:
            ref = a[i:j] @ b[e].T
            off = (out[i:j].double() - ref).abs() - product_bound(a[i:j], b[e], ref)
            assert not (off > 0).any() and out[i:j].isfinite().all(), (e, i, j, float(off.max()))
    for part in (slice(0, at[0]), slice(at[-1], None)):
        assert torch.equal(out[part], before[part])


# groups, rows, features, cols: one tile and less, ragged tiles, odd features, sums that end
# inside a stage or a product, more tiles than SMs, sums cut into parts
SIZES = [(1, 1, 1, 32), (1, 1, 128, 256), (1, 16, 128, 512), (1, 5, 130, 96), (1, 128, 256, 1024),
         (1, 256, 128, 256), (1, 257, 256, 288), (3, 300, 200, 544), (5, 700, 1000, 416),
         (7, 40, 77, 160), (1, 33, 64, 7168), (1, 300, 128, 4096), (64, 90, 2048, 1024),
         (2, 3000, 1536, 320), (1, 2000, 4096, 512), (300, 900, 136, 64),
         # rows of scales that are not whole 16 bytes, in sums long enough to be copied first
         (4, 3000, 1536, 7136), (24, 200, 1500, 7136),
         # pairs of CTAs with groups of few rows, and with features that end inside a pair
         (40, 6000, 512, 288), (40, 6000, 333, 256), (30, 4500, 650, 512)]


@pytest.mark.parametrize("E,T,N,K", SIZES)
@pytest.mark.parametrize("each", [True, False])
def test_nvfp4_product(ws, E, T, N, K, each):
    rng = np.random.default_rng(E + T + N + K)
    x, w = randn(1, T + 9, K), randn(2, E, N, K, size=K ** -0.5)
    start = starts(ragged(rng, E, T), first=4)
    status = torch.zeros(1, **I32)
    if each:
        a = nv.nvfp4_quantize_per_token(x, dequant=False)
        a_amax = a["row_amax"]
    else:
        a_amax = nv.nvfp4_amax(x)
        a = nv.nvfp4_quantize(x, a_amax, dequant=False)["row"]
    b_amax = nv.nvfp4_amax(w)
    b = nv.nvfp4_quantize(w, b_amax, dequant=False)["row"]
    before = randn(3, T + 9, N)
    out = nv.nvfp4_grouped_matmul(a, a_amax, b, b_amax, start, out=before.clone(), workspace=ws,
                                  status=status)
    av = fp4_values(a["codes"].view(T + 9, -1), a["scales"].view(T + 9, -1),
                    a_amax.expand(T + 9))
    bv = fp4_values(b["codes"], b["scales"], b_amax[:, None])
    check_rows(out, before, av, bv, start)
    assert status.item() == 0 and not ws[:384].any()


@pytest.mark.parametrize("E,T,N,K", SIZES)
def test_mx_product(ws, E, T, N, K):
    rng = np.random.default_rng(E + T + N + K)
    x, w = randn(1, T + 9, K), randn(2, E, N, K, size=K ** -0.5)
    start = starts(ragged(rng, E, T), first=4)
    status = torch.zeros(1, **I32)
    cfg = nv.Config(blocks=nv.BLOCKS_ROW)
    a, b = nv.nvfp4_mx_quantize(x, cfg)["row"], nv.nvfp4_mx_quantize(w, cfg)["row"]
    before = randn(3, T + 9, N)
    out = nv.nvfp4_mx_grouped_matmul(a, b, start, out=before.clone(), workspace=ws, status=status)
    check_rows(out, before, mx_values(a["codes"], a["scales"])[0],
               mx_values(b["codes"], b["scales"]), start)
    assert status.item() == 0 and not ws[:384].any()


@pytest.mark.parametrize("E,T,N,K", [(1, 32, 1, 1), (1, 64, 130, 77), (1, 128, 256, 128),
                                     (3, 320, 200, 100), (4, 960, 1000, 544), (1, 4096, 128, 128),
                                     (16, 4096, 512, 300), (40, 640, 33, 64), (2, 32, 300, 256),
                                     (2, 8160, 2048, 2000)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_mx_weight_gradient(ws, E, T, N, K, dtype):
    rng = np.random.default_rng(E + T + N + K)
    pad = 64  # rows in front of the first and behind the last group
    g, x = randn(1, T + pad, N), randn(2, T + pad, K)
    start = starts(ragged(rng, E, T, unit=32), first=32)
    status = torch.zeros(1, **I32)
    cfg = nv.Config(blocks=nv.BLOCKS_COL)
    gt, xt = nv.nvfp4_mx_quantize(g, cfg)["col"], nv.nvfp4_mx_quantize(x, cfg)["col"]
    out = nv.nvfp4_mx_grouped_wgrad(gt, xt, start, out_dtype=dtype, workspace=ws, status=status)
    gv, xv = mx_values(gt["codes"], gt["scales"])[0], mx_values(xt["codes"], xt["scales"])[0]
    at = start.tolist()
    assert out.shape == (E, N, K) and out.dtype == dtype
    for e in range(E):
        ga, xa = gv[:, at[e]:at[e + 1]], xv[:, at[e]:at[e + 1]]
        ref = ga @ xa.T
        off = (out[e].double() - ref).abs() - product_bound(ga, xa, ref, dtype == torch.float32)
        assert not (off > 0).any() and out[e].isfinite().all(), (e, float(off.max()))
    assert status.item() == 0 and not ws[:384].any()
