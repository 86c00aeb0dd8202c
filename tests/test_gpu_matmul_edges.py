"""The grouped products where they can go wrong: groups out of range, sums over nothing, scales
that are no numbers beside a group's rows, other outer maxima, many groups, streams and graphs."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_02_gb300 as nv
from linear_ref import fp4_values, mx_values, product_bound, ragged
from test_gpu_matmul import I32, check_rows, randn, starts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ws():
    return nv.grouped_matmul_workspace("cuda")


def fp4_operands(T, E, N, K, cfg=None, seed=1):
    cfg = cfg or nv.Config()
    x, w = randn(seed, T, K), randn(seed + 1, E, N, K, size=K ** -0.5)
    a = nv.nvfp4_quantize_per_token(x, cfg, dequant=False)
    b_amax = nv.nvfp4_amax(w)
    b = nv.nvfp4_quantize(w, b_amax, cfg, dequant=False)["row"]
    M = 256.0 if cfg.four_over_six else cfg.scale_max or 448.0
    return (a, a["row_amax"], b, b_amax,
            fp4_values(a["codes"].view(T, -1), a["scales"].view(T, -1), a["row_amax"], M),
            fp4_values(b["codes"], b["scales"], b_amax[:, None], M))


def mx_operands(T, E, N, K, seed=1):
    cfg = nv.Config(blocks=nv.BLOCKS_ROW)
    a = nv.nvfp4_mx_quantize(randn(seed, T, K), cfg)["row"]
    b = nv.nvfp4_mx_quantize(randn(seed + 1, E, N, K, size=K ** -0.5), cfg)["row"]
    return a, b, mx_values(a["codes"], a["scales"])[0], mx_values(b["codes"], b["scales"])


def columns(rows, n, k, seed=1):
    cfg = nv.Config(blocks=nv.BLOCKS_COL)
    g = nv.nvfp4_mx_quantize(randn(seed, rows, n), cfg)["col"]
    x = nv.nvfp4_mx_quantize(randn(seed + 1, rows, k), cfg)["col"]
    return g, x, mx_values(g["codes"], g["scales"])[0], mx_values(x["codes"], x["scales"])[0]


# group 1 ends before it begins, group 3 ends behind the rows, group 5 begins before them
BAD = [0, 32, 0, 64, 1 << 20, -32, 96]


def test_groups_out_of_range_are_left_out(ws):
    E, T, N, K = 6, 96, 200, 256
    a, aa, b, ba, av, bv = fp4_operands(T, E, N, K)
    start = torch.tensor(BAD, **I32)
    good = [e for e in range(E) if 0 <= BAD[e] <= BAD[e + 1] <= T]
    assert good == [0, 2]
    for mx in (False, True):
        status = torch.zeros(1, **I32)
        before = randn(3, T, N)
        out = before.clone()
        if mx:
            a, b, av, bv = mx_operands(T, E, N, K)
            nv.nvfp4_mx_grouped_matmul(a, b, start, out=out, workspace=ws, status=status)
        else:
            nv.nvfp4_grouped_matmul(a, aa, b, ba, start, out=out, workspace=ws, status=status)
        assert status.item() == nv.DEV_BAD_INDEX
        # rows 0 .. 63 belong to group 2 (0 .. 31 to group 0 too: either may be there)
        ref = [av[32:64] @ bv[2].T]
        off = (out[32:64].double() - ref[0]).abs() - product_bound(av[32:64], bv[2], ref[0])
        assert not (off > 0).any() and torch.equal(out[64:], before[64:])
    g, x, gv, xv = columns(T, N, K)
    status = torch.zeros(1, **I32)
    before = randn(4, E, N, K)
    out = before.clone()
    nv.nvfp4_mx_grouped_wgrad(g, x, start, out=out, workspace=ws, status=status)
    assert status.item() == nv.DEV_BAD_INDEX
    for e in range(E):
        if e in good:
            ga, xa = gv[:, BAD[e]:BAD[e + 1]], xv[:, BAD[e]:BAD[e + 1]]
            ref = ga @ xa.T
            assert ((out[e].double() - ref).abs() <= product_bound(ga, xa, ref)).all()
        else:
            assert torch.equal(out[e], before[e])
    # a border that is no multiple of 32
    status.zero_()
    nv.nvfp4_mx_grouped_wgrad(g, x, torch.tensor([0, 32, 48, 96], **I32), out=out[:3].clone(),
                              workspace=ws, status=status)
    assert status.item() == nv.DEV_BAD_INDEX
    assert not ws[:384].any()


def test_sums_over_nothing(ws):
    """A weights' gradient of groups without rows, and of no rows at all, is zero; a product of
    no rows writes nothing."""
    g, x, gv, xv = columns(64, 130, 77)
    for dtype in (torch.bfloat16, torch.float32):
        out = torch.full((5, 130, 77), 7.0, dtype=dtype, device="cuda")
        nv.nvfp4_mx_grouped_wgrad(g, x, torch.tensor([0, 0, 32, 32, 64, 64], **I32), out=out,
                                  workspace=ws)
        assert not out[0].any() and not out[2].any() and not out[4].any()
        ref = gv[:, 32:] @ xv[:, 32:].T
        assert ((out[3].double() - ref).abs() <= product_bound(
            gv[:, 32:], xv[:, 32:], ref, dtype == torch.float32)).all()
        empty = {"codes": torch.empty(130, 0, dtype=torch.uint8, device="cuda"),
                 "scales": torch.empty(130, 0, dtype=torch.uint8, device="cuda")}
        ex = {"codes": torch.empty(77, 0, dtype=torch.uint8, device="cuda"),
              "scales": torch.empty(77, 0, dtype=torch.uint8, device="cuda")}
        out.fill_(7)
        nv.nvfp4_mx_grouped_wgrad(empty, ex, torch.zeros(6, **I32), out=out, workspace=ws)
        assert not out.any()
        one = nv.nvfp4_mx_grouped_wgrad(empty, ex, out_dtype=dtype, workspace=ws)
        assert one.shape == (1, 130, 77) and not one.any()
    a, aa, b, ba, av, bv = fp4_operands(40, 3, 64, 256)
    before = randn(5, 40, 64)
    out = before.clone()
    nv.nvfp4_grouped_matmul(a, aa, b, ba, torch.full((4,), 17, **I32), out=out, workspace=ws)
    assert torch.equal(out, before)
    none = {"codes": a["codes"][:0], "scales": a["scales"][:0]}
    assert nv.nvfp4_grouped_matmul(none, aa[:1], b, ba, torch.zeros(4, **I32)).shape == (0, 64)


@pytest.mark.parametrize("cols", [256, 96, 1056])
def test_scales_that_are_no_numbers_stay_in_their_rows(ws, cols):
    """NaN scale bytes of rows outside a group, of other groups' rows and weights, and behind the
    last value of a row reach no other result; those of a row and of a weight reach theirs."""
    E, T, N = 3, 70, 136
    a, aa, b, ba, av, bv = fp4_operands(T, E, N, cols)
    start = torch.tensor([3, 20, 41, 60], **I32)
    clean = nv.nvfp4_grouped_matmul(a, aa, b, ba, start, out=torch.zeros(
        T, N, dtype=torch.bfloat16, device="cuda"), workspace=ws)
    for t in (2, 60, 69):  # rows that no group owns
        a["scales"].view(T, -1)[t] = 0x7F
    a["scales"].view(T, -1)[25, -1] = 0x7F          # a row of group 1
    b["scales"][2, 5, 0] = 0x7F                     # a weight of group 2
    out = nv.nvfp4_grouped_matmul(a, aa, b, ba, start, out=torch.zeros_like(clean), workspace=ws)
    want = clean.clone()
    want[25] = float("nan")
    want[41:60, 5] = float("nan")
    assert torch.equal(out.isnan(), want.isnan())
    assert torch.equal(out[~want.isnan()], clean[~want.isnan()])


def test_scales_of_other_groups_rows_stay_out_of_a_gradient(ws):
    g, x, gv, xv = columns(160, 140, 130)
    start = torch.tensor([32, 96, 128], **I32)
    clean = nv.nvfp4_mx_grouped_wgrad(g, x, start, workspace=ws)
    for t in (0, 4):  # blocks of rows 0 .. 31 and 128 .. 159: no group's
        g["scales"][..., t] = 0xFF
        x["scales"][..., t] = 0xFF
    assert torch.equal(nv.nvfp4_mx_grouped_wgrad(g, x, start, workspace=ws), clean)
    x["scales"][0, 7, 3] = 0xFF  # rows 96 .. 127: group 1
    out = nv.nvfp4_mx_grouped_wgrad(g, x, start, workspace=ws)
    assert torch.equal(out[0], clean[0]) and out[1, :, 7].isnan().all()
    keep = torch.arange(130, device="cuda") != 7
    assert torch.equal(out[1][:, keep], clean[1][:, keep])


@pytest.mark.parametrize("cfg", [nv.Config(four_over_six=1), nv.Config(scale_max=300.0)])
def test_other_outer_maxima(ws, cfg):
    a, aa, b, ba, av, bv = fp4_operands(50, 2, 72, 288, cfg)
    start = torch.tensor([0, 30, 50], **I32)
    out = nv.nvfp4_grouped_matmul(a, aa, b, ba, start, a_cfg=cfg, b_cfg=cfg, workspace=ws)
    check_rows(out, out, av, bv, start)


def test_rows_of_zeros_and_bad_amax(ws):
    a, aa, b, ba, av, bv = fp4_operands(8, 1, 40, 256)
    x = randn(1, 8, 256)
    x[3] = 0
    z = nv.nvfp4_quantize_per_token(x, dequant=False)
    out = nv.nvfp4_grouped_matmul(z, z["row_amax"], b, ba, workspace=ws)
    assert not out[3].any() and out.isfinite().all()
    for bad in (float("nan"), float("inf"), -1.0):
        for which in (0, 1):
            status = torch.zeros(1, **I32)
            am, bm = aa.clone(), ba.clone()
            (am if which == 0 else bm)[0] = bad
            nv.nvfp4_grouped_matmul(a, am, b, bm, workspace=ws, status=status)
            assert status.item() == nv.DEV_BAD_AMAX


def test_most_groups(ws):
    E, T, N, K = 1024, 1500, 24, 64
    n = ragged(np.random.default_rng(3), E, T, empty=0.4)
    a, aa, b, ba, av, bv = fp4_operands(T, E, N, K)
    out = nv.nvfp4_grouped_matmul(a, aa, b, ba, starts(n), workspace=ws)
    check_rows(out, out, av, bv, starts(n))
    g, x, gv, xv = columns(2048, 40, 33)
    n = ragged(np.random.default_rng(4), E, 2048, empty=0.95, unit=32)
    start = starts(n)
    out = nv.nvfp4_mx_grouped_wgrad(g, x, start, workspace=ws)
    at = start.tolist()
    for e in range(E):
        ref = gv[:, at[e]:at[e + 1]] @ xv[:, at[e]:at[e + 1]].T
        assert ((out[e].double() - ref).abs() <= product_bound(
            gv[:, at[e]:at[e + 1]], xv[:, at[e]:at[e + 1]], ref)).all()


def test_same_bits_again_and_on_two_streams():
    """Two calls at a time on streams of their own, each with its workspace, give the bits of a
    call alone; so do sums that are cut into parts."""
    cases = [(300, 4, 512, 1024), (40, 1, 130, 7168), (2000, 1, 1000, 512)]
    work = []
    for i, (T, E, N, K) in enumerate(cases):
        a, aa, b, ba, _, _ = fp4_operands(T, E, N, K, seed=10 * i)
        start = starts(ragged(np.random.default_rng(i), E, T))
        work.append((a, aa, b, ba, start))
    alone = [nv.nvfp4_grouped_matmul(*w) for w in work]
    g, x, _, _ = columns(4096, 128, 100)
    gw = nv.nvfp4_mx_grouped_wgrad(g, x, out_dtype=torch.float32)
    side = [torch.cuda.Stream() for _ in range(2)]
    spaces = [nv.grouped_matmul_workspace("cuda") for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[], []]
    for rep in range(5):
        for s in (0, 1):
            with torch.cuda.stream(side[s]):
                for w in (work if s else work[::-1]):
                    outs[s].append(nv.nvfp4_grouped_matmul(*w, workspace=spaces[s]))
                outs[s].append(nv.nvfp4_mx_grouped_wgrad(g, x, out_dtype=torch.float32,
                                                         workspace=spaces[s]))
    torch.cuda.synchronize()
    for s in (0, 1):
        want = (alone if s else alone[::-1]) + [gw]
        for i, o in enumerate(outs[s]):
            assert torch.equal(o, want[i % 4])
        assert not spaces[s][:384].any()


def test_captured_and_replayed_with_other_groups(ws):
    """A graph's groups are read when it runs: borders and inputs change between replays."""
    E, T, N, K = 5, 200, 384, 512
    a, aa, b, ba, av, bv = fp4_operands(T, E, N, K)
    a2, b2, av2, bv2 = mx_operands(T, E, N, K, seed=7)
    g, x, gv, xv = columns(T - T % 32, N, 100, seed=9)
    start, start32 = torch.zeros(E + 1, **I32), torch.zeros(E + 1, **I32)
    out, out2 = (torch.zeros(T, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    gw = torch.zeros(E, N, 100, dtype=torch.float32, device="cuda")

    def step():
        nv.nvfp4_grouped_matmul(a, aa, b, ba, start, out=out, workspace=ws)
        nv.nvfp4_mx_grouped_matmul(a2, b2, start, out=out2, workspace=ws)
        nv.nvfp4_mx_grouped_wgrad(g, x, start32, out=gw, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        rng = np.random.default_rng(i)
        start.copy_(starts(ragged(rng, E, T)))
        start32.copy_(starts(ragged(rng, E, 192, unit=32)))
        out.fill_(3)
        before = out.clone()
        graph.replay()
        check_rows(out, before, av, bv, start)
        check_rows(out2, out2, av2, bv2, start)
        at = start32.tolist()
        for e in range(E):
            ga, xa = gv[:, at[e]:at[e + 1]], xv[:, at[e]:at[e + 1]]
            ref = ga @ xa.T
            assert ((gw[e].double() - ref).abs() <= product_bound(ga, xa, ref, True)).all()


def test_past_32_bits(ws):
    """Weights and results whose byte offsets pass 32 bits."""
    E, N, K = 9, 33000, 16384
    x = randn(1, 40, K)
    a = nv.nvfp4_quantize_per_token(x, dequant=False)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    codes = torch.randint(0, 256, (E, N, K // 2), generator=g, dtype=torch.uint8, device="cuda")
    scales = torch.randint(0x30, 0x50, (E, N, K // 16), generator=g, dtype=torch.uint8,
                           device="cuda")
    ba = torch.ones(E, device="cuda")
    start = torch.tensor([0, 0, 0, 0, 0, 0, 0, 0, 20, 40], **I32)
    out = nv.nvfp4_grouped_matmul(a, a["row_amax"], {"codes": codes, "scales": scales}, ba, start,
                                  workspace=ws)
    av = fp4_values(a["codes"].view(40, -1), a["scales"].view(40, -1), a["row_amax"])
    for e, i in ((7, 0), (8, 20)):
        for n in (0, N - 300):
            bv = fp4_values(codes[e, n:n + 300], scales[e, n:n + 300], ba[e].expand(300))
            ref = av[i:i + 20] @ bv.T
            assert ((out[i:i + 20, n:n + 300].double() - ref).abs()
                    <= product_bound(av[i:i + 20], bv, ref)).all()
    del codes, scales, out
    # 2.2 billion gradients
    E, N, K = 40, 8192, 6720
    g, x, gv, xv = columns(64, N, K)
    start = torch.tensor([0] * 39 + [32, 64], **I32)
    out = nv.nvfp4_mx_grouped_wgrad(g, x, start, workspace=ws)
    for e, i in ((38, 0), (39, 32)):
        ref = gv[-200:, i:i + 32] @ xv[:, i:i + 32].T
        assert ((out[e, -200:].double() - ref).abs()
                <= product_bound(gv[-200:, i:i + 32], xv[:, i:i + 32], ref)).all()
    assert not out[37, -1].any()


@pytest.mark.parametrize("E,T,N,K", [(5, 320, 33, 64), (3, 96, 130, 304), (2, 4096, 96, 272),
                                     (8, 2048, 500, 1040)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gradients_stay_in_their_place(ws, E, T, N, K, dtype):
    """Results at 16-byte and at 32-byte boundaries of a larger buffer: the same bits, nothing
    around them."""
    g, x, _, _ = columns(T, N, K)
    start = starts(ragged(np.random.default_rng(N), E, T, unit=32))
    want = nv.nvfp4_mx_grouped_wgrad(g, x, start, out_dtype=dtype, workspace=ws)
    n = E * N * K
    for at in (8, 16, 32):
        buf = torch.full((n + 64,), 7.0, dtype=dtype, device="cuda")
        out = buf[at:at + n].view(E, N, K)
        nv.nvfp4_mx_grouped_wgrad(g, x, start, out=out, workspace=ws)
        assert torch.equal(out, want)
        assert (buf[:at] == 7).all() and (buf[at + n:] == 7).all()


@pytest.mark.parametrize("N,K", [(130, 80), (300, 528), (32, 16)])
def test_rows_of_gradients_of_nothing_and_of_bad_groups(ws, N, K):
    """Results that leave row by row: groups without rows and calls without rows give zeros, bad
    groups leave theirs, in a graph as well."""
    g, x, gv, xv = columns(96, N, K)
    out = torch.full((6, N, K), 7.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, **I32)
    start = torch.tensor([0, 0, 32, 48, 64, 32, 96], **I32)  # 48 no border, 64 .. 32 backwards
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        nv.nvfp4_mx_grouped_wgrad(g, x, start, out=out, workspace=ws, status=status)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        nv.nvfp4_mx_grouped_wgrad(g, x, start, out=out, workspace=ws, status=status)
    for _ in range(2):
        assert status.item() == nv.DEV_BAD_INDEX
        assert not out[0].any() and (out[2:5] == 7).all()
        for e, a, b in ((1, 0, 32), (5, 32, 96)):
            ref = gv[:, a:b] @ xv[:, a:b].T
            assert ((out[e].double() - ref).abs()
                    <= product_bound(gv[:, a:b], xv[:, a:b], ref)).all()
        out.fill_(7)
        status.zero_()
        graph.replay()
    none = [{"codes": torch.empty(n, 0, dtype=torch.uint8, device="cuda"),
             "scales": torch.empty(n, 0, dtype=torch.uint8, device="cuda")} for n in (N, K)]
    nv.nvfp4_mx_grouped_wgrad(*none, torch.zeros(7, **I32), out=out, workspace=ws)
    assert not out.any()


def test_a_matrix_with_itself(ws):
    """One encoding, and one outer scale, as both operands."""
    x = randn(1, 300, 416)
    amax = nv.nvfp4_amax(x)
    q = nv.nvfp4_quantize(x, amax, nv.Config(), dequant=False)["row"]
    out = nv.nvfp4_grouped_matmul(q, amax, q, amax, workspace=ws)
    v = fp4_values(q["codes"].view(300, -1), q["scales"].view(300, -1), amax.expand(300))
    ref = v @ v.T
    assert ((out.double() - ref).abs() <= product_bound(v, v, ref)).all()
    m = nv.nvfp4_mx_quantize(x, nv.Config(blocks=nv.BLOCKS_ROW))["row"]
    out = nv.nvfp4_mx_grouped_matmul(m, m, workspace=ws)
    v = mx_values(m["codes"], m["scales"])[0]
    ref = v @ v.T
    assert ((out.double() - ref).abs() <= product_bound(v, v, ref)).all()
    m = nv.nvfp4_mx_quantize(x[:288], nv.Config(blocks=nv.BLOCKS_COL))["col"]
    out = nv.nvfp4_mx_grouped_wgrad(m, m, out_dtype=torch.float32, workspace=ws)
    v = mx_values(m["codes"], m["scales"])[0]
    ref = v @ v.T
    assert ((out[0].double() - ref).abs() <= product_bound(v, v, ref, True)).all()


def test_on_inputs_device_and_refusals():
    a, aa, b, ba, _, _ = fp4_operands(8, 2, 40, 64)
    st = torch.tensor([0, 4, 8], **I32)
    good = lambda **k: nv.nvfp4_grouped_matmul(**{**dict(  # noqa: E731
        a=a, a_amax=aa, b=b, b_amax=ba, group_start=st), **k})
    good()
    for k in (dict(group_start=None), dict(group_start=st[:2]), dict(a_amax=aa[:3]),
              dict(b_amax=ba[:1]), dict(a={"codes": a["codes"], "scales": a["scales"][:4]}),
              dict(b={"codes": b["codes"][:, :, :16].contiguous(), "scales": b["scales"]}),
              dict(out=torch.empty(8, 41, dtype=torch.bfloat16, device="cuda")),
              dict(a_cfg=nv.Config(scale_fmt=nv.SCALE_UE5M3))):
        with pytest.raises(ValueError):
            good(**k)
    for k in (dict(group_start=st.long()), dict(a_amax=aa.double()),
              dict(out=torch.empty(8, 40, device="cuda"))):
        with pytest.raises(TypeError):
            good(**k)
    with pytest.raises(nv.Nvfp4Error):
        good(workspace=torch.zeros(16, **I32))
    with pytest.raises(ValueError):
        good(b={"codes": b["codes"].cpu(), "scales": b["scales"]})


# rows of each group: few or many rows, then a dozen and more groups without any for every CTA,
# then rows again; rows of scales of whole 16 bytes (multiples of 512 rows) and not
GAPS = [[64] + [0] * 20 + [448], [160] + [0] * 20 + [96], [0] * 3 + [2048] + [0] * 20 + [512],
        [0] * 20 + [1000 * 32] + [0] * 20 + [32], [32, 0, 0, 96] * 4 + [0] * 30 + [32, 0] * 5]


@pytest.mark.parametrize("rows", GAPS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("wide", [True, False])
def test_many_groups_without_rows_between_others(ws, rows, dtype, wide):
    """Tiles without sums between tiles with sums, by pairs of CTAs (wide results) and by single
    ones: every result is there, and no wait runs out."""
    n, k = (1024, 2048) if wide else (96, 8192)
    if not wide:  # more groups, for as many pieces of a CTA
        rows = [r for r in rows for _ in range(1 if r else 3)]
    total = sum(rows)
    g, x, gv, xv = columns(total, n, k, seed=total)
    status = torch.zeros(1, **I32)
    out = torch.full((len(rows), n, k), 7.0, dtype=dtype, device="cuda")
    nv.nvfp4_mx_grouped_wgrad(g, x, starts(rows), out=out, workspace=ws, status=status)
    assert status.item() == 0 and not ws[:384].any()
    at = np.concatenate([[0], np.cumsum(rows)])
    for e, r in enumerate(rows):
        if r == 0:
            assert not out[e].any(), e
        else:
            ga, xa = gv[:, at[e]:at[e + 1]], xv[:, at[e]:at[e + 1]]
            ref = ga @ xa.T
            off = (out[e].double() - ref).abs() - product_bound(ga, xa, ref,
                                                                dtype == torch.float32)
            assert not (off > 0).any() and out[e].isfinite().all(), e


@pytest.mark.parametrize("E,T,N,K", [(1, 8192, 1000, 64), (1, 4096, 128, 16), (1, 16384, 200, 160),
                                     (2, 8192, 64, 528), (4, 1024, 1000, 1040)])
def test_gradients_bits_do_not_depend_on_alignment(ws, E, T, N, K):
    """Sums that are cut into parts too: the same order at 16-byte as at larger boundaries."""
    g, x, gv, xv = columns(T, N, K)
    start = torch.tensor([T // E // 32 * 32 * e for e in range(E)] + [T], **I32)
    want = nv.nvfp4_mx_grouped_wgrad(g, x, start, workspace=ws)
    at, n = start.tolist(), E * N * K
    for e in range(E):
        ga, xa = gv[:, at[e]:at[e + 1]], xv[:, at[e]:at[e + 1]]
        ref = ga @ xa.T
        assert ((want[e].double() - ref).abs() <= product_bound(ga, xa, ref)).all()
    for first in (8, 16, 24):
        buf = torch.full((n + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
        nv.nvfp4_mx_grouped_wgrad(g, x, start, out=buf[first:first + n].view(E, N, K), workspace=ws)
        assert torch.equal(buf[first:first + n].view(E, N, K), want)
        assert (buf[:first] == 7).all() and (buf[first + n:] == 7).all()


@pytest.mark.parametrize("T", [300, 1 << 30])
def test_groups_that_share_rows(ws, T):
    """Borders that go back and forth: every other of 1024 groups has all rows (with 2^30 of them
    2^31 tiles, past 32 bits), the others are out of order. All have the same weights, so that the
    results are known; nothing around them is written."""
    E, K = 1024, 32
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    codes = torch.empty(T, K // 2, dtype=torch.uint8, device="cuda")
    codes.random_(0, 256, generator=g)
    scales = torch.empty(T, K // 16, dtype=torch.uint8, device="cuda")
    scales.random_(0x30, 0x50, generator=g)
    bc = torch.randint(0, 256, (1, 1, K // 2), generator=g, dtype=torch.uint8, device="cuda")
    bs = torch.randint(0x30, 0x50, (1, 1, K // 16), generator=g, dtype=torch.uint8, device="cuda")
    one = torch.full((1,), 2688.0, device="cuda")  # outer scales of 1
    b = {"codes": bc.expand(E, 1, -1).contiguous(), "scales": bs.expand(E, 1, -1).contiguous()}
    start = torch.tensor([0, T] * (E // 2) + [0], **I32)
    status = torch.zeros(1, **I32)
    buf = torch.full((T + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    nv.nvfp4_grouped_matmul({"codes": codes, "scales": scales}, one, b, one.expand(E).contiguous(),
                            start, out=buf[32:32 + T].view(T, 1), workspace=ws, status=status)
    assert status.item() == nv.DEV_BAD_INDEX
    assert (buf[:32] == 7).all() and (buf[32 + T:] == 7).all()
    n = min(T, 1 << 20)
    bv = fp4_values(bc[0], bs[0], one)
    for at in (0, (T - n) // 2, T - n):
        av = fp4_values(codes[at:at + n], scales[at:at + n], one.expand(n))
        ref = av @ bv.T
        out = buf[32 + at:32 + at + n, None].double()
        assert ((out - ref).abs() <= product_bound(av, bv, ref)).all()
