"""Attention over the paged NVFP4 cache against the 64-bit form.

Bounds, per row, with A = max over keys of scale * sum |q_d k_d| and B = sum p
|v|, C = the largest p times sum |v|: a score is an fp32 sum of exact products, off by at most 2^-19 A (D / 16
accumulation steps, some of them truncating); a probability is off by that, by
2^-20 (exponential, running rescales) and by 2^-11 for its rounding to f16; the
output is rounded to bf16 once (half an ulp). So |out - exact| <= half an ulp +
(2^-11 + 2^-18 A + 2^-19) B and |lse - exact| <= 2^-18 A + 2^-19 + 2^-22 |lse|."""
import numpy as np
import pytest
import torch

import kv_ref
import nvfp4_block_scaled_02_gb300 as nv

pytestmark = pytest.mark.gpu


def _state(new, total, hq, hk, D, P, seed, q_size=1.0, junk=True, fos=False):
    """A cache of random codes and scale bytes; places that no request holds and
    the slots past a request's length hold NaN scale bytes."""
    r = np.random.default_rng(seed)
    new, total = np.asarray(new), np.asarray(total)
    held = -(-total // P)
    pages = int(held.sum()) + 2
    cols = max(1, int(held.max(initial=0)) + 1)
    order = r.permutation(pages)
    table = np.full((len(new), cols), -1, np.int32)
    table[np.arange(cols)[None, :] < held[:, None]] = order[: int(held.sum())]
    c = {"four_over_six": int(fos)}
    for n in ("k", "v"):
        c[n + "_codes"] = r.integers(0, 256, (pages, hk, P, D // 2)).astype(np.uint8)
        # block scales from 2^-3 to 2^3, a few zeros and a few subnormals
        s = r.integers(32, 81, (pages, hk, P, D // 16)).astype(np.uint8)
        s[r.random(s.shape) < 0.02] = 0
        s[r.random(s.shape) < 0.02] = 3
        if junk:
            live = np.zeros((pages, P), bool)
            for b in range(len(total)):
                for j in range(int(held[b])):
                    live[table[b, j], : min(P, int(total[b]) - j * P)] = True
            s.transpose(0, 2, 1, 3)[~live] = 0x7F
        c[n + "_scales"] = s
        c[n + "_amax"] = r.uniform(100, 900, hk).astype(np.float32)
    T = int(new.sum())
    q = torch.from_numpy((q_size * r.standard_normal((T, hq, D))).astype(np.float32)).to(torch.bfloat16)
    return dict(new=new, total=total, table=table, cache=c, q=q, P=P, hk=hk, D=D,
                q_start=np.concatenate([[0], np.cumsum(new)]).astype(np.int32))


def _dev(s):
    c = {n: torch.from_numpy(v).cuda() if isinstance(v, np.ndarray) else v
         for n, v in s["cache"].items()}
    return (s["q"].cuda(), c, torch.from_numpy(s["table"]).cuda(),
            torch.from_numpy(s["total"].astype(np.int32)).cuda(),
            torch.from_numpy(s["q_start"]).cuda(), int(max(s["new"], default=0)))


def _ref(s, scale, window):
    c, M = s["cache"], 256.0 if s["cache"]["four_over_six"] else 448.0

    def of(n):
        def get(b):
            L = int(s["total"][b])
            pg = s["table"][b, : -(-L // s["P"])]
            x = [kv_ref.decode(c[n + "_codes"][pg, h].reshape(-1, s["D"] // 2)[:L],
                               c[n + "_scales"][pg, h].reshape(-1, s["D"] // 16)[:L],
                               float(c[n + "_amax"][h]) / (6 * M)) for h in range(s["hk"])]
            return np.stack(x)
        return get
    return kv_ref.attention(s["q"].double().numpy(), of("k"), of("v"), s["q_start"], s["total"],
                            scale, window)


def _check(got, want):
    out, lse, absv, size, allv = want
    o, z = got["out"].double().cpu().numpy(), got["lse"].double().cpu().numpy()
    A = size[..., None]
    tol = (2.0 ** -11 + 2.0 ** -18 * A + 2.0 ** -19) * absv + 2.0 ** -31 * allv
    tol += kv_ref.half_ulp_bf16(np.abs(out) + tol)
    err = np.abs(o - out)
    assert (err <= tol).all(), f"out: {np.nanmax(err / tol)} of the bound, {np.isnan(o).sum()} NaN"
    empty = np.isinf(lse)
    assert np.array_equal(empty, np.isinf(z)) and (z[empty] < 0).all()
    lt = 2.0 ** -18 * size + 2.0 ** -19 + 2.0 ** -22 * np.abs(np.where(empty, 0, lse))
    le = np.abs(np.where(empty, 0, z) - np.where(empty, 0, lse))
    assert (le <= lt).all(), f"lse: {(le / lt).max()} of the bound"


def _go(s, scale=None, window=0, ws=None):
    scale = s["D"] ** -0.5 if scale is None else scale
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = nv.nvfp4_kv_attention(*_dev(s), scale=scale, window=window, status=st, workspace=ws)
    assert int(st.item()) == 0
    return got


CASES = [
    # new, total, q_heads, kv_heads, D, P
    ([1], [1], 1, 1, 64, 16), ([1], [1], 8, 1, 128, 16), ([1], [2], 4, 2, 128, 16),
    ([1, 1], [15, 16], 8, 2, 64, 16), ([1, 1, 1], [17, 31, 33], 6, 2, 128, 16),
    ([1, 1], [100, 1000], 32, 8, 128, 64), ([1] * 5, [48, 49, 95, 97, 47], 7, 7, 64, 48),
    ([1], [20000], 8, 2, 128, 64), ([1], [9999], 5, 1, 64, 32),
    ([1] * 40, list(range(0, 400, 10)), 10, 2, 128, 16),
    ([1, 0, 1], [0, 40, 70], 4, 1, 128, 16),                  # an empty and an idle request
    ([3], [2], 4, 2, 64, 16),                                 # the first row sees nothing
    ([2, 4, 3], [30, 4, 3000], 8, 2, 128, 16), ([5, 1], [5, 700], 21, 7, 64, 32),
    ([4], [4], 16, 4, 128, 16), ([16, 17], [16, 400], 4, 4, 128, 64), ([40], [100], 3, 1, 64, 16),
    ([1, 130], [300, 130], 8, 2, 128, 16), ([257, 5], [300, 900], 4, 1, 128, 64),
    ([300], [1500], 8, 2, 64, 32), ([129, 128, 127], [129, 500, 1000], 6, 2, 128, 128),
    ([1], [77], 64, 2, 128, 16), ([33], [64], 40, 1, 64, 16), ([600], [601], 1, 1, 128, 80),
]


@pytest.mark.parametrize("window", [0, 1, 20, 10**9])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_matches_the_formula(case, window):
    new, total, hq, hk, D, P = CASES[case]
    s = _state(new, total, hq, hk, D, P, seed=case)
    _check(_go(s, window=window), _ref(s, D ** -0.5, window))


@pytest.mark.parametrize("window", [1000, 129])
def test_long_windows(window):
    s = _state([3, 70, 1], [5000, 3000, 1100], 8, 2, 128, 64, seed=window)
    _check(_go(s, window=window), _ref(s, 128 ** -0.5, window))


@pytest.mark.parametrize("new,total", [([1, 2], [500, 900]), ([200], [700])])
@pytest.mark.parametrize("q_size,scale", [(1e-30, 1e28), (1e30, 1e-32), (100.0, 0.09), (1.0, 0.0),
                                          (1.0, -0.5), (300.0, 1.0)])
def test_query_ranges_and_peaked_rows(new, total, q_size, scale):
    """Rows of tiny and huge queries (the product with the scale is ordinary), rows
    whose softmax is nearly one key, a zero and a negative scale."""
    s = _state(new, total, 8, 2, 128, 16, seed=7, q_size=q_size)
    _check(_go(s, scale=scale), _ref(s, scale, 0))


def test_one_query_row_with_values_far_apart():
    s = _state([1, 150], [400, 400], 8, 2, 64, 16, seed=9)
    q = s["q"].float()
    q[:, :, ::3] *= 2.0 ** -20
    q[:, 1] = 0
    s["q"] = q.to(torch.bfloat16)
    _check(_go(s), _ref(s, 64 ** -0.5, 0))


def test_four_over_six_cache_and_strided_queries():
    s = _state([1, 20, 200], [99, 333, 500], 8, 2, 128, 16, seed=10, fos=True)
    want = _go(s)
    _check(want, _ref(s, 128 ** -0.5, 0))
    q, *rest = _dev(s)
    wide = torch.zeros(q.shape[0], 12, 128, dtype=torch.bfloat16, device="cuda")
    wide[:, 2:10] = q
    got = nv.nvfp4_kv_attention(wide[:, 2:10], *rest)
    assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])


def test_same_bits_again_with_a_shared_workspace():
    ws = nv.kv_attention_workspace("cuda")
    states = [_state([1] * 3, [5000, 70, 900], 32, 8, 128, 16, seed=1),
              _state([2, 300, 1], [800, 2000, 0], 8, 2, 64, 32, seed=2),
              _state([1], [30000], 8, 1, 128, 64, seed=3)]
    first = [_go(s, ws=ws) for s in states]
    for s, a in zip(states, first):
        b = _go(s, ws=ws)
        assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])
        c = _go(s)
        assert torch.equal(a["out"], c["out"]) and torch.equal(a["lse"], c["lse"])


def test_data_errors_are_flagged():
    s = _state([1, 2], [40, 60], 4, 1, 64, 16, seed=4, junk=False)

    def status(change, **kw):
        a = list(_dev(s))
        change(a)
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        nv.nvfp4_kv_attention(*a, status=st, **kw)
        return int(st.item())
    assert status(lambda a: None) == 0

    def page(x):
        def f(a):
            a[2][1, 2] = x
        return f
    assert status(page(-1)) == nv.DEV_BAD_INDEX
    assert status(page(10**6)) == nv.DEV_BAD_INDEX

    def length(x):
        def f(a):
            a[3][0] = x
        return f
    assert status(length(10**6)) == nv.DEV_BAD_INDEX
    assert status(length(-1)) == nv.DEV_BAD_INDEX

    def start(x):
        def f(a):
            a[4][2] = x
        return f
    assert status(start(100)) == nv.DEV_BAD_INDEX
    assert status(start(0)) == nv.DEV_BAD_INDEX

    def most(a):
        a[5] = 1
    assert status(most) == nv.DEV_BAD_INDEX

    def q(x):
        def f(a):
            a[0][1, 1, 3] = x
        return f
    assert status(q(float("nan"))) & nv.DEV_NONFINITE_INPUT
    assert status(q(float("inf"))) & nv.DEV_NONFINITE_INPUT

    def amax(a):
        a[1]["v_amax"][0] = -1
    assert status(amax) == nv.DEV_BAD_AMAX


def test_rows_no_request_owns_are_left_alone():
    s = _state([1, 2], [40, 60], 4, 1, 64, 16, seed=5)
    q, *rest = _dev(s)
    pad = torch.cat([q, q[:2]])
    out = torch.full((5, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((5, 4), 7.0, device="cuda")
    nv.nvfp4_kv_attention(pad, *rest, out=out, lse=lse)
    want = _go(s)
    assert torch.equal(out[:3], want["out"]) and (out[3:] == 7).all() and (lse[3:] == 7).all()


@pytest.mark.parametrize("requests", [15, 17, 40, 130, 700])
def test_batches_of_every_kind_of_request(requests):
    """Single rows, up to 8, 9 to 16 and more rows per KV head, empty requests, one without
    keys and rows before the first key in one call: fewer and more requests than
    threads share the work of finding them."""
    r = np.random.default_rng(requests)
    new = np.resize([1, 0, 3, 17, 5, 20, 8, 2, 33, 1, 140], requests)
    total = new + r.integers(0, 60, requests)
    total[4] = 0
    total[3::11] = 10  # 17 rows, 10 keys
    _check(_go(_state(new, total, 2, 1, 64, 16, 5)), _ref(_state(new, total, 2, 1, 64, 16, 5), 64 ** -0.5, 0))


@pytest.mark.parametrize("window", [0, 300])
def test_a_long_prompt_among_short_ones(window):
    """Items of very different lengths: the runs are cut inside long ones and hold many
    short ones."""
    new, total = [1100, 17, 40, 1, 300, 18], [1500, 17, 45, 900, 300, 2000]
    s = _state(new, total, 8, 2, 128, 32, 9)
    _check(_go(s, window=window), _ref(s, 128 ** -0.5, window))
