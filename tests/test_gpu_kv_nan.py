"""NaN scale bytes in the NVFP4 cache matter to the rows that see their key and to no
other: a key in front of a row's window, or after its position, must not reach the row,
not even as 0 x NaN. A row that sees a key with a NaN V scale has NaN in the 16 values
of that block and numbers elsewhere; one that sees a NaN K scale has NaN everywhere.

The numbers are held to the bounds of test_gpu_kv_attn.py (derived there)."""
import numpy as np
import pytest
import torch

import kv_ref
import nvfp4_block_scaled_02_gb300 as nv
import test_gpu_kv_attn as plain

pytestmark = pytest.mark.gpu

NAN = (0x7F, 0xFF)


def _spoil(s, name, marks):
    """Scale byte of (request, position, head, block) of K or V to NaN."""
    for i, (b, pos, h, block) in enumerate(marks):
        s["cache"][name + "_scales"][s["table"][b, pos // s["P"]], h, pos % s["P"], block] = NAN[i % 2]


def _seen(s, b, pos, window):
    """Which rows of request b see the key."""
    n, L = int(s["new"][b]), int(s["total"][b])
    at = np.arange(n) + L - n
    return (pos <= at) & ((pos > at - window) if window else True)


def _want(s, scale, window, k_marks, v_marks):
    """The 64-bit result without the NaN blocks, and where NaN has to stand."""
    clean = dict(s, cache=dict(s["cache"]))
    for name, marks in (("k", k_marks), ("v", v_marks)):
        sc = clean["cache"][name + "_scales"] = s["cache"][name + "_scales"].copy()
        for b, pos, h, block in marks:
            sc[s["table"][b, pos // s["P"]], h, pos % s["P"], block] = 0
    want = plain._ref(clean, scale, window)
    G, nan_out = s["q"].shape[1] // s["hk"], np.zeros(want[0].shape, bool)
    nan_lse = np.zeros(want[1].shape, bool)
    for marks, every in ((k_marks, True), (v_marks, False)):
        for b, pos, h, block in marks:
            rows = np.flatnonzero(_seen(s, b, pos, window)) + int(s["q_start"][b])
            heads = slice(h * G, (h + 1) * G)
            nan_out[rows, heads, slice(None) if every else slice(16 * block, 16 * block + 16)] = True
            if every:
                nan_lse[rows, heads] = True
    return want, nan_out, nan_lse


def _test(s, window, k_marks, v_marks):
    scale = s["D"] ** -0.5
    _spoil(s, "k", k_marks)
    _spoil(s, "v", v_marks)
    (out, lse, absv, size, allv), nan_out, nan_lse = _want(s, scale, window, k_marks, v_marks)
    got = plain._go(s, scale=scale, window=window)
    o, z = got["out"].double().cpu().numpy(), got["lse"].double().cpu().numpy()
    assert np.array_equal(np.isnan(o), nan_out), (
        f"{(np.isnan(o) & ~nan_out).sum()} values are NaN that should be numbers, "
        f"{(~np.isnan(o) & nan_out).sum()} the other way round")
    assert np.array_equal(np.isnan(z), nan_lse)
    # the numbers, where a row has them
    o, z = np.where(nan_out, out, o), np.where(nan_lse, lse, z)
    plain._check({"out": torch.from_numpy(o), "lse": torch.from_numpy(z)},
                 (out, lse, absv, size, allv))


SHAPES = [  # new, total, q_heads, kv_heads, D, P
    ([1, 3, 1], [700, 333, 40], 8, 2, 128, 16), ([5, 1], [700, 900], 7, 7, 64, 32),
    ([4, 2], [4, 1000], 16, 4, 128, 64), ([40], [100], 3, 1, 64, 16),
    ([300, 1], [1500, 900], 8, 2, 64, 32), ([257, 5], [300, 900], 4, 1, 128, 64),
    ([129, 128], [600, 128], 6, 2, 128, 128), ([600], [4000], 4, 2, 128, 64),
    ([2], [20000], 8, 2, 128, 64),
]


@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("window", [1, 20, 300])
def test_in_front_of_every_window(shape, window):
    """Every key that no row sees is NaN, in K and in V: nothing changes."""
    new, total, hq, hk, D, P = SHAPES[shape]
    s = plain._state(new, total, hq, hk, D, P, seed=shape)
    marks = []
    for b in range(len(new)):
        lowest = max(0, total[b] - new[b] + 1 - window)
        marks += [(b, pos, h, (pos + h) % (D // 16)) for pos in range(lowest) for h in range(hk)]
    _spoil(s, "k", marks)
    _spoil(s, "v", marks)
    got = plain._go(s, window=window)
    for n in ("k", "v"):
        sc = s["cache"][n + "_scales"]
        sc[(sc & 0x7F) == 0x7F] = 0
    plain._check(got, plain._ref(s, D ** -0.5, window))


@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("window", [0, 1, 20, 300])
def test_seen_by_some_rows(shape, window):
    """A few NaN blocks of V among the newest tokens and behind them: rows before
    such a token, rows whose window has passed it and rows that see it."""
    new, total, hq, hk, D, P = SHAPES[shape]
    s = plain._state(new, total, hq, hk, D, P, seed=20 + shape)
    r = np.random.default_rng(shape)
    marks = []
    for b in range(len(new)):
        lowest = max(0, total[b] - new[b] - 30)
        for pos in {total[b] - 1, lowest, *r.integers(lowest, total[b], 3).tolist()}:
            marks.append((b, int(pos), int(r.integers(hk)), int(r.integers(D // 16))))
    _test(s, window, [], marks)


@pytest.mark.parametrize("shape", [0, 2, 3, 4, 5, 7])
@pytest.mark.parametrize("window", [0, 20])
def test_in_keys_and_values(shape, window):
    new, total, hq, hk, D, P = SHAPES[shape]
    s = plain._state(new, total, hq, hk, D, P, seed=40 + shape)
    b = int(np.argmax(new))
    last = total[b] - 1
    mid = total[b] - (new[b] + 1) // 2
    _test(s, window, [(b, mid, 0, 1)], [(b, last, hk - 1, D // 16 - 1), (b, max(0, mid - 40), 0, 0)])


@pytest.mark.parametrize("new", [1, 30])
def test_a_part_with_a_vanishing_weight(new):
    """The NaN lies in a part of the keys (another CTA's) whose weight in the whole
    is 0 in 32 bits: the formula still gives NaN."""
    D, P, L = 128, 64, 12000
    s = plain._state([new], [L], 8, 1, D, P, seed=60 + new)
    pg = s["table"][0, : -(-L // P)]
    s["cache"]["k_scales"][pg, 0] = 0x38       # 1
    s["cache"]["k_codes"][pg, 0] = 0x22        # 1
    s["cache"]["k_codes"][pg[:2], 0] = 0x77    # 6: the first 128 keys
    s["cache"]["k_amax"][:] = 6 * 448
    s["q"] = torch.full_like(s["q"], 4.0)      # scores of 45 and 271: a weight of 2^-326
    _test(s, 0, [], [(0, L - new - 200, 0, 3)])


def test_a_token_appended_with_nan_leaves_with_the_window():
    """A V row with a NaN goes into the cache (and is flagged): rows see it until their
    window has passed it, and never before its position."""
    H, D, P, T, W = 2, 128, 16, 90, 24
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v, q = (torch.randn((T, H, D), generator=g, device="cuda", dtype=torch.bfloat16)
               for _ in range(3))
    amax = torch.full((H,), 6.0, device="cuda")
    caches, at = [], 37
    for bad in (False, True):
        x = v.clone()
        x[at, 1, 20] = float("nan") if bad else 0.0
        c = nv.alloc_kv_cache(6, P, H, D, amax, amax)
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        nv.nvfp4_kv_append(c, k, x, torch.arange(T, device="cuda"), status=st)
        assert int(st.item()) == (nv.DEV_NONFINITE_INPUT if bad else 0)
        caches.append(c)
    table = torch.arange(6, dtype=torch.int32, device="cuda")[None]

    def attend(c, first, last):
        i32 = dict(dtype=torch.int32, device="cuda")
        return nv.nvfp4_kv_attention(q[first:last], c, table, torch.tensor([last], **i32),
                                     torch.tensor([0, last - first], **i32), last - first,
                                     window=W)["out"]
    for first, last in ((0, T), (0, 40), *((i, i + 1) for i in range(30, 70)),
                        *((i, i + 4) for i in range(30, 70, 3))):
        want, got = attend(caches[0], first, last), attend(caches[1], first, last)
        row = torch.arange(first, last)
        sees = (row >= at) & (row < at + W)
        assert torch.isnan(got[sees][:, 1, 16:32]).all()
        got, want = got.clone(), want.clone()
        got[sees, 1, 16:32] = want[sees, 1, 16:32] = 0
        assert torch.equal(got, want), (first, last)


@pytest.mark.parametrize("new", [1, 2, 30])
@pytest.mark.parametrize("total", [60, 12000])
@pytest.mark.parametrize("what", ["every key", "a query"])
def test_rows_whose_scores_are_all_nan(new, total, what):
    """NaN, not the 0 and -infinity of a row that sees no key, in one CTA and where
    several share the keys."""
    s = plain._state([new, 1], [total, 50], 8, 2, 128, 64, seed=total + new)
    if what == "every key":
        pg = s["table"][0, : -(-total // 64)]
        s["cache"]["k_scales"][pg, 1] = 0x7F
        rows, heads = slice(0, new), slice(4, 8)
    else:
        s["q"][new - 1, 5, 77] = float("nan")
        rows, heads = slice(new - 1, new), slice(5, 6)
    got = nv.nvfp4_kv_attention(*plain._dev(s))
    o, z = got["out"].float().cpu(), got["lse"].cpu()
    assert torch.isnan(o[rows, heads]).all() and torch.isnan(z[rows, heads]).all()
    o[rows, heads], z[rows, heads] = 0, 0
    assert torch.isfinite(o).all() and torch.isfinite(z).all()
