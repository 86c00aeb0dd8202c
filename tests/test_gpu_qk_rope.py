"""Head norms with rotation and their gradient against 64-bit forms.

Bounds. An output is rounded to bf16 once (half an ulp); before that it is a sum
of two products of values that carry a few fp32 roundings each (the mean's sum
of D squares in a tree, rsqrt within 2 ulp, three products): below 2^-19 of the
pair's magnitudes. The weight gradient adds N terms in fp32 in trees and short
runs: 2^-20 of the sum of magnitudes for the N used here (runs of at most 64,
then trees)."""
import numpy as np
import pytest
import torch

import kv_ref
import nvfp4_block_scaled_02_gb300 as nv

pytestmark = pytest.mark.gpu
EPS = 1e-6


def _bf16(a):
    return torch.from_numpy(np.asarray(a, np.float32)).to(torch.bfloat16)


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _inputs(T, hq, hk, D, R, seed, norm="qk", packed=True):
    r = np.random.default_rng(seed)
    qkv = _bf16(r.standard_normal((T, (hq + 2 * hk) * D)) * 3).cuda()
    q, k = qkv[:, : hq * D].unflatten(1, (hq, D)), qkv[:, hq * D: (hq + hk) * D].unflatten(1, (hk, D))
    if not packed:
        q, k = q.contiguous(), k.contiguous()
    length = 3 * T + 50
    a = np.outer(np.arange(length), 10000.0 ** (-np.arange(0, R, 2) / R))
    cs = torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1)).float().cuda()
    pos = torch.from_numpy(r.integers(0, length, T).astype(np.int32)).cuda()
    w = [_bf16(1 + 0.3 * r.standard_normal(D)).cuda() if n in norm else None for n in "qk"]
    gq, gk = _bf16(r.standard_normal((T, hq, D))).cuda(), _bf16(r.standard_normal((T, hk, D))).cuda()
    return q, k, pos, cs, w[0], w[1], gq, gk


def _pair_size(x, R, il):
    """|a| + |b| of each value's rotated pair."""
    y, a = np.abs(x), np.abs(x).copy()
    if il:
        s = y[..., 0:R:2] + y[..., 1:R:2]
        a[..., 0:R:2], a[..., 1:R:2] = s, s
    else:
        s = y[..., : R // 2] + y[..., R // 2: R]
        a[..., : R // 2], a[..., R // 2: R] = s, s
    return a


def _close(got, want, size, what):
    err = np.abs(_np(got) - want)
    tol = kv_ref.half_ulp_bf16(np.abs(want) + 2.0 ** -19 * size) + 2.0 ** -19 * size
    assert (err <= tol).all(), f"{what}: {np.max(err / tol)} of the bound"


SHAPES = [(1, 1, 0, 64, 64), (1, 0, 1, 128, 128), (1, 32, 8, 128, 128), (3, 5, 1, 64, 32),
          (33, 15, 5, 64, 64), (7, 8, 2, 128, 48), (130, 7, 7, 128, 16), (257, 4, 4, 64, 64),
          (1000, 3, 1, 128, 128), (2049, 2, 1, 64, 16)]


@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("norm", ["qk", "q", "k", ""])
@pytest.mark.parametrize("T,hq,hk,D,R", SHAPES)
def test_forward(T, hq, hk, D, R, norm, il):
    q, k, pos, cs, qw, kw, _, _ = _inputs(T, hq, hk, D, R, seed=T + hq, norm=norm)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = nv.nvfp4_qk_norm_rope(q, k, pos, cs, qw, kw, eps=EPS, interleaved=il, status=st)
    c = _np(cs)[_np(pos).astype(int)]
    for name, x, w in (("q", q, qw), ("k", k, kw)):
        if x.shape[1] == 0:
            continue
        want = kv_ref.norm_rope(_np(x), _np(w), c, EPS, il)
        plain = kv_ref.norm_rope(_np(x), _np(w), np.tile(np.r_[np.ones(R // 2), np.zeros(R // 2)],
                                                         (T, 1)), EPS, il)
        _close(got[name], want, _pair_size(plain, R, il), name)
    assert int(st.item()) == 0


@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("norm", ["qk", "q", "k", ""])
@pytest.mark.parametrize("T,hq,hk,D,R", SHAPES)
def test_gradient(T, hq, hk, D, R, norm, il):
    q, k, pos, cs, qw, kw, gq, gk = _inputs(T, hq, hk, D, R, seed=T + hk, norm=norm)
    ws = nv.qk_norm_rope_workspace("cuda")
    got = nv.nvfp4_qk_norm_rope_bwd(gq, gk, q, k, pos, cs, qw, kw, eps=EPS, interleaved=il,
                                    workspace=ws)
    again = nv.nvfp4_qk_norm_rope_bwd(gq, gk, q, k, pos, cs, qw, kw, eps=EPS, interleaved=il,
                                      workspace=ws)
    c = _np(cs)[_np(pos).astype(int)]
    for name, x, w, gy in (("q", q, qw, gq), ("k", k, kw, gk)):
        if x.shape[1] == 0:
            continue
        x, w, gy = _np(x), _np(w), _np(gy)
        gx, gw = kv_ref.norm_rope_bwd(gy, x, w, c, EPS, il)
        size = _pair_size(gy, R, il)
        if w is not None:  # r (|w u| + |x| r^2 mean |w u x|): the terms before they cancel
            r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + EPS)
            wu = np.abs(w) * size
            size = r * (wu + np.abs(x) * r * r * (wu * np.abs(x)).mean(-1, keepdims=True))
            u = kv_ref.norm_rope_bwd(gy, x, None, c, EPS, il)[0]
            tol = 2.0 ** -20 * np.abs(_pair_size(gy, R, il) * x * r).sum((0, 1)) + 1e-38
            err = np.abs(_np(got[f"g{name}_weight"]) - (u * x * r).sum((0, 1)))
            assert (err <= tol).all() and np.allclose((u * x * r).sum((0, 1)), gw), name
        _close(got["g" + name], gx, size, name)
    for n in got:
        assert (got[n] is None) == (again[n] is None)
        assert got[n] is None or torch.equal(got[n], again[n]), n


@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("D,R", [(64, 64), (128, 64)])
def test_gradient_against_differences(D, R, il):
    """The loss sum(gy * y) of the 64-bit forward, moved by +-h in one input."""
    T, hq, hk = 2, 2, 1
    q, k, pos, cs, qw, kw, gq, gk = _inputs(T, hq, hk, D, R, seed=D + R)
    got = nv.nvfp4_qk_norm_rope_bwd(gq, gk, q, k, pos, cs, qw, kw, eps=EPS, interleaved=il)
    c = _np(cs)[_np(pos).astype(int)]
    h = 1e-5
    for name, x, w, gy in (("q", q, qw, gq), ("k", k, kw, gk)):
        x, w, gy = _np(x), _np(w), _np(gy)

        def loss(x, w):
            return (gy * kv_ref.norm_rope(x, w, c, EPS, il)).sum()

        def slope(a, at, f):
            up, down = a.copy(), a.copy()
            up[at] += h
            down[at] -= h
            return (f(up) - f(down)) / (2 * h)
        gx, gw = _np(got["g" + name]), _np(got[f"g{name}_weight"])
        r = 1 / np.sqrt((x * x).mean(-1) + EPS)
        for at in [(0, 0, 0), (1, 0, 5), (0, x.shape[1] - 1, R // 2), (1, 0, D - 1)]:
            want = slope(x, at, lambda a: loss(a, w))
            # bf16 of the gradient, the formula's own error (above) and the difference's h^2
            tol = 2.0 ** -8 * abs(want) + 2.0 ** -19 * 10 * r[at[:2]] * np.abs(gy).max() + 1e-7
            assert abs(gx[at] - want) <= tol, (name, at)
        for d in (0, R // 2, D - 1):
            want = slope(w, (d,), lambda a: loss(x, a))
            assert abs(gw[d] - want) <= 2.0 ** -18 * np.abs(gy).sum() + 1e-7, (name, d)


def test_in_place_and_contiguous_inputs_give_the_same_bits():
    q, k, pos, cs, qw, kw, _, _ = _inputs(65, 6, 2, 128, 64, seed=1)
    want = nv.nvfp4_qk_norm_rope(q, k, pos, cs, qw, kw)
    c = nv.nvfp4_qk_norm_rope(q.contiguous(), k.contiguous(), pos, cs, qw, kw)
    nv.nvfp4_qk_norm_rope(q, k, pos, cs, qw, kw, q_out=q, k_out=k)
    for n, x in (("q", q), ("k", k)):
        assert torch.equal(want[n], c[n]) and torch.equal(want[n], x)


def test_gradient_in_place_of_the_output_gradients():
    q, k, pos, cs, qw, kw, gq, gk = _inputs(65, 6, 2, 64, 64, seed=2)
    want = nv.nvfp4_qk_norm_rope_bwd(gq, gk, q, k, pos, cs, qw, kw)
    got = nv.nvfp4_qk_norm_rope_bwd(gq, gk, q, k, pos, cs, qw, kw, gq=gq, gk=gk)
    for n in want:
        assert torch.equal(want[n], got[n]), n


def test_zero_heads_and_large_values():
    """A head of zeros stays zero (eps keeps its norm finite); large inputs do
    not overflow where their mean square fits fp32."""
    q, k, pos, cs, qw, kw, gq, gk = _inputs(2, 2, 1, 64, 64, seed=3, packed=False)
    q[0, 1] = 0
    k[1] *= 1e16
    got = nv.nvfp4_qk_norm_rope(q, k, pos, cs, qw, kw, eps=EPS)
    assert (got["q"][0, 1] == 0).all() and torch.isfinite(got["k"]).all()
    b = nv.nvfp4_qk_norm_rope_bwd(gq, gk, q, k, pos, cs, qw, kw, eps=EPS)
    assert all(torch.isfinite(v).all() for v in b.values())


def test_a_position_outside_the_table_is_flagged():
    q, k, pos, cs, qw, kw, _, _ = _inputs(4, 2, 1, 64, 64, seed=5)
    for bad in (-1, cs.shape[0]):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        p = pos.clone()
        p[2] = bad
        nv.nvfp4_qk_norm_rope(q, k, p, cs, qw, kw, status=st)
        assert int(st.item()) == nv.DEV_BAD_INDEX


def test_no_tokens_zero_the_weight_gradients():
    q, k, pos, cs, qw, kw, gq, gk = _inputs(3, 2, 1, 64, 64, seed=6)
    r = nv.nvfp4_qk_norm_rope_bwd(gq[:0], gk[:0], q[:0], k[:0], pos[:0], cs, qw, kw)
    assert (r["gq_weight"] == 0).all() and (r["gk_weight"] == 0).all()
    assert nv.nvfp4_qk_norm_rope(q[:0], k[:0], pos[:0], cs, qw, kw)["q"].shape == (0, 2, 64)
