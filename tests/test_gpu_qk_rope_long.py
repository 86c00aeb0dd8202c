"""Head norms with rotation over many tokens, where a warp takes several heads of a token
one after the other (weights and angles kept from the first, an uneven last step), in
both directions.

Bounds of the outputs: as in test_gpu_qk_rope.py. Weight gradients: a term u x r carries
at most 16 roundings of 2^-24 of its pair's magnitudes (two products of the rotation, the
mean of D squares in a tree, rsqrt, the products); a lane adds a run of them one after the
other (a warp's tasks and their steps), then two to four values side by side in the
warp, 16 warps, up to 19 CTAs of a group and 8 or 16 groups. The error is at most (16 + the number of
additions) x 2^-24 of the sum of the magnitudes."""
import numpy as np
import pytest
import torch

import kv_ref
import nvfp4_block_scaled_02_gb300 as nv
from test_gpu_qk_rope import EPS, _close, _inputs, _np, _pair_size

pytestmark = pytest.mark.gpu

# 4 steps of 15 + 5 heads of 128 (the last of 8 and of 3 with a head missing), 6 and 2 steps of 21 + 7
# heads of 64, 16 and 4 steps of 32 + 8 heads (gradient: at most 8 in a task), queries alone
SHAPES = [(4099, 15, 5, 128, 128), (9733, 21, 7, 64, 32), (5003, 32, 8, 128, 128),
          (4801, 37, 0, 64, 64)]


@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("norm", ["qk", ""])
@pytest.mark.parametrize("T,hq,hk,D,R", SHAPES)
def test_forward(T, hq, hk, D, R, norm, il):
    q, k, pos, cs, qw, kw, _, _ = _inputs(T, hq, hk, D, R, seed=T + hq, norm=norm)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = nv.nvfp4_qk_norm_rope(q, k, pos, cs, qw, kw, eps=EPS, interleaved=il, status=st)
    c = _np(cs)[_np(pos).astype(int)]
    unit = np.tile(np.r_[np.ones(R // 2), np.zeros(R // 2)], (T, 1))
    for name, x, w in (("q", q, qw), ("k", k, kw)):
        if x.shape[1] == 0:
            continue
        plain = kv_ref.norm_rope(_np(x), _np(w), unit, EPS, il)
        want = kv_ref.norm_rope(_np(x), _np(w), c, EPS, il)
        _close(got[name], want, _pair_size(plain, R, il), name)
    assert int(st.item()) == 0


@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("norm", ["qk", "k"])
@pytest.mark.parametrize("T,hq,hk,D,R", SHAPES)
def test_gradient(T, hq, hk, D, R, norm, il):
    q, k, pos, cs, qw, kw, gq, gk = _inputs(T, hq, hk, D, R, seed=T + hk, norm=norm)
    got = nv.nvfp4_qk_norm_rope_bwd(gq, gk, q, k, pos, cs, qw, kw, eps=EPS, interleaved=il)
    again = nv.nvfp4_qk_norm_rope_bwd(gq, gk, q, k, pos, cs, qw, kw, eps=EPS, interleaved=il)
    c = _np(cs)[_np(pos).astype(int)]
    warps = 16 * torch.cuda.get_device_properties(0).multi_processor_count
    side = 32 // (D // 8)  # heads side by side in a warp
    for name, x, w, gy in (("q", q, qw, gq), ("k", k, kw, gk)):
        if x.shape[1] == 0:
            continue
        steps = -(-x.shape[1] // side)
        x, w, gy = _np(x), _np(w), _np(gy)
        gx, gw = kv_ref.norm_rope_bwd(gy, x, w, c, EPS, il)
        size = _pair_size(gy, R, il)
        if w is not None:  # r (|w u| + |x| r^2 mean |w u x|): the terms before they cancel
            r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + EPS)
            run = (-(-T * -(-steps // 8) // warps) + 1) * 8  # tasks of at most 8 steps a warp
            adds = run + side + 16 + 19 + 16
            tol = (16 + adds) * 2.0 ** -24 * np.abs(size * x * r).sum((0, 1)) + 1e-38
            assert (np.abs(_np(got[f"g{name}_weight"]) - gw) <= tol).all(), name
            wu = np.abs(w) * size
            size = r * (wu + np.abs(x) * r * r * (wu * np.abs(x)).mean(-1, keepdims=True))
        _close(got["g" + name], gx, size, name)
    for n in got:
        assert (got[n] is None) == (again[n] is None)
        assert got[n] is None or torch.equal(got[n], again[n]), n
