"""Values at the ends of the ranges that the KV-cache operators take."""
import numpy as np
import pytest
import torch

import kv_ref
import nvfp4_block_scaled_02_gb300 as nv
from test_gpu_qk_rope import _inputs, _np

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_norm_gradient_of_tiny_heads_without_eps(D, il):
    """Heads of values +-2^-65 with eps 0: r = 2^65, whose square is past fp32, but the
    gradient r (w u - x r^2 mean(w u x)) is not. Every term in it is at most |r| (|w u| +
    mean |w u|), exact products apart from 16 roundings; the result is rounded to bf16."""
    q, k, pos, cs, qw, kw, gq, gk = _inputs(5, 3, 1, D, D, seed=D, packed=False)
    q, k = (torch.sign(x.float()).mul(2.0 ** -65).to(torch.bfloat16) for x in (q, k))
    got = nv.nvfp4_qk_norm_rope_bwd(gq, gk, q, k, pos, cs, qw, kw, eps=0.0, interleaved=il)
    c = _np(cs)[_np(pos).astype(int)]
    for name, x, w, gy in (("q", q, qw, gq), ("k", k, kw, gk)):
        gx, gw = kv_ref.norm_rope_bwd(_np(gy), _np(x), _np(w), c, 0.0, il)
        u = np.abs(kv_ref.norm_rope_bwd(_np(gy), _np(x), None, c, 0.0, il)[0]) * np.abs(_np(w))
        size = 2.0 ** 65 * (u + u.mean(-1, keepdims=True) + np.abs(_np(gy)).max())
        tol = 2.0 ** -20 * size
        err = np.abs(_np(got["g" + name]) - gx)
        assert (err <= tol + kv_ref.half_ulp_bf16(np.abs(gx) + tol)).all(), name
        # 15 or 5 rows and the roundings of a term
        assert (np.abs(_np(got[f"g{name}_weight"]) - gw) <= 2.0 ** -19 * np.abs(_np(gy)).max()
                * 2 * gy.shape[0] * gy.shape[1]).all(), name
