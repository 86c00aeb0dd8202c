"""Values at the ends of the ranges that the KV-cache operators take."""
import numpy as np
import pytest
import torch

import kv_ref
import nvfp4_block_scaled_02_gb300 as nv
import test_gpu_kv_attn as plain
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


@pytest.mark.parametrize("new,total", [([1, 2], [700, 12000]), ([40], [700]), ([30], [12000])])
@pytest.mark.parametrize("size", [2.0 ** e for e in (8, 10, 12, 13)])
def test_large_scores(new, total, size):
    """Scores of up to 2^21, where fp32 holds them to a quarter: the rows are nearly one key's V.
    The bounds of test_gpu_kv_attn.py allow for the scores' error, which is above 1 here, so
    that the output is only held to the range of the values: a mean of them, rounded to bf16
    (and the probabilities to f16)."""
    s = plain._state(new, total, 8, 2, 128, 64, seed=int(np.log2(size)), q_size=size)
    got = nv.nvfp4_kv_attention(*plain._dev(s), scale=0.5)
    _, lse, _, a, _ = plain._ref(s, 0.5, 0)
    assert np.abs(lse).max() < 2.0 ** 21
    o, z = got["out"].double().cpu().numpy(), got["lse"].double().cpu().numpy()
    assert (np.abs(z - lse) <= 2.0 ** -18 * a + 2.0 ** -19 + 2.0 ** -22 * np.abs(lse)).all()
    c = s["cache"]
    for b in range(len(new)):
        pg = s["table"][b, : -(-total[b] // 64)]
        rows = slice(s["q_start"][b], s["q_start"][b + 1])
        for h in range(2):
            v = np.abs(kv_ref.decode(c["v_codes"][pg, h].reshape(-1, 64)[: total[b]],
                                     c["v_scales"][pg, h].reshape(-1, 8)[: total[b]],
                                     float(c["v_amax"][h]) / (6 * 448))).max(0)
            assert (np.abs(o[rows, 4 * h: 4 * h + 4]) <= v * (1 + 2.0 ** -7)).all(), (b, h)
