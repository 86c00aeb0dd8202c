"""Plain forms in 64 bits of the quantised linear layer's operators, and the bounds that
follow from their arithmetic."""
import numpy as np
import torch

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def fp4_values(codes, scales, amax, M=448.0):
    """fp64 values of an NVFP4 row encoding [..., rows, cols/2]; amax broadcasts over its rows."""
    lut = torch.tensor(E2M1 + tuple(-m for m in E2M1), dtype=torch.float64, device=codes.device)
    x = torch.stack([lut[(codes & 15).long()], lut[(codes >> 4).long()]], -1).flatten(-2)
    amax = amax.double()
    g = torch.where(amax > 0, amax / (6 * M), torch.ones_like(amax))[..., None]
    d = scales.view(torch.float8_e4m3fn).double() * g
    return x * d.repeat_interleave(16, -1)


def mx_values(codes, scales):
    e = scales.double() - 127
    return codes.view(torch.float8_e4m3fn).double() * torch.exp2(e).repeat_interleave(32, -1)


def product_bound(a, b, ref, fp32_out=False):
    """|error| of a product a @ b.T of the tensor cores: every step of 32 or 64 values adds its
    exact products to the sum in fp32 arithmetic, which cuts at most 2^-22 of the magnitudes'
    sum (a rounding toward zero of the largest term's 24 bits, in the step and in the sum); the
    outer scales are two roundings of 2^-24 and their own, bf16 half a step of 2^-8."""
    size = a.abs() @ b.abs().T
    steps = a.shape[1] / 32 + 2
    return size * steps * 2.0 ** -22 + ref.abs() * (2.0 ** -21 if fp32_out else 2.0 ** -8 * 1.001)


def ragged(rng, groups, rows, empty=0.2, unit=1):
    """Rows of each group, some without any; their sum is `rows` (in units)."""
    w = rng.random(groups) ** 2
    w[rng.random(groups) < empty] = 0
    if w.sum() == 0:
        w[-1] = 1
    edge = np.floor(np.cumsum(w) / w.sum() * (rows // unit) + 0.5).astype(np.int64)
    edge[-1] = rows // unit
    return np.diff(edge, prepend=0) * unit
