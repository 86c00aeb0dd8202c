"""Appends of many tokens and of wide tokens: several batches per thread with odd
tails, and tokens of more lanes than a block has threads. Bytes as in
test_gpu_kv_append.py (the oracle's), and the de-quantised rows bit for bit, signs
included; only a zero's sign is free (with 4/6 a select by fma can turn -0 into +0)."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_02_gb300 as nv
from helpers import host_u16
from test_gpu_kv_append import _cache, _rows

pytestmark = pytest.mark.gpu


def _signed(bits):
    """bf16 bits with -0 as +0."""
    return np.where(bits & 0x7FFF, bits, 0)


# (T, H, D, P): 8 heads of 128 take 2 tokens at a time, 33 of 64 and 20 of 128 have lanes past
# 256, 1 head of 64 takes 32 tokens at a time. The long ones give a thread several tokens.
@pytest.mark.parametrize("fos", [False, True])
@pytest.mark.parametrize("T,H,D,P", [(5003, 8, 128, 64), (16381, 8, 128, 64), (9731, 33, 64, 16),
                                     (10007, 20, 128, 48), (3, 20, 128, 16), (77, 33, 64, 32),
                                     (80021, 1, 64, 64), (39001, 2, 64, 16)])
def test_matches_the_oracle(orc, T, H, D, P, fos):
    k, v = _rows(T, H, D, seed=T + H)
    pages = T // P + 3
    c = _cache(pages, P, H, D, fos, seed=T + 1)
    r = np.random.default_rng(T)
    slots = r.permutation(pages * P)[:T].astype(np.int64)
    slots[r.random(T) < 0.1] = -1
    at = np.flatnonzero(slots >= 0)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = nv.nvfp4_kv_append(c, k, v, torch.from_numpy(slots).cuda(), dequant=True, status=st)
    assert int(st.item()) == 0
    for n, x in (("k", k), ("v", v)):
        bits = host_u16(x.transpose(0, 1).contiguous())  # [H][T][D]
        ref = orc.quantize(bits, c[n + "_amax"].cpu().numpy(), four_over_six=int(fos))
        for name, want in (("_codes", ref["row_codes"].reshape(H, T, D // 2)),
                           ("_scales", ref["row_scales"].reshape(H, T, D // 16))):
            full = np.full(c[n + name].shape, 0xA5, np.uint8)
            full[slots[at] // P, :, slots[at] % P] = want[:, at].transpose(1, 0, 2)
            assert np.array_equal(c[n + name].cpu().numpy(), full), n + name
        dq = host_u16(got[n].transpose(0, 1).contiguous()).reshape(-1)
        assert np.array_equal(_signed(dq), _signed(ref["row_dq"].reshape(-1))), n


@pytest.mark.parametrize("fos", [False, True])
@pytest.mark.parametrize("T,H,D", [(1, 1, 64), (333, 3, 128), (4001, 8, 128)])
def test_signs_of_the_dequantised_rows(T, H, D, fos):
    """Every value that is not 0 has its input's sign."""
    k, v = _rows(T, H, D, seed=T)
    c = _cache(T // 16 + 1, 16, H, D, fos, seed=5)
    got = nv.nvfp4_kv_append(c, k, v, torch.arange(T, device="cuda"), dequant=True)
    for x, y in ((k, got["k"]), (v, got["v"])):
        assert ((y == 0) | (torch.signbit(x) == torch.signbit(y))).all() and (y != 0).any()
