"""Rows quantised into the paged cache: byte for byte the oracle's row encoding
of each head (one slice per head), at the slot the map names, and no other byte
of the cache touched."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_02_gb300 as nv
from helpers import host_u16

pytestmark = pytest.mark.gpu


def _rows(T, H, D, seed):
    r = np.random.default_rng(seed)
    x = r.standard_normal((T, 3 * H * D)) * np.exp(r.standard_normal((T, 1)))
    x[r.random(x.shape) < 0.02] *= 20
    x[r.random((T, 1)).repeat(x.shape[1], 1) < 0.1] = 0
    t = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).cuda()
    return [t[:, i * H * D:(i + 1) * H * D].unflatten(1, (H, D)) for i in (1, 2)]


def _cache(pages, P, H, D, fos, seed):
    r = np.random.default_rng(seed)
    am = [torch.from_numpy(r.uniform(1, 9, H).astype(np.float32)).cuda() for _ in range(2)]
    c = nv.alloc_kv_cache(pages, P, H, D, am[0], am[1], four_over_six=fos)
    for n in ("k", "v"):
        for w in ("_codes", "_scales"):
            c[n + w].fill_(0xA5)
    return c


@pytest.mark.parametrize("fos", [False, True])
@pytest.mark.parametrize("T,H,D,P", [(1, 1, 64, 16), (1, 8, 128, 16), (5, 3, 64, 48), (48, 8, 128, 64),
                                     (333, 2, 128, 16), (200, 5, 64, 32)])
def test_matches_the_oracle(orc, T, H, D, P, fos):
    k, v = _rows(T, H, D, seed=T)
    pages = T // P + 3
    c = _cache(pages, P, H, D, fos, seed=T + 1)
    slots = np.random.default_rng(T).permutation(pages * P)[:T].astype(np.int64)
    skip = np.random.default_rng(T + 5).random(T) < 0.15
    slots[skip] = -1
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = nv.nvfp4_kv_append(c, k, v, torch.from_numpy(slots).cuda(), dequant=True, status=st)
    assert int(st.item()) == 0
    for n, x in (("k", k), ("v", v)):
        bits = host_u16(x.transpose(0, 1).contiguous())  # [H][T][D]
        ref = orc.quantize(bits, c[n + "_amax"].cpu().numpy(), four_over_six=int(fos))
        codes, scales = ref["row_codes"].reshape(H, T, D // 2), ref["row_scales"].reshape(H, T, D // 16)
        wc, wsc = (np.full(c[n + w].shape, 0xA5, np.uint8) for w in ("_codes", "_scales"))
        for t in range(T):
            if slots[t] >= 0:
                wc[slots[t] // P, :, slots[t] % P] = codes[:, t]
                wsc[slots[t] // P, :, slots[t] % P] = scales[:, t]
        assert np.array_equal(c[n + "_codes"].cpu().numpy(), wc)
        assert np.array_equal(c[n + "_scales"].cpu().numpy(), wsc)
        dq = host_u16(got[n].transpose(0, 1).contiguous()).reshape(-1)
        assert np.array_equal(dq & 0x7FFF, ref["row_dq"].reshape(-1) & 0x7FFF)


def test_contiguous_rows_and_no_dequant():
    k, v = _rows(20, 4, 64, seed=3)
    slots = torch.arange(20, device="cuda") + 7
    a, b = _cache(3, 16, 4, 64, False, 1), _cache(3, 16, 4, 64, False, 1)
    assert nv.nvfp4_kv_append(a, k, v, slots) == {"k": None, "v": None}
    nv.nvfp4_kv_append(b, k.contiguous(), v.contiguous(), slots, dequant=True)
    for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert torch.equal(a[n], b[n])


def test_data_errors():
    k, v = (x.contiguous() for x in _rows(4, 2, 64, seed=4))
    slots = torch.arange(4, device="cuda")

    def status(c, k, v, slots):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        nv.nvfp4_kv_append(c, k, v, slots, status=st)
        return int(st.item())
    c = _cache(2, 16, 2, 64, False, 2)
    before = c["k_codes"].clone()
    assert status(c, k, v, torch.tensor([32, -2, 1 << 40, -1], device="cuda")) == nv.DEV_BAD_INDEX
    assert torch.equal(before, c["k_codes"])
    for x in (float("nan"), float("inf")):
        bad = v.clone()
        bad[2, 1, 9] = x
        assert status(c, k, bad, slots) == nv.DEV_NONFINITE_INPUT
    c["v_amax"][1] = float("inf")
    assert status(c, k, v, slots) == nv.DEV_BAD_AMAX
