"""A cache whose byte offsets pass 32 bits (codes of more than 4 GB each for K and V):
rows in its last pages are written and read as in a cache of a few pages, and its first
pages stay as they were."""
import pytest
import torch

import nvfp4_block_scaled_02_gb300 as nv

pytestmark = pytest.mark.gpu

P, HK, HQ, D = 64, 8, 16, 128
FAR = (1 << 32) // (P * HK * D // 2)  # pages that 4 GB of codes hold


@pytest.mark.parametrize("new", [1, 7, 100])
def test_last_pages_of_a_large_cache(new):
    g = torch.Generator(device="cuda").manual_seed(new)
    k, v = (torch.randn((100, HK, D), generator=g, device="cuda", dtype=torch.bfloat16)
            for _ in range(2))
    q = torch.randn((new, HQ, D), generator=g, device="cuda", dtype=torch.bfloat16)
    amax = [x.float().abs().amax((0, 2)) for x in (k, v)]
    slots = torch.arange(100, device="cuda")
    seen = []
    for pages, first in ((4, 2), (FAR + 4, FAR + 2)):
        cache = nv.alloc_kv_cache(pages, P, HK, D, *amax)
        nv.nvfp4_kv_append(cache, k, v, slots + first * P)
        for n in ("k_codes", "v_codes", "k_scales", "v_scales"):
            assert not cache[n][:2].any()
        table = torch.tensor([[first, first + 1]], dtype=torch.int32, device="cuda")
        r = nv.nvfp4_kv_attention(q, cache, table, torch.full((1,), 100, dtype=torch.int32,
                                                              device="cuda"),
                                  torch.tensor([0, new], dtype=torch.int32, device="cuda"), new,
                                  lse=torch.empty((new, HQ), device="cuda"))
        seen.append([cache[n][first:first + 2].clone()
                     for n in ("k_codes", "v_codes", "k_scales", "v_scales")] + [r["out"], r["lse"]])
        del cache
    for a, b in zip(*seen):
        assert a.any() and torch.equal(a, b)
