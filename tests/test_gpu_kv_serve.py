"""The cache operators together: prompts, then single tokens, through the layer of
examples/attention_layer.py, each output against the 64-bit attention over what the
cache then holds; a decode step from a CUDA graph, on another stream, and from two
streams at once."""
import os
import sys

import numpy as np
import pytest
import torch

import kv_ref
import nvfp4_block_scaled_02_gb300 as nv
from conftest import ROOT

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(ROOT, "examples"))

HQ, HK, D, P = 6, 2, 64, 16


def _layer(requests, max_len):
    from attention_layer import AttentionLayer
    torch.manual_seed(requests)
    return AttentionLayer(requests, max_len, q_heads=HQ, kv_heads=HK, head_dim=D, page_size=P)


def _rows(n, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(n, (HQ + 2 * HK) * D, generator=g, device="cuda").to(torch.bfloat16)


def _check(layer, qkv, new, before, out):
    """The layer's output from the queries' 64-bit norm and rotation and the cache."""
    T, total = qkv.shape[0], before + new
    start = np.concatenate([[0], np.cumsum(new)])
    pos = np.concatenate([np.arange(b, b + n) for b, n in zip(before, new)]).astype(int)
    cs = layer.cos_sin.double().cpu().numpy()[pos]
    q = qkv[:, : HQ * D].unflatten(1, (HQ, D)).double().cpu().numpy()
    q = kv_ref.norm_rope(q, np.ones(D), cs, 1e-6, False)
    # the attention call gets the queries in bf16
    q = torch.from_numpy(q).to(torch.bfloat16).double().numpy()
    table = layer.table.cpu().numpy()
    c = {n: t.cpu().numpy() for n, t in layer.cache.items() if isinstance(t, torch.Tensor)}

    def of(n):
        def get(b):
            L = int(total[b])
            pg = table[b, : -(-L // P)]
            assert (pg >= 0).all()
            return np.stack([kv_ref.decode(c[n + "_codes"][pg, h].reshape(-1, D // 2)[:L],
                                           c[n + "_scales"][pg, h].reshape(-1, D // 16)[:L],
                                           float(c[n + "_amax"][h]) / (6 * 448)) for h in range(HK)])
        return get
    want, _, absv, _, allv = kv_ref.attention(q, of("k"), of("v"), start, total, D ** -0.5, 0)
    o = out.double().cpu().numpy()
    # As the attention's own bound, plus a query value that the fp32 norm rounds to the
    # other bf16 neighbour: 2^-8 of it, at most 2^-8 sqrt(D) |k| / sqrt(D) <= 2^-5 of a score
    # for the |k| < 8 here, so a probability off by 2^-5 in the worst row.
    tol = 2.0 ** -5 * 2 * absv + 2.0 ** -31 * allv
    assert (np.abs(o - want) <= tol + kv_ref.half_ulp_bf16(np.abs(want) + tol)).all()
    # and nearly every row far inside it: no row's bf16 queries differ in all values
    rel = np.linalg.norm(o - want) / np.linalg.norm(want)
    assert rel < 2.0 ** -8, rel


def test_prompts_then_single_tokens():
    layer = _layer(5, 300)
    before = np.zeros(5, int)
    for step, new in enumerate(([40, 1, 0, 130, 17], [1, 1, 90, 1, 1], [1] * 5, [3, 0, 2, 1, 5])):
        new = np.array(new)
        qkv = _rows(int(new.sum()), step)
        out = layer(qkv, torch.tensor(new, dtype=torch.int32, device="cuda"), int(new.max()))
        assert int(layer.status.item()) == 0
        _check(layer, qkv, new, before, out)
        before = before + new
        assert layer.lengths.tolist() == before.tolist()
    held = layer.table[layer.table >= 0].tolist()
    assert len(set(held)) == len(held) == int(sum(-(-b // P) for b in before))


def test_decode_steps_from_a_graph_and_on_another_stream():
    layer, same = _layer(3, 200), _layer(3, 200)
    new = torch.tensor([30, 70, 5], dtype=torch.int32, device="cuda")
    one = torch.ones(3, dtype=torch.int32, device="cuda")
    for x in (layer, same):
        x.free_pages.copy_(torch.arange(x.free_pages.numel(), device="cuda", dtype=torch.int32))
        x(_rows(105, 1), new, 70)
    qkv = _rows(3, 2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # another stream than the tensors' own
        first = layer(qkv, one, 1)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first, same(qkv, one, 1))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = layer(qkv, one, 1)
    for seed in range(3, 23):  # past several page boundaries
        x = _rows(3, seed)
        qkv.copy_(x)
        g.replay()
        assert torch.equal(out, same(x, one, 1))
    assert layer.lengths.tolist() == same.lengths.tolist() == [51, 91, 26]
    assert torch.equal(layer.table, same.table) and int(layer.status.item()) == 0


def test_two_streams_with_their_own_workspaces():
    layers = [_layer(4, 400) for _ in range(2)]
    alone = [_layer(4, 400) for _ in range(2)]
    new = torch.tensor([200, 3, 90, 31], dtype=torch.int32, device="cuda")
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    rows = [[_rows(324, 10 * i + j) for j in range(2)] for i in range(2)]
    torch.cuda.synchronize()
    for j in range(2):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(layers[i](rows[i][0], new, 200) if j == 0 else
                              layers[i](rows[i][1][:4], torch.ones_like(new), 1))
    torch.cuda.synchronize()
    for i in range(2):
        want = [alone[i](rows[i][0], new, 200), alone[i](rows[i][1][:4], torch.ones_like(new), 1)]
        for a, b in zip(got[i], want):
            assert torch.equal(a, b)


def test_entry_points_by_keyword():
    q, k = _rows(2, 1)[:, : HQ * D].unflatten(1, (HQ, D)), _rows(2, 1)[:, -HK * D:].unflatten(1, (HK, D))
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    cs = torch.cat([torch.ones(4, 16), torch.zeros(4, 16)], 1).cuda()
    r = nv.nvfp4_qk_norm_rope(q=q, k=k, positions=pos, cos_sin=cs)
    assert torch.equal(r["q"], q) and torch.equal(r["k"], k)  # no weight, angle 0
