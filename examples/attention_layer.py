"""The attention of one decoder layer served from an NVFP4 KV cache.

    python examples/attention_layer.py [--requests 8] [--prompt 700] [--steps 32]

Every batch, prompts and single tokens alike, goes through four calls: block
tables and slots from the requests' lengths, norm and rotation of the query and
key heads, the K and V rows into the cache, attention over it. A decode step is
captured in a CUDA graph once and replayed: every length it needs is on the
device and moves on by itself.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import nvfp4_block_scaled_02_gb300 as nv  # noqa: E402


class AttentionLayer:
    """Cache, block table and buffers of one layer for a fixed number of requests."""

    def __init__(self, requests, max_len, q_heads=32, kv_heads=8, head_dim=128, page_size=64,
                 k_amax=8.0, v_amax=8.0, device="cuda"):
        i32 = dict(dtype=torch.int32, device=device)
        cols = -(-max_len // page_size)
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        self.page_size, self.requests = page_size, requests
        amax = [torch.full((kv_heads,), a, dtype=torch.float32, device=device)
                for a in (k_amax, v_amax)]
        self.cache = nv.alloc_kv_cache(requests * cols, page_size, kv_heads, head_dim, *amax)
        self.table = torch.full((requests, cols), -1, **i32)
        self.free = torch.randperm(requests * cols, device=device).to(torch.int32)
        self.free_pages = self.free.clone()
        self.lengths = torch.zeros(requests, **i32)
        self.status = torch.zeros(1, **i32)
        self.workspace = nv.kv_attention_workspace(device)
        self.q_weight, self.k_weight = (torch.ones(head_dim, dtype=torch.bfloat16, device=device)
                                        for _ in range(2))
        f = 10000.0 ** (-torch.arange(0, head_dim, 2, device=device) / head_dim)
        a = torch.arange(max_len, device=device)[:, None] * f
        self.cos_sin = torch.cat([a.cos(), a.sin()], 1).float().contiguous()

    def __call__(self, qkv, new, max_new):
        """qkv: bf16 [tokens, (q_heads + 2 kv_heads) head_dim], the requests' rows one
        after the other; new: int32 [requests], each request's rows (on the device);
        max_new: an upper bound of them. Returns bf16 [tokens, q_heads, head_dim]."""
        d, hq, hk = self.head_dim, self.q_heads, self.kv_heads
        q, k, v = qkv.split([hq * d, hk * d, hk * d], dim=1)
        q, k, v = q.unflatten(1, (hq, d)), k.unflatten(1, (hk, d)), v.unflatten(1, (hk, d))
        plan = nv.nvfp4_kv_plan(self.lengths, new, self.table, self.free_pages, self.page_size,
                                qkv.shape[0], status=self.status)
        r = nv.nvfp4_qk_norm_rope(q, k, plan["positions"], self.cos_sin, self.q_weight,
                                  self.k_weight, status=self.status)
        nv.nvfp4_kv_append(self.cache, r["k"], v, plan["slots"], status=self.status)
        o = nv.nvfp4_kv_attention(r["q"], self.cache, self.table, plan["seq_lens"],
                                  plan["q_start"], max_new, workspace=self.workspace,
                                  status=self.status)
        # the pages taken leave the free list, on the device: no host round trip
        n = self.free_pages.numel()
        at = torch.arange(n, device=qkv.device) + plan["pages_used"]
        self.free_pages.copy_(torch.where(at < n, self.free_pages[at.clamp(max=n - 1)], -1))
        self.lengths.copy_(plan["seq_lens"])
        return o["out"]


def main():
    ap = argparse.ArgumentParser(description=__doc__,
                                 formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=700)
    ap.add_argument("--steps", type=int, default=32)
    a = ap.parse_args()
    torch.manual_seed(0)
    layer = AttentionLayer(a.requests, a.prompt + a.steps + 8)
    width = (layer.q_heads + 2 * layer.kv_heads) * layer.head_dim

    def rows(n):
        return torch.randn(n, width, dtype=torch.bfloat16, device="cuda")

    # prompts of different lengths in one batch
    new = torch.randint(1, a.prompt + 1, (a.requests,), dtype=torch.int32)
    layer(rows(int(new.sum())), new.cuda(), int(new.max()))

    # one token of every request a step, from a graph
    one, x = torch.ones(a.requests, dtype=torch.int32, device="cuda"), rows(a.requests)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(x, one, 1)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(x, one, 1)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(a.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print(f"{a.requests} requests, {int(layer.lengths.sum())} cached tokens, "
          f"{start.elapsed_time(end) / a.steps * 1e3:.1f} us a decode step, "
          f"status {int(layer.status.item())}, output {tuple(out.shape)}")


if __name__ == "__main__":
    main()
