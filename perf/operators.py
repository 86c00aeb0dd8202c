"""Performance cases of the attention operators around the NVFP4 KV cache.

Four operators, each with its plain form in elementary torch operations:

- ``plan``: block tables and slot maps of a paged cache, built on the GPU from
  the requests' lengths (``nvfp4_kv_plan``);
- ``rope`` and ``rope_bwd``: RMS norm of every query and key head with the
  position rotation in the same pass, and its gradient
  (``nvfp4_qk_norm_rope``, ``nvfp4_qk_norm_rope_bwd``);
- ``append``: K and V rows quantised into the paged NVFP4 cache
  (``nvfp4_kv_append``);
- ``attend``: attention over that cache, for single tokens, a few tokens per
  request and whole prompts (``nvfp4_kv_attention``).

``own`` chooses the path that ``run`` takes: the plain forms or the library.
"""
import math

import numpy as np
import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
FP8_MAX = 448.0
EPS = 1e-6


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one decode step of a small server: 64 running requests, one new token each
        dict(name="plan decode 64", op="plan", requests=64, page=16, new_lo=1, new_hi=1,
             cached_hi=8000),
        # chunked prompts and single tokens scheduled together on a large server
        dict(name="plan mixed 1500", op="plan", requests=1500, page=64, new_lo=1, new_hi=1024,
             cached_hi=30000),
        # the projections of one decode step of 32 requests
        dict(name="rope decode 32", op="rope", tokens=32, q_heads=32, kv_heads=8, dim=128,
             rotary=128, interleaved=False, norm=True),
        # a prompt (or a training step's forward) of 8192 tokens, hidden size 4096
        dict(name="rope prompt 8192", op="rope", tokens=8192, q_heads=32, kv_heads=8, dim=128,
             rotary=128, interleaved=False, norm=True),
        # the gradient of that step
        dict(name="rope_bwd train 8192", op="rope_bwd", tokens=8192, q_heads=32, kv_heads=8,
             dim=128, rotary=128, interleaved=False, norm=True),
        # a short odd sequence with a partial interleaved rotation of narrow heads
        dict(name="rope_bwd odd 1021", op="rope_bwd", tokens=1021, q_heads=15, kv_heads=5, dim=64,
             rotary=32, interleaved=True, norm=True),
        # one token of each of 48 requests into the cache
        dict(name="append decode 48", op="append", tokens=48, kv_heads=8, dim=128, page=16,
             q_heads=32),
        # a prompt of 16381 tokens into the cache
        dict(name="append prompt 16381", op="append", tokens=16381, kv_heads=8, dim=128, page=64,
             q_heads=32),
        # latency: four short conversations, one token each
        dict(name="attend decode 4", op="attend", requests=4, idle=0, new_lo=1, new_hi=1,
             len_lo=300, len_hi=1100, q_heads=32, kv_heads=8, dim=128, page=16, window=0),
        # throughput: 64 ragged conversations up to 32768 tokens, and two idle places of the batch
        dict(name="attend decode 64 long", op="attend", requests=64, idle=2, new_lo=1, new_hi=1,
             len_lo=1000, len_hi=32768, q_heads=32, kv_heads=8, dim=128, page=64, window=0),
        # a few drafted tokens per request, narrow heads, a sliding window
        dict(name="attend draft window", op="attend", requests=24, idle=1, new_lo=2, new_hi=5,
             len_lo=40, len_hi=9001, q_heads=21, kv_heads=7, dim=64, page=32, window=1000),
        # chunks of prompts behind cached prefixes
        dict(name="attend prompt 4x2048", op="attend", requests=4, idle=0, new_lo=1500,
             new_hi=2048, len_lo=3000, len_hi=10000, q_heads=32, kv_heads=8, dim=128, page=64,
             window=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "rope", "rope_bwd", "append", "attend", "attend", "attend"])
    if op == "plan":
        return dict(op=op, requests=_log(rng, 1, 1500), page=rng.choice([16, 32, 64, 128]),
                    new_lo=1, new_hi=_log(rng, 1, 1000), cached_hi=_log(rng, 1, 30000))
    dim = rng.choice([64, 128])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8])
    kv = rng.choice([1, 2, 3, 4, 5, 8])
    if op in ("rope", "rope_bwd"):
        return dict(op=op, tokens=_log(rng, 1, 8000), q_heads=kv * group if kv < 8 else 32,
                    kv_heads=kv, dim=dim, rotary=rng.choice([32, dim]),
                    interleaved=rng.random() < 0.5, norm=rng.random() < 0.75)
    if op == "append":
        return dict(op=op, tokens=_log(rng, 1, 16000), kv_heads=kv, dim=dim,
                    page=rng.choice([16, 32, 64, 128]), q_heads=kv * group)
    kind = rng.choice(["one", "few", "prompt"])
    page = rng.choice([16, 32, 64, 128])
    window = rng.choice([0, 0, _log(rng, 1, 4000)])
    if kind == "prompt":
        hi = _log(rng, 17, 1500)
        return dict(op="attend", requests=rng.randint(1, 4), idle=0, new_lo=rng.randint(1, hi),
                    new_hi=hi, len_lo=hi, len_hi=hi + _log(rng, 1, 8000), q_heads=kv * min(group, 4),
                    kv_heads=kv, dim=dim, page=page, window=window)
    hi = 1 if kind == "one" else rng.randint(2, 8)
    length = _log(rng, 16, 32000)
    requests = _log(rng, 1, max(2, min(64, 400000 // length)))
    return dict(op="attend", requests=requests, idle=rng.randint(0, 2), new_lo=1, new_hi=hi,
                len_lo=max(1, length // rng.randint(1, 20)), len_hi=length, q_heads=kv * group,
                kv_heads=kv, dim=dim, page=page, window=window)


def _spread(n, lo, hi):
    """n lengths from lo to hi, even on their logarithm: a case's lengths are
    the same whatever the seed (the seed gives their order)."""
    at = (np.arange(n) + 0.5) / max(n, 1)
    return np.clip(np.round(lo * (hi / lo) ** at), lo, hi).astype(np.int64)


def _lengths(case):
    """(new tokens, total length) of every request of an `attend` case."""
    n, idle = case["requests"], case["idle"]
    new, total = _spread(n, case["new_lo"], case["new_hi"]), _spread(n, case["len_lo"], case["len_hi"])
    total = np.maximum(total, new)
    # an idle place of the batch: one query row, an empty cache
    return np.concatenate([new, np.ones(idle, np.int64)]), np.concatenate(
        [total, np.zeros(idle, np.int64)])


def _plan_lengths(case):
    n = case["requests"]
    new = _spread(n, case["new_lo"], case["new_hi"])
    cached = _spread(n, 1, case["cached_hi"])
    return np.roll(cached, n // 3), new


def work(case):
    op = case["op"]
    if op == "plan":
        cached, new = _plan_lengths(case)
        P = case["page"]
        pages = (-(-(cached + new) // P) - -(-cached // P)).sum()
        # lengths read; totals, row starts written; per token a slot and a position; per page
        # the free page read and the table entry written; a partly filled last page read
        return dict(bytes=float(16 * len(new) + 12 * new.sum() + 8 * pages
                                + 4 * (cached % P != 0).sum()),
                    flops=float(new.sum()))
    D = case["dim"]
    if op in ("rope", "rope_bwd"):
        T, n = case["tokens"], case["q_heads"] + case["kv_heads"]
        values = T * n * D
        side = T * (case["rotary"] * 4 + 4)
        if op == "rope":
            return dict(bytes=float(4 * values + side), flops=float(10 * values))
        return dict(bytes=float(6 * values + side + 8 * D), flops=float(20 * values))
    if op == "append":
        values = 2 * case["tokens"] * case["kv_heads"] * D
        return dict(bytes=float(values * (2 + 0.5 + 1 / 16 + 2) + 8 * case["tokens"]),
                    flops=float(6 * values))
    new, total = _lengths(case)
    W = case["window"]
    seen = 0
    read = 0
    for n, t in zip(new.tolist(), total.tolist()):
        last = np.arange(t - n, t, dtype=np.int64)  # positions of the query rows
        keys = last + 1 if W == 0 else np.minimum(last + 1, W)
        seen += int(np.maximum(keys, 0).sum())
        read += t if W == 0 else max(0, min(t, n - 1 + W))
    rows = int(new.sum()) * case["q_heads"]
    return dict(bytes=float(read * case["kv_heads"] * D * 1.125 + rows * (4 * D + 4)
                            + 4 * (total // case["page"]).sum()),
                flops=float(4 * D * case["q_heads"] * seen))


# ----------------------------------------------------------------- inputs --

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed & 0x7FFFFFFF)
    return g


def _heads(g, tokens, heads, dim):
    """Activations of projection outputs: normal, every head with its own size."""
    size = torch.exp(0.5 * torch.randn(heads, 1, generator=g, device="cuda"))
    return torch.randn(tokens, heads, dim, generator=g, device="cuda") * size


def _packed(g, case):
    """q, k, v as strided views of one projection's output [tokens, (q + 2 kv) * dim]."""
    T, hq, hk, D = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]
    qkv = _heads(g, T, hq + 2 * hk, D).to(torch.bfloat16).view(T, -1)
    q, k, v = qkv.split([hq * D, hk * D, hk * D], dim=1)
    return q.unflatten(1, (hq, D)), k.unflatten(1, (hk, D)), v.unflatten(1, (hk, D))


def _cos_sin(rotary, length):
    f = 10000.0 ** (-torch.arange(0, rotary, 2, dtype=torch.float64, device="cuda") / rotary)
    a = torch.arange(length, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def _encode(x, amax):
    """NVFP4 code bytes, scale bytes and values of x [..., heads, rows, dim] (blocks of 16 along
    the last dimension, the outer scale of each head from amax [heads])."""
    g = (amax / (6 * FP8_MAX))[:, None, None, None]
    b = x.float().unflatten(-1, (-1, 16))
    t = b.abs().amax(-1, keepdim=True) * (1 / (6 * g))
    s8 = t.clamp(max=FP8_MAX).to(torch.float8_e4m3fn)
    d = s8.float() * g
    inv = torch.where(d > 0, 1 / d, torch.zeros_like(d))
    y = b * inv
    a = y.abs()
    # nearest of the eight magnitudes, ties to the even code
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
            + (a >= 3.5) + (a > 5))
    val = torch.tensor(E2M1, device=x.device)[code.int()] * d
    val = torch.where(torch.signbit(y), -val, val).flatten(-2)
    code = (code + 8 * torch.signbit(y).to(torch.uint8)).flatten(-2)
    return code[..., 0::2] + 16 * code[..., 1::2], s8.view(torch.uint8).squeeze(-1), val


def _cache(g, pages, heads, page, dim, fill):
    shape = (pages, heads, page)
    c = {}
    for n in ("k", "v"):
        if fill:
            size = torch.exp(0.5 * torch.randn(heads, 1, dim, generator=g, device="cuda"))
            x = (torch.randn(*shape, dim, generator=g, device="cuda") * size).to(torch.bfloat16)
            c[n + "_amax"] = x.abs().amax((0, 2, 3)).float()
            c[n + "_codes"], c[n + "_scales"], _ = _encode(x, c[n + "_amax"])
        else:
            c[n + "_amax"] = 4 + 4 * torch.rand(heads, generator=g, device="cuda")
            c[n + "_codes"] = torch.zeros(*shape, dim // 2, dtype=torch.uint8, device="cuda")
            c[n + "_scales"] = torch.zeros(*shape, dim // 16, dtype=torch.uint8, device="cuda")
    return {k: v.contiguous() for k, v in c.items()}


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", torch.int32)


def prepare(case, seed):
    g, r = _gen(seed), np.random.default_rng(seed)
    op, s = case["op"], {"case": dict(case), "op": case["op"]}
    if op == "plan":
        cached, new = _plan_lengths(case)
        n, P = case["requests"], case["page"]
        order = r.permutation(n)
        cached, new = cached[order], new[order]
        held, total = -(-cached // P), -(-(cached + new) // P)
        most = int(total.max()) + 3  # a table as wide as its longest request, and some more
        pages = r.permutation(int(held.sum() + (total - held).sum()) + 17)
        table = np.full((n, most), -1, np.int64)
        at = np.arange(most)[None, :] < held[:, None]
        table[at] = pages[: int(held.sum())]
        s.update(cached=_i32(cached), new=_i32(new), table=_i32(table),
                 free=_i32(pages[int(held.sum()):]), page=P, tokens=int(new.sum()))
        return s
    if op in ("rope", "rope_bwd"):
        T, D = case["tokens"], case["dim"]
        length = 2 * T + 100
        s["q"], s["k"], _ = _packed(g, case)
        s["cos_sin"] = _cos_sin(case["rotary"], length)
        start = int(r.integers(0, length - T + 1))
        s["positions"] = torch.arange(start, start + T, dtype=torch.int32, device="cuda")
        w = [(1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16)
             for _ in range(2)]
        s["qw"], s["kw"] = w if case["norm"] else (None, None)
        s["interleaved"] = case["interleaved"]
        if op == "rope_bwd":
            s["gq"] = _heads(g, T, case["q_heads"], D).mul(1e-2).to(torch.bfloat16)
            s["gk"] = _heads(g, T, case["kv_heads"], D).mul(1e-2).to(torch.bfloat16)
        return s
    P, hk, D = case["page"], case["kv_heads"], case["dim"]
    if op == "append":
        T = case["tokens"]
        _, s["k"], s["v"] = _packed(g, case)
        pages = -(-T // P) + 5
        s["cache"] = _cache(g, pages, hk, P, D, fill=False)
        # a prompt's tokens fill whole pages in order, the pages lie anywhere
        order = r.permutation(pages)
        t = np.arange(T) + int(r.integers(0, P))
        s["slots"] = torch.from_numpy(order[t // P] * P + t % P).to("cuda", torch.int64)
        return s
    new, total = _lengths(case)
    order = r.permutation(len(new))
    new, total = new[order], total[order]
    held = -(-total // P)
    pages = int(held.sum()) + 3
    most = max(1, int(held.max()))
    table = np.full((len(new), most), -1, np.int64)
    table[np.arange(most)[None, :] < held[:, None]] = r.permutation(pages)[: int(held.sum())]
    s["cache"] = _cache(g, pages, hk, P, D, fill=True)
    T = int(new.sum())
    s["q"] = torch.randn(T, case["q_heads"], D, generator=g, device="cuda").to(torch.bfloat16)
    s.update(table=_i32(table), seq_lens=_i32(total), max_q=int(new.max()), window=case["window"],
             max_len=max(1, int(total.max())), q_start=_i32(np.concatenate([[0], np.cumsum(new)])),
             scale=1 / math.sqrt(D))
    return s


# ------------------------------------------------------------ plain forms --

def _plain_plan(s):
    P, cached, new = s["page"], s["cached"].long(), s["new"].long()
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    held, total = (cached + P - 1) // P, (cached + new + P - 1) // P
    q_start = torch.cat([zero, new.cumsum(0)])
    p_start = torch.cat([zero, (total - held).cumsum(0)])
    col = torch.arange(s["table"].shape[1], device="cuda")[None, :]
    taken = (p_start[:-1, None] + col - held[:, None]).clamp(0, s["free"].numel() - 1)
    fresh = (col >= held[:, None]) & (col < total[:, None])
    table = torch.where(fresh, s["free"][taken], s["table"])
    t = torch.arange(s["tokens"], device="cuda")
    req = torch.searchsorted(q_start[1:], t, right=True)
    pos = cached[req] + t - q_start[req]
    slots = table[req, pos // P].long() * P + pos % P
    return {"table": table, "seq_lens": (cached + new).int(), "q_start": q_start.int(),
            "slots": slots, "positions": pos.int(), "pages_used": p_start[-1:].int()}


def _pairs(x, rotary, interleaved):
    """The two members of every rotated pair, and what is not rotated."""
    r, rest = x[..., :rotary], x[..., rotary:]
    if interleaved:
        return r[..., 0::2], r[..., 1::2], rest
    return r[..., : rotary // 2], r[..., rotary // 2:], rest


def _unpair(a, b, rest, interleaved):
    r = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([r, rest], -1)


def _cs(s):
    cs = s["cos_sin"][s["positions"].long()][:, None, :]
    h = cs.shape[-1] // 2
    return cs[..., :h], cs[..., h:], 2 * h


def _plain_rope(s):
    c, n, rotary = _cs(s)

    def one(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
        a, b, rest = _pairs(x, rotary, s["interleaved"])
        return _unpair(a * c - b * n, b * c + a * n, rest, s["interleaved"]).to(torch.bfloat16)

    return {"q": one(s["q"], s["qw"]), "k": one(s["k"], s["kw"])}


def _plain_rope_bwd(s):
    c, n, rotary = _cs(s)

    def one(gy, x, w):
        gy, x = gy.float(), x.float()
        a, b, rest = _pairs(gy, rotary, s["interleaved"])
        u = _unpair(a * c + b * n, b * c - a * n, rest, s["interleaved"])
        if w is None:
            return u.to(torch.bfloat16), None
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        wu = u * w.float()
        gx = r * (wu - x * r * r * (wu * x).mean(-1, keepdim=True))
        return gx.to(torch.bfloat16), (u * x * r).sum((0, 1))

    gq, gqw = one(s["gq"], s["q"], s["qw"])
    gk, gkw = one(s["gk"], s["k"], s["kw"])
    return {"gq": gq, "gk": gk, "gq_weight": gqw, "gk_weight": gkw}


def _append_outputs(s, k, v):
    c = s["cache"]
    # what the rows now stand for, and the cache's block scales as the values they are
    return {"k": k, "v": v, "k_scales": c["k_scales"].view(torch.float8_e4m3fn),
            "v_scales": c["v_scales"].view(torch.float8_e4m3fn)}


def _plain_append(s):
    c, P = s["cache"], s["case"]["page"]
    page, off = s["slots"] // P, s["slots"] % P

    def one(x, n):
        codes, scales, val = _encode(x.transpose(0, 1), c[n + "_amax"])
        c[n + "_codes"][page, :, off] = codes.transpose(0, 1)
        c[n + "_scales"][page, :, off] = scales.transpose(0, 1)
        return val.transpose(0, 1).contiguous().to(torch.bfloat16)

    return _append_outputs(s, one(s["k"], "k"), one(s["v"], "v"))


def _plain_attend(s):
    c, P = s["cache"], s["case"]["page"]
    T, hq, D = s["q"].shape
    hk = s["case"]["kv_heads"]
    G, L, N = hq // hk, s["max_len"], s["max_q"]
    key = torch.arange(L, device="cuda")
    page, off = s["table"][:, key // P].clamp(min=0).long(), (key % P)[None, :]
    lut = torch.tensor(E2M1 + tuple(-m for m in E2M1), device="cuda")

    def rows(n):  # [requests, heads, L, D] in 32 bits
        b = c[n + "_codes"][page, :, off]
        x = torch.stack([lut[(b & 15).int()], lut[(b >> 4).int()]], -1).flatten(-2)
        d = c[n + "_scales"].view(torch.float8_e4m3fn)[page, :, off].float()
        d = d * (c[n + "_amax"] / (6 * FP8_MAX))[None, None, :, None]
        return (x.unflatten(-1, (-1, 16)) * d[..., None]).flatten(-2).transpose(1, 2)

    start, length = s["q_start"].long(), s["seq_lens"].long()
    i = torch.arange(N, device="cuda")[None, :]
    tok = (start[:-1, None] + i).clamp(max=T - 1)
    q = s["q"].float()[tok]  # [requests, N, heads, D]
    q = q.unflatten(2, (hk, G)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    score = torch.matmul(q, rows("k").transpose(2, 3)) * s["scale"]
    pos = length[:, None] - (start[1:] - start[:-1])[:, None] + i  # [requests, N]
    seen = (key <= pos[..., None]) & (key < length[:, None, None])
    if s["window"]:
        seen &= key > pos[..., None] - s["window"]
    score = score.unflatten(2, (N, G)).masked_fill(~seen[:, None, :, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), rows("v")).unflatten(2, (N, G))
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (total.log() + top).squeeze(-1)
    t = torch.arange(T, device="cuda")
    req = torch.searchsorted(start[1:], t, right=True)
    at = t - start[req]
    return {"out": o.transpose(1, 2)[req, at].flatten(1, 2).to(torch.bfloat16),
            "lse": lse.transpose(1, 2)[req, at].flatten(1, 2)}


# --------------------------------------------------------------- the calls --

def run(s):
    op = s["op"]
    if not own:
        return {"plan": _plain_plan, "rope": _plain_rope, "rope_bwd": _plain_rope_bwd,
                "append": _plain_append, "attend": _plain_attend}[op](s)
    import nvfp4_block_scaled_02_gb300 as nv
    if op == "plan":
        return nv.nvfp4_kv_plan(s["cached"], s["new"], s["table"], s["free"], s["page"],
                                s["tokens"])
    if op == "rope":
        return nv.nvfp4_qk_norm_rope(s["q"], s["k"], s["positions"], s["cos_sin"], s["qw"],
                                     s["kw"], eps=EPS, interleaved=s["interleaved"])
    if op == "rope_bwd":
        if "ws" not in s:
            s["ws"] = nv.qk_norm_rope_workspace(s["q"].device)
        return nv.nvfp4_qk_norm_rope_bwd(s["gq"], s["gk"], s["q"], s["k"], s["positions"],
                                         s["cos_sin"], s["qw"], s["kw"], eps=EPS,
                                         interleaved=s["interleaved"], workspace=s["ws"])
    if op == "append":
        r = nv.nvfp4_kv_append(s["cache"], s["k"], s["v"], s["slots"], dequant=True)
        return _append_outputs(s, r["k"], r["v"])
    if "ws" not in s:
        s["ws"] = nv.kv_attention_workspace(s["q"].device)
    return nv.nvfp4_kv_attention(s["q"], s["cache"], s["table"], s["seq_lens"], s["q_start"],
                                 s["max_q"], scale=s["scale"], window=s["window"],
                                 workspace=s["ws"])


# ------------------------------------------------------- 64-bit definition --

def _exact_rope(s, back):
    pos = s["positions"].long()
    cs = s["cos_sin"].double()[pos]
    h = cs.shape[1] // 2
    z = torch.complex(cs[:, :h], cs[:, h:])[:, None, :]  # a rotation is a product by e^(i angle)

    def turn(x, w):
        r = x[..., : 2 * h]
        x = x.clone()
        if s["interleaved"]:
            y = torch.complex(r[..., 0::2].contiguous(), r[..., 1::2].contiguous()) * w
            x[..., 0: 2 * h: 2], x[..., 1: 2 * h: 2] = y.real, y.imag
        else:
            y = torch.complex(r[..., :h].contiguous(), r[..., h:].contiguous()) * w
            x[..., :h], x[..., h: 2 * h] = y.real, y.imag
        return x

    def norm(x):
        return x / ((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()

    out = {}
    for n in ("q", "k"):
        x, w = s[n].double(), s[n + "w"]
        if not back:
            out[n] = turn(x if w is None else norm(x) * w.double(), z)
            continue
        u = turn(s["g" + n].double(), z.conj())
        if w is None:
            out["g" + n], out["g" + n + "_weight"] = u, None
            continue
        y = norm(x)
        out["g" + n + "_weight"] = (u * y).sum((0, 1))
        u = u * w.double()
        size = ((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()
        out["g" + n] = (u - y * (u * y).sum(-1, keepdim=True) / x.shape[-1]) / size
    return out


def _exact_append(s):
    c, P = s["cache"], s["case"]["page"]
    mags = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    # every finite E4M3 value >= 0 by its code
    e4m3 = torch.arange(127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()
    out = {}

    def nearest(x, grid):  # index of the nearest grid value, ties to the even index
        hi = torch.searchsorted(grid, x).clamp(1, len(grid) - 1)
        lo = hi - 1
        a, b = x - grid[lo], grid[hi] - x
        return torch.where((b < a) | ((a == b) & (hi % 2 == 0)), hi, lo)

    for n in ("k", "v"):
        g = (c[n + "_amax"].double() / (6 * FP8_MAX))[None, :, None]
        b = s[n].double().unflatten(-1, (-1, 16))
        code = nearest((b.abs().amax(-1) / (6 * g)).clamp(max=FP8_MAX).contiguous(), e4m3)
        d = (e4m3[code] * g)[..., None]
        y = torch.where(d > 0, b / d.clamp(min=1e-300), torch.zeros_like(b))
        m = mags[nearest(y.abs().clamp(max=6).contiguous(), mags)]
        out[n] = (torch.copysign(m, b) * d).flatten(-2)
        scales = c[n + "_scales"].view(torch.float8_e4m3fn).double()
        scales[s["slots"] // P, :, s["slots"] % P] = e4m3[code]
        out[n + "_scales"] = scales
    return out


def _exact_attend(s):
    c, P = s["cache"], s["case"]["page"]
    T, hq, D = s["q"].shape
    hk = s["case"]["kv_heads"]
    out = torch.zeros(T, hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64, device="cuda")
    mags = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    start, lens, table = (s[n].tolist() for n in ("q_start", "seq_lens", "table"))
    for b, L in enumerate(lens):
        pages = torch.tensor(table[b][: -(-L // P)], dtype=torch.int64, device="cuda")
        if L == 0:
            continue
        pos = torch.arange(start[b + 1] - start[b], device="cuda") + L - (start[b + 1] - start[b])
        key = torch.arange(L, device="cuda")[None, :]
        hide = key > pos[:, None]
        if s["window"]:
            hide = hide | (key <= pos[:, None] - s["window"])
        for h in range(hk):
            kv = []
            for n in ("k", "v"):
                by = c[n + "_codes"][pages, h].reshape(-1, D // 2)[:L].long()
                code = torch.stack([by % 16, by // 16], 2).view(L, D)
                x = mags[code % 8] * (1 - 2 * (code // 8))
                sc = c[n + "_scales"][pages, h].reshape(-1, D // 16)[:L]
                sc = sc.view(torch.float8_e4m3fn).double() * c[n + "_amax"][h].double()
                kv.append(x * sc.repeat_interleave(16, 1) / (6 * FP8_MAX))
            for j in range(h * (hq // hk), (h + 1) * (hq // hk)):
                q = s["q"][start[b]: start[b + 1], j].double()
                x = (q @ kv[0].T * s["scale"]).masked_fill(hide, -math.inf)
                z = torch.logsumexp(x, 1)
                p = torch.exp(x - z.clamp(min=-1e300)[:, None])
                out[start[b]: start[b + 1], j] = p @ kv[1]
                lse[start[b]: start[b + 1], j] = z
    return {"out": out, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "plan":
        return None  # whole numbers
    if op in ("rope", "rope_bwd"):
        return _exact_rope(s, op == "rope_bwd")
    return _exact_append(s) if op == "append" else _exact_attend(s)
