"""64-bit reference forms of the operators around the NVFP4 KV cache, in plain
numpy: the definitions, with loops over requests and heads."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)
E2M1 = np.concatenate([E2M1, -E2M1])


def half_ulp_bf16(y: np.ndarray) -> np.ndarray:
    """Half the distance of neighbouring bf16 values (8 significant bits) at y's
    magnitude: how far round-to-nearest moves y at most."""
    _, e = np.frexp(np.abs(y))  # |y| in [2^(e-1), 2^e)
    return np.ldexp(1.0, np.maximum(e, -125) - 9)


def e4m3(b: np.ndarray) -> np.ndarray:
    b = np.asarray(b, np.int64)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7.0))
    v = np.where((b & 0x7F) == 0x7F, np.nan, v)
    return np.where(b & 0x80, -v, v)


def decode(codes: np.ndarray, scales: np.ndarray, g: float) -> np.ndarray:
    """Values of code bytes [..., D/2] and scale bytes [..., D/16]."""
    v = np.stack([E2M1[codes & 15], E2M1[codes >> 4]], -1).reshape(*codes.shape[:-1], -1)
    return v * np.repeat(e4m3(scales) * g, 16, axis=-1)


def plan(cached, new, table, free, P, tokens):
    """(table, seq_lens, q_start, slots, positions, used) of valid lengths; a page
    missing from the free list is -1."""
    table, taken, starts = table.copy(), 0, [0]
    slots, positions = np.full(tokens, -1, np.int64), np.zeros(tokens, np.int32)
    for b in range(len(cached)):
        held, total = -(-int(cached[b]) // P), -(-int(cached[b] + new[b]) // P)
        for j in range(held, total):
            table[b, j] = free[taken] if taken < len(free) else -1
            taken += 1
        for i in range(int(new[b])):
            t, pos = starts[-1] + i, int(cached[b]) + i
            if t < tokens:
                page = table[b, pos // P]
                slots[t] = -1 if page < 0 else int(page) * P + pos % P
                positions[t] = pos
        starts.append(starts[-1] + int(new[b]))
    return (table, np.asarray(cached + new, np.int32), np.minimum(starts, tokens).astype(np.int32),
            slots, positions, min(taken, len(free)))


def _rotate(x, cs, interleaved, sign=1.0):
    """x [tokens, heads, D] rotated by cs [tokens, R]."""
    R = cs.shape[1]
    c, s = cs[:, None, : R // 2], sign * cs[:, None, R // 2:]
    y = x.copy()
    a, b = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def norm_rope(x, w, cs, eps, interleaved):
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    return _rotate(x, cs, interleaved)


def norm_rope_bwd(gy, x, w, cs, eps, interleaved):
    u = _rotate(gy, cs, interleaved, -1.0)
    if w is None:
        return u, None
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    gx = r * (w * u - x * r * r * (w * u * x).mean(-1, keepdims=True))
    return gx, (u * x * r).sum((0, 1))


def attention(q, k_of, v_of, q_start, seq_lens, scale, window):
    """out, lse and, for error bounds, sum p |v|, max |q| . |k| scale of each row and
    its largest p times sum |v|.
    k_of(b), v_of(b): [heads, length, D] of request b. q: [tokens, q_heads, D]."""
    T, hq, D = q.shape
    out, absv, allv = np.zeros((T, hq, D)), np.zeros((T, hq, D)), np.zeros((T, hq, D))
    lse, size = np.full((T, hq), -np.inf), np.zeros((T, hq))
    for b, L in enumerate(seq_lens):
        q0, q1 = int(q_start[b]), int(q_start[b + 1])
        if L == 0 or q0 == q1:
            continue
        k, v = k_of(b), v_of(b)
        G = hq // k.shape[0]
        pos = np.arange(q0, q1) - q1 + L
        key = np.arange(L)
        seen = key[None, :] <= pos[:, None]
        if window:
            seen &= key[None, :] > pos[:, None] - window
        some = seen.any(1)
        for h in range(hq):
            x = scale * (q[q0:q1, h] @ k[h // G].T)
            x = np.where(seen, x, -np.inf)
            top = np.where(some, x.max(1), 0.0)
            p = np.where(seen, np.exp(x - top[:, None]), 0.0)
            z = p.sum(1)
            zs = np.where(some, z, 1.0)
            out[q0:q1, h] = np.where(some[:, None], (p @ v[h // G]) / zs[:, None], 0)
            absv[q0:q1, h] = np.where(some[:, None], (p @ np.abs(v[h // G])) / zs[:, None], 0)
            allv[q0:q1, h] = np.where(some[:, None], (seen @ np.abs(v[h // G])) / zs[:, None], 0)
            lse[q0:q1, h] = np.where(some, np.log(zs) + top, -np.inf)
            a = abs(scale) * (np.abs(q[q0:q1, h]) @ np.abs(k[h // G]).T)
            size[q0:q1, h] = np.where(seen, a, 0).max(1)
    return out, lse, absv, size, allv
