"""Refusals of the KV-cache operators, without a GPU: the library's argument
errors (returned before any CUDA call) and the binding's checks of tensors."""
import ctypes as C

import pytest
import torch

import nvfp4_block_scaled_02_gb300 as nv
from nvfp4_block_scaled_02_gb300 import kv

FAKE = 0x100000  # a 16-byte aligned, never dereferenced address
OK, NULL, SHAPE, ALIGN, ENUM = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def L():
    nv.build()
    return nv.lib()


def rows(ptr=FAKE, stride=1024):
    return kv._Rows(ptr, stride)


def test_plan_argument_errors(L):
    def plan(cached=FAKE, new=FAKE, B=4, table=FAKE, cols=8, P=16, free=FAKE, n_free=9, T=4,
             seq=FAKE, start=FAKE, slots=FAKE, pos=FAKE, used=FAKE, status=None):
        return L.nvfp4_kv_plan(cached, new, B, table, cols, P, free, n_free, T, seq, start, slots,
                               pos, used, status, None)
    for bad in (dict(B=-1), dict(B=1 << 31), dict(cols=-1), dict(cols=1 << 31), dict(P=0),
                dict(P=-16), dict(n_free=-1), dict(n_free=1 << 31), dict(T=-1), dict(T=1 << 31)):
        assert plan(**bad) == SHAPE, bad
    for name in ("cached", "new", "table", "free", "seq", "start", "slots", "pos", "used"):
        assert plan(**{name: None}) == NULL, name
        assert plan(**{name: FAKE + 2}) == ALIGN, name
    assert plan(slots=FAKE + 4) == ALIGN and plan(status=FAKE + 1) == ALIGN


def qk(**kw):
    d = dict(tokens=4, q_heads=2, kv_heads=1, head_dim=64, rotary_dim=64, interleaved=0, eps=1e-6,
             q_weight=FAKE, k_weight=FAKE, positions=FAKE, cos_sin=FAKE, max_pos=10)
    d.update(kw)
    return kv._QkConfig(*[d[n] for n, _ in kv._QkConfig._fields_])


QK_BAD = [(dict(tokens=-1), SHAPE), (dict(tokens=1 << 31), SHAPE), (dict(q_heads=-1), SHAPE),
          (dict(kv_heads=-1), SHAPE), (dict(q_heads=1 << 17), SHAPE), (dict(head_dim=96), SHAPE),
          (dict(head_dim=0), SHAPE), (dict(rotary_dim=0), SHAPE), (dict(rotary_dim=24), SHAPE),
          (dict(rotary_dim=80), SHAPE), (dict(max_pos=0), SHAPE), (dict(interleaved=2), ENUM),
          (dict(eps=-1.0), ENUM), (dict(eps=float("nan")), ENUM), (dict(eps=float("inf")), ENUM),
          (dict(positions=None), NULL), (dict(cos_sin=None), NULL), (dict(positions=FAKE + 2), ALIGN),
          (dict(cos_sin=FAKE + 4), ALIGN), (dict(q_weight=FAKE + 8), ALIGN),
          (dict(k_weight=FAKE + 2), ALIGN)]


def test_norm_rope_argument_errors(L):
    def fwd(cfg=None, q=rows(), k=rows(), qo=rows(), ko=rows(), status=None, **kw):
        return L.nvfp4_qk_norm_rope(C.byref(cfg or qk(**kw)), q, k, qo, ko, status, None)
    assert L.nvfp4_qk_norm_rope(None, rows(), rows(), rows(), rows(), None, None) == NULL
    for bad, want in QK_BAD:
        assert fwd(**bad) == want, bad
    for n in ("q", "k", "qo", "ko"):
        assert fwd(**{n: rows(None)}) == NULL
        assert fwd(**{n: rows(FAKE + 8)}) == ALIGN
        assert fwd(**{n: rows(stride=1028)}) == SHAPE      # not a multiple of 8
        assert fwd(**{n: rows(stride=56)}) == SHAPE        # below one token's heads
    assert fwd(status=FAKE + 2) == ALIGN
    assert fwd(tokens=0, positions=None, q=rows(None)) == OK
    assert fwd(q_heads=0, kv_heads=0) == OK


def test_norm_rope_bwd_argument_errors(L):
    size = L.nvfp4_qk_norm_rope_ws_bytes()

    def bwd(r=None, gqw=FAKE, gkw=FAKE, ws=FAKE, n=size, status=None, at=None, **kw):
        a = [rows() for _ in range(6)]
        if at is not None:
            a[at] = r
        return L.nvfp4_qk_norm_rope_bwd(C.byref(qk(**kw)), *a, gqw, gkw, ws, n, status, None)
    for bad, want in QK_BAD:
        assert bwd(**bad) == want, bad
    for at in range(6):
        assert bwd(rows(None), at=at) == NULL
        assert bwd(rows(FAKE + 2), at=at) == ALIGN
        assert bwd(rows(stride=8), at=at) == SHAPE
    assert bwd(gqw=None) == NULL and bwd(gkw=None) == NULL          # a weight without its gradient
    assert bwd(q_weight=None) == NULL and bwd(k_weight=None) == NULL  # and the other way round
    assert bwd(ws=None) == NULL and bwd(n=size - 1) == SHAPE and bwd(ws=FAKE + 4) == ALIGN
    assert bwd(gqw=FAKE + 2) == ALIGN and bwd(status=FAKE + 2) == ALIGN


def cache(**kw):
    d = dict(k_codes=FAKE, k_scales=FAKE, v_codes=FAKE, v_scales=FAKE, k_amax=FAKE, v_amax=FAKE,
             pages=4, kv_heads=2, page_size=16, head_dim=64, four_over_six=0)
    d.update(kw)
    return kv._Cache(*[d[n] for n, _ in kv._Cache._fields_])


CACHE_BAD = [(dict(pages=-1), SHAPE), (dict(pages=1 << 58), SHAPE), (dict(kv_heads=0), SHAPE),
             (dict(kv_heads=1 << 17), SHAPE), (dict(page_size=0), SHAPE), (dict(page_size=24), SHAPE),
             (dict(page_size=-16), SHAPE), (dict(head_dim=32), SHAPE), (dict(head_dim=256), SHAPE),
             (dict(four_over_six=2), ENUM), (dict(four_over_six=-1), ENUM)]
CACHE_BAD += [(dict([(n, None)]), NULL) for n in ("k_codes", "k_scales", "v_codes", "v_scales",
                                                  "k_amax", "v_amax")]
CACHE_BAD += [(dict([(n, FAKE + 8)]), ALIGN) for n in ("k_codes", "k_scales", "v_codes", "v_scales")]
CACHE_BAD += [(dict([(n, FAKE + 2)]), ALIGN) for n in ("k_amax", "v_amax")]


def test_append_argument_errors(L):
    def app(c=None, k=rows(), v=rows(), slots=FAKE, T=3, kd=None, vd=None, status=None):
        return L.nvfp4_kv_append(C.byref(c or cache()), k, v, slots, T, kd, vd, status, None)
    assert L.nvfp4_kv_append(None, rows(), rows(), FAKE, 3, None, None, None, None) == NULL
    for bad, want in CACHE_BAD:
        assert app(cache(**bad)) == want, bad
    for n in ("k", "v"):
        assert app(**{n: rows(None)}) == NULL and app(**{n: rows(FAKE + 8)}) == ALIGN
        assert app(**{n: rows(stride=120)}) == SHAPE
    assert app(slots=None) == NULL and app(slots=FAKE + 4) == ALIGN
    assert app(T=-1) == SHAPE and app(T=1 << 31) == SHAPE
    assert app(kd=FAKE + 8) == ALIGN and app(vd=FAKE + 8) == ALIGN and app(status=FAKE + 1) == ALIGN
    assert app(T=0, slots=None) == OK


def test_attention_argument_errors(L):
    size = L.nvfp4_kv_attention_ws_bytes()

    def cfg(**kw):
        d = dict(block_table=FAKE, seq_len=FAKE, q_start=FAKE, requests=3, table_cols=4, tokens=5,
                 q_heads=4, max_q=2, window=0, scale=0.1)
        d.update(kw)
        return kv._AttentionConfig(*[d[n] for n, _ in kv._AttentionConfig._fields_])

    def att(c=None, q=rows(), out=FAKE, lse=FAKE, ws=FAKE, n=size, status=None, **kw):
        return L.nvfp4_kv_attention(C.byref(c or cache()), C.byref(cfg(**kw)), q, out, lse, ws, n,
                                    status, None)
    for bad, want in CACHE_BAD:
        assert att(cache(**bad)) == want, bad
    assert L.nvfp4_kv_attention(C.byref(cache()), None, rows(), FAKE, None, FAKE, size, None,
                                None) == NULL
    for bad in (dict(requests=-1), dict(requests=(1 << 31) - 1), dict(table_cols=-1),
                dict(table_cols=1 << 31), dict(tokens=-1), dict(tokens=1 << 31), dict(max_q=-1),
                dict(window=-1), dict(q_heads=0), dict(q_heads=3), dict(q_heads=1 << 17),
                dict(max_q=(1 << 31) - 1), dict(n=size - 1), dict(q=rows(stride=248)),
                dict(q=rows(stride=260))):
        assert att(**bad) == SHAPE, bad
    for bad in (float("nan"), float("inf")):
        assert att(scale=bad) == ENUM
    for bad in (dict(block_table=None), dict(seq_len=None), dict(q_start=None), dict(out=None),
                dict(ws=None), dict(q=rows(None))):
        assert att(**bad) == NULL, bad
    for bad in (dict(block_table=FAKE + 2), dict(seq_len=FAKE + 1), dict(q_start=FAKE + 2),
                dict(out=FAKE + 8), dict(ws=FAKE + 8), dict(q=rows(FAKE + 8)), dict(lse=FAKE + 2),
                dict(status=FAKE + 2)):
        assert att(**bad) == ALIGN, bad
    assert att(tokens=0, out=None) == OK and att(requests=0, out=None) == OK


# ---- the binding: checks come before the library, so CPU tensors will do -----

def _cpu_cache():
    return nv.alloc_kv_cache(2, 16, 2, 64, torch.ones(2), torch.ones(2))


def _bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_binding_checks_rows():
    with pytest.raises(TypeError, match="q must hold bf16"):
        kv._rows(torch.zeros(2, 2, 64), "q", 2, 2, 64)
    with pytest.raises(ValueError, match=r"q must be \[2, 2, 64\]"):
        kv._rows(_bf(2, 3, 64), "q", 2, 2, 64)
    with pytest.raises(ValueError, match="contiguous"):
        kv._rows(_bf(2, 64, 2).transpose(1, 2), "q", 2, 2, 64)
    with pytest.raises(ValueError, match="contiguous"):
        kv._rows(_bf(2, 2, 128)[:, :, :64], "q", 2, 2, 64)
    for t in (_bf(2, 2, 64), _bf(2, 4, 64)[:, :2]):
        with pytest.raises(ValueError, match="CUDA"):
            kv._rows(t, "q", 2, 2, 64)


def test_binding_checks_of_the_entry_points():
    c, i32 = _cpu_cache(), torch.int32
    slots = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        nv.nvfp4_kv_append(c, _bf(3, 2, 64), _bf(3, 2, 64), slots)
    bad = dict(c, v_scales=c["v_scales"][:1])
    with pytest.raises(ValueError):
        nv.nvfp4_kv_append(bad, _bf(3, 2, 64), _bf(3, 2, 64), slots)
    with pytest.raises(ValueError, match="k_codes"):
        nv.nvfp4_kv_append(dict(c, k_codes=c["k_codes"][0]), _bf(3, 2, 64), _bf(3, 2, 64), slots)
    n = torch.zeros(2, dtype=i32)
    with pytest.raises(ValueError, match="table"):
        nv.nvfp4_kv_plan(n, n, n, n, 16, 4)
    with pytest.raises(ValueError, match="tokens"):
        nv.nvfp4_kv_plan(n, n, torch.zeros(2, 3, dtype=i32), n, 16, -1)
    with pytest.raises(TypeError, match="cached"):
        nv.nvfp4_kv_plan(n.long(), n, torch.zeros(2, 3, dtype=i32), n, 16, 4)
    q, k, pos, cs = _bf(3, 2, 64), _bf(3, 1, 64), torch.zeros(3, dtype=i32), torch.zeros(9, 64)
    for args, what in (((_bf(3, 128), k, pos, cs), "q and k"), ((q, k, pos, cs[0]), "cos_sin"),
                       ((q, k, pos, cs, _bf(32)), "q_weight"),
                       ((q, k, pos, cs, None, torch.zeros(64)), "k_weight"),
                       ((q, k, pos[:2], cs), "positions")):
        with pytest.raises(ValueError, match=what):
            nv.nvfp4_qk_norm_rope(*args)
    with pytest.raises(TypeError, match="cos_sin"):
        nv.nvfp4_qk_norm_rope(q, k, pos, cs.double())


def test_binding_checks_of_attention():
    """Argument order of the checks: shapes first, devices with the pointers."""
    c = {n: v for n, v in _cpu_cache().items()}
    with pytest.raises(ValueError, match="CUDA"):
        nv.nvfp4_kv_attention(_bf(2, 4, 64), c, torch.zeros(1, 2, dtype=torch.int32),
                              torch.ones(1, dtype=torch.int32),
                              torch.tensor([0, 2], dtype=torch.int32), 2)
