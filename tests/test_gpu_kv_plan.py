"""Block tables and slot maps against a loop over requests and tokens: whole
numbers, so every output must be equal."""
import numpy as np
import pytest
import torch

import kv_ref
import nvfp4_block_scaled_02_gb300 as nv

pytestmark = pytest.mark.gpu


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def _case(B, P, hi_new, hi_cached, seed, spare=3):
    r = np.random.default_rng(seed)
    new = r.integers(0, hi_new + 1, B)
    cached = r.integers(0, hi_cached + 1, B)
    held, total = -(-cached // P), -(-(cached + new) // P)
    cols = int(total.max(initial=0)) + 2
    pages = r.permutation(int(total.sum()) + spare)
    table = np.full((B, cols), -7, np.int32)
    at = np.arange(cols)[None, :] < held[:, None]
    table[at] = pages[: int(held.sum())]
    return new, cached, table, pages[int(held.sum()):].astype(np.int32)


def _run(cached, new, table, free, P, tokens):
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = nv.nvfp4_kv_plan(_i32(cached), _i32(new), _i32(table), _i32(free), P, tokens, status=st)
    return {k: v.cpu().numpy() for k, v in r.items()}, int(st.item())


def _same(got, want):
    for name, w in zip(("table", "seq_lens", "q_start", "slots", "positions"), want):
        assert np.array_equal(got[name], w), name
    assert int(got["pages_used"][0]) == want[5]


@pytest.mark.parametrize("B,P,hi_new,hi_cached", [
    (1, 16, 1, 0), (1, 16, 5000, 100), (3, 16, 40, 40), (64, 16, 1, 500), (65, 17, 9, 300),
    (1023, 64, 3, 200), (1024, 32, 2, 50), (1025, 1, 4, 9), (2500, 128, 7, 1000),
    (40, 64, 700, 3000), (5, 48, 0, 77)])
def test_matches_the_loops(B, P, hi_new, hi_cached):
    new, cached, table, free = _case(B, P, hi_new, hi_cached, seed=B + P)
    for pad in (0, 1, 2049):  # rows past the last new token
        tokens = int(new.sum()) + pad
        got, st = _run(cached, new, table, free, P, tokens)
        _same(got, kv_ref.plan(cached, new, table, free, P, tokens))
        assert st == 0


def test_no_requests_and_no_tokens():
    e = np.zeros(0, np.int64)
    got, st = _run(e, e, np.zeros((0, 4)), np.arange(3), 16, 5)
    assert st == 0 and got["q_start"].tolist() == [0] and got["slots"].tolist() == [-1] * 5
    assert got["positions"].tolist() == [0] * 5 and got["pages_used"].tolist() == [0]
    got, st = _run(np.array([5, 0]), np.array([0, 0]), np.full((2, 1), 9), e, 16, 0)
    assert st == 0 and got["q_start"].tolist() == [0, 0, 0] and got["seq_lens"].tolist() == [5, 0]


def test_free_pages_run_out():
    new, cached, table, free = _case(30, 16, 60, 100, seed=4)
    free = free[:20]
    got, st = _run(cached, new, table, free, 16, int(new.sum()))
    _same(got, kv_ref.plan(cached, new, table, free, 16, int(new.sum())))
    assert st == nv.DEV_NO_PAGES and int(got["pages_used"][0]) == 20


def test_bad_lengths_are_flagged_and_write_nothing_out_of_range():
    # a table too narrow: its columns are filled, tokens past them have no slot
    got, st = _run(np.array([0]), np.array([50]), np.full((1, 2), -1), np.arange(9), 16, 50)
    assert st == nv.DEV_BAD_INDEX and got["table"].tolist() == [[0, 1]]
    assert got["slots"][:32].tolist() == list(range(32)) and (got["slots"][32:] == -1).all()
    # a negative length counts as 0
    got, st = _run(np.array([3, -4]), np.array([-1, 2]), np.full((2, 2), 8), np.arange(5), 16, 4)
    assert st == nv.DEV_BAD_INDEX and got["q_start"].tolist() == [0, 0, 2]
    assert got["slots"].tolist() == [0, 1, -1, -1] and got["seq_lens"].tolist() == [3, 2]
    # more new tokens than rows
    got, st = _run(np.array([0]), np.array([40]), np.full((1, 3), -1), np.arange(9), 16, 10)
    assert st == nv.DEV_BAD_INDEX and got["slots"].tolist() == list(range(10))
    assert got["q_start"].tolist() == [0, 10]


def test_repeating_the_call_changes_nothing():
    new, cached, table, free = _case(200, 16, 20, 90, seed=8)
    t = _i32(table)
    args = (_i32(cached), _i32(new), t, _i32(free), 16, int(new.sum()))
    a = nv.nvfp4_kv_plan(*args)
    first = {k: v.clone() for k, v in a.items()}
    b = nv.nvfp4_kv_plan(*args, out=a)
    for k in first:
        assert torch.equal(first[k], b[k]), k
