"""spec_page_plan against the oracle (everything has to be equal): requests
that open pages and that do not, batches over one cluster's CTAs and over one
chunk of requests, and what is skipped and reported."""

import numpy as np
import pytest
import torch

import gpu_helpers as gh
from kv8_helpers import page_layout
from oracle import kv8
from self_speculative_verification_gb300 import binding as bn

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    gh.require_gpu()
    bn.spec_get_status()


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def plan(S, new, ps, table, free, head=0, extra=5, n_pages=None, n_slots=None, status=0):
    S, new = np.asarray(S, dtype=np.int32), np.asarray(new, dtype=np.int32)
    n = int(np.maximum(new, 0).sum()) + extra if n_slots is None else n_slots
    B = len(S)
    tab, fh = dev(table), dev(np.array([head], dtype=np.int32))
    cu = torch.full((B + 1,), -3, dtype=torch.int32, device="cuda")
    slots = torch.full((n,), -9, dtype=torch.int64, device="cuda")
    ln = torch.full((B,), -3, dtype=torch.int32, device="cuda")
    bn.spec_page_plan(ps, n_pages or 10 ** 6, dev(S), dev(new), tab, dev(free), fh, cu, slots, ln)
    assert bn.spec_get_status() == status
    got = tuple(x.cpu().numpy() for x in (tab, cu, slots, ln)) + (int(fh),)
    t, h, c, s, l = kv8.page_plan(S, new, table, free, head, ps, n)
    for g, w in zip(got, (t, c, s, l)):
        assert np.array_equal(g, w)
    assert got[4] == h
    return got


@pytest.mark.parametrize("ps", [16, 48, 128, 1])
@pytest.mark.parametrize("B,hi,held", [(1, 1, 0), (1, 0, 5), (3, 40, 20), (64, 9, 300), (200, 700, 500),
                                       (2048, 3, 30), (2049, 40, 30), (5000, 2, 9)])
def test_plan(B, hi, held, ps):
    rng = np.random.default_rng(B + ps)
    S = rng.integers(0, held + 1, size=B)
    new = rng.integers(0, hi + 1, size=B)
    maxp = max(1, -(-(held + hi) // ps))
    _, table, free = page_layout(rng, S, maxp, ps, int((-(-(S + new) // ps)).sum()) + 3)
    plan(S, new, ps, table, free, head=2 if len(free) > 2 else 0)


def test_a_plan_without_requests_or_slots():
    z = np.zeros(0, dtype=np.int32)
    plan(z, z, 16, np.zeros((0, 4), dtype=np.int32), np.arange(3, dtype=np.int32), extra=7)
    plan([4], [0], 16, np.array([[2, -1]], dtype=np.int32), np.zeros(0, dtype=np.int32), extra=0)


def test_what_is_skipped():
    table = np.full((4, 3), -1, dtype=np.int32)
    table[:, 0] = [0, 1, 2, 3]
    free = np.arange(10, 20, dtype=np.int32)
    # over the table's 48 tokens
    plan([10, 40, 16, 16], [3, 9, 17, 0], 16, table, free, status=bn.SPEC_DEV_CAPACITY)
    plan([10, -5, 16, 100], [3, 9, 17, 0], 16, table, free, status=bn.SPEC_DEV_SEQ_OVERFLOW)
    # too few free pages: nothing
    got = plan([10, 16, 16, 16], [3, 9, 17, 1], 16, table, free[:3], status=bn.SPEC_DEV_CAPACITY)
    assert np.all(got[2] == -1) and got[4] == 0
    plan([10, 16, 16, 16], [3, 9, 17, 1], 16, table, free, head=8, status=bn.SPEC_DEV_CAPACITY)
    plan([10, 16, 16, 16], [3, 9, 17, 1], 16, table, free, head=-1, status=bn.SPEC_DEV_CAPACITY)
    # fewer slots than tokens
    plan([10, 16, 16, 16], [3, 9, 17, 1], 16, table, free, n_slots=11, status=bn.SPEC_DEV_BAD_INDEX)


def test_negative_requests_and_bad_pages():
    table = np.array([[0, -1], [1, -1]], dtype=np.int32)
    free = np.array([7, 99, 5], dtype=np.int32)
    S, new = dev(np.array([16, 16], dtype=np.int32)), dev(np.array([2, 2], dtype=np.int32))
    i32 = dict(dtype=torch.int32, device="cuda")
    tab, fh, cu = dev(table), torch.zeros(1, **i32), torch.zeros(3, **i32)
    slots = torch.zeros(6, dtype=torch.int64, device="cuda")
    bn.spec_page_plan(16, 8, S, new, tab, dev(free), fh, cu, slots)
    assert bn.spec_get_status() == bn.SPEC_DEV_BAD_PAGE
    assert slots.tolist() == [112, 113, -1, -1, -1, -1] and tab[1].tolist() == [1, -1]
    new[0] = -4
    fh.zero_()
    bn.spec_page_plan(16, 8, S, new, tab, dev(free), fh, cu, slots)
    assert bn.spec_get_status() == bn.SPEC_DEV_BAD_INDEX
    assert cu.tolist() == [0, 0, 2] and slots.tolist()[:2] == [112, 113]


def test_too_many_tokens_are_refused():
    B = 3
    S = torch.zeros(B, dtype=torch.int32, device="cuda")
    new = torch.full((B,), 1 << 30, dtype=torch.int32, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    tab = torch.full((B, 4), -1, **i32)
    fh, cu, ln = torch.zeros(1, **i32), torch.full((B + 1,), 5, **i32), torch.zeros(B, **i32)
    slots = torch.zeros(100, dtype=torch.int64, device="cuda")
    bn.spec_page_plan(1 << 28, 100, S, new, tab, torch.arange(20, **i32), fh, cu, slots, ln)
    assert bn.spec_get_status() == bn.SPEC_DEV_BAD_INDEX
    assert cu.tolist() == [0] * 4 and torch.all(slots == -1) and int(fh) == 0
    assert torch.all(tab == -1) and torch.all(ln == 0)


def test_plan_graph_replay():
    rng = np.random.default_rng(3)
    S, new = rng.integers(0, 50, size=30), rng.integers(0, 2000, size=30)
    _, table, free = page_layout(rng, S, 130, 16, 4000)
    i32 = dict(dtype=torch.int32, device="cuda")
    tab0 = dev(table)
    tab, fh, cu, ln = tab0.clone(), torch.zeros(1, **i32), torch.zeros(31, **i32), torch.zeros(30, **i32)
    slots = torch.zeros(int(new.sum()), dtype=torch.int64, device="cuda")
    args = (16, 10 ** 6, dev(S.astype(np.int32)), dev(new.astype(np.int32)), tab, dev(free), fh, cu,
            slots, ln)
    bn.spec_page_plan(*args)
    want = [x.clone() for x in (tab, fh, cu, slots, ln)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tab.copy_(tab0)
        fh.zero_()
        bn.spec_page_plan(*args)
    slots.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert bn.spec_get_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(want, (tab, fh, cu, slots, ln)))
