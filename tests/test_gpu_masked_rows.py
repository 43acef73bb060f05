"""Judged rows whose mask allows nothing: the vocabulary reduction names no
token, and no acceptance takes one there."""

import numpy as np
import pytest
import torch

import gpu_helpers as gh
from self_speculative_verification_gb300 import binding as bn

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.fixture(autouse=True)
def _gpu():
    gh.require_gpu()
    bn.spec_get_status()


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Rows:
    """One request of 4 nodes in a chain whose tokens are all 0, judged by
    rows that want token 0 but for row `masked`, which allows nothing."""

    def __init__(self, V, dtype, masked):
        self.V, self.dt = V, torch.bfloat16 if dtype == "bf16" else torch.float32
        self.z = torch.randn((1, 4, V), device="cuda").to(self.dt)
        self.z[:, :, 0] = 20.0
        # by the operator that masks, in place
        bits = torch.zeros((1, (V + 31) // 32), dtype=torch.int32, device="cuda")
        rows = torch.full((1, 4), -1, dtype=torch.int32, device="cuda")
        rows[0, masked] = 0
        bn.spec_logits_adjust(bn.logits_desc(1, 4, V, bn.spec_dtype(self.z), n_masks=1), self.z, self.z,
                              mask_bits=bits, row_mask=rows)
        self.tokens, self.parent, self.n = i32([0] * 4), i32([-1, 0, 1, 2]), i32(4)
        self.am = torch.full((1, 4), 77, dtype=torch.int32, device="cuda")
        self.lse, self.zp = torch.zeros((1, 4), device="cuda"), torch.zeros((1, 4), device="cuda")
        self.acc, self.next, self.last = i32(9), i32(9), i32(9)
        self.path = torch.full((1, 4), 9, dtype=torch.int32, device="cuda")

    def accept(self, mode):
        d = bn.accept_desc(mode, 0.5, 1, 4, self.V, bn.spec_dtype(self.z), 4, 4)
        tree = mode == bn.SPEC_ACCEPT_GREEDY_TREE
        bn.spec_accept(d, self.z, self.tokens, self.parent if tree else None, None, self.n, self.am, self.lse,
                       self.zp, self.acc, self.path, self.next, self.last)
        assert bn.spec_get_status() == 0
        return int(self.acc), self.path[0].tolist(), int(self.next), int(self.last)


CASES = [(V, dt) for V in (1, 7, 4000, 4001, 50272) for dt in ("bf16", "f32")]


@pytest.mark.parametrize("V,dtype", CASES)
@pytest.mark.parametrize("masked", [0, 2])
def test_reduction_and_acceptance(V, dtype, masked):
    r = Rows(V, dtype, masked)
    bn.spec_vocab_reduce(r.z.view(4, V), r.tokens.view(-1), r.am.view(-1), r.lse.view(-1), r.zp.view(-1))
    assert r.am[0].tolist() == [-1 if j == masked else 0 for j in range(4)]
    assert float(r.lse[0, masked]) == -INF and torch.isfinite(r.lse[0, 1]).all()
    # the walk ends at the node that the masked row judges; it follows no child
    n = masked + 1
    got = r.accept(bn.SPEC_ACCEPT_GREEDY_TREE)
    assert got == (n, list(range(n)) + [-1] * (4 - n), -1, masked)
    # a chain's masked row accepts no proposal and has no other token to offer
    got = r.accept(bn.SPEC_ACCEPT_THRESH_CHAIN)
    assert got == (masked, list(range(masked)) + [-1] * (4 - masked), -1, masked - 1)


@pytest.mark.parametrize("V,dtype", CASES[2:])
@pytest.mark.parametrize("draft_rows", [0, 4])
def test_soft_matching(V, dtype, draft_rows):
    r = Rows(V, dtype, 2)
    d = bn.soft_desc(1, 4, draft_rows, V, bn.spec_dtype(r.z), 4, 4)
    draft = torch.randn((1, max(draft_rows, 1), V), device="cuda").to(r.dt)
    u = torch.full((1, 4), 0.25, device="cuda")
    for us in (0.0, 0.5, 0.99):
        bn.spec_accept_soft(d, r.z, draft[:, :draft_rows], r.tokens, r.parent, None,
                            torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4) if draft_rows else None,
                            r.n, u, torch.full((1,), us, device="cuda"), r.lse, torch.zeros((1, 4), device="cuda"),
                            r.acc, r.path, r.next, r.last)
        assert bn.spec_get_status() == 0
        # p(token 0) is 1 - 1e-4 at rows 0 and 1, so their children are taken
        assert int(r.acc) == 3 and r.path[0].tolist() == [0, 1, 2, -1] and int(r.last) == 2
        assert int(r.next) == -1


def test_a_row_of_nan_names_no_token_either():
    z = torch.full((2, 4000), float("nan"), device="cuda")
    z[1, 5] = 1.0
    am, lse = i32(3, 3), torch.zeros(2, device="cuda")
    bn.spec_vocab_reduce(z, None, am, lse, None)
    assert am.tolist() == [-1, 5] and np.isnan(lse.cpu().numpy()).all()
