"""spec_verify_attn_kv8 for rows that see their prefix alone (no block or
soft-prompt column), where units are cut between CTAs right ahead of the
block's tile, after calls that left other contents on the SMs."""

import numpy as np
import pytest
import torch

import gpu_helpers as gh
from kv8_helpers import Attn
from self_speculative_verification_gb300 import binding as bn

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    gh.require_gpu()
    bn.spec_get_status()


def blind(a):
    """Every second row loses its block and soft-prompt columns."""
    a.vis[:, ::2] = False
    a.sees[:, ::2] = False
    a.words[:, ::2] = 0
    a.d_vis.copy_(torch.from_numpy(a.words))
    a.d_flags.copy_(torch.from_numpy((a.valid * 1 + a.sees * 2).astype(np.uint8)))


@pytest.mark.parametrize("n_soft", [0, 5])
@pytest.mark.parametrize("before,R", [(2, 8), (4, 8), (16, 8), (2, 4), (8, 4), (8, 2), (16, 2), (2, 16)])
def test_prefix_rows_of_cut_units(before, R, n_soft):
    rng = np.random.default_rng(before * 100 + R)
    # units of 3 .. 9 steps over all of the GPU's CTAs: cuts fall on every
    # step of a unit, the last among them
    S = rng.integers(200, 1000, size=40)
    other = Attn(2, B=20, Hq=16, Hkv=4, R=before, S=rng.integers(1, 300, size=20), mask="tree")
    a = Attn(3, B=40, Hq=16, Hkv=4, R=R, S=S, n_soft=n_soft, mask="tree", pad=False)
    blind(a)
    for _ in range(3):
        other.run()
        a.run()
        torch.cuda.synchronize()
        assert bn.spec_get_status() == 0
        assert torch.isfinite(a.o).all() and torch.isfinite(a.lse).all()
    a.check(requests=range(0, 40, 7))
