"""Chunk attention of rows whose scores are -inf over whole steps, with units cut
there: a non-finite value that such a row sees reaches it, as it does where one
CTA has the unit whole."""

import numpy as np
import pytest
import torch

import gpu_helpers as gh
from chunk_helpers import Chunk
from kv8_helpers import pack
from self_speculative_verification_gb300 import binding as bn

pytestmark = pytest.mark.gpu

DIM, HEAD = 5, 0                                      # -inf in this element of this head's keys


@pytest.fixture(autouse=True)
def _gpu():
    gh.require_gpu()
    bn.spec_get_status()


def put(c, which, b, h, t, x, what):
    """One element of a key or value, on the device and in the oracle's rows."""
    host, device = (c.k, c.d_k) if which == "k" else (c.v, c.d_v)
    host[b][h, t, x] = what
    ps = device.shape[3]
    if c.kind == "paged":
        device[c.table[b, t // ps], h, x // 64, t % ps, x % 64] = what
    else:
        device[b, h, t, x] = what


def unseen(c, lo, hi):
    """Scores of -inf for tokens lo .. hi - 1 of request 0, head HEAD."""
    G = c.shape[2] // c.shape[3]
    c.q[:, HEAD * G:(HEAD + 1) * G, DIM] = 1.0
    c.d_q[:, HEAD * G:(HEAD + 1) * G, DIM] = 1.0
    for t in range(lo, hi):
        put(c, "k", 0, HEAD, t, DIM, -np.inf)


# (held: steps of 128 and of 64 keys, shared out one by one; a single step)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["paged", "contiguous"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("held,lo,hi", [(2999, 1280, 1536), (2999, 0, 3000), (2999, 0, 2944), (59, 0, 60), (59, 7, 30)])
@pytest.mark.parametrize("what", [None, np.nan, np.inf])
def test_values_behind_scores_of_minus_infinity(dtype, kind, d, held, lo, hi, what):
    c = Chunk(held + d, kind, dtype, d, 4, 2, (1, 2), (held, 9), ps=16)
    unseen(c, lo, hi)
    t, x = lo + 10, d - 3
    if what is not None:
        put(c, "v", 0, HEAD, t, x, what)
    c.run()
    assert bn.spec_get_status() == 0
    O, L, A, big = c.oracle()
    n = int(c.cu[-1])
    got, lse = c.o.double().cpu().numpy()[:n], c.lse.double().cpu().numpy()[:n]
    none = lo == 0 and hi == held + 1                 # no other score
    assert np.array_equal(np.isneginf(lse), np.isneginf(L[:n])) and np.isneginf(lse[0, :2]).all() == none
    hit = np.zeros(got.shape[:2], dtype=bool)
    hit[0, :2] = what is not None
    assert not np.isfinite(got[0, :2, x][hit[0, :2]]).any()
    # (-inf elements: what bounds an error is the other keys' sizes)
    big = np.where(np.isfinite(big), big, 40.0)
    to, tl = c.tolerance(np.nan_to_num(O[:n]), np.where(np.isfinite(L[:n]), L[:n], 0.0), np.nan_to_num(A[:n]), big[:n])
    assert (np.abs(got - O[:n])[~hit] <= to[~hit]).all()
    fin = np.isfinite(L[:n])
    assert np.isfinite(lse[fin]).all() and (np.abs(lse[fin] - L[:n][fin]) <= tl[fin]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("held", [1999, 59])
@pytest.mark.parametrize("bad", [False, True])
def test_a_nan_value_scale_behind_scores_of_minus_infinity(dtype, held, bad):
    """8 bits: an infinite query element against keys that are all negative there."""
    c = Chunk(held, "kv8", dtype, 128, 4, 2, (1, 2), (held, 9), ps=16)
    c.codes[:, HEAD, 0, :, DIM] = 0x80 | 0x38                                # -1 of its scale
    c.d_kv.copy_(pack(c.codes))
    c.d_q[0, :2, DIM] = float("inf")
    if bad:
        c.d_scales[int(c.table[0, 2]), HEAD, 1] = float("nan")
    c.run()
    assert bn.spec_get_status() == 0
    assert torch.isneginf(c.lse[0, :2]).all() and torch.isfinite(c.lse[0, 2:]).all()
    if bad:
        assert torch.isnan(c.o[0, :2]).all()
    else:
        assert (c.o[0, :2] == 0).all()
    assert torch.isfinite(c.o[0, 2:]).all() and torch.isfinite(c.o[1:3, 2:]).all()
