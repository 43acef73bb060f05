"""Chunk attention where consecutive units of a CTA differ in their tiles: last units
with one query tile, parts that a request's earlier tokens are through with, behind
histories of many steps, over pages that requests share."""

import numpy as np
import pytest
import torch

import gpu_helpers as gh
from chunk_helpers import Chunk, dev
from self_speculative_verification_gb300 import binding as bn
from test_gpu_chunk_step import double_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    gh.require_gpu()
    bn.spec_get_status()


def share_prefix(c, tokens, ps):
    """The first `tokens` (a multiple of ps) of every request lie in the first one's
    pages."""
    for b in range(1, len(c.new)):
        c.table[b, :tokens // ps] = c.table[0, :tokens // ps]
        c.k[b][:, :tokens], c.v[b][:, :tokens] = c.k[0][:, :tokens], c.v[0][:, :tokens]
    c.d_table.copy_(dev(c.table))


# tokens of a tile: 32 (of 4 query heads a KV head).  n mod 64 in 1 .. 32: a last unit
# of one tile
@pytest.mark.parametrize("kind,ps,prefix", [("paged", 16, 2048), ("paged", 64, 1024), ("contiguous", 0, 0),
                                            ("kv8", 16, 2048)])
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("new,held", [
    ((84,) * 10, (3000,) * 10),                                  # two units, one tile and a half
    ((65, 96, 212, 33, 1, 160, 70, 81), (2900, 2500, 2111, 3300, 2800, 2222, 2047 + 64, 3071)),
    ((276, 276, 276), (2048, 2100, 2175))])
def test_last_units_of_one_tile(kind, ps, prefix, d, new, held):
    c = Chunk(len(new) + d, kind, "bf16", d, 32, 8, new, held, ps=ps or 16)
    if prefix:
        share_prefix(c, prefix, ps)
    c.run()
    assert bn.spec_get_status() == 0
    rng = np.random.default_rng(0)
    n = int(c.cu[-1])
    rows = np.unique(np.concatenate([c.cu[:-1], c.cu[1:] - 1, rng.integers(0, n, 60)]))
    O, A, L, big = double_attention(c, rows)
    to, tl = c.tolerance(O, L, A, big)
    got, lse = c.o.double().cpu().numpy(), c.lse.double().cpu().numpy()
    assert np.isfinite(got[:n]).all() and np.isfinite(lse[:n]).all()
    assert (got[n:] == 7.0).all() and (lse[n:] == 7.0).all()
    assert (np.abs(got[rows] - O) <= to).all() and (np.abs(lse[rows] - L) <= tl).all()
    assert np.linalg.norm(got[rows] - O) <= 2.0 ** -8 * np.linalg.norm(O)
    o, lse = c.o.clone(), c.lse.clone()
    for _ in range(30):
        c.run()
        assert torch.equal(c.o, o) and torch.equal(c.lse, lse)
    assert bn.spec_get_status() == 0
