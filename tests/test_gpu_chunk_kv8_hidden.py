"""Non-finite values of the 8-bit cache that lie in a chunk itself: rows before them
are as if they were not there."""

import numpy as np
import pytest

import gpu_helpers as gh
from chunk_helpers import Chunk
from kv8_helpers import NAN_CODE, pack
from self_speculative_verification_gb300 import binding as bn

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    gh.require_gpu()
    bn.spec_get_status()


# (request, head, token; None: the value scale of its page, else this dimension's code)
PLACES = {
    "two tiles, a scale": [(0, 0, 64, None)],
    "two tiles, a code": [(0, 1, 90, 7)],
    "two heads, a scale of the first": [(1, 0, 48, None)],
    "two heads, a scale of the second": [(1, 1, 48, None)],
    "two heads, a code of the first": [(1, 0, 61, 120)],
    "two heads, a code of the second": [(1, 1, 61, 0)],
    "the last token": [(0, 0, 159, 3), (1, 1, 79, 3), (2, 0, 304, 3)],
    "several": [(0, 0, 130, 1), (0, 0, 96, None), (0, 1, 12, 5), (1, 0, 33, 9), (1, 1, 32, None), (2, 1, 288, None)],
    "one of a step behind whole ones": [(2, 0, 290, 60), (2, 1, 303, 1)],
}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("ps", [16, 32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("places", PLACES)
def test_rows_before_a_non_finite_value(dtype, ps, d, places):
    """Two query heads a KV head: a tile is 64 tokens, so the second and third
    requests' units are pairs of heads."""
    c = Chunk(80 + ps, "kv8", dtype, d, 4, 2, (150, 60, 40), (10, 20, 265), ps=ps)
    ref = c.oracle()                                             # of the finite cache
    first = {}                                                   # its first bad token, per (request, head)
    n = int(c.cu[-1])
    must = np.zeros((n, 4, d), dtype=bool)                       # places that have to be NaN
    for b, h, t, x in PLACES[places]:
        page = int(c.table[b, t // ps])
        x = x if x is None else x % d
        if x is None:
            t = t // ps * ps                                     # all of the page
            c.d_scales[page, h, 1] = float("nan")
        else:
            c.codes[page, h, 1, t % ps, x] = NAN_CODE
        first[b, h] = min(first.get((b, h), 1 << 30), t)
        rows = slice(int(c.cu[b]) + max(0, t - int(c.held[b])), int(c.cu[b + 1]))
        must[rows, 2 * h:2 * h + 2, slice(None) if x is None else x] = True
    c.d_kv.copy_(pack(c.codes))
    free = np.ones((n, 4), dtype=bool)                           # rows that see no such place
    for (b, h), t in first.items():
        free[int(c.cu[b]) + max(0, t - int(c.held[b])):int(c.cu[b + 1]), 2 * h:2 * h + 2] = False
    assert free.any() and must.any()
    c.run()
    assert bn.spec_get_status() == 0
    O, L, A, big = (x[:n] for x in ref)
    to, tl = c.tolerance(O, L, A, big)
    got, lse = c.o.double().cpu().numpy()[:n], c.lse.double().cpu().numpy()[:n]
    assert (np.abs(got - O)[free] <= to[free]).all()
    assert np.isnan(got[must]).all()
    assert np.isfinite(lse).all() and (np.abs(lse - L) <= tl).all()     # (values do not reach it)
